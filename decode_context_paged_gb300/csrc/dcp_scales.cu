// dcp_scales.cu -- block scales of an 8-bit cache, from the CP layer split to the DCP ranks.
//
// "Serving Macaron-V1 at Scale: Page-Level 2D KV Resharding", 2, 5.1, 6.3: a page of layer l moves
// from the CP rank that owns l to rank v mod N_dcp at slot v div N_dcp.  The scales of a
// block-scaled page (64 / g fp32 values, contiguous) take the same way: source
// [layers of r][source pages][64 / g], destination [layers][slots][64 / g] per rank.
//
// A gather and a scatter of 4 to 256 bytes per (layer, page).  One thread owns one vector (16 bytes,
// or a whole page's scales where they are fewer, or what every rank's start is a multiple of: a rank's
// scales may be a slice of a larger tensor) of one page and moves it for kLayersPerThread
// layers: the page's two table entries and its division are paid once, and the loads of all those
// layers are in flight together.  Bound: HBM for whole batches (neighbouring threads cover a
// page's 256 contiguous bytes; 184 MB of scales in 58.5 us = 6.5 TB/s, 98% of the copy rate), latency
// for one request (2.0 us).
#include <cuda_runtime.h>

#include "dcp_internal.h"
#include "dcp_ptx.cuh"

namespace dcp {
namespace {

constexpr int kScaleThreads = 256;
constexpr int kLayersPerThread = 4;

template <typename V>
__global__ void __launch_bounds__(kScaleThreads) scales_kernel(const __grid_constant__ ScalesArgs a, int vecs) {
    grid_dep_wait();
    grid_dep_launch();
    const long long id = (long long)blockIdx.x * kScaleThreads + threadIdx.x;
    const long long p = id / vecs;
    const int part = (int)(id - p * vecs);
    // entries behind the last request's are padding
    if (p >= a.num_pages || p >= (long long)__ldg(a.req_page_ptr + a.num_requests)) return;
    const int v = __ldg(a.dst_vpages + p), src = __ldg(a.src_pages + p);
    const int d = v < 0 ? -1 : v % a.n_dcp;
    const long long slot = v / a.n_dcp;
    if (d < 0 || slot >= a.dst_slots || src < 0 || src >= a.src_pool_pages) {
        if (part == 0 && blockIdx.y == 0 && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_OUT_OF_RANGE);
        return;
    }
    const int l0 = blockIdx.y * kLayersPerThread;
    V *dst = reinterpret_cast<V *>(a.dst_scales[d]) + slot * vecs + part;
    V x[kLayersPerThread];
    int r = 0;
#pragma unroll
    for (int i = 0; i < kLayersPerThread; ++i) {
        const int l = l0 + i;
        if (l < a.num_layers) {
            while (l >= a.layer_start[r + 1]) ++r;
            x[i] = __ldg(reinterpret_cast<const V *>(a.src_scales[r]) +
                         ((long long)(l - a.layer_start[r]) * a.src_pool_pages + src) * vecs + part);
        }
    }
#pragma unroll
    for (int i = 0; i < kLayersPerThread; ++i)
        if (l0 + i < a.num_layers) dst[(long long)(l0 + i) * a.dst_slots * vecs] = x[i];
}

}  // namespace

cudaError_t launch_scales(const ScalesArgs &a, cudaStream_t stream) {
    if (a.num_pages <= 0 || a.num_layers <= 0) return cudaSuccess;
    int vec = a.groups >= 4 ? 4 : a.groups;  // floats per thread
    uintptr_t starts = 0;
    for (int r = 0; a.layer_start[r] < a.num_layers; ++r) starts |= reinterpret_cast<uintptr_t>(a.src_scales[r]);
    for (int d = 0; d < a.n_dcp; ++d) starts |= reinterpret_cast<uintptr_t>(a.dst_scales[d]);
    while (starts % (4 * vec)) vec /= 2;  // (every start is a multiple of 4 bytes)
    const int vecs = a.groups / vec;
    const long long blocks = (a.num_pages * vecs + kScaleThreads - 1) / kScaleThreads;
    const int ly = (a.num_layers + kLayersPerThread - 1) / kLayersPerThread;
    if (blocks > 0x7fffffffLL || ly > 65535) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks, (unsigned)ly), block(kScaleThreads);
    if (vec == 4) return launch_pdl(scales_kernel<float4>, grid, block, 0, stream, a, vecs);
    if (vec == 2) return launch_pdl(scales_kernel<float2>, grid, block, 0, stream, a, vecs);
    return launch_pdl(scales_kernel<float>, grid, block, 0, stream, a, vecs);
}

}  // namespace dcp
