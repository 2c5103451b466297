// dcp_append.cu -- new tokens' key rows into the paged DCP pools, with the rotary embedding and
// (8-bit pools) the quantisation on the way.
//
// "Serving Macaron-V1 at Scale: Page-Level 2D KV Resharding", 5.1 (page value v lives on rank
// v mod N_dcp at slot v div N_dcp), 5.3 (rows are 512 latent + 64 rope = 576 elements); "SGLang's
// path" (the token-interleaved layout).
//
// Per new token at position p:  row = [ latent (512) | R(p) rope (64) ].  R(p) turns the pairs
// (x_2i, x_2i+1), or (x_i, x_i+32), by the angle p * inv_freq[i].
//
// The angle.  An fp32 product p * inv_freq loses the angle of far positions (p = 10^6 leaves 2^-4
// rad).  inv_freq / (2 pi) is taken as a 64-bit fixed-point fraction of a turn instead, p times it
// wraps modulo 2^64 exactly as angles do, and the top 32 bits make the angle, right to about 2^-30
// turns for every p below 2^31, in integer instructions (the fp64 units are slow).
//
// Quantisation.  Block scales: the scale of g consecutive rows of a page is the smallest power of
// two s with max|x| <= 448 s (non-finite values do not count), held to [2^-40, 2^48]: the attention takes
// larger scales as 2^48, so elements above 448 * 2^48 saturate here instead.  A power of two makes
// x / s exact, costs no precision in E4M3's normal range, and lets a block's rows be coded again
// with one more rounding only where they turn subnormal.  A call that goes on a block holding rows
// of earlier tokens never shrinks its scale; where the scale grows the earlier rows are coded again.
//
// Work split.  One CTA per (request, part of a page of one rank) with new tokens: the CTA owns the
// part's new rows and their scale blocks, so there are no atomics on global memory and no order to
// matter.  A part is 16 rows, or a scale block where that is larger; a warp takes four rows, all
// loaded before the first is used.
// Its first warp finds the request by a 32-way search over new_ptr: request b's units start at
// floor(new_ptr[b] / W) + 2 b (W = the part's rows; times N and W = N rows for the token layout), which
// bounds the pages its tokens can touch without a scan or a host copy.  Further CTAs of the same
// launch rotate the queries.  Bound: launch latency for a decode step (64 tokens with 64 query
// heads: 4.0 us a call of a captured sequence), the latency of loads and barriers for prompts (69K tokens into E4M3 with blocks of
// 16: 26.0 us = 4.55 TB/s, 68% of the copy rate).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "dcp_internal.h"
#include "dcp_ptx.cuh"
#include "dcp_search.cuh"

namespace dcp {
namespace {

constexpr int kRowsPerWarp = 4;
constexpr int kQHeads = 8;              // heads one warp rotates: its loads are in flight together
constexpr int kMinScaleExp = -40, kMaxScaleExp = 48;

// inv_freq / (2 pi) mod 1 as a 64-bit fraction.  x = m 2^(e - 1075) with an integer m < 2^53;
// C = round(2^64 / (2 pi)); the fraction is m C 2^(e - 1075) as an integer modulo 2^64.
__device__ __forceinline__ unsigned long long turn_fraction(double x) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(x);
    const int e = (int)((bits >> 52) & 0x7ff);
    if (e == 0 || e == 0x7ff) return 0;  // zero, subnormal; infinity and NaN are not frequencies
    const unsigned long long m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
    const unsigned long long C = 0x28be60db9391054aull;
    const unsigned long long hi = __umul64hi(m, C), lo = m * C;
    const int sh = 1075 - e;  // right shift of the 128-bit product
    unsigned long long f;
    if (sh <= 0) f = -sh < 64 ? lo << (-sh) : 0;
    else if (sh < 64) f = (hi << (64 - sh)) | (lo >> sh);
    else f = sh < 128 ? hi >> (sh - 64) : 0;
    return (bits >> 63) ? 0ull - f : f;
}

struct Turn {
    float c0, s0, c1, s1;
};

// The lane's cosines and sines at position pos.  Interleaved: lane l turns pair l (c0, s0).
// Halves: lane l holds elements 2l and 2l + 1, whose frequencies are 2 (l mod 16) and the next.
__device__ __forceinline__ Turn turn_at(long long pos, unsigned long long f0, unsigned long long f1, bool interleaved,
                                        float scale) {
    Turn t;
    // radians in [-pi, pi) from the top 32 bits, three roundings of 2^-24 of at most pi; there the
    // hardware sine and cosine are off by at most 2^-21.1: about 1e-6 in all, against the outputs' half
    // steps of 2^-8 and more
    auto radians = [](unsigned long long ph) { return (float)(int)(ph >> 32) * 1.4629180792671596e-9f; };  // 2 pi 2^-32
    const float a = radians(f0 * (unsigned long long)pos);
    t.s0 = t.s1 = __sinf(a) * scale;
    t.c0 = t.c1 = __cosf(a) * scale;
    if (!interleaved) {
        const float b = radians(f1 * (unsigned long long)pos);
        t.s1 = __sinf(b) * scale;
        t.c1 = __cosf(b) * scale;
    }
    return t;
}

// The warp's 64 rotary elements, two per lane (2l, 2l + 1), turned.
__device__ __forceinline__ float2 turned(uint32_t raw, const Turn &t, bool interleaved, int lane) {
    const float a = __uint_as_float(raw << 16), b = __uint_as_float(raw & 0xffff0000u);
    if (interleaved) return make_float2(a * t.c0 - b * t.s0, b * t.c0 + a * t.s0);
    const uint32_t other = __shfl_xor_sync(0xffffffffu, raw, 16);
    const float oa = __uint_as_float(other << 16), ob = __uint_as_float(other & 0xffff0000u);
    return lane < 16 ? make_float2(a * t.c0 - oa * t.s0, b * t.c1 - ob * t.s1)
                     : make_float2(a * t.c0 + oa * t.s0, b * t.c1 + ob * t.s1);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// E4M3 codes of a lane's part of a row (16 latent elements, two rope) divided by s.  kPow2: s is a
// power of two and the product with 1 / s exact; otherwise (a pool scale, a user's block scale) a
// division each.  The choice is made once per row: decided per element it cost more than the codes.
template <bool kPow2>
__device__ __forceinline__ void quantise(const uint4 &u, const uint4 &v, float2 r, float s, float inv, uint2 &lo, uint2 &hi, uint32_t &tail) {
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xffff0000u);
        o[i] = kPow2 ? e4m3x2(a * inv, b * inv) : e4m3x2(a / s, b / s);
    }
    lo = make_uint2(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410));
    hi = make_uint2(__byte_perm(o[4], o[5], 0x5410), __byte_perm(o[6], o[7], 0x5410));
    tail = kPow2 ? e4m3x2(r.x * inv, r.y * inv) : e4m3x2(r.x / s, r.y / s);
}

// 1 / s of a power of two (with a normal reciprocal), else 0.
__device__ __forceinline__ float exact_inverse(float s) {
    const uint32_t b = __float_as_uint(s);
    return (b & 0x807fffffu) == 0 && b >= 0x00800000u && b < 0x7f000000u ? __uint_as_float(0x7f000000u - b) : 0.f;
}

// Codes of a coarser scale: ratio = old scale / new scale.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float ratio) {
    uint32_t o = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        o |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * i);
    }
    return o;
}

// The largest finite magnitude of a lane's part of a row, as float bits (order-preserving).
__device__ __forceinline__ uint32_t finite_amax(const uint4 &a, const uint4 &b, float2 r) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    uint32_t x = max(m & 0xffffu, m >> 16);
    if (x >= 0x7f80u) {  // some element is infinite or NaN: leave those out one by one
        x = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
            if (lo < 0x7f80u) x = max(x, lo);
            if (hi < 0x7f80u) x = max(x, hi);
        }
    }
    x <<= 16;
    const uint32_t r0 = __float_as_uint(r.x) & 0x7fffffffu, r1 = __float_as_uint(r.y) & 0x7fffffffu;
    if (r0 < 0x7f800000u) x = max(x, r0);
    if (r1 < 0x7f800000u) x = max(x, r1);
    return x;
}

// Smallest power of two s >= 2^-40 with amax <= 448 s (448 = 1.75 * 2^8), at most 2^48.
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23) - 127;
    const int k = e - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(min(max(k, kMinScaleExp), kMaxScaleExp) + 127) << 23);
}

__device__ void rotate_queries(const AppendArgs &a, long long task, int lane) {
    const uint32_t chunks = (uint32_t)(a.num_heads + kQHeads - 1) / kQHeads;
    const long long tok = (uint32_t)task / chunks;  // (rows times chunks are below 2^31)
    const int h0 = (int)((uint32_t)task - (uint32_t)tok * chunks) * kQHeads;
    if (tok >= a.num_new) return;
    uint32_t x[kQHeads];
    const __nv_bfloat16 *src = a.q_rope + tok * a.q_tok_stride + 2 * lane;
#pragma unroll
    for (int i = 0; i < kQHeads; ++i)  // (plain loads: q_out may be q_rope, and this warp alone writes these rows)
        x[i] = h0 + i < a.num_heads ? *reinterpret_cast<const uint32_t *>(src + (h0 + i) * a.q_head_stride) : 0u;
    const int b = warp_search(a.num_requests, tok, lane, [&](int i) { return (long long)__ldg(a.new_ptr + i); });
    if (b < 0) return;
    const long long n0 = __ldg(a.new_ptr + b), n1 = __ldg(a.new_ptr + b + 1);
    if (n0 < 0 || tok >= n1 || n1 > a.num_new) return;  // a row no request has
    const long long start = (long long)__ldg(a.seq_lens + b) - (n1 - n0);
    if (start < 0) return;  // (reported beside the units)
    const int fi = a.interleaved ? lane : 2 * (lane & 15);
    const unsigned long long f0 = turn_fraction(__ldg(a.inv_freq + fi));
    const unsigned long long f1 = a.interleaved ? 0 : turn_fraction(__ldg(a.inv_freq + fi + 1));
    const Turn t = turn_at(start + tok - n0, f0, f1, a.interleaved, a.rope_scale);
    __nv_bfloat16 *dst = a.q_out + tok * a.qo_tok_stride + 2 * lane;
#pragma unroll
    for (int i = 0; i < kQHeads; ++i) {
        const float2 y = turned(x[i], t, a.interleaved, lane);
        if (h0 + i < a.num_heads) *reinterpret_cast<uint32_t *>(dst + (h0 + i) * a.qo_head_stride) = pack2(y.x, y.y);
    }
}

// TOK: the token-interleaved layout.  Every offset and position is below 2^31 (larger ones are refused
// or reported), so the divisions by the rank count are 32-bit, and the page layout has shifts only:
// 64-bit divisions, seven per warp, were a third of the kernel's instructions.
// U: rows of a unit, a part of a page that holds whole scale blocks; U / 4 warps, four rows each.
template <bool F8, bool SC, bool TOK, int U>
__global__ void __launch_bounds__(U * 8, 768 / (U * 8)) append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kWarps = U / kRowsPerWarp, kParts = kPage / U;
    __shared__ uint32_t amax[kPage];
    __shared__ float2 scale_of[kPage];  // a block's scale, and its reciprocal where it is a power of two, else 0
    __shared__ float again;  // old scale / new scale of the first block where it grew, else -1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    if ((long long)blockIdx.x >= a.n_units) {
        rotate_queries(a, ((long long)blockIdx.x - a.n_units) * kWarps + warp, lane);
        return;
    }
    const uint32_t ns = TOK ? (uint32_t)a.tok_n : 1u;  // ranks that share a request's pages token by token
    // Warp 0 finds the unit's rows, then its page while the others load; warp 1 the turn fractions.
    __shared__ struct {
        long long tok0, pos0;  // token and position of row lo; + ns per row
        long long slot;
        int lo, hi, d;
    } unit;
    __shared__ unsigned long long fraction[32];
    int lo = 0, hi = 0, d0 = 0;
    long long p0 = 0, p1 = 0;  // the request's page table
    uint32_t jj = 0;
    auto fits = [&](long long n0, long long n1, int len) { return n0 >= 0 && n0 <= n1 && n1 <= a.num_new && n1 - n0 <= len; };
    if (warp == 0) {
        // x / (U ns): a unit's span of tokens
        auto spans = [&](uint32_t x) -> uint32_t { return TOK ? x / U / ns : x / U; };
        auto first_unit = [&](long long x, int i) -> long long {
            return ns * (spans(x < 0 ? 0u : x > 0x7fffffff ? 0x7fffffffu : (uint32_t)x) + 2LL * i);
        };
        const long long u = blockIdx.x;
        // Up to 32 requests are left (a coarse search in larger batches): each lane loads all that its
        // request needs at once, so that the page's entry and the rows are two round trips away, not four.
        int r0 = 0, r1 = a.num_requests;
        while (r1 - r0 > 32) {
            const int step = (r1 - r0 + 31) / 32, i = r0 + lane * step;
            const unsigned m = __ballot_sync(0xffffffffu, i < r1 && first_unit(__ldg(a.new_ptr + i), i) <= u);
            const int c = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
            if (c == 0) break;  // (only where the first unit is behind u, or offsets decrease)
            r0 += (c - 1) * step;
            r1 = min(r1, r0 + step);
        }
        const int mine = min(r0 + lane, a.num_requests - 1);
        const long long ptr0 = __ldg(a.new_ptr + mine), ptr1 = __ldg(a.new_ptr + mine + 1);
        const long long page0 = __ldg(a.req_page_ptr + mine), page1 = __ldg(a.req_page_ptr + mine + 1);
        const int len = __ldg(a.seq_lens + mine);
        const unsigned m = __ballot_sync(0xffffffffu, r0 + lane < r1 && first_unit(ptr0, mine) <= u);
        const int at = m == 0xffffffffu ? 31 : __ffs(~m) - 2;
        if (at >= 0) {
            const long long n0 = __shfl_sync(0xffffffffu, ptr0, at), n1 = __shfl_sync(0xffffffffu, ptr1, at);
            p0 = __shfl_sync(0xffffffffu, page0, at);
            p1 = __shfl_sync(0xffffffffu, page1, at);
            const int end = __shfl_sync(0xffffffffu, len, at);
            const uint32_t k = (uint32_t)(u - first_unit(n0, r0 + at));
            if (fits(n0, n1, end) && n1 > n0) {
                const int start = end - (int)(n1 - n0);
                jj = spans((uint32_t)start) + (TOK ? k / ns : k);
                d0 = TOK ? (int)(k % ns) : 0;
                // rows [lo, hi) of the page are new: row i of the unit holds position (U jj + i) ns + d0
                auto first_row = [&](int p) -> int {
                    const long long x = TOK ? (p <= d0 ? 0 : ((uint32_t)(p - d0) + ns - 1) / ns) : (uint32_t)p;
                    const long long i = x - (long long)U * jj;
                    return (int)(jj % kParts) * U + (int)(i < 0 ? 0 : i > U ? U : i);
                };
                lo = first_row(start);
                hi = first_row(end);
                if (lane == 0) {
                    unit.pos0 = ((long long)U * jj + lo - (int)(jj % kParts) * U) * ns + d0;
                    unit.tok0 = n0 + unit.pos0 - start;
                }
            }
        }
        if (lane == 0) {
            unit.lo = lo;
            unit.hi = hi;
        }
    } else if (warp == 1) {
        fraction[lane] = turn_fraction(__ldg(a.inv_freq + lane));
    } else if (warp == 2 && a.dev_error) {
        // Requests that do not fit are reported here, 32 to a CTA (a request has two units at least): their
        // offsets may lead to no unit at all.
        const long long i = (long long)blockIdx.x * 32 + lane;
        if (i < a.num_requests) {
            const long long n0 = __ldg(a.new_ptr + i), n1 = __ldg(a.new_ptr + i + 1);
            if (n0 != n1 && !fits(n0, n1, __ldg(a.seq_lens + i))) atomicOr(a.dev_error, DCP_DEVERR_OUT_OF_RANGE);
        }
    }
    __syncthreads();
    lo = unit.lo;
    hi = unit.hi;
    if (lo >= hi) return;
    const long long tok0 = unit.tok0;
    // this warp's rows, all in flight
    uint4 x0[kRowsPerWarp], x1[kRowsPerWarp];
    uint32_t xr[kRowsPerWarp];
    const __nv_bfloat16 *ls = a.latent + (tok0 + (long long)warp * ns) * a.latent_stride + 8 * lane;
    const __nv_bfloat16 *rs = a.rope + (tok0 + (long long)warp * ns) * a.rope_stride + 2 * lane;
    const long long l_step = a.latent_stride * kWarps * ns, r_step = a.rope_stride * kWarps * ns;
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        x0[r] = x1[r] = make_uint4(0, 0, 0, 0);
        xr[r] = 0;
        if (lo + warp + kWarps * r < hi) {
            x0[r] = __ldg(reinterpret_cast<const uint4 *>(ls));
            x1[r] = __ldg(reinterpret_cast<const uint4 *>(ls) + 32);
            xr[r] = __ldg(reinterpret_cast<const uint32_t *>(rs));
        }
        ls += l_step;
        rs += r_step;
    }
    if (warp == 0) {
        const long long e = (long long)(jj / kParts) * ns + d0;
        int d = -1;
        long long slot = 0;
        if (e < p1 - p0 && p0 >= 0 && p0 + e < a.num_pages) {
            const int v = __ldg(a.dst_vpages + p0 + e);
            d = v < 0 ? -1 : v % a.n_dcp;
            slot = v / a.n_dcp;
        }
        if (d < 0 || slot >= a.slots_per_rank || (TOK && d != d0)) {  // no such page: skip its rows
            if (lane == 0 && a.dev_error) atomicOr(a.dev_error, DCP_DEVERR_OUT_OF_RANGE);
            d = -1;
        }
        if (lane == 0) {
            unit.d = d;
            unit.slot = slot;
        }
    }
    if (SC && threadIdx.x < kPage) amax[threadIdx.x] = 0;
    __syncthreads();
    const int d = unit.d;
    if (d < 0) return;
    const long long slot = unit.slot;
    const int g = a.scale_block, g_shift = 31 - __clz(g | 1);
    float *scales = nullptr;
    float old = 0.f;
    if (SC) {
        scales = a.kv_scales[d] + slot * (kPage >> g_shift);
        if (threadIdx.x == (unsigned)(lo >> g_shift)) old = scales[lo >> g_shift];  // (threads 0..63)
    }
    const int fi = a.interleaved ? lane : 2 * (lane & 15);
    const unsigned long long f0 = fraction[fi], f1 = fraction[a.interleaved ? lane : fi + 1];
    float2 y[kRowsPerWarp];
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        const int row = lo + warp + kWarps * r;
        if (row >= hi) break;  // (warp-uniform)
        const Turn t = turn_at(unit.pos0 + (long long)(row - lo) * ns, f0, f1, a.interleaved, a.rope_scale);
        y[r] = turned(xr[r], t, a.interleaved, lane);
        if (SC) {
            const uint32_t m = __reduce_max_sync(0xffffffffu, finite_amax(x0[r], x1[r], y[r]));
            if (lane == 0) atomicMax(&amax[row >> g_shift], m);
        }
    }
    uint8_t *page = a.kv_pools[d] + slot * (long long)kPage * kKDim * (F8 ? 1 : 2);
    if (SC) {
        __syncthreads();
        const int blk = threadIdx.x;
        if (blk >= lo / g && blk <= (hi - 1) / g) {
            float s = block_scale(amax[blk]);
            if (blk == lo / g) {
                const bool holds = lo % g != 0;  // rows of earlier tokens
                float ratio = -1.f;
                if (holds) {
                    if (s > old) ratio = old / s;
                    else s = old;
                }
                again = ratio;
            }
            scale_of[blk] = make_float2(s, exact_inverse(s));
            scales[blk] = s;
        }
        __syncthreads();
        const float ratio = again;
        if (ratio >= 0.f) {
            for (int row = lo / g * g + warp; row < lo; row += kWarps) {
                uint32_t *c = reinterpret_cast<uint32_t *>(page + row * kKDim);
#pragma unroll
                for (int i = 0; i < 5; ++i) {
                    const int at = lane + 32 * i;
                    if (at < kKDim / 4) c[at] = recode4(c[at], ratio);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRowsPerWarp; ++r) {
        const int row = lo + warp + kWarps * r;
        if (row >= hi) break;
        if (F8) {
            const float2 s = SC ? scale_of[row >> g_shift] : make_float2(a.kv_scale, a.kv_scale_inv);
            uint2 lo8, hi8;
            uint32_t tail;
            if (s.y != 0.f) quantise<true>(x0[r], x1[r], y[r], s.x, s.y, lo8, hi8, tail);
            else quantise<false>(x0[r], x1[r], y[r], s.x, s.y, lo8, hi8, tail);
            uint8_t *dst = page + row * kKDim;
            *reinterpret_cast<uint2 *>(dst + 8 * lane) = lo8;
            *reinterpret_cast<uint2 *>(dst + 256 + 8 * lane) = hi8;
            *reinterpret_cast<uint16_t *>(dst + kVDim + 2 * lane) = (uint16_t)tail;
        } else {
            uint4 *dst = reinterpret_cast<uint4 *>(page + row * kKDim * 2);
            dst[lane] = x0[r];
            dst[32 + lane] = x1[r];
            reinterpret_cast<uint32_t *>(page + row * kKDim * 2 + kVDim * 2)[lane] = pack2(y[r].x, y[r].y);
        }
    }
}

}  // namespace

template <bool F8, bool SC, int U>
static cudaError_t launch_unit(AppendArgs &a, cudaStream_t stream) {
    const long long ns = a.tok_n > 0 ? a.tok_n : 1;
    a.n_units = ns * (a.num_new / (U * ns) + 2LL * a.num_requests);
    const long long chunks = (a.num_heads + kQHeads - 1) / kQHeads;
    const long long q_blocks = (a.num_new * chunks + U / kRowsPerWarp - 1) / (U / kRowsPerWarp);
    const long long blocks = a.n_units + q_blocks;
    if (blocks > 0x7fffffffLL || a.num_new * chunks > 0x7fffff00LL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)blocks), block(U * 8);
    return a.tok_n > 0 ? launch_pdl(append_kernel<F8, SC, true, U>, grid, block, 0, stream, a)
                       : launch_pdl(append_kernel<F8, SC, false, U>, grid, block, 0, stream, a);
}

cudaError_t launch_append(const AppendArgs &args, cudaStream_t stream) {
    AppendArgs a = args;
    uint32_t b;
    memcpy(&b, &a.kv_scale, 4);
    int e;
    a.kv_scale_inv = std::frexp(a.kv_scale, &e) == 0.5f && b >= 0x00800000u && b < 0x7f000000u ? 1.f / a.kv_scale : 0.f;
    if (a.dtype == DCP_KV_BF16) return launch_unit<false, false, 16>(a, stream);
    if (a.scale_block == 0) return launch_unit<true, false, 16>(a, stream);
    // as small as the scale block allows: 16-row units overlap their loads, arithmetic and stores with
    // those of others on the SM (69K tokens, blocks of 16: 26.5 us against 31 us in units of 64 rows)
    if (a.scale_block <= 16) return launch_unit<true, true, 16>(a, stream);
    if (a.scale_block == 32) return launch_unit<true, true, 32>(a, stream);
    return launch_unit<true, true, 64>(a, stream);
}

}  // namespace dcp
