// dcp_prefill.cu -- expanded latent attention over packed prompts.
//
// The prompt form of the latent attention the decode side runs absorbed ("Serving Macaron-V1 at
// Scale: Page-Level 2D KV Resharding", 5.3: 512 latent + 64 rope dims; per head 128 + 64 key dims
// and 128 value dims).  For head h of request b, query i and key j:
//     s_ij = softmax_scale * (q_i[0:128] . k_nope_j,h + q_i[128:192] . k_rope_j)
//     O_i = sum_j exp(s_ij - LSE_i) v_j,h,   LSE_i = ln sum_j exp(s_ij)
// over the keys j <= n_k - n_q + i (causal: the queries are the request's last tokens) or all keys.
// A row that sees no key gives O = 0, LSE = -inf, one with a NaN or +inf score NaN.  k_rope is one row per token, shared by the heads,
// and is read in place: no concatenated key is made.
//
// Design (GB300 / sm_103a).  Bound: the tensor cores (640 flops per key and query).  Measured: 8192
// rows x 64 heads, causal, 753 us = 1.82 PFLOP/s, 95% of cuBLAS's BF16 rate, at burst clocks, 820 to
// 860 us under the power cap; eight packed prompts of 1 to 2048 rows x 64 heads 143 us = 1.18 PFLOP/s,
// 154 to 159 us capped; 256 rows over 33,024 keys x 16 heads 73 us = 1.18 PFLOP/s and 3.8 TB/s.
//  * A work unit is 256 query rows (two tiles of 128) of one request and head.  Per 128-key tile
//    tcgen05 computes S_t = Q_t K^T (12 MMAs of 128 x 128 x 16) into TMEM, one softmax warpgroup per
//    tile turns its S into P, and tcgen05 adds P_t V (8 MMAs, P read from TMEM) to O_t.  The two
//    tiles alternate on the tensor cores: P_0 V, S_0 of the next keys, P_1 V, S_1 of the next keys;
//    while one tile's products run the other tile's softmax does.  TMEM: S_0 S_1 O_0 O_1, 128 columns
//    each, P over its S.
//  * Thread = query row (TMEM lane): row maxima and sums need no shuffles.  A lazy maximum: the
//    reference moves, and O is rescaled, only when a row's maximum passes it by more than 2^8.
//    Statistics and O are fp32; P is rounded to BF16 (at most 2^-8 of itself, as the inputs were).
//  * Q (96 KB) stays for the unit; K and V tiles go through a ring of eight 16 KB blocks (K: two
//    blocks of 64 nope dims, one of rope dims; V: two of 64 dims) filled by TMA, so K of the next
//    tile and more is in flight while V of this one is used.
//  * Units are taken by resident CTAs (one per SM) through cluster launch control, groups of heads
//    outermost (their K and V are in L2 at a time) and a request's last rows, its longest units,
//    first.  No work counter, no host copy of the offsets: request b's units start at slot
//    floor(q_ptr[b] / 256) + b, found by a 32-way search.
//  * Few rows over long keys: the keys are split into `splits` ranges whose partials a second kernel
//    merges (exact, ascending).
//  * V rows behind a request's last key are cleared in shared memory before P*V reads them (they
//    belong to the next request, or to nobody, and 0 x NaN is NaN).
//  * Every mbarrier wait is bounded; on timeout the CTA stops, drains its in-flight copies and MMAs,
//    frees TMEM and reports DCP_DEVERR_TIMEOUT.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "dcp_internal.h"
#include "dcp_merge_row.cuh"
#include "dcp_ptx.cuh"
#include "dcp_search.cuh"

namespace dcp {
namespace {

constexpr int kTile = 128;                    // query rows of a tile, keys of a step
constexpr int kUnitRows = 2 * kTile;
static_assert(kUnitRows == 1 << 8, "decode_unit shifts by 8");
constexpr int kQkDim = 192, kNope = 128, kRopeDim = 64, kV = 128;
constexpr uint32_t kBlock = 16384;            // 128 rows x 64 dims BF16, 128-byte swizzle
constexpr int kSlots = 8;
constexpr uint32_t kQTile = 3 * kBlock;
constexpr uint32_t kOffRing = 2 * kQTile;
constexpr uint32_t kOffCtl = kOffRing + kSlots * kBlock;
constexpr int kThreads = 512;                 // warps 0-3, 4-7 softmax of tiles 0, 1; 8-11 outputs; 12 loads; 13 MMAs
constexpr int kLoadWarp = 12, kMmaWarp = 13;
constexpr int kCached = 64;                   // requests whose offsets are kept in shared memory
constexpr int kConsumers = 13;                // arrivals that free a unit record: 8 softmax, 4 output warps, MMA
constexpr uint32_t kSCol = 0, kOCol = 256;    // TMEM columns of S_t (+ 128 t) and O_t
constexpr float kTau = 8.f;                   // margin of the lazy maximum (log2)
constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, 0, 1);

struct Unit {
    int valid, head, split;
    int rows;                 // 1 .. 256
    int n_k;                  // keys of the request
    int tile0;                // first key tile of this split
    int nt[2];                // key tiles of each query tile
    int lim0;                 // keys row 0 sees (causal: + 1 per row), may be <= 0
    int k_row;                // first key row of the request
    int q_row;                // first query row of the unit
};

struct __align__(16) Ctl {
    uint4 answer;
    uint64_t answer_bar;
    uint64_t full[kSlots], empty[kSlots], vland;
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2], p_full2[2], o_full[2], o_free[2];  // p_full2: P of keys 64-127
    uint64_t stat_full[2], stat_free[2];
    uint64_t unit_full[2], unit_empty[2];
    uint64_t drain;
    Unit unit[2];
    uint32_t tmem_base;
    int abort_flag;
    float2 stat[2][kTile];  // per row of a finished tile: the reference maximum and the sum of the weights
    int q_off[kCached + 1], k_off[kCached + 1];  // the offsets, where there are few enough
};
constexpr size_t kSmem = kOffCtl + sizeof(Ctl);
static_assert(kSmem <= 232448, "shared memory budget");

struct Maps {
    CUtensorMap q, kn, kr, v;
};

struct Params {
    const int64_t *q_ptr, *k_ptr;
    int B, H, slots, splits, causal;
    int group;                // heads taken together
    long long n_q, n_k;
    float c2;                 // softmax_scale * log2(e)
    void *out;
    int out_bf16;
    float *lse, *part_o, *part_lse;
    int32_t *dev_error;
    unsigned long long wait_limit_ns;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A warp's bounded wait, short because it stands at many places: false after `lim` ns, or when another
// role gave up.  (The role that sees false leaves its loops and calls give_up.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t lim) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t t0 = global_timer_ns();
#pragma unroll 1
        do ok = mbar_try_wait(bar, parity);
        while (!ok && !*abort && global_timer_ns() - t0 < lim);
    }
    return __all_sync(0xffffffffu, ok) != 0;
}

__device__ __forceinline__ void give_up(volatile int *abort, int32_t *err) {
    *abort = 1;
    if (err) atomicOr(err, DCP_DEVERR_TIMEOUT);
}

// Four 16-byte chunks per lane: afterwards lane q of four holds chunk q of each of the four lanes' rows
// (position i: lane i's).
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[16], int lane) {
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1) {
        const bool up = (lane & bit) != 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c & bit) continue;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t &lo = w[4 * c + x], &hi = w[4 * (c | bit) + x];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
                lo = up ? got : lo;
                hi = up ? hi : got;
            }
        }
    }
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

struct Cta {  // a unit: grid (slots x heads of a group, groups, splits)
    uint32_t x, y, z;
};

__device__ __forceinline__ bool offsets_fit(const Params &p, long long q0, long long q1, long long k0, long long k1) {
    return q0 >= 0 && q0 <= q1 && q1 <= p.n_q && k0 >= 0 && k0 <= k1 && k1 <= p.n_k;
}

// Offsets that do not fit may lead to no slot at all: the slots of head 0 report them, 32 requests each
// (there are as many slots as requests, and more).  Called when a unit's loads are on their way.
__device__ __noinline__ void report_offsets(const Params &p, Cta c, int lane) {
    const uint32_t turn = c.x / (uint32_t)p.group;
    const long long i = (long long)turn * 32 + lane;
    if (c.x == turn * p.group && i < p.B && !offsets_fit(p, p.q_ptr[i], p.q_ptr[i + 1], p.k_ptr[i], p.k_ptr[i + 1]))
        atomicOr(p.dev_error, DCP_DEVERR_OUT_OF_RANGE);
}

// A unit's rows and key tiles; false: the slot holds no rows.  (Warp-uniform.)
template <typename T>
__device__ __forceinline__ bool decode_unit(const Params &p, const T *q_ptr, const T *k_ptr, Cta c, int lane, Unit &u) {
    u.split = (int)c.z;
    const int turn = (int)(c.x / (uint32_t)p.group);
    u.head = (int)c.y * p.group + (int)c.x - turn * p.group;
    if (u.head >= p.H) return false;
    const int slot = p.slots - 1 - turn;  // last rows first
    const int b = warp_search(p.B, slot, lane, [&](int i) { return (long long)(q_ptr[i] >> 8) + i; });
    if (b < 0) return false;
    const long long q0 = q_ptr[b], q1 = q_ptr[b + 1], k0 = k_ptr[b], k1 = k_ptr[b + 1];
    const long long r0 = (slot - ((q0 >> 8) + b)) * kUnitRows;
    if (!offsets_fit(p, q0, q1, k0, k1)) return false;
    const int nq = (int)(q1 - q0), nk = (int)(k1 - k0);
    if (r0 >= nq) return false;
    u.valid = 1;
    u.rows = min(kUnitRows, nq - (int)r0);
    u.n_k = nk;
    u.lim0 = p.causal ? nk - nq + (int)r0 + 1 : nk;
    u.k_row = (int)k0;
    u.q_row = (int)(q0 + r0);
    int tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int rows = min(kTile, u.rows - kTile * t);
        int keys = p.causal ? min(nk, u.lim0 + kTile * t + rows - 1) : nk;
        if (rows <= 0) keys = 0;
        tiles[t] = keys > 0 ? (keys + kTile - 1) / kTile : 0;
    }
    const int all = max(tiles[0], tiles[1]);
    u.tile0 = 0;
    int end = all;
    if (p.splits > 1) {  // (at most 2^23 tiles, 64 splits)
        u.tile0 = (int)((uint32_t)all * (uint32_t)u.split / (uint32_t)p.splits);
        end = (int)((uint32_t)all * (uint32_t)(u.split + 1) / (uint32_t)p.splits);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) u.nt[t] = max(0, min(end, tiles[t]) - u.tile0);
    return true;
}

__global__ void __launch_bounds__(kThreads, 1)
prefill_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem[];
    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled blocks need 1024-byte alignment (uniform)
        if (threadIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, DCP_DEVERR_LAYOUT);
        return;
    }
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + kOffCtl);
    // (the shuffle tells the compiler that a warp has one role)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    volatile int *abort_flag = &ctl->abort_flag;
    const uint64_t lim = p.wait_limit_ns;
    if (threadIdx.x == 0) {
        mbar_init(&ctl->answer_bar, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        mbar_init(&ctl->vland, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&ctl->q_full[t], 1);
            mbar_init(&ctl->q_empty[t], 1);
            mbar_init(&ctl->s_full[t], 1);
            mbar_init(&ctl->p_full[t], 4);
            mbar_init(&ctl->p_full2[t], 4);
            mbar_init(&ctl->o_full[t], 1);
            mbar_init(&ctl->o_free[t], 4);
            mbar_init(&ctl->stat_full[t], 4);
            mbar_init(&ctl->stat_free[t], 4);
            mbar_init(&ctl->unit_full[t], 1);
            mbar_init(&ctl->unit_empty[t], kConsumers);
        }
        mbar_init(&ctl->drain, 1);
        ctl->abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_dep_wait();
    grid_dep_launch();
    // All 512 columns are this CTA's, so they start at column 0 (checked): constant addresses.
    constexpr uint32_t tmem = 0;
    if (ctl->tmem_base != 0) {
        if (threadIdx.x == 0 && p.dev_error) atomicOr(p.dev_error, DCP_DEVERR_LAYOUT);
        ctl->abort_flag = 1;
    }

    if (warp < 8) {
        // ----------------------------------------------------------------------- softmax
        const int t = warp >> 2;
        const int row = (warp & 3) * 32 + lane;  // of the tile = TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lanes + kSCol + 128 * t, o_tmem = tmem + lanes + kOCol + 128 * t;
        uint32_t k = 0, s_cnt = 0, st_cnt = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return warp_wait(bar, parity, abort_flag, lim);
        };
        const float c2 = p.c2, tau = fminf(kTau / p.c2, 3e38f);
        bool ok = true;
        while (ok) {
            const int e = k & 1;
            ok = wait(&ctl->unit_full[e], (k >> 1) & 1);
            if (!ok) break;
            const Unit *rec = &ctl->unit[e];
            const int valid = rec->valid, rows = rec->rows - kTile * t, nt = rec->nt[t];
            // keys of this split's range that the row sees
            const int seen = min(rec->n_k, p.causal ? rec->lim0 + kTile * t + row : rec->lim0) - kTile * rec->tile0;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->unit_empty[e]);
            ++k;
            if (!valid) break;
            if (rows <= 0) continue;
            float m = -INFINITY;
            uint64_t sum2 = pack_f32x2(0.f, 0.f);
            for (int j = 0; j < nt; ++j) {
                ok = wait(&ctl->s_full[t], s_cnt & 1);
                if (!ok) break;
                ++s_cnt;
                tc_fence_after();
                // S is read twice, 64 columns at a time in rolled loops: the row's maximum, then the weights
                // (the whole row in registers needs twice the code, which the warps' roles cannot keep in
                // the instruction cache).
                const int n = seen - kTile * j;
                float top = -INFINITY;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    float s[2][32];
                    tmem_ld32(s_tmem + 64 * half, s[0]);
                    tmem_ld32(s_tmem + 64 * half + 32, s[1]);
                    tmem_wait_ld();
                    const int c = n - 64 * half;  // columns of this half that the row sees
                    if (__any_sync(0xffffffffu, c < 64)) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
#pragma unroll
                            for (int x = 0; x < 32; ++x) s[i][x] = 32 * i + x < c ? s[i][x] : -INFINITY;
                            tmem_st32(s_tmem + 64 * half + 32 * i, s[i]);  // for the second reading
                        }
                    }
                    float mx[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
#pragma unroll
                    for (int x = 2; x < 32; x += 2) {
                        mx[0] = fmaxf(mx[0], s[0][x]);
                        mx[1] = fmaxf(mx[1], s[0][x + 1]);
                        mx[2] = fmaxf(mx[2], s[1][x]);
                        mx[3] = fmaxf(mx[3], s[1][x + 1]);
                    }
                    top = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                }
                tmem_wait_st();
                const bool up = top > m + tau;
                if (__any_sync(0xffffffffu, up)) {
                    const float corr = up ? exp2_approx((m - top) * c2) : 1.f;
                    m = up ? top : m;
                    if (j > 0) {  // P*V of the previous keys is complete: S was issued after it
                        sum2 = mul_f32x2(sum2, pack_f32x2(corr, corr));
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            float o[32];
                            tmem_ld32(o_tmem + 32 * i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x) o[x] *= corr;
                            tmem_st32(o_tmem + 32 * i, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : -__fmul_rn(m, c2);
                const uint64_t ref2 = pack_f32x2(ref, ref), c22 = pack_f32x2(c2, c2);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    float s[2][32];
                    tmem_ld32(s_tmem + 64 * half, s[0]);
                    tmem_ld32(s_tmem + 64 * half + 32, s[1]);
                    tmem_wait_ld();
                    uint32_t w[32];
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        float a, b;
                        unpack_f32x2(fma_f32x2(pack_f32x2(s[x / 16][2 * (x % 16)], s[x / 16][2 * (x % 16) + 1]), c22, ref2), a, b);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        sum2 = add_f32x2(sum2, pack_f32x2(a, b));
                        w[x] = bf16x2(a, b);
                    }
                    tmem_st32_u(s_tmem + 32 * half, w);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    // P*V begins on the first 64 keys while the weights of the others are computed
                    if (lane == 0) mbar_arrive(half == 0 ? &ctl->p_full[t] : &ctl->p_full2[t]);
                }
            }
            if (!ok) break;
            float la, lb;
            unpack_f32x2(sum2, la, lb);
            ok = wait(&ctl->stat_free[t], (st_cnt & 1) ^ 1);
            if (!ok) break;
            ++st_cnt;
            ctl->stat[t][row] = make_float2(m, la + lb);
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->stat_full[t]);
        }
        if (!ok && lane == 0) give_up(abort_flag, p.dev_error);
    } else {
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------------------- loads
            if (lane == 0) {
                prefetch_tmap(&maps.q);
                prefetch_tmap(&maps.kn);
                prefetch_tmap(&maps.kr);
                prefetch_tmap(&maps.v);
            }
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return warp_wait(bar, parity, abort_flag, lim);
            };
            // Offsets of few requests are read once (each unit's decoding asks for them twice in a row).
            const bool cached = p.B <= kCached;
            for (int i = lane; cached && i <= p.B; i += 32) {
                // (offsets that fit no tensor become -1, which fits no tensor either)
                const long long a = p.q_ptr[i], b = p.k_ptr[i];
                ctl->q_off[i] = a < 0 || a > p.n_q ? -1 : (int)a;
                ctl->k_off[i] = b < 0 || b > p.n_k ? -1 : (int)b;
            }
            __syncwarp();
            uint32_t slot = 0, phase = 0;   // ring slot, bit per slot: uses so far mod 2
            uint32_t fphase = 0;            // bit per slot: loads that landed on its full barrier mod 2
            uint64_t *last_bar = nullptr;   // the barrier of the latest group of loads
            bool open = false;              // that group is not wholly issued
            uint32_t q_used = 0, qphase = 0;  // bit per query tile: ever loaded, loads mod 2
            uint32_t k = 0, land_cnt = 0, tries = 0;
            bool ok = true, land_pending = false, have = true;
            Cta idx = {blockIdx.x, blockIdx.y, blockIdx.z};
            while (ok && have) {
                // The next unit is asked for when the loads of this one's last tiles begin: early enough to
                // hide the answer's latency, late enough not to hold a unit while other SMs run dry.
                bool asked = false;
                auto ask = [&]() {
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&ctl->answer_bar, 16);
                        try_cancel(&ctl->answer, &ctl->answer_bar);
                    }
                    ++tries;
                    asked = true;
                };
                Unit u;
                if (cached ? decode_unit(p, ctl->q_off, ctl->k_off, idx, lane, u) : decode_unit(p, p.q_ptr, p.k_ptr, idx, lane, u)) {
                    const int e = k & 1;
                    if (!wait(&ctl->unit_empty[e], ((k >> 1) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        ctl->unit[e] = u;
                        mbar_arrive(&ctl->unit_full[e]);
                    }
                    ++k;
                    const int nt = max(u.nt[0], u.nt[1]);
                    // Q of tile t as soon as the previous unit's last scores of that tile are done
                    auto load_q = [&](int t) -> bool {
                        if (u.nt[t] == 0) return true;
                        if (!wait(&ctl->q_empty[t], ((qphase >> t) & 1) ^ 1)) return false;
                        qphase ^= 1u << t;
                        q_used |= 1u << t;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&ctl->q_full[t], kQTile);
#pragma unroll 1
                            for (int kb = 0; kb < 3; ++kb)
                                tma_load_3d(smem + t * kQTile + kb * kBlock, &maps.q, &ctl->q_full[t], kb * 64, u.head,
                                            u.q_row + kTile * t);
                        }
                        return true;
                    };
                    if (!load_q(0)) {
                        ok = false;
                        break;
                    }
#pragma unroll 1
                    for (int j = 0; j < nt && ok; ++j) {
                        if (!asked && j + 2 >= nt) ask();
                        const int key = kTile * (u.tile0 + j);
                        const int row = u.k_row + key;
                        const bool tail = u.n_k - key < kTile;
#pragma unroll 1
                        for (int grp = 0; grp < 2 && ok; ++grp) {  // K's three blocks, V's two
                            if (j == 0 && grp == 1 && !load_q(1)) {
                                ok = false;
                                break;
                            }
                            const uint32_t first = slot;
                            const int blocks = grp == 0 ? 3 : 2;
                            const bool via = tail && grp == 1;
                            // V's dims 64-127 lie behind dims 0-63: where its two blocks wrap around the
                            // ring (slots 7, 0) they are swapped, seven slots apart instead of one
                            const int swap = slot == kSlots - 1 ? 1 : 0;
                            uint64_t *bar = via ? &ctl->vland : &ctl->full[first];
#pragma unroll 1
                            for (int blk = 0; blk < blocks; ++blk) {
                                if (!wait(&ctl->empty[slot], ((phase >> slot) & 1) ^ 1)) {
                                    ok = false;
                                    break;
                                }
                                phase ^= 1u << slot;
                                open = blk + 1 < blocks;  // bytes are expected, the arrival is to come
                                if (blk == 0) {
                                    last_bar = bar;
                                    if (via) land_pending = true;
                                    else fphase ^= 1u << first;
                                }
                                if (lane == 0) {
                                    uint8_t *dst = smem + kOffRing + slot * kBlock;
                                    if (open) mbar_expect_tx(bar, kBlock);
                                    else mbar_arrive_expect_tx(bar, kBlock);
                                    if (grp == 1) tma_load_3d(dst, &maps.v, bar, 64 * (blk ^ swap), u.head, row);
                                    else if (blk < 2) tma_load_3d(dst, &maps.kn, bar, 64 * blk, u.head, row);
                                    else tma_load_2d(dst, &maps.kr, bar, 0, row);
                                }
                                slot = (slot + 1) % kSlots;
                            }
                            if (!ok || !via) continue;
                            ok = wait(&ctl->vland, land_cnt & 1);
                            if (!ok) continue;
                            ++land_cnt;
                            land_pending = false;
                            // 128-byte rows of a block are contiguous whatever the swizzle
#pragma unroll 1
                            for (int blk = 0; blk < 2; ++blk) {
                                uint4 *v = reinterpret_cast<uint4 *>(smem + kOffRing + (first + blk) % kSlots * kBlock);
#pragma unroll 1
                                for (int i = 8 * (u.n_k - key) + lane; i < kTile * 8; i += 32) v[i] = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&ctl->full[first]);
                            fphase ^= 1u << first;
                        }
                    }
                    if (!ok) break;
                }
                if (!asked) ask();
                if (p.dev_error && (idx.y | idx.z) == 0) report_offsets(p, idx, lane);
                if (!wait(&ctl->answer_bar, (tries - 1) & 1)) {
                    ok = false;
                    break;
                }
                have = cancelled_cta(&ctl->answer, idx.x, idx.y, idx.z);
                fence_proxy_async_smem();  // the answer is read before the next one is written
                __syncwarp();
            }
            if (ok) {  // the end of the work
                const int e = k & 1;
                ok = wait(&ctl->unit_empty[e], ((k >> 1) & 1) ^ 1);
                if (ok && lane == 0) {
                    ctl->unit[e].valid = 0;
                    mbar_arrive(&ctl->unit_full[e]);
                }
                if (!ok && lane == 0) give_up(abort_flag, p.dev_error);
            } else {  // let issued copies and a pending answer land before the CTA can exit (bounded)
                if (lane == 0) give_up(abort_flag, p.dev_error);
                int never = 0;
                const uint64_t lim = p.wait_limit_ns > 100000000ull ? p.wait_limit_ns : 100000000ull;
                if (open && last_bar && lane == 0) mbar_arrive(last_bar);  // (its issued part can complete)
                __syncwarp();
                // (a barrier no load has used has completed the phase before its first: no wait)
#pragma unroll 1
                for (uint32_t s = 0; s < (uint32_t)kSlots; ++s) mbar_wait(&ctl->full[s], ((fphase >> s) & 1) ^ 1, &never, nullptr, lim);
                if (land_pending) mbar_wait(&ctl->vland, land_cnt & 1, &never, nullptr, lim);
                for (int t = 0; t < 2; ++t)
                    if ((q_used >> t) & 1u) mbar_wait(&ctl->q_full[t], ((qphase >> t) & 1) ^ 1, &never, nullptr, lim);
                if (tries > 0) mbar_wait(&ctl->answer_bar, (tries - 1) & 1, &never, nullptr, lim);
            }
        } else if (warp == kMmaWarp) {
            // -------------------------------------------------------------------------- MMAs
            // The whole warp runs in step and one elected lane issues: under a lane's branch the issue
            // of 20 MMAs took 1800 cycles, more than the 1280 they run.
            // low words of the operands' descriptors: the address / 16 and the leading offset / 16
            const uint32_t v_lo = (smem_u32(smem) + kOffRing) >> 4, ring_lo = v_lo + (1u << 16);
            const uint32_t q_lo = (smem_u32(smem) >> 4) + (1u << 16);
            constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (kSwizzle128 << 29);
            const uint32_t go = warp_elect();
            uint32_t slot = 0, phase = 0, k = 0;
            uint32_t p_cnt[2] = {0, 0}, of_cnt[2] = {0, 0}, q_cnt[2] = {0, 0};
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return warp_wait(bar, parity, abort_flag, lim);
            };
            // The next three ring blocks (K of a tile) or two (V), loaded: they land on the first one's
            // barrier (a wait costs about 70 cycles even when it is over).
            uint32_t ks[3], vs[2];
            auto take_k = [&]() -> bool {
                ks[0] = slot;
                if (!wait(&ctl->full[ks[0]], (phase >> ks[0]) & 1)) return false;
                ks[1] = (slot + 1) % kSlots;
                ks[2] = (slot + 2) % kSlots;
                phase ^= 1u << ks[0];
                slot = (slot + 3) % kSlots;
                return true;
            };
            auto take_v = [&]() -> bool {
                vs[0] = slot;
                if (!wait(&ctl->full[vs[0]], (phase >> vs[0]) & 1)) return false;
                vs[1] = (slot + 1) % kSlots;
                phase ^= 1u << vs[0];
                slot = (slot + 2) % kSlots;
                return true;
            };
            auto scores = [&](int t, bool last, bool end) {  // end: the unit's last scores of tile t
#pragma unroll
                for (int kb = 0; kb < 3; ++kb) {
                    mma_f16_ss_x4(go, tmem + kSCol + 128 * t, q_lo + (t * kQTile + kb * kBlock) / 16,
                                  ring_lo + ks[kb] * (kBlock / 16), kDescHi, kIdescQK, kb != 0);
                    if (last) mma_commit_if(go, &ctl->empty[ks[kb]]);
                }
                mma_commit_if(go, &ctl->s_full[t]);
                if (end) mma_commit_if(go, &ctl->q_empty[t]);
            };
            // Step j of a unit: P_t V of its key tile j and the scores of key tile j + 1, tile 0 then tile 1.
            // The last step takes the first scores of the next unit in their place, so that they run while
            // the tile with more keys (tile 1 of a causal unit) is still in its last softmax.
            int c[2] = {0, 0}, nx[2] = {0, 0};  // key tiles of this unit and of the next
            int j = -1;
            bool have = false, done = false;    // the next unit is known; there is none
            auto fetch = [&](bool block) -> bool {
                while (!have && !done) {
                    const int e = k & 1;
                    if (block) {
                        if (!wait(&ctl->unit_full[e], (k >> 1) & 1)) return false;
                    } else if (!__all_sync(0xffffffffu, mbar_try_wait(&ctl->unit_full[e], (k >> 1) & 1))) {
                        return true;
                    }
                    done = __shfl_sync(0xffffffffu, ctl->unit[e].valid, 0) == 0;
                    nx[0] = __shfl_sync(0xffffffffu, ctl->unit[e].nt[0], 0);
                    nx[1] = __shfl_sync(0xffffffffu, ctl->unit[e].nt[1], 0);
                    __syncwarp();
                    if (go) mbar_arrive(&ctl->unit_empty[e]);
                    ++k;
                    have = !done && (nx[0] > 0 || nx[1] > 0);  // (a unit without keys has no products)
                }
                return true;
            };
#pragma unroll 1
            while (ok) {
                const int n = max(c[0], c[1]);
                const bool end = j == n - 1;
                if (j >= 0) ok = take_v();
                bool k_here = false, first0 = false;  // K of these scores is here; tile 0's of the next unit are issued
                auto first_scores = [&](int t) -> bool {  // of the next unit
                    if (!k_here && !take_k()) return false;
                    k_here = true;
                    if (!wait(&ctl->q_full[t], q_cnt[t] & 1)) return false;
                    ++q_cnt[t];
                    tc_fence_after();
                    return true;
                };
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (ok && j >= 0 && j < c[t]) {
                        if (j == 0) {  // O of the previous unit is read
                            ok = wait(&ctl->o_free[t], (of_cnt[t] & 1) ^ 1);
                            ++of_cnt[t];
                        }
                        // dims 64-127 lie one slot on, or (swapped, slots 7 and 0) seven: the leading offset
                        const uint32_t v = vs[0] < vs[1] ? v_lo + vs[0] * (kBlock / 16) + ((kBlock / 16) << 16)
                                                         : v_lo + (((kSlots - 1) * kBlock / 16) << 16);
                        ok = ok && wait(&ctl->p_full[t], p_cnt[t] & 1);
                        if (!ok) continue;
                        tc_fence_after();
                        mma_f16_ts_x4(go, tmem + kOCol + 128 * t, tmem + kSCol + 128 * t, v, kDescHi, kIdescPV, j != 0);
                        ok = wait(&ctl->p_full2[t], p_cnt[t] & 1);  // the second half of P
                        ++p_cnt[t];
                        if (!ok) continue;
                        tc_fence_after();
                        mma_f16_ts_x4(go, tmem + kOCol + 128 * t, tmem + kSCol + 128 * t + 32, v + 512, kDescHi, kIdescPV, 1);
                        if (t == 1 || j >= c[1]) {  // last reader of V
                            mma_commit_if(go, &ctl->empty[vs[0]]);
                            mma_commit_if(go, &ctl->empty[vs[1]]);
                        }
                        if (j == c[t] - 1) mma_commit_if(go, &ctl->o_full[t]);
                    }
                    bool issue = !end && j + 1 < c[t];
                    if (ok && end) {
                        ok = fetch(t == 1);  // (before tile 1's P only if it is there already)
                        if (ok && t == 1 && have && nx[0] > 0 && !first0) {
                            ok = first_scores(0);
                            if (ok) scores(0, nx[1] == 0, nx[0] == 1);
                        }
                        issue = have && nx[t] > 0;
                        if (ok && issue) ok = first_scores(t);
                        if (t == 0) first0 = ok && issue;
                    } else if (ok && issue && !k_here) {
                        ok = take_k();
                        k_here = true;
                        tc_fence_after();
                    }
                    if (ok && issue)
                        scores(t, t == 1 || (end ? nx[1] == 0 : j + 1 >= c[1]), (end ? nx[t] == 1 : j + 2 == c[t]));
                }
                if (!end) {
                    ++j;
                } else {
                    if (!have) break;
                    c[0] = nx[0];
                    c[1] = nx[1];
                    have = false;
                    j = 0;
                }
            }
            __syncwarp();
            if (!ok && lane == 0) give_up(abort_flag, p.dev_error);
            mma_commit_if(go, &ctl->drain);
            int never = 0;
            mbar_wait(&ctl->drain, 0, &never, nullptr, 100000000ull);
            __syncwarp();
        } else if (warp < kLoadWarp) {
            // ----------------------------------------------------------------------- outputs
            // O of a finished tile, scaled and stored, while its softmax warps go on with the next unit.
            const int quad = warp & 3, row = quad * 32 + lane;
            const uint32_t lanes = (uint32_t)(quad * 32) << 16;
            uint32_t k = 0, s_phase = 0, o_phase = 0;
            const bool part = p.splits > 1, wide = part || !p.out_bf16;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                return warp_wait(bar, parity, abort_flag, lim);
            };
            while (ok) {
                const int e = k & 1;
                ok = wait(&ctl->unit_full[e], (k >> 1) & 1);
                if (!ok) break;
                const Unit *rec = &ctl->unit[e];
                const int valid = rec->valid, all_rows = rec->rows, nt0 = rec->nt[0], nt1 = rec->nt[1];
                const long long q_row = rec->q_row;
                const int head = rec->head, split = rec->split;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->unit_empty[e]);
                ++k;
                if (!valid) break;
#pragma unroll 1
                for (int t = 0; t < 2 && all_rows > kTile * t; ++t) {
                    const int rows = all_rows - kTile * t, nt = t == 0 ? nt0 : nt1;
                    const uint32_t o_tmem = tmem + lanes + kOCol + 128 * t;
                    ok = wait(&ctl->stat_full[t], (s_phase >> t) & 1);
                    if (!ok) break;
                    s_phase ^= 1u << t;
                    const float2 ml = ctl->stat[t][row];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->stat_free[t]);
                    const bool live = ml.y != 0.f;  // (a NaN sum is no empty row)
                    const float inv = live ? 1.f / ml.y : 0.f;
                    const long long at = (q_row + kTile * t + row) * p.H + head;
                    const long long prow = (long long)split * p.n_q * p.H + at;
                    if (row < rows)
                        (part ? p.part_lse + prow : p.lse + at)[0] =
                            live ? (__fmul_rn(ml.x, p.c2) + log2f(ml.y)) * 0.69314718055994531f : -INFINITY;
                    if (nt > 0) {
                        ok = wait(&ctl->o_full[t], (o_phase >> t) & 1);
                        if (!ok) break;
                        o_phase ^= 1u << t;
                        tc_fence_after();
                    }
                    // 16 words of a row at a time (16 columns FP32, 32 BF16): each four lanes exchange theirs,
                    // so that a store writes 64 contiguous bytes of 8 rows, not 16 bytes of 32.  (An empty
                    // partial's zeros are not read back.)
                    const int row4 = row & ~3;
                    const long long row_bytes = wide ? 4 * kV : 2 * kV, stride = (long long)p.H * row_bytes;
                    uint8_t *dst = (part ? reinterpret_cast<uint8_t *>(p.part_o) + prow * row_bytes
                                         : static_cast<uint8_t *>(p.out) + at * row_bytes) -
                                   (row - row4) * stride + 16 * (lane & 3);
                    const uint32_t keep = live ? 0xffffffffu : 0u;  // (an empty row's O may hold anything)
#pragma unroll 1
                    for (int g = 0; g < (wide ? 8 : 4); ++g) {
                        uint32_t w[16];
                        if (nt == 0) {
#pragma unroll
                            for (int x = 0; x < 16; ++x) w[x] = 0;
                        } else if (wide) {
                            float o[16];
                            tmem_ld16(o_tmem + 16 * g, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * inv) & keep;
                        } else {
                            float o[32];
                            tmem_ld32(o_tmem + 32 * g, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) w[x] = bf16x2(o[2 * x] * inv, o[2 * x + 1] * inv) & keep;
                        }
                        quad_transpose(w, lane);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row4 + i < rows)
                                *reinterpret_cast<uint4 *>(dst + stride * i + 64 * g) =
                                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                        __syncwarp();
                    }
                    if (nt > 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl->o_free[t]);
                    }
                }
            }
            if (!ok && lane == 0) give_up(abort_flag, p.dev_error);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// The splits' partials, merged in ascending order: one warp per row, a float4 per lane.
__global__ void __launch_bounds__(256) prefill_merge_kernel(int splits, long long rows, const float *__restrict__ part_o,
                                                            const float *__restrict__ part_lse, void *out, int out_bf16,
                                                            float *lse, const int64_t *__restrict__ q_ptr, int B, int H) {
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    // rows of no request keep what they hold (and have no partials)
    if (row >= rows || row / H < (long long)__ldg(q_ptr) || row / H >= (long long)__ldg(q_ptr + B)) return;
    float mx = -INFINITY;
    for (int i = lane; i < splits; i += 32) mx = max_or_nan(mx, __ldg(part_lse + i * rows + row));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = max_or_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (mx != -INFINITY) {
        for (int i = 0; i < splits; ++i) {
            const float l = __ldg(part_lse + i * rows + row);
            if (l == -INFINITY) continue;
            const float w = expf(l - mx);
            const float4 x = __ldg(reinterpret_cast<const float4 *>(part_o) + (i * rows + row) * (kV / 4) + lane);
            sum += w;
            acc.x = fmaf(w, x.x, acc.x);
            acc.y = fmaf(w, x.y, acc.y);
            acc.z = fmaf(w, x.z, acc.z);
            acc.w = fmaf(w, x.w, acc.w);
        }
    }
    const float inv = mx != -INFINITY ? 1.f / sum : 0.f;  // (sum >= 1, or NaN)
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (out_bf16) static_cast<uint2 *>(out)[row * (kV / 4) + lane] = make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
    else static_cast<float4 *>(out)[row * (kV / 4) + lane] = acc;
    if (lane == 0) lse[row] = mx != -INFINITY ? mx + logf(sum) : -INFINITY;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// [rows][heads][width] BF16 with given strides (elements), boxes of 128 rows x 1 head x 64 dims;
// heads == 0: [rows][width].
bool map3(CUtensorMap *m, const void *ptr, int64_t rows, int heads, int width, int64_t row_stride, int64_t head_stride) {
    const EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!enc) return false;
    const bool two = heads == 0;
    const cuuint64_t tok = (cuuint64_t)row_stride * 2, head = (cuuint64_t)head_stride * 2;
    const cuuint64_t dims[3] = {(cuuint64_t)width, two ? (cuuint64_t)rows : (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {two ? tok : head, tok};
    const cuuint32_t box[3] = {64, two ? (cuuint32_t)kTile : 1u, (cuuint32_t)kTile};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, two ? 2 : 3, const_cast<void *>(ptr), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Ranges of keys per unit: enough for every SM to have a unit, each of at least four key tiles (a
// range costs a partial's round trip and a restart).  The host knows only the totals: requests are
// taken as equally long.
int prefill_splits(int num_requests, int64_t n_q, int64_t n_k, int num_heads, int num_sms) {
    if (num_requests < 1 || n_q < 1 || n_k < 1 || num_heads < 1) return 1;
    const int64_t per = (n_q + num_requests - 1) / num_requests;
    const int64_t units = (per + kUnitRows - 1) / kUnitRows * num_requests * num_heads;
    const int64_t tiles = (n_k / num_requests + kTile - 1) / kTile;
    return (int)std::max<int64_t>(1, std::min<int64_t>({num_sms / units, tiles / 4, 64}));
}

size_t prefill_workspace(int splits, int64_t n_q, int num_heads) {
    if (splits <= 1) return 0;
    const size_t rows = (size_t)splits * n_q * num_heads;
    return up256(rows * kV * sizeof(float)) + up256(rows * sizeof(float));
}

int launch_prefill(const PrefillArgs &a, int num_sms, cudaStream_t stream) {
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    // without keys the key maps are never used (every row is empty): any valid pointer will do
    const int64_t nk = std::max<int64_t>(a.n_k, 1);
    const void *kn = a.n_k ? a.k_nope : a.q, *kr = a.n_k ? a.k_rope : a.q, *v = a.n_k ? a.v : a.q;
    if (!map3(&maps.q, a.q, a.n_q, a.num_heads, kQkDim, a.q_tok, a.q_head) ||
        !map3(&maps.kn, kn, nk, a.num_heads, kNope, a.kn_tok, a.kn_head) ||
        !map3(&maps.kr, kr, nk, 0, kRopeDim, a.kr_tok, 0) || !map3(&maps.v, v, nk, a.num_heads, kV, a.v_tok, a.v_head))
        return DCP_ERR_CUDA;
    Params p;
    p.q_ptr = a.q_ptr;
    p.k_ptr = a.k_ptr;
    p.B = a.num_requests;
    p.H = a.num_heads;
    p.slots = (int)(a.n_q / kUnitRows + a.num_requests);
    p.splits = a.splits;
    p.causal = a.causal;
    p.n_q = a.n_q;
    p.n_k = a.n_k;
    p.c2 = a.softmax_scale * 1.4426950408889634f;
    p.out = a.out;
    p.out_bf16 = a.out_bf16;
    p.lse = a.lse;
    const size_t rows = (size_t)a.splits * a.n_q * a.num_heads;
    p.part_o = reinterpret_cast<float *>(a.workspace);
    p.part_lse = reinterpret_cast<float *>(a.workspace + up256(rows * kV * sizeof(float)));
    p.dev_error = a.dev_error;
    p.wait_limit_ns = a.wait_limit_ns;
    // Heads are taken in equal groups whose keys and values (512 bytes a key, of a request of average
    // length) stay in L2, all slots of a group before the next group, a slot's heads side by side:
    // longest units first within the group, so that the last group ends evenly.  Measured: 8192 x 64
    // heads 754 us with 48 MB groups, 778 with 24, 763 with 96, 800 with one group; 4096 x 32 heads 109
    // us with equal groups against 127 with a full and a small one; eight requests of 2048 x 16 heads
    // 124 us with one group against 134 with three.
    const int64_t keys = std::max<int64_t>(1, a.n_k / a.num_requests);
    const int most = (int)std::max<int64_t>(1, std::min<int64_t>(a.num_heads, (48ll << 20) / (512 * keys)));
    const int groups = (a.num_heads + most - 1) / most;
    p.group = (a.num_heads + groups - 1) / groups;
    const long long grid_x = (long long)p.slots * p.group;
    if (grid_x > 0x7fffffffLL || groups > 65535) return DCP_ERR_INVALID_ARG;
    static std::atomic<uint64_t> allowed{0};
    if (allow_smem(prefill_kernel, kSmem, allowed) != cudaSuccess) return DCP_ERR_CUDA;
    if (launch_pdl(prefill_kernel, dim3((unsigned)grid_x, groups, a.splits), dim3(kThreads), kSmem, stream, maps, p) != cudaSuccess)
        return DCP_ERR_CUDA;
    if (a.splits > 1) {
        const long long out_rows = (long long)a.n_q * a.num_heads;
        if (launch_pdl(prefill_merge_kernel, dim3((unsigned)((out_rows + 7) / 8)), dim3(256), 0, stream, a.splits, out_rows,
                       (const float *)p.part_o, (const float *)p.part_lse, a.out, a.out_bf16, a.lse, a.q_ptr,
                       a.num_requests, a.num_heads) != cudaSuccess)
            return DCP_ERR_CUDA;
    }
    return DCP_OK;
}

}  // namespace dcp
