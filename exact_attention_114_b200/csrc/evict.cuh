// evict.cuh -- eviction from a KV cache by accumulated attention weight.  Per (batch, kv head) and
// key j the weight is a_j = sum of P_ij over all query rows i of the head's group that have attended
// so far; a cache over its budget keeps its newest keys and the heaviest of the others.
//
//   key_weights_kernel     a_j += sum_i exp(scale q_i.k_j - LSE_i) for any number of rows, from the
//                          saved LSE (the recomputation of P that the backward does, without its
//                          gradients)
//   key_weights_add_kernel adds the sums of a launch whose rows were shared between CTAs
//   (the split-KV decode leaves its scores behind instead: decode_weights_kernel)
//   evict_select_kernel    the kept keys of each (batch, kv head), in order
//   evict_gather_kernel    their rows of K and V, moved to the front of a new cache
#pragma once

#include <climits>
#include <type_traits>

#include "sm100.cuh"
#include "fa_kernels.h"

namespace fa {

struct KeyWeightParams {
    const float* lse;      // [B, Hq, Nq]
    const float* w_in;     // [B, Hkv, Nk] or nullptr (zeros)
    float* w_out;          // [B, Hkv, Nk]
    float* part;           // [nsp][B * Hkv * Nk] sums of the shares (nsp > 1)
    int B, Hkv, Nq, Nk;
    int heads;             // query heads walked one after another: G, or 1 where the group's
                           // G * Nq rows are one run (row r at position r % Nq)
    int rows;              // rows of each: Nq, or G * Nq
    int causal;
    int nsp;               // CTAs that share a key block's steps
    float scale_log2;
};

// 2^x for both lanes on the FMA pipe: x = n + f, f in [-1/2, 1/2], times the degree-5 polynomial
// through 2^f at the six Chebyshev nodes cos((2 k + 1) pi / 12) / 2 (relative error 2.4e-7; the
// degree-4 one of the forward has 3.6e-6, which sums of weights in fp32 would show).  2^n is a factor
// of its own, bits (n + 127) << 23: 0 for n = -127, at which x is held (so what lies below -126.5 is 0,
// -inf too), and a NaN x stays NaN.
constexpr float kKeyExp2C0 = 1.0000001192092896f, kKeyExp2C1 = 0.69314718246459961f,
                kKeyExp2C2 = 0.24022106826305389f, kKeyExp2C3 = 0.055503569543361664f,
                kKeyExp2C4 = 0.009676031768321991f, kKeyExp2C5 = 0.0013390863314270973f;

__device__ __forceinline__ float2 key_weight_exp2(float2 x)
{
    x.x = fmax_nan(x.x, -127.f);
    x.y = fmax_nan(x.y, -127.f);
    const float2 t = fadd2(x, make_float2(12582912.f, 12582912.f));
    const float2 f = fadd2(x, fadd2(make_float2(12582912.f, 12582912.f), make_float2(-t.x, -t.y)));
    float2 q = ffma2(make_float2(kKeyExp2C5, kKeyExp2C5), f, make_float2(kKeyExp2C4, kKeyExp2C4));
    q = ffma2(q, f, make_float2(kKeyExp2C3, kKeyExp2C3));
    q = ffma2(q, f, make_float2(kKeyExp2C2, kKeyExp2C2));
    q = ffma2(q, f, make_float2(kKeyExp2C1, kKeyExp2C1));
    q = ffma2(q, f, make_float2(kKeyExp2C0, kKeyExp2C0));
    return fmul2(q, make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3F800000),
                                __int_as_float((__float_as_int(t.y) << 23) + 0x3F800000)));
}

// pairs in four whose exponentials go to the FMA pipe
constexpr int kKeyPoly = 1;

template <int D>
struct KeyWCfg {
    static constexpr int kCtas = D == 256 ? 1 : 2;       // per SM
    static constexpr int kGroups = 4 / kCtas;            // consumer warpgroups, each with a TMEM buffer
    static constexpr int kThreads = kGroups * 128 + 64;
    static constexpr int kPanels = D / 64;
    static constexpr int kPanelBytes = 128 * 128;        // 128 rows x 64 elements
    static constexpr int kTileBytes = kPanels * kPanelBytes;
    static constexpr int kStages = D == 64 ? 4 : 2;
    static constexpr int kOffK = 0;
    static constexpr int kOffQ = kTileBytes;
    static constexpr int kOffVec = kOffQ + kStages * kTileBytes;   // per group: [2][128] -LSE log2(e), then positions
    static constexpr int kOffSum = kOffVec + kGroups * 2 * 128 * 8;   // [kGroups][128] sums
    static constexpr int kOffBar = kOffSum + kGroups * 512;
    static constexpr int kSmemBytes = kOffBar + 256 + 1024;
    static_assert((1 + 2 * kStages + 9) * 8 + 8 <= 256, "barrier area");
    static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory per SM");
};

// One CTA per (key block of 128, batch and kv head, share of the steps), two per SM (one at d = 256):
// one starts or ends while the other computes.  A step is 128 query rows: S^T = K Q^T (keys along TMEM
// lanes) goes to a TMEM buffer, and the consumer warpgroups take the steps in turn: thread r holds
// key r, so a step's sum over rows is a sum over the thread's own registers, and no two threads ever
// add to the same key.  The exponentials bound it (128 x 128 of them against 2 x 128 x 128 x d flops): one pair in four goes to the FMA pipe, and
// four warps per scheduler keep both pipes fed across the waits for TMEM and barriers.  GQA 32 / 8,
// 4096 rows, d = 128, causal: 89 us (without the mask 165 us: 3.3e12 exponentials a second, 0.75 of the
// MUFU's own rate; with the mask a CTA has 1 to 32 steps, each with the same set-up); 95 behind a forward
// in a loop at the power limit.
template <int D, typename T>
__global__ void __launch_bounds__(KeyWCfg<D>::kThreads, KeyWCfg<D>::kCtas)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       KeyWeightParams p)
{
    using C = KeyWCfg<D>;
    griddep_launch_dependents();   // the addition of the shares may be scheduled
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    uint64_t* bar_k = reinterpret_cast<uint64_t*>(smem + C::kOffBar);   // K landed
    uint64_t* bar_full = bar_k + 1;                 // [kStages] Q slot landed
    uint64_t* bar_empty = bar_full + C::kStages;    // [kStages] Q slot read
    uint64_t* bar_s = bar_empty + C::kStages;       // [kGroups] S^T of a step in TMEM
    uint64_t* bar_free = bar_s + 4;                 // [kGroups] read out (count 4)
    uint64_t* bar_drain = bar_free + 4;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    constexpr int kTma = C::kGroups * 4, kMma = kTma + 1;   // warps
    const int warp = warp_id(), lane = lane_id();
    const int BH = p.B * p.Hkv;
    // blocks of the first keys, which most rows see, first
    const int kb = (int)blockIdx.x / (BH * p.nsp);
    const int kvh = ((int)blockIdx.x % (BH * p.nsp)) / p.nsp;
    const int sp = (int)blockIdx.x % p.nsp;
    const int delta = p.Nk - p.Nq;
    int qb0 = 0, nqb = (p.rows + 127) / 128;
    if (p.causal) {
        const int first = kb * 128 - delta;   // first position that sees a key of the block
        if (first >= p.Nq)
            nqb = 0;
        else if (p.rows == p.Nq && first > 0)
            qb0 = first / 128;
        nqb = max(0, nqb - qb0);
    }
    const long long n_all = (long long)p.heads * nqb;
    const int it_lo = (int)(sp * n_all / p.nsp);
    const int n_it = (int)((sp + 1) * n_all / p.nsp) - it_lo;
    // row tile (tile head, first row) of the CTA's step it
    auto step = [&](int it, int& th, int& row0) {
        const int g = it_lo + it;
        th = kvh * p.heads + g / nqb;
        row0 = (qb0 + g % nqb) * 128;
    };

    if (threadIdx.x == 0) {
        mbar_init(bar_k, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], 1);
        }
        for (int b = 0; b < C::kGroups; ++b) {
            mbar_init(&bar_s[b], 1);
            mbar_init(&bar_free[b], 4);
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMma) {
        tmem_alloc(tmem_slot, 128 * C::kGroups);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp >= kTma) {
        if (warp == kTma && lane == 0 && n_it > 0) {
            // ------------------------------------------------------------ TMA producer
            mbar_arrive_expect_tx(bar_k, C::kTileBytes);
            for (int i = 0; i < C::kPanels; ++i)
                tma_load_3d(smem + C::kOffK + i * C::kPanelBytes, &tmK, bar_k, i * 64, kb * 128, kvh);
            int issued = 0;
            for (int it = 0; it < n_it; ++it) {
                const int s = it % C::kStages;
                if (!mbar_wait(&bar_empty[s], (uint32_t)((it / C::kStages) & 1) ^ 1u, abort_flag))
                    break;
                int th, row0;
                step(it, th, row0);
                mbar_arrive_expect_tx(&bar_full[s], C::kTileBytes);
                for (int pn = 0; pn < C::kPanels; ++pn)
                    tma_load_3d(smem + C::kOffQ + s * C::kTileBytes + pn * C::kPanelBytes, &tmQ, &bar_full[s], pn * 64,
                                row0, th);
                ++issued;
            }
            if (*abort_flag) {
                // let the loads in flight land before the block exits
                mbar_wait_limited(bar_k, 0, FA_WAIT_LIMIT_CYCLES);
                for (int i = max(0, issued - C::kStages); i < issued; ++i)
                    mbar_wait_limited(&bar_full[i % C::kStages], (uint32_t)((i / C::kStages) & 1), FA_WAIT_LIMIT_CYCLES);
            }
        } else if (warp == kMma && n_it > 0) {
            // ------------------------------------------------------------ MMA issuer
            const uint32_t id = idesc_f16kind(Elt<T>::kMmaFmt, 128, 128, false, false);
            const uint64_t dK = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
            const uint64_t dQ = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
            bool ok = mbar_wait_w(bar_k, 0, abort_flag);
            for (int it = 0; ok && it < n_it; ++it) {
                const int s = it % C::kStages;
                if (!(ok = mbar_wait_w(&bar_full[s], (uint32_t)((it / C::kStages) & 1), abort_flag)))
                    break;
                const int b = it % C::kGroups;
                if (!(ok = mbar_wait_w(&bar_free[b], (uint32_t)((it / C::kGroups) & 1) ^ 1u, abort_flag)))
                    break;
                tc_fence_after();
#pragma unroll 4
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (uint32_t)((kk >> 2) * C::kPanelBytes + (kk & 3) * 32);
                    mma_ss_w(tmem + 128u * (uint32_t)b, dK + (uint64_t)(o >> 4),
                             dQ + (uint64_t)((o + (uint32_t)(s * C::kTileBytes)) >> 4), id, kk > 0 ? 1u : 0u);
                }
                mma_commit_w(&bar_s[b]);
                mma_commit_w(&bar_empty[s]);
            }
            if (!ok) {
                mma_commit_w(bar_drain);
                mbar_wait_limited(bar_drain, 0, FA_WAIT_LIMIT_CYCLES);
            }
        }
    } else {
        // ------------------------------------------------------------ exponentials and sums
        const int g = warp >> 2, c0 = threadIdx.x & 127;
        const int r = ((warp & 3) << 5) + lane;            // key within its tile = TMEM lane
        const int key = kb * 128 + r;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        float* vec = reinterpret_cast<float*>(smem + C::kOffVec) + g * 512;   // [2][128] floats, then [2][128] ints
        int* pos = reinterpret_cast<int*>(vec + 256);
        const float sl2 = p.scale_log2;
        const float2 sl22 = make_float2(sl2, sl2);
        float sum = 0.f;
        bool ok = true;
        // the group's next step: tile head th, query block qb of its nqb
        int th = 0, qb = 0;
        if (n_it > 0) {
            th = kvh * p.heads + (it_lo + g) / nqb;
            qb = (it_lo + g) % nqb;
        }
        // LSE of this thread's row of the next step (loaded a step ahead)
        auto next_lse = [&](int it) {
            const int row = (qb0 + qb) * 128 + c0;
            return it < n_it && row < p.rows ? __ldg(p.lse + (size_t)th * p.rows + row) : -INFINITY;
        };
        float lse_next = next_lse(g);
        for (int it = g, u = 0; it < n_it; it += C::kGroups, ++u) {
            const int row0 = (qb0 + qb) * 128, row = row0 + c0;
            // -LSE log2(e) of the step's rows: -inf (P = 0) for rows that see no key
            const float nl = (lse_next == -INFINITY) ? -INFINITY : -lse_next * 1.4426950408889634f;
            for (qb += C::kGroups; qb >= nqb; qb -= nqb)
                ++th;
            lse_next = next_lse(it + C::kGroups);
            float* v = vec + (u & 1) * 128;
            int* ps = pos + (u & 1) * 128;
            v[c0] = nl;
            // the last step of a head may end past its rows: those see nothing (32 of them at a time are left out)
            const int n_rows = p.rows - row0;
            if (p.causal || n_rows < 128)
                ps[c0] = row >= p.rows ? INT_MIN : !p.causal ? INT_MAX : (p.rows == p.Nq ? row : row % p.Nq) + delta;
            // (nobody still reads the buffer of two steps ago; the four warps go on or stop together)
            ok = named_bar_and(1 + g, 128, ok);
            if (!ok)
                break;
            const int b = g;
            ok = mbar_wait(&bar_s[b], (uint32_t)(u & 1), abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                continue;
            tc_fence_after();
            // rows whose position does not reach the key: only in the blocks on the diagonal
            // (every block of a run of short groups)
            const bool masked = p.causal && (p.rows != p.Nq || row0 + delta < kb * 128 + 127);
            const float4* v4 = reinterpret_cast<const float4*>(v);
            float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t sr[32];
                tmem_ld32(tmem + lane_off + 128u * (uint32_t)b + 32u * h, sr);
                if (h == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(&bar_free[b]);
                }
                if (32 * h >= n_rows)
                    continue;
                if (!masked && 32 * h + 32 <= n_rows) {
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        const float4 n0 = v4[8 * h + (c >> 2)], n1 = v4[8 * h + (c >> 2) + 1];
                        const float2 x0 = ffma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl22,
                                                make_float2(n0.x, n0.y));
                        const float2 x1 = ffma2(make_float2(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sl22,
                                                make_float2(n0.z, n0.w));
                        const float2 x2 = ffma2(make_float2(__uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5])), sl22,
                                                make_float2(n1.x, n1.y));
                        const float2 x3 = ffma2(make_float2(__uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7])), sl22,
                                                make_float2(n1.z, n1.w));
                        a0 = fadd2(a0, make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
                        a1 = fadd2(a1, make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
                        a0 = fadd2(a0, kKeyPoly >= 2 ? key_weight_exp2(x2) : make_float2(ex2_approx(x2.x), ex2_approx(x2.y)));
                        a1 = fadd2(a1, kKeyPoly >= 1 ? key_weight_exp2(x3) : make_float2(ex2_approx(x3.x), ex2_approx(x3.y)));
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 n4 = v4[8 * h + (c >> 2)];
                        const int4 p4 = *reinterpret_cast<const int4*>(ps + 32 * h + c);
                        float2 x0 = ffma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl22,
                                          make_float2(n4.x, n4.y));
                        float2 x1 = ffma2(make_float2(__uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3])), sl22,
                                          make_float2(n4.z, n4.w));
                        x0.x = p4.x >= key ? x0.x : -INFINITY;
                        x0.y = p4.y >= key ? x0.y : -INFINITY;
                        x1.x = p4.z >= key ? x1.x : -INFINITY;
                        x1.y = p4.w >= key ? x1.y : -INFINITY;
                        a0 = fadd2(a0, make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
                        a1 = fadd2(a1, make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
                    }
                }
            }
            sum += (a0.x + a0.y) + (a1.x + a1.y);
        }
        // the groups' sums, in a fixed order
        float* sums = reinterpret_cast<float*>(smem + C::kOffSum);
        sums[g * 128 + r] = sum;
        named_bar_sync(C::kGroups + 1, C::kGroups * 128);
        if (g == 0 && ok && !*abort_flag && key < p.Nk) {
            const size_t at = (size_t)kvh * p.Nk + key;
            for (int k = 1; k < C::kGroups; ++k)
                sum += sums[k * 128 + r];
            if (p.nsp > 1)
                p.part[(size_t)sp * BH * p.Nk + at] = sum;
            else
                p.w_out[at] = (p.w_in ? p.w_in[at] : 0.f) + sum;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 128 * C::kGroups);
    }
}

// w_out = w_in + the shares' sums, in share order.
__global__ void __launch_bounds__(256) key_weights_add_kernel(KeyWeightParams p)
{
    griddep_wait();   // the sums are complete once key_weights_kernel has finished
    const size_t n = (size_t)p.B * p.Hkv * p.Nk;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        float s = 0.f;
        for (int sp = 0; sp < p.nsp; ++sp)
            s += p.part[(size_t)sp * n + i];
        p.w_out[i] = (p.w_in ? p.w_in[i] : 0.f) + s;
    }
}

// ----------------------------------------------------------------------------
// selection
// ----------------------------------------------------------------------------
struct EvictParams {
    const float* w;        // [BH, Nk]
    const int* seq_lens;   // [B] or nullptr (all Nk)
    const uint4* k;        // [BH, Nk, d] as 16-byte chunks
    const uint4* v;
    uint4* k_out;          // [BH, keep, d]
    uint4* v_out;
    float* w_out;          // [BH, keep] or nullptr
    int* index;            // [BH, keep]
    int BH, Hkv, Nk, chunks;   // chunks: d * 2 / 16
    int keep, recent;
};

// A weight as an unsigned number of the same order: -0 and 0 alike, NaN above all.
__device__ __forceinline__ uint32_t evict_order(float w)
{
    if (w != w)
        return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.f);   // -0 becomes 0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block's threads (1024, in thread order), `warp_sum` [32] in shared memory.
__device__ __forceinline__ int evict_prefix(int v, int* warp_sum)
{
    const int warp = warp_id(), lane = lane_id();
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off)
            incl += x;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    int before = lane < warp ? warp_sum[lane] : 0;   // the warps before this one
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        before += __shfl_xor_sync(0xffffffffu, before, off);
    return before + incl - v;
}

// One block per (batch, kv head).  Of its n keys the newest `recent` stay, and of the m before them
// the `need` = keep - recent heaviest.  The need-th largest weight T is found digit by digit from the
// highest (11, 11 and 10 bits): a histogram of the digit, and the bin in which the count from above
// reaches what is left.  The first digit takes the sign, the exponent and two bits of the mantissa, so
// that few keys are left for the next ones; they are listed in shared memory (where they fit).  Then
// every warp walks its own contiguous part of the keys: a key stays if it is above T, or equal to T
// with fewer than the remaining number of equal ones before it.  Its place is the number of kept keys
// before it, so the kept keys stay in order.
// FUSED: the block also moves the kept rows, where they are few: a launch less (small caches are bound
// by the launches).
constexpr int kEvictThreads = 1024;
constexpr int kEvictCache = 40 * 1024;   // keys whose order numbers are held in shared memory
constexpr int kEvictList = 8 * 1024;     // keys listed after the first digit
constexpr int kEvictBins = 2048;

template <bool FUSED>
__global__ void __launch_bounds__(kEvictThreads, 1) evict_select_kernel(EvictParams p)
{
    extern __shared__ uint32_t s_mem[];
    uint32_t* s_list = s_mem;                 // [kEvictList]
    uint32_t* s_cache = s_mem + kEvictList;
    __shared__ int s_hist[kEvictBins];
    __shared__ int s_warp[32], s_eq[32];
    __shared__ uint32_t s_digit;
    __shared__ int s_left, s_count, s_listed;
    griddep_launch_dependents();
    const int row = (int)blockIdx.x, tid = (int)threadIdx.x, warp = warp_id(), lane = lane_id();
    const int n = p.seq_lens ? max(0, min(__ldg(p.seq_lens + row / p.Hkv), p.Nk)) : p.Nk;
    const float* w = p.w + (size_t)row * p.Nk;
    int* index = p.index + (size_t)row * p.keep;
    float* w_out = p.w_out ? p.w_out + (size_t)row * p.keep : nullptr;
    if (n <= p.keep) {   // all of them
        for (int i = tid; i < n; i += kEvictThreads) {
            index[i] = i;
            if (w_out)
                w_out[i] = w[i];
        }
    } else {
        const int m = n - p.recent;             // recent <= keep < n
        const int need = p.keep - p.recent;     // < m
        const bool cached = m <= kEvictCache;
        // eight keys' order numbers, `step` apart, their loads in flight together (0 past `end`)
        constexpr int kAtOnce = 8;
        auto orders = [&](uint32_t (&u)[kAtOnce], int i, int step, int end) {
            if (cached) {
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    u[k] = i + k * step < end ? s_cache[i + k * step] : 0u;
            } else {
                float x[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    x[k] = i + k * step < end ? __ldg(w + i + k * step) : 0.f;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    u[k] = evict_order(x[k]);
            }
        };
        uint32_t T = 0xFFFFFFFFu;   // need = 0: nothing is above it, and none of the equal ones stays
        int left = 0;               // how many of the keys equal to T stay
        // count one key's digit: one addition where a warp's keys agree (equal weights)
        auto count = [&](bool in, int digit) {
            const unsigned who = __ballot_sync(0xffffffffu, in);
            int same;
            __match_all_sync(0xffffffffu, in ? digit : -1, &same);
            if (same) {
                if (in && lane == 0)
                    atomicAdd(&s_hist[digit], __popc(who));
            } else if (in) {
                atomicAdd(&s_hist[digit], 1);
            }
        };
        // the bin, from the highest, in which `left` keys are reached, and its count (s_count: the
        // histogram itself may be cleared by another thread once this returns); two bins per thread
        auto find = [&]() {
            __syncthreads();
            const int hi = kEvictBins - 1 - 2 * tid, a = s_hist[hi], b = s_hist[hi - 1];
            const int before = evict_prefix(a + b, s_warp);
            if (before < left && left <= before + a) {
                s_digit = (uint32_t)hi;
                s_left = left - before;
                s_count = a;
            } else if (before + a < left && left <= before + a + b) {
                s_digit = (uint32_t)(hi - 1);
                s_left = left - before - a;
                s_count = b;
            }
            __syncthreads();
            left = s_left;
            return s_digit;
        };
        auto clear = [&]() {
            s_hist[tid] = 0;
            s_hist[tid + kEvictThreads] = 0;
            __syncthreads();
        };
        static_assert(kEvictBins == 2 * kEvictThreads, "two bins per thread");
        if (tid == 0)
            s_listed = 0;
        clear();
        if (need > 0 || cached) {
            for (int i0 = 0; i0 < m; i0 += kAtOnce * kEvictThreads) {
                float x[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int i = i0 + k * kEvictThreads + tid;
                    x[k] = i < m ? __ldg(w + i) : 0.f;
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int i = i0 + k * kEvictThreads + tid;
                    if (i0 + k * kEvictThreads >= m)
                        break;
                    const uint32_t u = evict_order(x[k]);
                    if (cached && i < m)
                        s_cache[i] = u;
                    count(i < m, (int)(u >> 21));
                }
            }
        }
        if (need > 0) {
            left = need;
            T = find() << 21;
            const int in_bin = s_count;   // the same for all threads: written again only after the next barriers
            const bool listed = in_bin <= kEvictList;
            if (listed) {
                for (int i0 = 0; i0 < m; i0 += kAtOnce * kEvictThreads) {
                    uint32_t u[kAtOnce];
                    orders(u, i0 + tid, kEvictThreads, m);
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k)
                        if (i0 + k * kEvictThreads + tid < m && (u[k] >> 21) == (T >> 21))
                            s_list[atomicAdd(&s_listed, 1)] = u[k];
                }
                __syncthreads();
            }
            const int c = listed ? in_bin : m;   // keys that the next digits look at
            for (int d = 0; d < 2; ++d) {
                const int shift = d == 0 ? 10 : 0, above = d == 0 ? 21 : 10;
                clear();
                const uint32_t digits = d == 0 ? 2047u : 1023u;
                if (listed) {
                    for (int i0 = 0; i0 < c; i0 += kEvictThreads) {
                        const int i = i0 + tid;
                        const uint32_t u = i < c ? s_list[i] : 0u;
                        count(i < c && (u >> above) == (T >> above), (int)((u >> shift) & digits));
                    }
                } else {
                    for (int i0 = 0; i0 < c; i0 += kAtOnce * kEvictThreads) {
                        uint32_t u[kAtOnce];
                        orders(u, i0 + tid, kEvictThreads, c);
#pragma unroll
                        for (int k = 0; k < kAtOnce; ++k)
                            count(i0 + k * kEvictThreads + tid < c && (u[k] >> above) == (T >> above),
                                  (int)((u[k] >> shift) & digits));
                    }
                }
                T |= find() << shift;
            }
        }
        // counts above and at T in each warp's part
        const int part = ((m + 31) / 32 + 31) / 32 * 32, lo = min(m, warp * part), hi = min(m, lo + part);
        int gt = 0, eq = 0;
        __syncthreads();
        for (int i0 = lo; i0 < hi; i0 += 32 * kAtOnce) {
            uint32_t u[kAtOnce];
            orders(u, i0 + lane, 32, hi);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const bool in = i0 + 32 * k + lane < hi;
                gt += in && u[k] > T;
                eq += in && u[k] == T;
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            gt += __shfl_xor_sync(0xffffffffu, gt, off);
            eq += __shfl_xor_sync(0xffffffffu, eq, off);
        }
        if (lane == 0) {
            s_warp[warp] = gt;
            s_eq[warp] = eq;
        }
        __syncthreads();
        gt = lane < warp ? s_warp[lane] : 0;
        eq = lane < warp ? s_eq[lane] : 0;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            gt += __shfl_xor_sync(0xffffffffu, gt, off);
            eq += __shfl_xor_sync(0xffffffffu, eq, off);
        }
        const unsigned below = (1u << lane) - 1u;
        for (int i0 = lo; i0 < hi; i0 += 32 * kAtOnce) {
            uint32_t u[kAtOnce];
            orders(u, i0 + lane, 32, hi);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = i0 + 32 * k + lane;
                const bool is_gt = i < hi && u[k] > T, is_eq = i < hi && u[k] == T;
                const unsigned bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
                const int eq_before = eq + __popc(be & below);
                if (is_gt || (is_eq && eq_before < left)) {
                    const int at = gt + __popc(bg & below) + min(eq_before, left);
                    index[at] = i;
                    if (w_out)
                        w_out[at] = w[i];
                }
                gt += __popc(bg);
                eq += __popc(be);
            }
        }
        for (int i = m + tid; i < n; i += kEvictThreads) {
            index[need + i - m] = i;
            if (w_out)
                w_out[need + i - m] = w[i];
        }
    }
    if constexpr (FUSED) {
        __syncthreads();   // the indices, written by this block
        const int moved = min(n, p.keep) * p.chunks;
        const size_t in = (size_t)row * p.Nk * p.chunks, out = (size_t)row * p.keep * p.chunks;
        for (int c = tid; c < moved; c += kEvictThreads) {
            const int j = c / p.chunks;
            const size_t from = in + (size_t)index[j] * p.chunks + (c - j * p.chunks);
            const uint4 a = p.k[from], b = p.v[from];
            p.k_out[out + c] = a;
            p.v_out[out + c] = b;
        }
    }
}

// The kept rows of K and V, 16 bytes per thread and tensor at a time; bound by HBM (each kept row
// read and written once: 268 MB in 41 us, 6.5 TB/s, for 128 caches cut to 2048 keys of d = 128).
constexpr int kGatherItems = 4;

__global__ void __launch_bounds__(256) evict_gather_kernel(EvictParams p)
{
    griddep_wait();   // the kept keys' indices are complete once the selection has finished
    const int per_row = p.keep * p.chunks;                      // chunks of a (batch, kv head)
    const int blocks = (per_row + 256 * kGatherItems - 1) / (256 * kGatherItems);
    const int row = (int)(blockIdx.x / (unsigned)blocks), blk = (int)(blockIdx.x % (unsigned)blocks);
    const int n = p.seq_lens ? max(0, min(__ldg(p.seq_lens + row / p.Hkv), p.Nk)) : p.Nk;
    const int count = min(n, p.keep) * p.chunks;
    const size_t in = (size_t)row * p.Nk * p.chunks, out = (size_t)row * per_row;
    const int* index = p.index + (size_t)row * p.keep;
    uint4 a[kGatherItems], b[kGatherItems];
#pragma unroll
    for (int t = 0; t < kGatherItems; ++t) {
        const int c = blk * 256 * kGatherItems + t * 256 + (int)threadIdx.x;
        if (c < count) {
            const int j = c / p.chunks;
            const size_t from = in + (size_t)index[j] * p.chunks + (c - j * p.chunks);
            a[t] = __ldcs(p.k + from);
            b[t] = __ldcs(p.v + from);
        }
    }
#pragma unroll
    for (int t = 0; t < kGatherItems; ++t) {
        const int c = blk * 256 * kGatherItems + t * 256 + (int)threadIdx.x;
        if (c < count) {
            p.k_out[out + c] = a[t];
            p.v_out[out + c] = b[t];
        }
    }
}

}  // namespace fa
