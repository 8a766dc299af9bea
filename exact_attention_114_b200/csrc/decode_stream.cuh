// decode_stream.cuh -- split-KV forward for few query rows per kv head (R = G * Nq <= 16) over
// lists of keys: a window with sinks, a padded or paged cache with a length per sequence, a shared
// prefix followed by own keys.  The recurrence and the warp MMAs are those of the split pass in
// decode.cuh; what differs is how the work is cut.
//
// Each (batch, kv head) is a unit: a list of 64-key tiles that hold at least one visible key.  The
// tiles of all units form one line, T tiles long, and CTA c of G takes the tiles
// [c T / G, (c + 1) T / G): as many as any other, whatever the lengths.  Its TMA warp runs through
// them without a pause, into the next unit while the other warps still end the last one, so the
// loads in flight (three stages of 32 KB, two CTAs per SM) never drain at a unit's end.  The pass is
// bound by HBM, and short lists (a window of 1024 keys is 17 tiles) would otherwise spend a third of
// their time starting and ending CTAs.
//
// A unit within one CTA is written out straight away.  A unit that continues in other CTAs leaves a
// partial (O_s normalised, lse_s, fp32) in each: in the CTA's slot 1 where the CTA starts the unit, in
// its slot 0 where it goes on with one, so two slots per CTA are enough.  Which CTAs hold a unit
// follows from T, G and the unit's first tile, and stream_combine_kernel merges them in order.
#pragma once

#include "decode.cuh"

namespace fa {

// Lists of keys
constexpr int kListAll = 0;     // the sequence's keys (dense cache, with or without lengths)
constexpr int kListWindow = 1;  // sliding window with sinks, dense cache
constexpr int kListPaged = 2;   // the same in a paged cache
constexpr int kListCat = 3;     // a shared prefix, then the sequence's own keys

struct StreamParams {
    const void* q;          // [B, Hq, Nq, d]
    void* o;                // [B, Hq, Nq, d]
    float* lse;             // [B, Hq, Nq] or nullptr
    float* part_o;          // [slots][R][128]: 2 per CTA, then (partial) one per unit
    float* part_lse;        // [slots][R], log2 units
    int* first;             // [B + 1] tiles of the sequences before b, per kv head (with lengths)
    const int* seq_lens;    // [B] or nullptr (Nk each)
    const int* block_table; // [B, max_pages] (kListPaged)
    int B, Hq, Hkv, Nq, Nk, G, R, d_io;
    int causal;
    int window, sinks;
    int np;                 // prefix keys (kListCat)
    int page_size, max_pages;
    int partial;            // every unit as a partial
    int after;              // launched as a dependent of a kernel it does not read from: wait for that
                            // one before ending, so that later kernels find both complete
    float scale_log2;
    float* scores;          // SCORES: [B * Hkv, R, score_stride]
    int score_stride;
};

struct StreamCfg {
    static constexpr int kThreads = 160;
    static constexpr int kStages = 3;
    static constexpr int kMergeRows = 4;               // rows of the four warps' states merged at a time
    static constexpr int kOffMerge = kStages * 2 * DecCfg::kTileBytes;
    static constexpr int kOffML = kOffMerge + 4 * kMergeRows * 128 * 4;   // [4 warps][16] m, then l
    static constexpr int kOffScan = kOffML + 2 * 64 * 4;                  // [128] ints
    static constexpr int kOffBar = kOffScan + 128 * 4;
    static constexpr int kSmemBytes = kOffBar + 128 + 1024;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

// A sequence's list of tiles.
struct StreamList {
    int len;      // keys of the sequence (own keys behind a prefix)
    int tiles;
    int seg;      // tiles of the first segment (sinks, prefix), whose keys start at 0
    int base;     // first key of the second segment
    int win_lo;   // window: the first row's first window key
};

template <int LIST>
__host__ __device__ __forceinline__ StreamList stream_list(const StreamParams& p, int len)
{
    StreamList l;
    l.len = len;
    l.seg = l.base = l.win_lo = 0;
    constexpr int kt = DecCfg::kKeys;
    if constexpr (LIST == kListWindow || LIST == kListPaged) {
        const int s = p.sinks < len ? p.sinks : len;
        const int first = len - p.Nq - p.window + 1;
        l.win_lo = first > 0 ? first : 0;
        l.seg = (s + kt - 1) / kt;
        // in a paged cache tiles keep to multiples of 64, so that none straddles a page
        const int from = LIST == kListPaged ? l.win_lo / kt * kt : l.win_lo;
        l.base = from > l.seg * kt ? from : l.seg * kt;
        l.tiles = l.seg + (len > l.base ? (len - l.base + kt - 1) / kt : 0);
    } else if constexpr (LIST == kListCat) {
        l.seg = (p.np + kt - 1) / kt;
        l.tiles = l.seg + (len + kt - 1) / kt;
    } else {
        l.tiles = (len + kt - 1) / kt;
    }
    return l;
}

__device__ __forceinline__ int stream_len(const StreamParams& p, int b)
{
    return p.seq_lens ? max(0, min(__ldg(p.seq_lens + b), p.Nk)) : p.Nk;
}

// The CTA that holds tile t of T, and CTA c's first tile.  Where the lengths leave fewer tiles than
// CTAs were launched, T of them take one each (none between two of a unit's CTAs is empty).
__host__ __device__ __forceinline__ int stream_cta(long long t, long long T, int grid)
{
    const long long g = grid < T ? grid : T;
    return (int)(((t + 1) * g - 1) / T);
}
__host__ __device__ __forceinline__ long long stream_tile(int c, long long T, int grid)
{
    const long long g = grid < T ? grid : T;
    return c < g ? c * T / g : T;
}

// Place in the line: kv head hk of sequence b, tile t of its list.
template <int LIST>
struct StreamPos {
    int b, hk, t;
    StreamList l;
    __device__ __forceinline__ void next_unit(const StreamParams& p)
    {
        t = 0;
        if (++hk < p.Hkv)
            return;
        hk = 0;
        do {
            if (++b >= p.B)
                return;
            l = stream_list<LIST>(p, stream_len(p, b));
        } while (l.tiles == 0);
    }
};

template <typename T, bool NARROW, int LIST, bool SCORES = false>
__global__ void __launch_bounds__(160, 2)
    decode_stream_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ CUtensorMap tmK0, const __grid_constant__ CUtensorMap tmV0, StreamParams p)
{
    using C = StreamCfg;
    constexpr int kt = DecCfg::kKeys;
    griddep_launch_dependents();   // the merge may be scheduled
    const int d_io = NARROW ? p.d_io : 128;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    uint64_t* bar_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
    uint64_t* bar_empty = bar_full + C::kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_empty + C::kStages);
    int* start = const_cast<int*>(abort_flag) + 1;   // [3] b, hk, t of the CTA's first tile
    int* scan = reinterpret_cast<int*>(smem + C::kOffScan);

    const int warp = warp_id(), lane = lane_id();
    const int cta = (int)blockIdx.x, grid = (int)gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], 4);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 128) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    // the line's length and the CTA's part of it
    long long total;
    StreamPos<LIST> at;
    if (p.seq_lens == nullptr) {
        at.l = stream_list<LIST>(p, p.Nk);
        total = (long long)at.l.tiles * p.B * p.Hkv;
        const long long t0 = stream_tile(cta, total, grid);
        const int unit = (int)(t0 / at.l.tiles);
        at.b = unit / p.Hkv;
        at.hk = unit % p.Hkv;
        at.t = (int)(t0 % at.l.tiles);
        __syncthreads();
    } else {
        // thread i of the first 128 sums the tiles of its share of the sequences
        const int per = (p.B + 127) / 128;
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        int mine = 0;
        if (threadIdx.x < 128) {
            for (int b = b0; b < b1; ++b)
                mine += stream_list<LIST>(p, stream_len(p, b)).tiles;
            scan[threadIdx.x] = mine;
        }
        __syncthreads();
        if (warp == 0) {
            int v[4], sum = 0;
            for (int k = 0; k < 4; ++k) {
                v[k] = sum;
                sum += scan[4 * lane + k];
            }
            int incl = sum;
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off)
                    incl += x;
            }
            __syncwarp();
            for (int k = 0; k < 4; ++k)
                scan[4 * lane + k] = v[k] + incl - sum;   // tiles before thread 4 lane + k's share
            if (lane == 31)
                start[3] = incl;
        }
        __syncthreads();
        total = (long long)start[3] * p.Hkv;
        const long long t0 = stream_tile(cta, total, grid);
        if (threadIdx.x < 128) {
            int before = scan[threadIdx.x];
            for (int b = b0; b < b1; ++b) {
                const int n = stream_list<LIST>(p, stream_len(p, b)).tiles;
                if (cta == 0)
                    p.first[b] = before;   // for the merge
                const long long lo = (long long)before * p.Hkv;
                if (n > 0 && lo <= t0 && t0 < lo + (long long)n * p.Hkv) {
                    start[0] = b;
                    start[1] = (int)((t0 - lo) / n);
                    start[2] = (int)((t0 - lo) % n);
                }
                before += n;
            }
            if (cta == 0 && threadIdx.x == 127)
                p.first[p.B] = start[3];
        }
        __syncthreads();
        at.b = start[0];
        at.hk = start[1];
        at.t = start[2];
        if (t0 < total)
            at.l = stream_list<LIST>(p, stream_len(p, at.b));
    }
    const int n_mine = (int)(stream_tile(cta + 1, total, grid) - stream_tile(cta, total, grid));   // tiles of the CTA
    int left = n_mine;

    if (warp == 4) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            const bool two = d_io > 64;   // the second 64-column panel only when the head has columns there
            const uint32_t bytes = (uint32_t)(two ? 4 : 2) * DecCfg::kPanelBytes;
            int n = 0;
            for (; left > 0; --left, ++n) {
                const int slot = n % C::kStages;
                if (!mbar_wait(&bar_empty[slot], ((uint32_t)(n / C::kStages) & 1u) ^ 1u, abort_flag))
                    break;
                uint8_t* dk = smem + slot * 2 * DecCfg::kTileBytes;
                uint8_t* dv = dk + DecCfg::kTileBytes;
                mbar_arrive_expect_tx(&bar_full[slot], bytes);
                const bool head_seg = at.t < at.l.seg;
                const int key0 = head_seg ? at.t * kt : at.l.base + (at.t - at.l.seg) * kt;
                if constexpr (LIST == kListPaged) {
                    // an out-of-range page id reads zeros (TMA bounds), never another buffer
                    const int page = __ldg(p.block_table + (size_t)at.b * p.max_pages + key0 / p.page_size);
                    const int off = key0 % p.page_size;
                    for (int pn = 0; pn < (two ? 2 : 1); ++pn) {
                        tma_load_4d(dk + pn * DecCfg::kPanelBytes, &tmK, &bar_full[slot], pn * 64, at.hk, off, page);
                        tma_load_4d(dv + pn * DecCfg::kPanelBytes, &tmV, &bar_full[slot], pn * 64, at.hk, off, page);
                    }
                } else {
                    const bool pre = LIST == kListCat && head_seg;
                    const CUtensorMap* mk = pre ? &tmK0 : &tmK;
                    const CUtensorMap* mv = pre ? &tmV0 : &tmV;
                    const int head = pre ? at.hk : at.b * p.Hkv + at.hk;
                    for (int pn = 0; pn < (two ? 2 : 1); ++pn) {
                        tma_load_3d(dk + pn * DecCfg::kPanelBytes, mk, &bar_full[slot], pn * 64, key0, head);
                        tma_load_3d(dv + pn * DecCfg::kPanelBytes, mv, &bar_full[slot], pn * 64, key0, head);
                    }
                }
                if (++at.t == at.l.tiles && left > 1)
                    at.next_unit(p);
            }
            if (*abort_flag)   // let the loads in flight land before the block exits
                for (int i = max(0, n - C::kStages); i < n; ++i)
                    mbar_wait_limited(&bar_full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u, FA_WAIT_LIMIT_CYCLES);
        }
        if (p.after)
            griddep_wait();
        return;   // the producer takes no part in the merges below
    }

    // ------------------------------------------------------------------ consumers
    const int g = lane >> 2, tq = lane & 3;   // mma fragment coordinates: rows g and g + 8
    const float sl2 = p.scale_log2;
    float* sm_o = reinterpret_cast<float*>(smem + C::kOffMerge);   // [4 warps][kMergeRows][128]
    float* sm_m = reinterpret_cast<float*>(smem + C::kOffML);      // [4][16]
    float* sm_l = sm_m + 64;
    int n = 0;   // tiles taken so far
    bool ok = true;
    while (left > 0) {
        const int unit = at.b * p.Hkv + at.hk, t_first = at.t;
        const int n_tiles = min(left, at.l.tiles - at.t);
        // the unit's query rows: row r is head hk * G + r / Nq, query r % Nq, and row r of its R
        uint32_t qa[8][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
                const int r = g + 8 * hr;
                qa[ks][hr] = qa[ks][hr + 2] = 0u;
                if (r < p.R && ks * 16 < d_io) {
                    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) +
                                                                             ((size_t)unit * p.R + r) * d_io);
                    qa[ks][hr] = __ldg(qrow + ks * 8 + tq);          // cols 16 ks + 2 tq, + 1
                    qa[ks][hr + 2] = __ldg(qrow + ks * 8 + 4 + tq);  // cols 16 ks + 8 + 2 tq, + 1
                }
            }
        // last visible key of the thread's two rows (own keys), of the prefix, and first window key
        int lim[2], low[2], pre[2];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const int x = at.l.len - p.Nq + (g + 8 * hr) % p.Nq;   // the row's position
            lim[hr] = p.causal ? min(at.l.len - 1, x) : at.l.len - 1;
            low[hr] = x - p.window + 1;
            pre[hr] = p.causal ? min(p.np - 1, p.np + x) : p.np - 1;
        }
        float o[16][4];
#pragma unroll
        for (int nd = 0; nd < 16; ++nd)
            o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int i = 0; i < n_tiles; ++i, ++n, ++at.t) {
            const int slot = n % C::kStages;
            ok = mbar_wait(&bar_full[slot], (uint32_t)(n / C::kStages) & 1u, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            uint8_t* tile = smem + slot * 2 * DecCfg::kTileBytes;
            const uint32_t kbase = smem_u32(tile), vbase = kbase + DecCfg::kTileBytes;
            const int key_w = warp * 16;   // this warp's 16 keys within the tile
            const bool head_seg = at.t < at.l.seg;
            const int key0 = (head_seg ? at.t * kt : at.l.base + (at.t - at.l.seg) * kt) + key_w;

            // S (16 rows x 16 keys) = Q K^T
            float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            {
                const int mi = lane >> 3, key = key_w + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    if (ks * 16 >= d_io)   // columns past the head: not loaded
                        break;
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4(kbase + dec_tile_off(key, 2 * ks + (mi & 1)), b0, b1, b2, b3);
                    mma_16816<T>(s[0], qa[ks], b0, b1);
                    mma_16816<T>(s[1], qa[ks], b2, b3);
                }
            }
            const bool in_prefix = LIST == kListCat && head_seg;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + nt * 8 + 2 * tq + (e & 1), hr = e >> 1;
                    bool out = key > (in_prefix ? pre[hr] : lim[hr]);
                    if constexpr (LIST == kListWindow || LIST == kListPaged)
                        out = out || (key < low[hr] && key >= p.sinks);
                    if (out)
                        s[nt][e] = -INFINITY;
                }
            // V rows of keys that no row sees (between the sinks and the window; past the sequence, in
            // its last page or in the padding) are zeroed: whatever they hold, 0 * V adds nothing
            if (!in_prefix) {
                constexpr bool kWin = LIST == kListWindow || LIST == kListPaged;
                const int len = at.l.len, win_lo = at.l.win_lo;
                if (key0 + 16 > len || (kWin && key0 < win_lo && key0 + 16 > p.sinks)) {
                    for (int j = lane; j < 256; j += 32) {
                        const int key = key0 + (j >> 4);
                        if (key >= len || (kWin && key >= p.sinks && key < win_lo))
                            *reinterpret_cast<uint4*>(tile + DecCfg::kTileBytes + dec_tile_off(key_w + (j >> 4), j & 15)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();   // before the slot is given back to the TMA
                    __syncwarp();
                }
            }
            if constexpr (SCORES) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int hr = 0; hr < 2; ++hr)
                        if (g + 8 * hr < p.R)
                            *reinterpret_cast<float2*>(p.scores + ((size_t)unit * p.R + g + 8 * hr) * p.score_stride + key0 +
                                                       nt * 8 + 2 * tq) = make_float2(s[nt][2 * hr] * sl2, s[nt][2 * hr + 1] * sl2);
            }
            // online softmax for rows g (e = 0, 1) and g + 8 (e = 2, 3)
            uint32_t pa[4];
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
                float mx = fmaxf(fmaxf(s[0][2 * hr], s[0][2 * hr + 1]), fmaxf(s[1][2 * hr], s[1][2 * hr + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float m_new = fmaxf(m[hr], mx * sl2);
                const float a = (m_new == -INFINITY) ? 1.f : ex2_approx(m[hr] - m_new);
                const float neg_m = (m_new == -INFINITY) ? 0.f : -m_new;
                m[hr] = m_new;
                const float p00 = ex2_approx(fmaf(s[0][2 * hr], sl2, neg_m));
                const float p01 = ex2_approx(fmaf(s[0][2 * hr + 1], sl2, neg_m));
                const float p10 = ex2_approx(fmaf(s[1][2 * hr], sl2, neg_m));
                const float p11 = ex2_approx(fmaf(s[1][2 * hr + 1], sl2, neg_m));
                l[hr] = l[hr] * a + (p00 + p01 + p10 + p11);
                pa[hr] = Elt<T>::pack(p00, p01);       // keys 2 tq, + 1
                pa[hr + 2] = Elt<T>::pack(p10, p11);   // keys 8 + 2 tq, + 1
#pragma unroll
                for (int nd = 0; nd < 16; ++nd) {
                    o[nd][2 * hr] *= a;
                    o[nd][2 * hr + 1] *= a;
                }
            }
            // O (16 rows x 128) += P (16 x 16 keys) V (16 keys x 128)
            {
                const int mi = lane >> 3, key = key_w + (mi & 1) * 8 + (lane & 7);
#pragma unroll
                for (int nd = 0; nd < 16; nd += 2) {
                    if (nd * 8 >= d_io)   // output columns past the head stay zero
                        break;
                    uint32_t b0, b1, b2, b3;
                    ldsm_x4_t(vbase + dec_tile_off(key, nd + (mi >> 1)), b0, b1, b2, b3);
                    mma_16816<T>(o[nd], pa, b0, b1);
                    mma_16816<T>(o[nd + 1], pa, b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&bar_empty[slot]);
        }
        // ---- merge the four warps' states, kMergeRows rows at a time
        ok = named_bar_and(1, 128, ok);   // (also: the last merge's shared memory is read out)
        if (!ok)
            break;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            float lt = l[hr];
            lt += __shfl_xor_sync(0xffffffffu, lt, 1);
            lt += __shfl_xor_sync(0xffffffffu, lt, 2);
            if (tq == 0) {
                sm_m[warp * 16 + g + 8 * hr] = m[hr];
                sm_l[warp * 16 + g + 8 * hr] = lt;
            }
        }
        const bool whole = t_first == 0 && at.t == at.l.tiles;
        const int dcol = threadIdx.x;   // 0..127
        for (int r0 = 0; r0 < p.R; r0 += C::kMergeRows) {
            if (r0 > 0)
                named_bar_sync(1, 128);   // the rows before are read out
#pragma unroll
            for (int hr = 0; hr < 2; ++hr)
                if (g + 8 * hr >= r0 && g + 8 * hr < r0 + C::kMergeRows) {
                    float* dst = sm_o + (warp * C::kMergeRows + g + 8 * hr - r0) * 128 + 2 * tq;
#pragma unroll
                    for (int nd = 0; nd < 16; ++nd)
                        *reinterpret_cast<float2*>(dst + nd * 8) = make_float2(o[nd][2 * hr], o[nd][2 * hr + 1]);
                }
            named_bar_sync(1, 128);
            for (int r = r0; r < min(p.R, r0 + C::kMergeRows); ++r) {
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    M = fmaxf(M, sm_m[w * 16 + r]);
                float L = 0.f, acc = 0.f;
                if (M != -INFINITY) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const float sc = ex2_approx(sm_m[w * 16 + r] - M);
                        L += sm_l[w * 16 + r] * sc;
                        acc += sm_o[(w * C::kMergeRows + r - r0) * 128 + dcol] * sc;
                    }
                }
                const float on = (L > 0.f) ? acc / L : 0.f;
                const float lse = (L > 0.f) ? M + __log2f(L) : -INFINITY;
                if (whole && !p.partial) {
                    const size_t row = (size_t)unit * p.R + r;
                    if (dcol < d_io)
                        static_cast<T*>(p.o)[row * d_io + dcol] = Elt<T>::from_float(on);
                    if (dcol == 0 && p.lse)
                        p.lse[row] = lse * 0.69314718055994530942f;
                } else {
                    const size_t slot = whole ? 2 * (size_t)grid + unit : 2 * (size_t)cta + (t_first == 0 ? 1 : 0);
                    p.part_o[(slot * p.R + r) * 128 + dcol] = on;
                    if (dcol == 0)
                        p.part_lse[slot * p.R + r] = lse;
                }
            }
        }
        left -= n_tiles;
        if (left > 0)
            at.next_unit(p);
    }
    if (p.after)
        griddep_wait();
}

// The parts of a unit that the pass has left: `n` of them, part i in slot slot(i).
struct StreamParts {
    const float* o;       // [slots][R][128]
    const float* lse;     // [slots][R], log2 units
    const int* first;     // [B + 1] or nullptr (tiles each)
    int tiles, B, Hkv, R, grid, partial;
    __device__ __forceinline__ int count(int unit, int& c0) const
    {
        long long base, n, total;
        if (first) {
            const int b = unit / Hkv, f = first[b];
            n = first[b + 1] - f;
            base = (long long)f * Hkv + (unit % Hkv) * n;
            total = (long long)first[B] * Hkv;
        } else {
            n = tiles;
            base = (long long)unit * n;
            total = (long long)B * Hkv * n;
        }
        c0 = 0;
        if (n == 0)
            return 0;
        c0 = stream_cta(base, total, grid);
        return stream_cta(base + n - 1, total, grid) - c0 + 1;
    }
    __device__ __forceinline__ size_t slot(int unit, int c0, int n, int i) const
    {
        return n == 1 ? 2 * (size_t)grid + unit : 2 * (size_t)(c0 + i) + (i == 0 ? 1 : 0);
    }
};

// One warp per row: the parts of units cut between CTAs; rows of units within one CTA are final,
// and rows of a sequence without keys get O = 0, LSE = -inf.
template <typename T>
__global__ void __launch_bounds__(128) stream_combine_kernel(StreamParts p, void* o_out, float* lse_out, int d_io)
{
    griddep_launch_dependents();
    griddep_wait();
    const int row = (int)(blockIdx.x * 4 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
    if (row >= p.B * p.Hkv * p.R)
        return;
    const int unit = row / p.R, r = row % p.R;
    int c0;
    const int n = p.count(unit, c0);
    if (n == 1)
        return;
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32)
        M = fmaxf(M, p.lse[p.slot(unit, c0, n, i) * p.R + r]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    if (M != -INFINITY) {
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const size_t at = p.slot(unit, c0, n, i) * p.R + r;
            const float w = ex2_approx(p.lse[at] - M);
            const float4 v = *reinterpret_cast<const float4*>(p.o + at * 128 + lane * 4);
            L += w;
            acc.x = fmaf(w, v.x, acc.x);
            acc.y = fmaf(w, v.y, acc.y);
            acc.z = fmaf(w, v.z, acc.z);
            acc.w = fmaf(w, v.w, acc.w);
        }
    }
    const float inv = (L > 0.f) ? 1.f / L : 0.f;
    if (lane * 4 < d_io)
        *reinterpret_cast<uint2*>(static_cast<T*>(o_out) + (size_t)row * d_io + lane * 4) =
            make_uint2(Elt<T>::pack(acc.x * inv, acc.y * inv), Elt<T>::pack(acc.z * inv, acc.w * inv));
    if (lane == 0 && lse_out)
        lse_out[row] = (L > 0.f) ? (M + __log2f(L)) * 0.69314718055994530942f : -INFINITY;
}

// The weights that the keys receive, from the scores that the pass has left and the rows' LSE:
// thread i takes four keys of a (batch, kv head).  Bound by reading the scores (mostly in L2).
struct DecodeWeightParams {
    const float* scores;    // [BH, R, stride]: log2 units, -inf where masked
    const float* lse;       // [BH, R]
    const float* w_in;      // [BH, Nk] or nullptr (zeros)
    float* w_out;
    int BH, R, Nk, stride;
};

__global__ void __launch_bounds__(128) decode_weights_kernel(DecodeWeightParams p)
{
    __shared__ float s_lse[16];
    griddep_wait();
    const int chunks = (p.Nk + 511) / 512;
    const int bh = (int)blockIdx.x / chunks, key = ((int)blockIdx.x % chunks) * 512 + (int)threadIdx.x * 4;
    if ((int)threadIdx.x < p.R) {
        const float l = p.lse[(size_t)bh * p.R + threadIdx.x];
        s_lse[threadIdx.x] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;   // P = 0 in a row without keys
    }
    __syncthreads();
    if (key >= p.Nk)
        return;
    const float* sc = p.scores + (size_t)bh * p.R * p.stride + key;   // stride: whole tiles of 64
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < p.R; ++r) {
        const float4 x = *reinterpret_cast<const float4*>(sc + (size_t)r * p.stride);
        const float l = s_lse[r];
        sum.x += ex2_approx(x.x - l);
        sum.y += ex2_approx(x.y - l);
        sum.z += ex2_approx(x.z - l);
        sum.w += ex2_approx(x.w - l);
    }
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
    const size_t at = (size_t)bh * p.Nk + key;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (key + k < p.Nk)
            p.w_out[at + k] = (p.w_in ? p.w_in[at + k] : 0.f) + v[k];
}

}  // namespace fa
