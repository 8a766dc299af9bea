// decode_stream.cuh -- split-KV forward for few query rows per kv head (R = G * Nq <= 16) over
// lists of keys: a window with sinks, a padded or paged cache with a length per sequence, a shared
// prefix followed by own keys.  The recurrence and the warp MMAs are those of the split pass in
// decode.cuh; what differs is how the work is cut.
//
// Each (batch, kv head) is a unit: a list of 64-key tiles that hold at least one visible key.  All
// units form one line, a place per tile and two more per unit (what ending one costs in tiles), T
// places long, and CTA c of G takes the places [c T / G, (c + 1) T / G): as much work as any other,
// whatever the lengths.  Its TMA warp runs through
// them without a pause, into the next unit while the other warps still end the last one, so the
// loads in flight (three stages of 32 KB, two CTAs per SM) never drain at a unit's end.  The pass is
// bound by HBM, and short lists (a window of 1024 keys is 17 tiles) would otherwise spend a third of
// their time starting and ending CTAs.
//
// 64 sequences, 8 kv heads, d = 128, a window of 1024 keys and 4 sinks: 53 us (dense cache) and 57 us
// (pages of 64) for 258 MB visible, 5.7 TB/s once running; 16 sequences with all 8192 keys: 88 us, 6.1 TB/s.
//
// A unit within one CTA is written out straight away.  A unit that continues in other CTAs leaves a
// partial (O_s normalised, lse_s, fp32) in each: in the CTA's slot 1 where the CTA starts the unit, in
// its slot 0 where it goes on with one, so two slots per CTA are enough.  Which CTAs hold a unit
// follows from T, G and the unit's first place, and stream_combine_kernel merges them in order.
#pragma once

#include "bwd.cuh"   // bulk_load
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
    int* first;             // [B + 1] places of the sequences before b, per kv head (with lengths)
    const int* seq_lens;    // [B] or nullptr (Nk each)
    const int* block_table; // [B, max_pages] (kListPaged)
    int B, Hq, Hkv, Nq, Nk, G, R, d_io;
    int causal;
    int window, sinks;
    int sink_rows;          // rows loaded of the last tile of sinks: sinks % 64 rounded up to 8, or 64
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
    static constexpr int kOffQ = kOffML + 2 * 64 * 4;                     // query rows of the next units
    static constexpr int kQBytes = 16 * 128 * 2;
    static constexpr int kQSlots = 4;                                     // at most (fewer where rows are many)
    static constexpr int kOffBar = kOffQ + kQBytes;
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

// Places of a unit with n tiles: a unit's end (the warps' merge, its stores, the next unit's start)
// takes about as long as two tiles.
constexpr int kUnitPlaces = 2;
__host__ __device__ __forceinline__ int stream_places(int n) { return n > 0 ? n + kUnitPlaces : 0; }

// The CTA that holds place t of T, and CTA c's first place.  Where the lengths leave fewer places than
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

// A CTA's walk along its part of the line: `left` places from place `off` of the unit (b, hk) on.
template <int LIST>
struct StreamWalk {
    int b, hk, off, left;
    StreamList l;
    // the unit's tiles in the part: [off, end())
    __device__ __forceinline__ int end() const { return min(l.tiles, off + left); }
    // on to the next unit with tiles; false at the part's end
    __device__ __forceinline__ bool next(const StreamParams& p)
    {
        left -= stream_places(l.tiles) - off;
        off = 0;
        if (left <= 0)
            return false;
        if (++hk < p.Hkv)
            return true;
        hk = 0;
        do {
            if (++b >= p.B)
                return false;
            l = stream_list<LIST>(p, stream_len(p, b));
        } while (l.tiles == 0);
        return true;
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
    uint64_t* bar_qfree = bar_empty + C::kStages + 1;   // [kQSlots] a unit's query rows are in registers (count 4)
    int* start = reinterpret_cast<int*>(bar_qfree + C::kQSlots);   // [3] b, hk, t of the CTA's first tile
    int* warp_sum = start + 3;                            // [4] tiles of the sequences of each warp's threads

    const int warp = warp_id(), lane = lane_id();
    const int cta = (int)blockIdx.x, grid = (int)gridDim.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], 4);
        }
        for (int s = 0; s < C::kQSlots; ++s)
            mbar_init(&bar_qfree[s], 4);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 128) {
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    // the line's length and the CTA's part of it
    long long total;
    StreamWalk<LIST> at;
    if (p.seq_lens == nullptr) {
        at.l = stream_list<LIST>(p, p.Nk);
        const int n = stream_places(at.l.tiles);
        total = (long long)n * p.B * p.Hkv;
        const long long t0 = stream_tile(cta, total, grid);
        const int unit = (int)(t0 / n);
        at.b = unit / p.Hkv;
        at.hk = unit % p.Hkv;
        at.off = (int)(t0 % n);
        __syncthreads();
    } else {
        // thread i of the first 128 takes a share of the sequences (their places in registers where it
        // has at most 4)
        const int per = (p.B + 127) / 128;
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        int mine = 0, before = 0, n4[4] = {0, 0, 0, 0};
        if (warp < 4) {
            if (per <= 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (b0 + k < b1)
                        n4[k] = stream_places(stream_list<LIST>(p, stream_len(p, b0 + k)).tiles);
                mine = n4[0] + n4[1] + n4[2] + n4[3];
            } else {
                for (int b = b0; b < b1; ++b)
                    mine += stream_places(stream_list<LIST>(p, stream_len(p, b)).tiles);
            }
            before = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, before, off);
                if (lane >= off)
                    before += x;
            }
            if (lane == 31)
                warp_sum[warp] = before;
            before -= mine;
        }
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            before += k < warp ? warp_sum[k] : 0;
            all += warp_sum[k];
        }
        total = (long long)all * p.Hkv;
        const long long t0 = stream_tile(cta, total, grid);
        if (warp < 4) {
            for (int b = b0; b < b1; ++b) {
                const int n = per <= 4 ? n4[0] : stream_places(stream_list<LIST>(p, stream_len(p, b)).tiles);
                n4[0] = n4[1];
                n4[1] = n4[2];
                n4[2] = n4[3];
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
                p.first[p.B] = all;
        }
        __syncthreads();
        at.b = start[0];
        at.hk = start[1];
        at.off = start[2];
        if (t0 < total)
            at.l = stream_list<LIST>(p, stream_len(p, at.b));
    }
    at.left = (int)(stream_tile(cta + 1, total, grid) - stream_tile(cta, total, grid));
    const bool any = at.left > 0;

    // slots for the units' query rows, so that the loads run ahead over units of a tile or two
    const int q_bytes = p.R * d_io * 2;
    const int q_slots = q_bytes * 4 <= C::kQBytes ? 4 : q_bytes * 2 <= C::kQBytes ? 2 : 1;

    if (warp == 4) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            const bool two = d_io > 64;   // the second 64-column panel only when the head has columns there
            const uint32_t row_bytes = (two ? 4u : 2u) * 128u;   // a key's K and V in a stage
            int n = 0, units = 0;
            bool go = any;
            while (go) {
                const int t0 = at.off, t1 = at.end();
                for (int t = t0; go && t < t1; ++t, ++n) {
                    const int slot = n % C::kStages;
                    go = mbar_wait(&bar_empty[slot], ((uint32_t)(n / C::kStages) & 1u) ^ 1u, abort_flag);
                    // the unit's query rows come with its first tile
                    if (go && t == t0)
                        go = mbar_wait(&bar_qfree[units % q_slots], ((uint32_t)(units / q_slots) & 1u) ^ 1u, abort_flag);
                    if (!go)
                        break;
                    uint8_t* dk = smem + slot * 2 * DecCfg::kTileBytes;
                    uint8_t* dv = dk + DecCfg::kTileBytes;
                    // the last tile of sinks, where the window has no key in it: only the sinks' rows
                    const bool few = (LIST == kListWindow || LIST == kListPaged) && t == at.l.seg - 1 && at.l.win_lo >= at.l.seg * kt;
                    mbar_arrive_expect_tx(&bar_full[slot],
                                          row_bytes * (uint32_t)(few ? p.sink_rows : kt) + (t == t0 ? (uint32_t)q_bytes : 0u));
                    if (t == t0) {
                        bulk_load(smem + C::kOffQ + (units % q_slots) * q_bytes,
                                  static_cast<const T*>(p.q) + (size_t)(at.b * p.Hkv + at.hk) * p.R * d_io, (uint32_t)q_bytes,
                                  &bar_full[slot]);
                        ++units;
                    }
                    const bool head_seg = t < at.l.seg;
                    const int key0 = head_seg ? t * kt : at.l.base + (t - at.l.seg) * kt;
                    if constexpr (LIST == kListPaged) {
                        // an out-of-range page id reads zeros (TMA bounds), never another buffer
                        const int page = __ldg(p.block_table + (size_t)at.b * p.max_pages + key0 / p.page_size);
                        const int off = key0 % p.page_size;
                        const CUtensorMap* mk = few ? &tmK0 : &tmK;
                        const CUtensorMap* mv = few ? &tmV0 : &tmV;
                        for (int pn = 0; pn < (two ? 2 : 1); ++pn) {
                            tma_load_4d(dk + pn * DecCfg::kPanelBytes, mk, &bar_full[slot], pn * 64, at.hk, off, page);
                            tma_load_4d(dv + pn * DecCfg::kPanelBytes, mv, &bar_full[slot], pn * 64, at.hk, off, page);
                        }
                    } else {
                        const bool pre = LIST == kListCat && head_seg;
                        const CUtensorMap* mk = pre || few ? &tmK0 : &tmK;
                        const CUtensorMap* mv = pre || few ? &tmV0 : &tmV;
                        const int head = pre ? at.hk : at.b * p.Hkv + at.hk;
                        for (int pn = 0; pn < (two ? 2 : 1); ++pn) {
                            tma_load_3d(dk + pn * DecCfg::kPanelBytes, mk, &bar_full[slot], pn * 64, key0, head);
                            tma_load_3d(dv + pn * DecCfg::kPanelBytes, mv, &bar_full[slot], pn * 64, key0, head);
                        }
                    }
                }
                go = go && at.next(p);
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
    int n = 0, units = 0;   // tiles and units taken so far
    bool ok = true;
    for (bool go = any; go; go = at.next(p)) {
        const int unit = at.b * p.Hkv + at.hk, t_first = at.off, t_end = at.end();
        if (t_first >= t_end)   // only places behind the unit's tiles
            continue;
        // the unit's query rows (row r is head hk * G + r / Nq, query r % Nq), landed with its first tile
        ok = mbar_wait(&bar_full[n % C::kStages], (uint32_t)(n / C::kStages) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        uint32_t qa[8][4];
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
                const int r = g + 8 * hr;
                qa[ks][hr] = qa[ks][hr + 2] = 0u;
                if (r < p.R && ks * 16 < d_io) {
                    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(smem + C::kOffQ + (units % q_slots) * q_bytes) + r * (d_io / 2);
                    qa[ks][hr] = qrow[ks * 8 + tq];          // cols 16 ks + 2 tq, + 1
                    qa[ks][hr + 2] = qrow[ks * 8 + 4 + tq];  // cols 16 ks + 8 + 2 tq, + 1
                }
            }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&bar_qfree[units % q_slots]);
        ++units;
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

        for (int t = t_first; ok && t < t_end; ++t, ++n) {
            const int slot = n % C::kStages;
            ok = mbar_wait(&bar_full[slot], (uint32_t)(n / C::kStages) & 1u, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                break;
            uint8_t* tile = smem + slot * 2 * DecCfg::kTileBytes;
            const uint32_t kbase = smem_u32(tile), vbase = kbase + DecCfg::kTileBytes;
            const int key_w = warp * 16;   // this warp's 16 keys within the tile
            const bool head_seg = t < at.l.seg;
            const int key0 = (head_seg ? t * kt : at.l.base + (t - at.l.seg) * kt) + key_w;

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
            // V of keys that no row sees (between the sinks and the window, where the stage may hold an
            // older tile's rows; past the sequence, in its last page or in the padding) is cleared in the operand registers: whatever is there,
            // 0 * V adds nothing.  A thread's operand words hold keys 2 tq, 2 tq + 1 (keep[0]) and 8
            // further on (keep[1]) of the warp's 16.
            uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
            bool clear = false;
            if (!in_prefix) {
                constexpr bool kWin = LIST == kListWindow || LIST == kListPaged;
                const int len = at.l.len, win_lo = at.l.win_lo;
                clear = key0 + 16 > len || (kWin && key0 < win_lo && key0 + 16 > p.sinks);
                if (clear) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + 8 * (e >> 1) + 2 * tq + (e & 1);
                        if (key >= len || (kWin && key >= p.sinks && key < win_lo))
                            keep[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
                    }
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
                    if (clear) {
                        b0 &= keep[0];
                        b1 &= keep[1];
                        b2 &= keep[0];
                        b3 &= keep[1];
                    }
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
        const bool whole = t_first == 0 && t_end == at.l.tiles;
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
            // a row per warp, four columns per lane
            const int r = r0 + warp, col = lane * 4;
            if (r >= p.R)
                continue;
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w)
                M = fmaxf(M, sm_m[w * 16 + r]);
            const float base = M == -INFINITY ? 0.f : M;   // a row without keys: l = 0, o = 0
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float sc = ex2_approx(sm_m[w * 16 + r] - base);
                const float4 x = *reinterpret_cast<const float4*>(sm_o + (w * C::kMergeRows + warp) * 128 + col);
                L = fmaf(sm_l[w * 16 + r], sc, L);
                acc.x = fmaf(x.x, sc, acc.x);
                acc.y = fmaf(x.y, sc, acc.y);
                acc.z = fmaf(x.z, sc, acc.z);
                acc.w = fmaf(x.w, sc, acc.w);
            }
            // 0 and -inf only for a row without keys; a NaN L stays one, in a partial too
            const float inv = L == 0.f ? 0.f : __frcp_rn(L);
            const float lse = L == 0.f ? -INFINITY : M + __log2f(L);
            if (whole && !p.partial) {
                const size_t row = (size_t)unit * p.R + r;
                if (col < d_io)
                    *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + row * d_io + col) =
                        make_uint2(Elt<T>::pack(acc.x * inv, acc.y * inv), Elt<T>::pack(acc.z * inv, acc.w * inv));
                if (lane == 0 && p.lse)
                    p.lse[row] = lse * 0.69314718055994530942f;
            } else {
                const size_t slot = whole ? 2 * (size_t)grid + unit : 2 * (size_t)cta + (t_first == 0 ? 1 : 0);
                *reinterpret_cast<float4*>(p.part_o + (slot * p.R + r) * 128 + col) =
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                if (lane == 0)
                    p.part_lse[slot * p.R + r] = lse;
            }
        }
    }
    if (p.after)
        griddep_wait();
}

// The parts of a unit that the pass has left.
struct StreamParts {
    const float* o;       // [slots][R][128]
    const float* lse;     // [slots][R], log2 units
    const int* first;     // [B + 1] or nullptr (tiles each)
    int tiles, B, Hkv, R, grid;   // tiles: of each unit (without lengths)
    // number of parts, and the CTA of the first; part i is in slot(unit, c0, n, i)
    __device__ __forceinline__ int count(int unit, int& c0) const
    {
        long long base, n, total;   // in places
        if (first) {
            const int b = unit / Hkv, f = first[b];
            n = first[b + 1] - f;
            base = (long long)f * Hkv + (unit % Hkv) * n;
            total = (long long)first[B] * Hkv;
        } else {
            n = stream_places(tiles);
            base = (long long)unit * n;
            total = (long long)B * Hkv * n;
        }
        c0 = 0;
        if (n == 0)
            return 0;
        c0 = stream_cta(base, total, grid);
        return stream_cta(base + n - kUnitPlaces - 1, total, grid) - c0 + 1;   // up to its last tile
    }
    __device__ __forceinline__ size_t slot(int unit, int c0, int n, int i) const
    {
        return n == 1 ? 2 * (size_t)grid + unit : 2 * (size_t)(c0 + i) + (i == 0 ? 1 : 0);
    }
};

// Adds up to AT_ONCE parts' rows at a time, their loads in flight together: part i has its row at
// row_of(i) (of both o and lse), lane l columns 4 l .. 4 l + 3.  Returns the running (M, L, acc).  A part
// whose lse is NaN makes L NaN (M leaves it out).
struct MergeState {
    float M, L;
    float4 acc;
};

template <int AT_ONCE, typename F>
__device__ __forceinline__ void merge_parts(MergeState& st, const float* o, const float* lse, int ld, int n, bool cols, F row_of)
{
    const int lane = lane_id();
    for (int i0 = 0; i0 < n; i0 += AT_ONCE) {
        float ls[AT_ONCE];
        float4 v[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            ls[k] = -INFINITY;
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + k < n) {
                const size_t at = row_of(i0 + k);
                ls[k] = lse[at];
                if (cols)
                    v[k] = *reinterpret_cast<const float4*>(o + at * ld + lane * 4);
            }
        }
        float M = st.M;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            M = fmaxf(M, ls[k]);
        const float base = M == -INFINITY ? 0.f : M;   // no part with a number yet
        const float a = ex2_approx(st.M - base);
        st.M = M;
        st.L *= a;
        st.acc.x *= a;
        st.acc.y *= a;
        st.acc.z *= a;
        st.acc.w *= a;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (ls[k] == -INFINITY)   // no key there: its row may never have been written
                continue;
            const float w = ex2_approx(ls[k] - base);
            st.L += w;
            st.acc.x = fmaf(w, v[k].x, st.acc.x);
            st.acc.y = fmaf(w, v[k].y, st.acc.y);
            st.acc.z = fmaf(w, v[k].z, st.acc.z);
            st.acc.w = fmaf(w, v[k].w, st.acc.w);
        }
    }
}

template <typename T>
__device__ __forceinline__ void merge_store(const MergeState& st, T* o, float* lse, size_t row, int d_io, int col)
{
    const float inv = st.L == 0.f ? 0.f : 1.f / st.L;
    if (col < d_io)
        *reinterpret_cast<uint2*>(o + row * d_io + col) = make_uint2(Elt<T>::pack(st.acc.x * inv, st.acc.y * inv),
                                                                    Elt<T>::pack(st.acc.z * inv, st.acc.w * inv));
    if (col == 0 && lse)
        lse[row] = st.L == 0.f ? -INFINITY : (st.M + __log2f(st.L)) * 0.69314718055994530942f;
}

// One warp per row: the parts of units cut between CTAs; rows of units within one CTA are final,
// and rows of a sequence without keys get O = 0, LSE = -inf.
template <typename T>
__device__ __forceinline__ void stream_combine_rows(const StreamParts& p, T* o_out, float* lse_out, int d_io, int block)
{
    const int row = block * 4 + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= p.B * p.Hkv * p.R)
        return;
    const int unit = row / p.R, r = row % p.R;
    int c0;
    const int n = p.count(unit, c0);
    if (n == 1)
        return;
    MergeState st{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    merge_parts<8>(st, p.o, p.lse, 128, n, lane * 4 < d_io, [&](int i) { return p.slot(unit, c0, n, i) * p.R + r; });
    merge_store(st, o_out, lse_out, (size_t)row, d_io, lane * 4);
}

template <typename T>
__global__ void __launch_bounds__(128) stream_combine_kernel(StreamParts p, void* o_out, float* lse_out, int d_io)
{
    griddep_launch_dependents();
    griddep_wait();
    stream_combine_rows(p, static_cast<T*>(o_out), lse_out, d_io, (int)blockIdx.x);
}

// The weights that the keys receive, from the scores that the pass has left and the rows' LSE:
// thread i takes four keys of a (batch, kv head).  Bound by reading the scores (mostly in L2).  The
// blocks after the keys' merge the units that are cut between CTAs, so that neither waits for the
// other: a keys' block takes the LSE of such a unit from its parts.
struct DecodeWeightParams {
    const float* scores;    // [BH, R, stride]: log2 units, -inf where masked
    float* lse;             // [BH, R]: final for units within one CTA, written by the merge for the others
    const float* w_in;      // [BH, Nk] or nullptr (zeros)
    float* w_out;
    void* o;
    int BH, R, Nk, stride, d_io;
    int key_blocks;         // BH * ceil(Nk / 512)
    StreamParts parts;
};

template <typename T>
__global__ void __launch_bounds__(128) decode_weights_kernel(DecodeWeightParams p)
{
    __shared__ float s_lse[16];
    griddep_wait();
    if ((int)blockIdx.x >= p.key_blocks) {
        stream_combine_rows(p.parts, static_cast<T*>(p.o), p.lse, p.d_io, (int)blockIdx.x - p.key_blocks);
        return;
    }
    const int chunks = (p.Nk + 511) / 512;
    const int bh = (int)blockIdx.x / chunks, key = ((int)blockIdx.x % chunks) * 512 + (int)threadIdx.x * 4;
    if ((int)threadIdx.x < p.R) {
        const int r = (int)threadIdx.x;
        int c0;
        const int n = p.parts.count(bh, c0);
        float l;   // log2 units
        if (n == 1) {
            l = p.lse[(size_t)bh * p.R + r] * 1.4426950408889634f;
        } else {
            float M = -INFINITY, L = 0.f;
            for (int i = 0; i < n; ++i)
                M = fmaxf(M, p.parts.lse[p.parts.slot(bh, c0, n, i) * p.R + r]);
            const float base = M == -INFINITY ? 0.f : M;
            for (int i = 0; i < n; ++i)
                L += ex2_approx(p.parts.lse[p.parts.slot(bh, c0, n, i) * p.R + r] - base);
            l = L == 0.f ? -INFINITY : M + __log2f(L);
        }
        s_lse[r] = l == -INFINITY ? INFINITY : l;   // P = 0 in a row without keys
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
        // a masked key gets nothing, of a row whose LSE is NaN neither
        sum.x += x.x == -INFINITY ? 0.f : ex2_approx(x.x - l);
        sum.y += x.y == -INFINITY ? 0.f : ex2_approx(x.y - l);
        sum.z += x.z == -INFINITY ? 0.f : ex2_approx(x.z - l);
        sum.w += x.w == -INFINITY ? 0.f : ex2_approx(x.w - l);
    }
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
    const size_t at = (size_t)bh * p.Nk + key;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (key + k < p.Nk)
            p.w_out[at + k] = (p.w_in ? p.w_in[at + k] : 0.f) + v[k];
}

}  // namespace fa
