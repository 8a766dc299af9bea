// prefix.cuh -- merge of a shared prefix's partials with those of the sequences' own keys.
//
// Where several sequences' rows fit a tile, their prefix is one tiled pass over the prefix's keys
// (fwd_kernel with kFwdPack: read and multiplied once for all of them) and the own keys are a second
// pass.  Both leave fp32 partials, merged here by the rescale-and-add of the online softmax (page
// "FlashAttention：为什么少搬数据，反而算得更快", §04).
// Bound by the latency of the parts' loads (17 parts of 512 bytes a row at 64 sequences on 8192 keys:
// 18 MB in 6 us, mostly from L2), so eight are in flight.
#pragma once

#include "decode_stream.cuh"
#include "fwd.cuh"

namespace fa {

struct PrefixMerge {
    const float* a_o;      // prefix: [na][rows][d_io]
    const float* a_lse;    // [na][rows], log2 units
    StreamParts own;       // own keys: what the split-KV pass left, or (tiled) one part per row, in row order
    int tiled, b_ld;       // floats per row of own.o
    int na, d_io;
    long long rows;
    void* o;
    float* lse;
};

// One warp per query row and 128 columns.
template <typename T>
__global__ void __launch_bounds__(128) prefix_merge_kernel(PrefixMerge p)
{
    const int per = (p.d_io + 127) / 128;   // warps per row
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const long long row = w / per;
    const int c = (int)(w % per) * 128, lane = threadIdx.x & 31;
    griddep_wait();
    if (row >= p.rows)
        return;
    const int unit = (int)(row / p.own.R), r = (int)(row % p.own.R);
    const bool cols = c + lane * 4 < p.d_io;
    MergeState st{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    merge_parts<8>(st, p.a_o + c, p.a_lse, p.d_io, p.na, cols, [&](int i) { return (size_t)i * p.rows + row; });
    if (p.tiled) {
        merge_parts<1>(st, p.own.o + c, p.own.lse, p.b_ld, 1, cols, [&](int) { return (size_t)row; });
    } else {
        int c0;
        const int n = p.own.count(unit, c0);
        merge_parts<4>(st, p.own.o + c, p.own.lse, p.b_ld, n, cols, [&](int i) { return p.own.slot(unit, c0, n, i) * p.own.R + r; });
    }
    merge_store(st, static_cast<T*>(p.o), p.lse, (size_t)row, p.d_io, c + lane * 4);
}

// Merge of the key shares of a split windowed or prefix-and-own forward (as fwd_combine_kernel), one
// warp per query row and 128 columns, AT_ONCE shares' loads in flight together.
template <int AT_ONCE, typename T>
__global__ void __launch_bounds__(128) share_merge_kernel(FwdParams p)
{
    const int per = (p.d_io + 127) / 128;   // warps per row
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const long long row = w / per;
    const int c = (int)(w % per) * 128, lane = threadIdx.x & 31;
    griddep_wait();
    if (row >= (long long)p.n_bh * p.rows)
        return;
    const int bh = (int)(row / p.rows), i = (int)(row % p.rows);
    // rows of whole units are final
    if ((long long)(p.n_pairs - 1 - i / p.pair_rows) * p.n_bh + bh < p.full_tiles)
        return;
    const bool cols = c + lane * 4 < p.d_io;
    MergeState st{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    merge_parts<AT_ONCE>(st, p.part_o + c, p.part_lse, p.d_io, p.kv_split, cols,
                         [&](int s) { return ((size_t)bh * p.kv_split + s) * p.rows + i; });
    merge_store(st, static_cast<T*>(p.o), p.lse, (size_t)row, p.d_io, c + lane * 4);
}

}  // namespace fa
