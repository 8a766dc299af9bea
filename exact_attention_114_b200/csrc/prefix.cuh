// prefix.cuh -- merge of a shared prefix's partials with those of the sequences' own keys.
//
// Where several sequences' rows fit a tile, their prefix is one tiled pass over the prefix's keys
// (fwd_kernel with kFwdPack: read and multiplied once for all of them) and the own keys are a second
// pass.  Both leave fp32 partials, merged here by the rescale-and-add of the online softmax (page
// "FlashAttention：为什么少搬数据，反而算得更快", §04).
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

// One warp per query row; lane l holds the weight of part l, 32 parts at a time, then all lanes add
// the parts' rows.
template <typename T>
__global__ void __launch_bounds__(128) prefix_merge_kernel(PrefixMerge p)
{
    griddep_wait();
    const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= p.rows)
        return;
    const int unit = (int)(row / p.own.R), r = (int)(row % p.own.R);
    int c0 = 0;
    const int nb = p.tiled ? 1 : p.own.count(unit, c0);
    const int n = p.na + nb;
    // row of part s among the own parts' rows
    auto own_row = [&](int s) { return p.tiled ? (size_t)row : p.own.slot(unit, c0, nb, s - p.na) * p.own.R + r; };
    auto lse_of = [&](int s) { return s < p.na ? p.a_lse[s * p.rows + row] : p.own.lse[own_row(s)]; };
    float M = -INFINITY;
    for (int s = lane; s < n; s += 32)
        M = fmaxf(M, lse_of(s));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    // lane l merges columns [c l, c l + c), c = d_io / 32
    const int c = p.d_io / 32;
    float acc[8], L = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        acc[k] = 0.f;
    for (int s0 = 0; s0 < n && M != -INFINITY; s0 += 32) {
        const float wl = s0 + lane < n ? ex2_approx(lse_of(s0 + lane) - M) : 0.f;
#pragma unroll 4
        for (int s = s0; s < min(n, s0 + 32); ++s) {
            const float w = __shfl_sync(0xffffffffu, wl, s - s0);
            if (w == 0.f)   // no key there (its O was never written) or a negligible share
                continue;
            L += w;
            const float* o = (s < p.na ? p.a_o + (s * p.rows + row) * p.d_io : p.own.o + own_row(s) * p.b_ld) + c * lane;
            if (c == 4) {
                const float4 v = *reinterpret_cast<const float4*>(o);
                acc[0] = fmaf(w, v.x, acc[0]);
                acc[1] = fmaf(w, v.y, acc[1]);
                acc[2] = fmaf(w, v.z, acc[2]);
                acc[3] = fmaf(w, v.w, acc[3]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < c)
                        acc[k] = fmaf(w, o[k], acc[k]);
            }
        }
    }
    const float inv = (L > 0.f) ? 1.f / L : 0.f;
    T* o = static_cast<T*>(p.o) + row * p.d_io + c * lane;
    if (c == 4) {
        *reinterpret_cast<uint2*>(o) = make_uint2(Elt<T>::pack(acc[0] * inv, acc[1] * inv),
                                                  Elt<T>::pack(acc[2] * inv, acc[3] * inv));
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < c)
                o[k] = Elt<T>::from_float(acc[k] * inv);
    }
    if (lane == 0 && p.lse)
        p.lse[row] = (L > 0.f) ? (M + __log2f(L)) * kLn2 : -INFINITY;
}

}  // namespace fa
