// What the kernels of second moments from captures held in few bits share (not installed).
#pragma once

#include "ops_internal.h"

namespace dobb {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

struct MomentTable {
    const i32x4 *codes[kMomentMats];
    const uint32_t *scales[kMomentMats];
    float *A[kMomentMats];
    int32_t n[kMomentMats];
    int32_t first[kMomentMats + 1];            // first block of each matrix
};

inline MomentTable moment_table(const MomentArgs &a, int64_t *blocks) {
    MomentTable t{};
    *blocks = 0;
    for (int i = 0; i < a.count; ++i) {
        t.codes[i] = (const i32x4 *)a.codes[i];
        t.scales[i] = (const uint32_t *)a.scales[i];
        t.A[i] = a.A[i];
        t.n[i] = (int32_t)a.n[i];
        t.first[i] = (int32_t)*blocks;
        *blocks += a.n[i] / a.nb;
    }
    t.first[a.count] = (int32_t)*blocks;
    return t;
}

// the splits' sums of the blocks that a launch has split (fp64), into A
hipError_t launch_moment_reduce(const MomentArgs &a, const MomentTable &t, int64_t blocks, hipStream_t s);

// beta A + (1 - beta)/N times the sum, rounded to fp32 once
__device__ __forceinline__ float moment_out(double beta, double scale, float A, double sum) {
    return (float)(beta > 0.0 ? beta * (double)A + scale * sum : scale * sum);
}

__device__ __forceinline__ int find_matrix(const MomentTable &t, int cnt, int blk) {
    int lo = 0, hi = cnt;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= blk) lo = mid; else hi = mid;
    }
    return lo;
}

// Loads before it are all issued before anything behind it: the compiler otherwise tends to wait for
// each load of a batch in turn, a memory latency apiece.
__device__ __forceinline__ void batch() { __builtin_amdgcn_sched_barrier(0); }

constexpr int kPairPad = 33;                   // row pitch of a 32x32 pair in LDS: rows and columns are read
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// One wave: a finished 32 x 32 pair at rows i0 and columns j0 of a block, in the accumulators' layout.
// read_pair takes its old entries of A; store_pair writes a split's partial sums as rows of the lower
// triangle, or the new entries of A as rows of the lower triangle and of the upper one, straight from the
// registers: a lane's four consecutive rows are 16 contiguous bytes of the mirrored row.  A load that
// follows a store waits for it (both count in order), so callers read for several pairs before they store
// the first: pair by pair, an exchange with memory each, the stores were most of a short call.
// (a block has at most 2^20 entries: 32-bit offsets from a scalar address)
__device__ __forceinline__ float *at(const float *base, int e) { return (float *)((char *)base + (uint32_t)e * 4u); }

__device__ __forceinline__ void read_pair(const float *out, int nb, int i0, int j0, float (&av)[16]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int i = min(i0 + acc_row(r, lane), nb - 1), j = min(j0 + (lane & 31), i);   // no branches
        av[r] = *at(out, i * nb + j);
    }
}

__device__ __forceinline__ void store_pair(float *out, int nb, int i0, int j0, const f32x16 &sum, const float (&av)[16], bool part,
                                           double beta, double scale) {
    const int lane = threadIdx.x & 63, j = j0 + (lane & 31);
    const bool inside = i0 + 32 <= nb && j0 < i0;                     // no bounds needed
    const int low = i0 * nb + j;                                      // + acc_row * nb: the pair's entries
    const int up = j * nb + i0 + 4 * (lane >> 5);                     // + 8 k: their mirrored ones, by fours
    if (part) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (inside || (i0 + acc_row(r, lane) < nb && j <= i0 + acc_row(r, lane))) *at(out, low + acc_row(r, lane) * nb) = sum[r];
        return;
    }
    float w[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) w[r] = moment_out(beta, scale, av[r], (double)sum[r]);
    if (inside) {
#pragma unroll
        for (int r = 0; r < 16; ++r) *at(out, low + acc_row(r, lane) * nb) = w[r];
#pragma unroll
        for (int k = 0; k < 4; ++k) *(f32x4u *)at(out, up + 8 * k) = f32x4u{w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]};
        return;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int i = i0 + acc_row(r, lane);
        if (i < nb && j <= i) *at(out, low + acc_row(r, lane) * nb) = w[r];
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int i = i0 + acc_row(r, lane);
        if (i < nb && j < i) *at(out, up + 8 * (r >> 2) + (r & 3)) = w[r];
    }
}

// Blocks 0 .. whole - 1 of a launch take their tokens in one go, the others in nsplit splits; nwg
// workgroups each.  The first kind come first.
struct Place {
    int blk, split, nsplit, wg;
};
__device__ __forceinline__ Place place(int whole, int nsplit, int nwg) {
    const int w = whole * nwg;
    Place p;
    if ((int)blockIdx.x < w) {
        const int id = xcd_remap(blockIdx.x, w);
        p.wg = id % nwg; p.blk = id / nwg; p.split = 0; p.nsplit = 1;
    } else {
        int id = xcd_remap(blockIdx.x - w, gridDim.x - w);
        p.wg = id % nwg; id /= nwg;
        p.split = id % nsplit; p.blk = whole + id / nsplit; p.nsplit = nsplit;
    }
    return p;
}

}  // namespace dobb
