// What the kernels of second moments from captures held in few bits share (not installed).
#pragma once

#include <algorithm>

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

// the splits' sums of the blocks that a launch has split (fp64), into A; `name` is the launch timer's
hipError_t launch_moment_reduce(const char *name, const MomentArgs &a, const MomentTable &t, int64_t blocks, hipStream_t s);

// The plan that run(workgroups, units), an estimate in us, makes fastest for blocks of nwg workgroups each: all blocks
// whole, those of whole rounds over the chip's slots whole and the rest split along their units of tokens, or all of
// them split (`some` false: all or none); at most `most` units in one go, `partial` us for a split's sums, and 5 us for the launch that adds them up.
template <class Run>
MomentPlan moment_plan(int64_t blocks, int64_t nwg, int64_t slots, int64_t units, int64_t most, double partial, Run run,
                       bool some = true) {
    const int64_t least = (units + most - 1) / most;
    MomentPlan best{0, 1};
    double cost = 1e300;
    const int64_t full = blocks * nwg / slots * slots / nwg;
    for (const int64_t whole : {blocks, full, (int64_t)0}) {
        if (whole > 0 && (least > 1 || (!some && whole < blocks))) continue;
        const int64_t rest = blocks - whole;
        for (int64_t ns = least; ns <= units && ns <= least + 63; ++ns) {
            const int64_t per = (units + ns - 1) / ns;
            if ((units + per - 1) / per != ns) continue;
            const double c = run(whole * nwg, units) + (rest ? run(rest * nwg * ns, per) : 0.0) +
                             (rest && ns > 1 ? 5.0 + partial * (double)(rest * ns) : 0.0);
            if (c < cost) { best = rest && ns > 1 ? MomentPlan{(int)whole, (int)ns} : MomentPlan{(int)blocks, 1}; cost = c; }
        }
    }
    if (cost == 1e300) {                                   // no even count of splits in the range
        const int64_t per = (units + least - 1) / least;
        best = {0, (int)((units + per - 1) / per)};
    }
    return best;
}

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

// What is left of a block of F fragments after four waves have summed a quarter of its tokens each: their sums of the
// PAIRS fragment pairs on or below the diagonal added up and stored.
template <int F>
struct PairSums {
    static constexpr int PAIRS = F * (F + 1) / 2;
    static constexpr int PH = PAIRS > 6 ? 5 : PAIRS;   // pairs that are added up at a time
    f32x4 sm[PH][3][4][64];                     // accumulators on their way from wave to wave, lane to lane
};
template <int F>
__device__ __forceinline__ void finish_pairs(const f32x16 (&acc)[F * (F + 1) / 2], PairSums<F> &lds, float *out, int nb, bool part,
                                             double beta, double scale) {
    constexpr int PAIRS = PairSums<F>::PAIRS, PH = PairSums<F>::PH;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    auto &sm = lds.sm;
    // Pair p ends up with wave p % 4: the others hand it their sums through LDS, and it adds them in
    // the order of the waves behind it and stores the pair.
    constexpr int OWN = (PAIRS + 3) / 4;        // pairs wave, wave + 4, ..
    int fi[OWN], fj[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        fi[o] = 0;
        fj[o] = 4 * o + wave;
        while (fj[o] > fi[o]) fj[o] -= ++fi[o];
    }
    const bool old = !part && beta > 0.0;
    float av[2][16];
    f32x16 own[OWN];
#pragma unroll
    for (int h = 0; h < PAIRS; h += PH) {
        if (h > 0) __syncthreads();
#pragma unroll
        for (int p = h; p < h + PH && p < PAIRS; ++p)
            if (wave != p % 4)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sm[p - h][(wave + 3 - p) & 3][k][lane] = f32x4{acc[p][4 * k], acc[p][4 * k + 1], acc[p][4 * k + 2], acc[p][4 * k + 3]};
        __syncthreads();
#pragma unroll
        for (int p = h; p < h + PH && p < PAIRS; ++p)
            if (wave == p % 4) {
                f32x4 x[3][4];
#pragma unroll
                for (int s = 0; s < 3; ++s)
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[s][k] = sm[p - h][s][k][lane];
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    own[p / 4][r] = ((acc[p][r] + x[0][r >> 2][r & 3]) + x[1][r >> 2][r & 3]) + x[2][r >> 2][r & 3];
            }
    }
#pragma unroll
    for (int o = 0; o < OWN; ++o) {             // the old entries of the next pair read before the stores of this one
        if (old && o == 0) read_pair(out, nb, 32 * fi[0], 32 * fj[0], av[0]);
        if (old && o + 1 < OWN) read_pair(out, nb, 32 * fi[o + 1], 32 * fj[o + 1], av[(o + 1) & 1]);
        batch();
        if (4 * o + wave < PAIRS) store_pair(out, nb, 32 * fi[o], 32 * fj[o], own[o], av[o & 1], part, beta, scale);
        batch();
    }
}

}  // namespace dobb
