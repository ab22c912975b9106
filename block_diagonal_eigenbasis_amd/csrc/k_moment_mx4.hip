// Second moments from captures in MXFP4:  A_b <- beta A_b + (1 - beta)/N sum_t x_t x_t^T  with the
// products on the scaled fp4 matrix instruction (mfma_scale_f32_32x32x64_f8f6f4).
//
// The capture's layout (dobb_ops.h) is the instruction's operand layout: 32 consecutive columns of one
// group are 512 contiguous bytes, one 16-byte piece a lane, and both sides of a product are the same
// kind of fragment.  The two half-waves of an instruction take the same group of two neighbouring token
// tiles (the order of the contraction is free as long as both sides agree): the scale bytes of a
// tile's four groups are then one 4-byte load for four instructions.  The unit of work along the tokens
// is such a pair of tiles, 256 tokens.
//
// k_moment_mx4_narrow (nb <= 128): a block's codes are read from HBM once, straight into operand
//   registers.  A workgroup owns one block; its four waves take every fourth tile pair, keep all
//   fragment pairs on or below the diagonal in registers and hand each other their sums through LDS at the
//   end.  Bound by HBM: 576 blocks of 100, 16384 tokens (501 MB of codes), in 110 us, 5.2 TB/s with A.
// k_moment_mx4_wide (128 < nb <= 1024): a workgroup of 8 waves stages the tile pair of a whole block
//   in LDS (through registers, one stage ahead) and each wave owns 2 x 4 of the fragment pairs on or
//   below the diagonal; a block with more than 8 such groups takes several workgroups, neighbours on one
//   XCD, so that its codes come from HBM once and from that XCD's L2 after that.  192 blocks of 400, 16384
//   tokens, in 280 us on average (254 at best); bound by the matrix cores' power: the clock falls to 1.8 GHz, and
//   codes that are all zero take a third less time.
// Rounding: fp32 sums of at most 4096 (narrow, then four of those in fp32) or 16384 tokens (wide) in
// the accumulators, token splits in fp64 (k_moment_mx4_reduce).  A product of two elements is a multiple of a
// quarter of their scales' product and at most 36 times it, so fp32 sums of them are exact unless a column's
// scales differ by large factors.  16384 tokens of sizes exp(0.3 N(0, 1)) and exp(N(0, 1)): every sum is exact;
// exp(2 N(0, 1)): the diagonal is off by 4.5e-8 (root mean square; 2.8e-7 at most).  Moving the diagonal entries
// into fp64 every four tile pairs made that 3.8e-8 (2.5e-7) and took 2 to 5 % more time: not done.
#include <algorithm>

#include "ops_internal.h"

namespace dobb {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kNarrow = 128;                   // widest block of the narrow kernel
constexpr int64_t kSplitPairs = 64;            // most tile pairs of one split: 16384 tokens

struct MomentTable {
    const i32x4 *codes[kMomentMats];
    const uint32_t *scales[kMomentMats];
    float *A[kMomentMats];
    int32_t n[kMomentMats];
    int32_t first[kMomentMats + 1];            // first block of each matrix
};

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

__device__ __forceinline__ i32x8 operand(const i32x4 &v) {
    return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}

// G: which byte of the scales, that is which group of the tiles
template <int G>
__device__ __forceinline__ f32x16 mfma_fp4(const i32x4 &a, const i32x4 &b, f32x16 c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, G, (int)sa, G, (int)sb);
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

// F = ceil(nb / 32) fragments; NT: the codes are read past the caches
template <int F, bool NT>
__global__ void __launch_bounds__(256, 2) k_moment_mx4_narrow(int cnt, int nb, int64_t tiles, int whole, int nsplit_, double beta,
                                                              double scale, float *partial, MomentTable t) {
    constexpr int PAIRS = F * (F + 1) / 2;
    constexpr int PH = PAIRS > 6 ? 5 : PAIRS;   // pairs that are added up at a time
    __shared__ f32x4 sm[PH][3][4][64];          // accumulators on their way from wave to wave, lane to lane
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    const Place pl = place(whole, nsplit_, 1);
    const int blk = pl.blk;
    const int mat = find_matrix(t, cnt, blk);
    const int64_t n = t.n[mat];
    const int64_t tp = (tiles + 1) / 2;
    const int64_t per = (tp + pl.nsplit - 1) / pl.nsplit;
    const int64_t p0 = per * pl.split, p1 = p0 + per < tp ? p0 + per : tp;
    const int64_t cb = (int64_t)(blk - t.first[mat]) * nb;
    const char *codes = (const char *)(t.codes[mat] + cb);
    const char *scales = (const char *)(t.scales[mat] + cb);
    // byte offsets of this lane's fragment columns (columns past the block repeat its last one: they fill
    // rows and columns that are not written) and of its half's tile
    uint32_t ci[F];
#pragma unroll
    for (int f = 0; f < F; ++f) ci[f] = (uint32_t)(32 * f + col < nb ? 32 * f + col : nb - 1) * 4;
    const uint32_t tile_b = half ? (uint32_t)(64 * n) : 0u;
    f32x16 acc[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) acc[p] = f32x16{};

    // A wave's operands are one tile pair ahead: once the products of a group are on their way, its
    // registers take the next pair's group, so loads are in flight all the time.
    uint32_t sa[F], sn[F];
    i32x4 a[4][F];
    const char *cp = nullptr;                   // of the pair that is being loaded
    uint32_t mine = 0;
    bool in = true;
    auto load_scales = [&](int64_t p) {
        const bool odd = 2 * p + 1 >= tiles;    // an odd last tile: the other half reads it too, and its
        in = !(odd && half);                    // scales become 2^-127, whose products vanish in fp32
        mine = odd ? 0u : tile_b;
        cp = codes + 2 * p * (64 * n);
        const char *sp = scales + 2 * p * (4 * n);
#pragma unroll
        for (int f = 0; f < F; ++f) sn[f] = *(const uint32_t *)(sp + (mine / 16 + ci[f]));
    };
    auto load_group = [&](int g) {
        const char *gp = cp + g * (16 * n);
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const i32x4 *x = (const i32x4 *)(gp + (mine + 4 * ci[f]));
            a[g][f] = NT ? __builtin_nontemporal_load(x) : *x;
        }
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int f = 0; f < F; ++f) sa[f] = in ? sn[f] : 0u;
    };
#define DOBB_MX4_GROUP(g, NEXT)                                                \
    {                                                                          \
        int q = 0;                                                             \
        _Pragma("unroll") for (int i = 0; i < F; ++i)                          \
            _Pragma("unroll") for (int j = 0; j <= i; ++j, ++q)                \
                acc[q] = mfma_fp4<g>(a[g][i], a[g][j], acc[q], sa[i], sa[j]);  \
        batch();                                                               \
        if (NEXT) load_group(g);                                               \
        batch();                                                               \
    }
    int64_t p = p0 + wave;
    if (p < p1) {
        load_scales(p);
#pragma unroll
        for (int g = 0; g < 4; ++g) load_group(g);
        batch();
        for (; p + 4 < p1; p += 4) {
            take_scales();
            load_scales(p + 4);
            DOBB_MX4_GROUP(0, true) DOBB_MX4_GROUP(1, true) DOBB_MX4_GROUP(2, true) DOBB_MX4_GROUP(3, true)
        }
        take_scales();
        DOBB_MX4_GROUP(0, false) DOBB_MX4_GROUP(1, false) DOBB_MX4_GROUP(2, false) DOBB_MX4_GROUP(3, false)
    }
#undef DOBB_MX4_GROUP

    // Pair p ends up with wave p % 4: the others hand it their sums through LDS, and it adds them in
    // the order of the waves behind it and stores the pair.
    const int64_t nbb = (int64_t)nb * nb;
    const bool part = pl.nsplit > 1;
    float *out = part ? partial + ((int64_t)(blk - whole) * pl.nsplit + pl.split) * nbb : t.A[mat] + (blk - t.first[mat]) * nbb;
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

// ---- wide ----------------------------------------------------------------------------------------
constexpr int kWideThreads = 512;
// 2 x 4 groups of fragment pairs with any on or below the diagonal
__host__ __device__ inline int wide_groups(int F) {
    int ng = 0;
    for (int i = 0; 2 * i < F; ++i) ng += ((2 * i + 2 < F ? 2 * i + 2 : F) + 3) / 4;
    return ng;
}

// GS groups of the tile pair a stage (4, or 2 where two stages of 4 would not fit the LDS: F > 16); PT 16-byte
// pieces of a stage a thread, ST scale words: what GS * 64 * F pieces and 64 * F words take
template <int GS, int PT>
__global__ void __launch_bounds__(kWideThreads, 2) k_moment_mx4_wide(int cnt, int nb, int F, int nwg, int64_t tiles, int whole,
                                                                     int nsplit_, double beta, double scale, float *partial, MomentTable t) {
    constexpr int ST = (PT * kWideThreads / GS + kWideThreads - 1) / kWideThreads;
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    const Place pl = place(whole, nsplit_, nwg);
    const int wg = pl.wg, blk = pl.blk;
    const int mat = find_matrix(t, cnt, blk);
    const int64_t n = t.n[mat];
    const int64_t tp = (tiles + 1) / 2;
    const int64_t per = (tp + pl.nsplit - 1) / pl.nsplit;
    const int64_t p0 = per * pl.split, p1 = p0 + per < tp ? p0 + per : tp;
    const int64_t cb = (int64_t)(blk - t.first[mat]) * nb;
    const char *codes = (const char *)(t.codes[mat] + cb);
    const uint32_t *scales = t.scales[mat] + cb;
    const int pieces = GS * 64 * F, words = 64 * F;       // of a stage: [group][half][column]
    const uint32_t stage = (uint32_t)pieces * 16 + (uint32_t)words * 4;

    // this thread's pieces: places in the stage (threads past the last piece repeat it: no branches),
    // byte offsets from the tile pair's first group, and which half they belong to
    uint32_t at[PT], off[PT], sat[ST], soff[ST], second = 0, ssecond = 0;
#pragma unroll
    for (int k = 0; k < PT; ++k) {
        const int e = min(k * kWideThreads + (int)threadIdx.x, pieces - 1);
        const int g = e / (64 * F), r = e - g * 64 * F;
        const int q = r >= 32 * F, c = r - q * 32 * F;
        at[k] = (uint32_t)e * 16;
        off[k] = (uint32_t)(((q * 4 + g) * n + (c < nb ? c : nb - 1)) * 16);
        second |= (uint32_t)q << k;
    }
#pragma unroll
    for (int k = 0; k < ST; ++k) {
        const int e = min(k * kWideThreads + (int)threadIdx.x, words - 1);
        const int q = e >= 32 * F, c = e - q * 32 * F;
        sat[k] = (uint32_t)pieces * 16 + (uint32_t)e * 4;
        soff[k] = (uint32_t)(q * n + (c < nb ? c : nb - 1)) * 4;
        ssecond |= (uint32_t)q << k;
    }
    i32x4 v[PT];
    uint32_t sv[ST];
    bool odd = false;                          // the second tile of the last pair is not there
    // stage s: groups GS * (s % (4 / GS)) on of tile pair p0 + s / (4 / GS)
    auto fetch = [&](int64_t s) {
        const int64_t p = p0 + s / (4 / GS);
        const int g0 = GS * (int)(s % (4 / GS));
        odd = 2 * p + 1 >= tiles;
        const char *cp = codes + (2 * p * 4 + g0) * n * 16;
        const char *sp = (const char *)(scales + 2 * p * n);
        const uint32_t back = odd ? (uint32_t)(64 * n) : 0u, sback = odd ? (uint32_t)(4 * n) : 0u;
#pragma unroll
        for (int k = 0; k < PT; ++k) v[k] = *(const i32x4 *)(cp + (off[k] - ((second >> k) & 1 ? back : 0u)));
#pragma unroll
        for (int k = 0; k < ST; ++k) sv[k] = *(const uint32_t *)(sp + (soff[k] - ((ssecond >> k) & 1 ? sback : 0u)));
    };
    auto store = [&](unsigned char *buf) {
#pragma unroll
        for (int k = 0; k < PT; ++k) *(i32x4 *)(buf + at[k]) = v[k];
#pragma unroll                                  // a missing tile's scales are 2^-127: its products vanish in fp32
        for (int k = 0; k < ST; ++k) *(uint32_t *)(buf + sat[k]) = odd && ((ssecond >> k) & 1) ? 0u : sv[k];
    };

    // this wave's group: rows 2 I, 2 I + 1 and columns 4 J .. 4 J + 3 of the fragments
    int I = -1, J = 0;
    {
        int left = wg * 8 + wave;
        for (int i = 0; 2 * i < F; ++i) {
            const int m = ((2 * i + 2 < F ? 2 * i + 2 : F) + 3) / 4;
            if (left < m) { I = i; J = left; break; }
            left -= m;
        }
    }
    uint32_t ra[2], rb[4];                                  // fragments' columns; past the last one: the last
#pragma unroll
    for (int i = 0; i < 2; ++i) ra[i] = (uint32_t)(min(2 * max(I, 0) + i, F - 1) * 32 + col + half * 32 * F);
#pragma unroll
    for (int j = 0; j < 4; ++j) rb[j] = (uint32_t)(min(4 * J + j, F - 1) * 32 + col + half * 32 * F);
    f32x16 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};

    // Stage s + 1 goes from registers to the other buffer, and stage s + 2 from memory to registers, after
    // the first group's products of stage s: the LDS takes the writes beside the other groups' products
    // and the loads have a whole stage to arrive.
    const int64_t stages = (p1 - p0) * (4 / GS);
    fetch(0);
    store(lds);
    if (stages > 1) fetch(1);
    __syncthreads();
    for (int64_t s = 0; s < stages; ++s) {
        unsigned char *cur = lds + (s & 1) * stage, *nxt = lds + ((s & 1) ^ 1) * stage;
        const i32x4 *cc = (const i32x4 *)cur;
        const uint32_t *cs = (const uint32_t *)(cur + (size_t)pieces * 16);
        uint32_t sa[2], sb[4];
        const int sh = GS == 4 ? 0 : 16 * (int)(s & 1);   // two groups a stage: the upper bytes second
#pragma unroll
        for (int i = 0; i < 2; ++i) sa[i] = cs[ra[i]] >> sh;
#pragma unroll
        for (int j = 0; j < 4; ++j) sb[j] = cs[rb[j]] >> sh;
#define DOBB_MX4_GROUP(g)                                                                              \
        if (g < GS && I >= 0) {                                                                        \
            i32x4 a[2], b[4];                                                                          \
            _Pragma("unroll") for (int i = 0; i < 2; ++i) a[i] = cc[g * 64 * F + ra[i]];               \
            _Pragma("unroll") for (int j = 0; j < 4; ++j) b[j] = cc[g * 64 * F + rb[j]];               \
            _Pragma("unroll") for (int i = 0; i < 2; ++i)                                              \
                _Pragma("unroll") for (int j = 0; j < 4; ++j)                                          \
                    acc[i][j] = mfma_fp4<g>(a[i], b[j], acc[i][j], sa[i], sb[j]);                      \
        }
        DOBB_MX4_GROUP(0)
        if (s + 1 < stages) store(nxt);
        if (s + 2 < stages) fetch(s + 2);
        DOBB_MX4_GROUP(1) DOBB_MX4_GROUP(2) DOBB_MX4_GROUP(3)
#undef DOBB_MX4_GROUP
        __syncthreads();
    }
    if (I < 0) return;
    const int64_t nbb = (int64_t)nb * nb;
    float av[2][16];
    if (pl.nsplit > 1) {
        float *out = partial + ((int64_t)(blk - whole) * pl.nsplit + pl.split) * nbb;
#define DOBB_MX4_STORE(p)                                                                                            \
        {                                                                                                            \
            const int i0 = 32 * (2 * I + ((p) >> 2)), j0 = 32 * (4 * J + ((p) & 3));                                  \
            if (i0 < nb && j0 <= i0) store_pair(out, nb, i0, j0, acc[(p) >> 2][(p) & 3], av[0], true, beta, scale);    \
        }
        DOBB_MX4_STORE(0) DOBB_MX4_STORE(1) DOBB_MX4_STORE(2) DOBB_MX4_STORE(3)
        DOBB_MX4_STORE(4) DOBB_MX4_STORE(5) DOBB_MX4_STORE(6) DOBB_MX4_STORE(7)
#undef DOBB_MX4_STORE
        return;
    }
    // pair by pair, the old entries of the next one read before the stores of this one
    float *out = t.A[mat] + (blk - t.first[mat]) * nbb;
    const bool old = beta > 0.0;
    if (old) read_pair(out, nb, 64 * I, 128 * J, av[0]);
#define DOBB_MX4_STORE(p)                                                                                            \
    {                                                                                                                \
        const int i0 = 32 * (2 * I + ((p) >> 2)), j0 = 32 * (4 * J + ((p) & 3));                                      \
        if (old && (p) < 7) read_pair(out, nb, 32 * (2 * I + (((p) + 1) >> 2)), 32 * (4 * J + (((p) + 1) & 3)), av[((p) + 1) & 1]); \
        batch();                                                                                                     \
        if (i0 < nb && j0 <= i0) store_pair(out, nb, i0, j0, acc[(p) >> 2][(p) & 3], av[(p) & 1], false, beta, scale); \
        batch();                                                                                                     \
    }
    DOBB_MX4_STORE(0) DOBB_MX4_STORE(1) DOBB_MX4_STORE(2) DOBB_MX4_STORE(3)
    DOBB_MX4_STORE(4) DOBB_MX4_STORE(5) DOBB_MX4_STORE(6) DOBB_MX4_STORE(7)
#undef DOBB_MX4_STORE
}

// The splits' sums of one 32 x 32 pair in fp64, in split order, for blocks whole .. of a launch; one
// workgroup a pair, thread t with column t % 32 and rows t / 32 + 8 u
__global__ void __launch_bounds__(256) k_moment_mx4_reduce(int cnt, int nb, int whole, int nsplit, int pairs, double beta,
                                                           double scale, const float *partial, MomentTable t) {
    __shared__ float tile[32][kPairPad];
    const int64_t nbb = (int64_t)nb * nb;
    const int blk = whole + blockIdx.x / pairs;
    int fi = 0, fj = blockIdx.x % pairs;
    while (fj > fi) fj -= ++fi;
    const int mat = find_matrix(t, cnt, blk);
    float *A = t.A[mat] + (blk - t.first[mat]) * nbb;
    const float *p = partial + (int64_t)(blk - whole) * nsplit * nbb;
    const int tr = threadIdx.x >> 5, tc = threadIdx.x & 31;
    int64_t at[4];
    float av[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int i = min(32 * fi + tr + 8 * u, nb - 1), j = min(32 * fj + tc, i);   // no branches
        at[u] = (int64_t)i * nb + j;
        if (beta > 0.0) av[u] = A[at[u]];
    }
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    for (int k0 = 0; k0 < nsplit; k0 += 4) {
        float x[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < 4; ++u) x[k][u] = p[min(k0 + k, nsplit - 1) * nbb + at[u]];
        batch();
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k0 + k < nsplit)
#pragma unroll
                for (int u = 0; u < 4; ++u) s[u] += (double)x[k][u];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int r = tr + 8 * u, i = 32 * fi + r, j = 32 * fj + tc;
        const float v = moment_out(beta, scale, av[u], s[u]);
        if (i < nb && j <= i) A[at[u]] = v;
        tile[r][tc] = v;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int c = tr + 8 * u, i = 32 * fi + tc, j = 32 * fj + c;
        if (i < nb && j < i) A[(int64_t)j * nb + i] = tile[tc][c];
    }
}

int wide_wgs(int64_t nb) { return (wide_groups((int)(nb + 31) / 32) + 7) / 8; }

template <int GS, int PT>
hipError_t launch_wide(const MomentMx4Args &a, const MomentTable &t, unsigned grid, int F, int nwg, double scale, hipStream_t s) {
    const size_t lds = 2 * ((size_t)GS * 1024 * F + 256 * (size_t)F);
    (void)hipFuncSetAttribute((const void *)k_moment_mx4_wide<GS, PT>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    DOBB_LAUNCH("moment_mx4_wide", s, (k_moment_mx4_wide<GS, PT>), dim3(grid), dim3(kWideThreads), lds, a.count, (int)a.nb, F, nwg,
                a.tiles, a.plan.whole, a.plan.nsplit, (double)a.beta, scale, a.partial, t);
    return hipGetLastError();
}

}  // namespace

// How a launch over `blocks` blocks splits their tokens: the plan that an estimate of the time makes
// smallest.  A launch runs in rounds of workgroups over the chip's slots (two narrow workgroups or one
// wide one a CU).  A tile pair takes a narrow workgroup 0.34 us (four at once; 1.8 us at 128 columns where all
// slots read at the memory's rate), a wide one 0.6 us and 0.1 us a fragment.  Whole rounds of blocks are
// left whole; those of the last round, which would leave slots empty, may be split, for the partial sums'
// traffic and a second launch (5 us).  Never more tile pairs than kSplitPairs in one go, never a split with
// none.  Measured, whole against split: 16384 tokens, 576 blocks of 100: 110 and 104 us; 192 blocks of 400: 320
// and 285; 48 blocks of 400: 116 and 84; 4096 tokens, 4 blocks of 192: 24 and 15; 192 blocks of 128: 18 and 25.
MomentPlan moment_mx4_plan(int64_t nb, int64_t blocks, int64_t tiles) {
    const int64_t tp = (tiles + 1) / 2;
    const bool narrow = nb <= kNarrow;
    const int64_t nwg = narrow ? 1 : wide_wgs(nb), slots = narrow ? 512 : 256;
    const double partial = (double)nb * nb * 8 / 5e6, tau = narrow ? 0.34 : 0.6 + 0.1 * (double)((nb + 31) / 32);
    auto run = [&](int64_t wgs, int64_t pairs) {           // us of wgs workgroups of so many tile pairs
        double t = 0.0;
        for (; wgs > 0; wgs -= std::min(wgs, slots)) {
            const double full = (double)std::min(wgs, slots) / 512 * 1.8 * nb / 128;
            t += narrow ? std::max(tau * ((pairs + 3) / 4) * 4, full * pairs) : tau * pairs;
            if (wgs > 64 * slots) return t * (double)wgs / slots;
        }
        return t;
    };
    const int64_t least = (tp + kSplitPairs - 1) / kSplitPairs;
    MomentPlan best{0, 1};
    double cost = 1e300;
    const int64_t full = blocks * nwg / slots * slots / nwg;
    for (const int64_t whole : {blocks, full, (int64_t)0}) {
        if (whole > 0 && least > 1) continue;
        const int64_t rest = blocks - whole;
        for (int64_t ns = least; ns <= tp && ns <= least + 63; ++ns) {
            const int64_t per = (tp + ns - 1) / ns;
            if ((tp + per - 1) / per != ns) continue;
            const double c = run(whole * nwg, tp) + (rest ? run(rest * nwg * ns, per) : 0.0) +
                             (rest && ns > 1 ? 5.0 + partial * (double)(rest * ns) : 0.0);
            if (c < cost) { best = rest && ns > 1 ? MomentPlan{(int)whole, (int)ns} : MomentPlan{(int)blocks, 1}; cost = c; }
        }
    }
    if (cost == 1e300) {                                   // no even count of splits in the range
        const int64_t per = (tp + least - 1) / least;
        best = {0, (int)((tp + per - 1) / per)};
    }
    return best;
}

size_t moment_mx4_ws(int64_t nb, int64_t blocks, int64_t tiles) {
    const MomentPlan p = moment_mx4_plan(nb, blocks, tiles);
    return (size_t)(blocks - p.whole) * (size_t)nb * (size_t)nb * 4 * (size_t)p.nsplit;
}

hipError_t launch_moment_mx4(const MomentMx4Args &a, hipStream_t s) {
    if (a.count < 1 || a.count > kMomentMats) return hipErrorInvalidValue;
    MomentTable t{};
    int64_t blocks = 0;
    for (int i = 0; i < a.count; ++i) {
        t.codes[i] = (const i32x4 *)a.codes[i];
        t.scales[i] = (const uint32_t *)a.scales[i];
        t.A[i] = a.A[i];
        t.n[i] = (int32_t)a.n[i];
        t.first[i] = (int32_t)blocks;
        blocks += a.n[i] / a.nb;
    }
    t.first[a.count] = (int32_t)blocks;
    const int nb = (int)a.nb, F = (nb + 31) / 32;
    const int nwg = nb <= kNarrow ? 1 : wide_wgs(nb);
    const int64_t rest = blocks - a.plan.whole, pairs = (int64_t)F * (F + 1) / 2;
    const int64_t wgs = (a.plan.whole + rest * a.plan.nsplit) * nwg;
    if (a.plan.whole < 0 || rest < 0 || wgs > 0x7fffffff || rest * pairs > 0x7fffffff) return hipErrorInvalidValue;
    const double scale = (1.0 - (double)a.beta) / (double)a.N;
    const unsigned grid = (unsigned)wgs;
    hipError_t e = hipSuccess;
    // Captures larger than half of the 256 MB cache behind the L2s are read past it: what the quantising
    // left there is gone by then (twelve GPT-2 XL layers, 16384 tokens: 403 us a call, 394 past it); a smaller set
    // may still be there (a 7B-style layer, 4096 tokens, 77 MB, right behind its quantising: the kernel takes 25.5 us,
    // 26.4 past it; the call on captures read before 23.2 and 26.0).
    const bool nt = blocks * a.nb * a.tiles * 68 > ((int64_t)128 << 20);
#define DOBB_MX4_NARROW_(F, NT)                                                                                       \
    DOBB_LAUNCH("moment_mx4_narrow", s, (k_moment_mx4_narrow<F, NT>), dim3(grid), dim3(256), 0, a.count, nb, a.tiles,    \
                a.plan.whole, a.plan.nsplit, (double)a.beta, scale, a.partial, t)
#define DOBB_MX4_NARROW(F)                     \
    do {                                       \
        if (nt) DOBB_MX4_NARROW_(F, true);     \
        else DOBB_MX4_NARROW_(F, false);       \
    } while (0)
    if (F == 1) DOBB_MX4_NARROW(1);
    else if (F == 2) DOBB_MX4_NARROW(2);
    else if (F == 3) DOBB_MX4_NARROW(3);
    else if (F == 4) DOBB_MX4_NARROW(4);
#undef DOBB_MX4_NARROW_
#undef DOBB_MX4_NARROW
    // a stage is 64 GS F pieces: as many a thread as that takes.  Rungs for every PT against 4, 6, 7 and 8 (GS = 4)
    // and 8 (GS = 2) alone, where threads load a piece twice: 64 blocks of 192, 16384 tokens, 37.7 and 39.1 us; 48 of
    // 320, 67.8 and 68.7; 8 of 768, 56.3 and 61.0; the same at 400, 512 and 1024.
#define DOBB_MX4_WIDE(GS, PT) else if (F <= 8 * (PT) / (GS)) e = launch_wide<GS, PT>(a, t, grid, F, nwg, scale, s)
    DOBB_MX4_WIDE(4, 3);
    DOBB_MX4_WIDE(4, 4);
    DOBB_MX4_WIDE(4, 5);
    DOBB_MX4_WIDE(4, 6);
    DOBB_MX4_WIDE(4, 7);
    DOBB_MX4_WIDE(4, 8);
    DOBB_MX4_WIDE(2, 5);
    DOBB_MX4_WIDE(2, 6);
    DOBB_MX4_WIDE(2, 7);
    DOBB_MX4_WIDE(2, 8);
#undef DOBB_MX4_WIDE
    else e = hipErrorInvalidValue;
    if (e == hipSuccess) e = hipGetLastError();
    if (e != hipSuccess || rest == 0) return e;
    DOBB_LAUNCH("moment_mx4_reduce", s, k_moment_mx4_reduce, dim3((unsigned)(rest * pairs)), dim3(256), 0, a.count, nb, a.plan.whole,
                a.plan.nsplit, (int)pairs, (double)a.beta, scale, a.partial, t);
    return hipGetLastError();
}

}  // namespace dobb
