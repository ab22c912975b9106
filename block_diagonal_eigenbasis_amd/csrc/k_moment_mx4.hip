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
//   fragment pairs on or below the diagonal in registers and add up through LDS at the end.
// k_moment_mx4_wide (128 < nb <= 1024): a workgroup of 8 waves stages the tile pair of a whole block
//   in LDS (through registers, one stage ahead) and each wave owns 2 x 4 of the fragment pairs on or
//   below the diagonal; a block with more than 8 such groups takes several workgroups, neighbours on one
//   XCD, so that its codes come from HBM once and from that XCD's L2 after that.
// Rounding: fp32 sums of at most 4096 (narrow, then four of those in fp32) or 16384 tokens (wide) in
// the accumulators, token splits in fp64 (k_moment_mx4_reduce).
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

constexpr int kPairPad = 33;                   // row pitch of a 32x32 pair in LDS: rows and columns are read

// grid: (split of block); F = ceil(nb / 32) fragments
template <int F>
__global__ void __launch_bounds__(256, 2) k_moment_mx4_narrow(int cnt, int nb, int64_t tiles, int nsplit, double beta, double scale,
                                                              float *partial, MomentTable t) {
    constexpr int PAIRS = F * (F + 1) / 2;
    constexpr int PP = PAIRS < 2 ? 1 : 2;       // fragment pairs that are added up at a time
    __shared__ float sm[4][PP][32][kPairPad];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    const int blk = id / nsplit, split = id % nsplit;
    const int mat = find_matrix(t, cnt, blk);
    const int64_t n = t.n[mat];
    const int64_t tp = (tiles + 1) / 2;
    const int64_t per = (tp + nsplit - 1) / nsplit;
    const int64_t p0 = per * split, p1 = p0 + per < tp ? p0 + per : tp;
    const int64_t cb = (int64_t)(blk - t.first[mat]) * nb;
    const i32x4 *codes = t.codes[mat] + cb;
    const uint32_t *scales = t.scales[mat] + cb;
    // columns past the block repeat its last one: they fill rows and columns that are not written
    uint32_t ci[F];
#pragma unroll
    for (int f = 0; f < F; ++f) ci[f] = 32 * f + col < nb ? 32 * f + col : nb - 1;
    f32x16 acc[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) acc[p] = f32x16{};

    for (int64_t p = p0 + wave; p < p1; p += 4) {
        const int64_t tl = 2 * p + half;
        const bool in = tl < tiles;             // an odd last tile: the other half's scales become 2^-127,
        const int64_t tt = in ? tl : tiles - 1; // whose products vanish in fp32
        const i32x4 *cp = codes + tt * 4 * n;
        const uint32_t *sp = scales + tt * n;
        uint32_t sa[F];
        i32x4 a[4][F];
#pragma unroll
        for (int f = 0; f < F; ++f) sa[f] = sp[ci[f]];
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int f = 0; f < F; ++f) a[g][f] = cp[g * n + ci[f]];
#pragma unroll
        for (int f = 0; f < F; ++f) sa[f] = in ? sa[f] : 0u;
#define DOBB_MX4_GROUP(g)                                                          \
        {                                                                          \
            int q = 0;                                                             \
            _Pragma("unroll") for (int i = 0; i < F; ++i)                          \
                _Pragma("unroll") for (int j = 0; j <= i; ++j, ++q)                \
                    acc[q] = mfma_fp4<g>(a[g][i], a[g][j], acc[q], sa[i], sa[j]);  \
        }
        DOBB_MX4_GROUP(0) DOBB_MX4_GROUP(1) DOBB_MX4_GROUP(2) DOBB_MX4_GROUP(3)
#undef DOBB_MX4_GROUP
    }

    // out: the split's partial sums, or A with both its triangles.  Thread t has column t % 32 and rows
    // t / 32 + 8 u of every pair; its entries of A are on their way while the waves' sums are added.
    const int64_t nbb = (int64_t)nb * nb;
    float *out = nsplit > 1 ? partial + ((int64_t)blk * nsplit + split) * nbb : t.A[mat] + (blk - t.first[mat]) * nbb;
    const int tr = threadIdx.x >> 5, tc = threadIdx.x & 31;
    const bool old = nsplit == 1 && beta > 0.0;
    float av[PAIRS][4];
    if (old) {
        int q = 0;
#pragma unroll
        for (int fi = 0; fi < F; ++fi)
#pragma unroll
            for (int fj = 0; fj <= fi; ++fj, ++q)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = min(32 * fi + tr + 8 * u, nb - 1), j = min(32 * fj + tc, i);   // no branches
                    av[q][u] = out[(int64_t)i * nb + j];
                }
    }
#pragma unroll
    for (int q0 = 0; q0 < PAIRS; q0 += PP) {
        if (q0 > 0) __syncthreads();
#pragma unroll
        for (int q = q0; q < q0 + PP && q < PAIRS; ++q)
#pragma unroll
            for (int r = 0; r < 16; ++r) sm[wave][q - q0][acc_row(r, lane)][col] = acc[q][r];
        __syncthreads();
#pragma unroll
        for (int q = q0; q < q0 + PP && q < PAIRS; ++q) {
            int fi = 0, fj = q;
            while (fj > fi) fj -= ++fi;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = tr + 8 * u, i = 32 * fi + r, j = 32 * fj + tc;
                const float sum = ((sm[0][q - q0][r][tc] + sm[1][q - q0][r][tc]) + sm[2][q - q0][r][tc]) + sm[3][q - q0][r][tc];
                const float v = nsplit > 1 ? sum : moment_out(beta, scale, old ? av[q][u] : 0.f, (double)sum);
                if (i < nb && j <= i) out[(int64_t)i * nb + j] = v;
                sm[0][q - q0][r][tc] = v;       // read by this thread only, until the barrier
            }
        }
        if (nsplit > 1) continue;
        __syncthreads();
#pragma unroll
        for (int q = q0; q < q0 + PP && q < PAIRS; ++q) {
            int fi = 0, fj = q;
            while (fj > fi) fj -= ++fi;
#pragma unroll
            for (int u = 0; u < 4; ++u) {       // the mirrored entries, rows of the upper triangle
                const int c = tr + 8 * u, i = 32 * fi + tc, j = 32 * fj + c;
                if (i < nb && j < i) out[(int64_t)j * nb + i] = sm[0][q - q0][tc][c];
            }
        }
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

// GS groups of the tile pair a stage (4, or 2 where four stages of 4 would not fit the LDS); PT 16-byte
// pieces of a stage a thread, ST scale words.  grid: (workgroup of split of block)
template <int GS, int PT, int ST>
__global__ void __launch_bounds__(kWideThreads, 2) k_moment_mx4_wide(int cnt, int nb, int F, int nwg, int64_t tiles, int nsplit,
                                                                     double beta, double scale, float *partial, MomentTable t) {
    extern __shared__ __align__(16) unsigned char lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    int id = xcd_remap(blockIdx.x, gridDim.x);
    const int wg = id % nwg; id /= nwg;
    const int split = id % nsplit, blk = id / nsplit;
    const int mat = find_matrix(t, cnt, blk);
    const int64_t n = t.n[mat];
    const int64_t tp = (tiles + 1) / 2;
    const int64_t per = (tp + nsplit - 1) / nsplit;
    const int64_t p0 = per * split, p1 = p0 + per < tp ? p0 + per : tp;
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
    // every pair leaves as rows of the lower triangle and, through a tile of LDS of the wave's own, of the
    // upper one; its 16 entries of A a lane are read before anything of it is written
    const int64_t nbb = (int64_t)nb * nb;
    float *out = nsplit > 1 ? partial + ((int64_t)blk * nsplit + split) * nbb : t.A[mat] + (blk - t.first[mat]) * nbb;
    float (*tile)[kPairPad] = (float (*)[kPairPad])(lds + wave * sizeof(float) * 32 * kPairPad);
#pragma unroll
    for (int fi = 0; fi < 2; ++fi)
#pragma unroll
        for (int fj = 0; fj < 4; ++fj) {
            const int i0 = 32 * (2 * I + fi), j0 = 32 * (4 * J + fj);
            if (i0 >= nb || j0 > i0) continue;
            float av[16];
            if (nsplit == 1 && beta > 0.0) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int i = min(i0 + acc_row(r, lane), nb - 1), j = min(j0 + col, i);   // no branches
                    av[r] = out[(int64_t)i * nb + j];
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int i = i0 + acc_row(r, lane), j = j0 + col;
                const float w = nsplit > 1 ? acc[fi][fj][r] : moment_out(beta, scale, av[r], (double)acc[fi][fj][r]);
                if (i < nb && j <= i) out[(int64_t)i * nb + j] = w;
                if (nsplit == 1) tile[acc_row(r, lane)][col] = w;
            }
            if (nsplit > 1) continue;
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = 2 * r + half, i = i0 + col, j = j0 + c;
                const float w = tile[col][c];
                if (i < nb && j < i) out[(int64_t)j * nb + i] = w;
            }
            __builtin_amdgcn_wave_barrier();
        }
}

// one thread per entry on or below the diagonal: the splits' sums in fp64, in split order
__global__ void __launch_bounds__(256) k_moment_mx4_reduce(int cnt, int nb, int nsplit, int chunks, double beta, double scale,
                                                           const float *partial, MomentTable t) {
    const int64_t nbb = (int64_t)nb * nb;
    const int blk = blockIdx.x / chunks;
    const int64_t at = (int64_t)(blockIdx.x % chunks) * 256 + threadIdx.x;
    if (at >= nbb) return;
    const int i = (int)(at / nb), j = (int)(at % nb);
    if (j > i) return;
    const float *p = partial + (int64_t)blk * nsplit * nbb + at;
    double s = 0.0;
    for (int k = 0; k < nsplit; ++k) s += (double)p[k * nbb];
    const int mat = find_matrix(t, cnt, blk);
    float *A = t.A[mat] + (blk - t.first[mat]) * nbb;
    const float v = moment_out(beta, scale, beta > 0.0 ? A[at] : 0.f, s);
    A[at] = v;
    if (i != j) A[(int64_t)j * nb + i] = v;
}

int wide_wgs(int64_t nb) { return (wide_groups((int)(nb + 31) / 32) + 7) / 8; }

template <int GS, int PT, int ST>
hipError_t launch_wide(const MomentMx4Args &a, const MomentTable &t, unsigned grid, int F, int nwg, double scale, hipStream_t s) {
    const size_t lds = 2 * ((size_t)GS * 1024 * F + 256 * (size_t)F);
    (void)hipFuncSetAttribute((const void *)k_moment_mx4_wide<GS, PT, ST>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    DOBB_LAUNCH("moment_mx4_wide", s, (k_moment_mx4_wide<GS, PT, ST>), dim3(grid), dim3(kWideThreads), lds, a.count, (int)a.nb, F, nwg,
                a.tiles, a.nsplit, (double)a.beta, scale, a.partial, t);
    return hipGetLastError();
}

}  // namespace

// Token splits of one launch over `blocks` blocks: the number that an estimate of the time makes
// smallest.  A split count costs rounds of workgroups over the chip's slots (two narrow workgroups or
// one wide one a CU) of so many tile pairs each, at 0.6 us (narrow: four at once) or 1.2 us (wide), and
// more than one split costs the partial sums' traffic and the reduction's launch.  Never more tile pairs
// than kSplitPairs a split, never a split with none.
int moment_mx4_splits(int64_t nb, int64_t blocks, int64_t tiles) {
    const int64_t tp = (tiles + 1) / 2;
    const bool narrow = nb <= kNarrow;
    const int64_t units = blocks * (narrow ? 1 : wide_wgs(nb)), slots = narrow ? 512 : 256;
    const double tau = narrow ? 0.15 : 1.2, partial = (double)blocks * nb * nb * 8 / 5e6;
    const int64_t least = (tp + kSplitPairs - 1) / kSplitPairs;
    int64_t best = least;
    double cost = 1e300;
    for (int64_t ns = least; ns <= tp && ns <= least + 64; ++ns) {
        const int64_t per = (tp + ns - 1) / ns;
        if ((tp + per - 1) / per != ns) continue;
        const double c = (double)((units * ns + slots - 1) / slots) * (narrow ? (per + 3) / 4 * 4 : per) * tau +
                         (ns > 1 ? 6.0 + partial * (double)ns : 0.0);
        if (c < cost) { best = ns; cost = c; }
    }
    const int64_t per = (tp + best - 1) / best;
    return (int)((tp + per - 1) / per);
}

size_t moment_mx4_ws(int64_t nb, int64_t blocks, int64_t tiles) {
    const int ns = moment_mx4_splits(nb, blocks, tiles);
    return ns > 1 ? (size_t)blocks * (size_t)nb * (size_t)nb * 4 * (size_t)ns : 0;
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
    const int64_t chunks = (a.nb * a.nb + 255) / 256;
    if (blocks * a.nsplit * nwg > 0x7fffffff || blocks * chunks > 0x7fffffff) return hipErrorInvalidValue;
    const double scale = (1.0 - (double)a.beta) / (double)a.N;
    const unsigned grid = (unsigned)(blocks * a.nsplit * nwg);
    hipError_t e = hipSuccess;
#define DOBB_MX4_NARROW(F)                                                                                             \
    DOBB_LAUNCH("moment_mx4_narrow", s, k_moment_mx4_narrow<F>, dim3(grid), dim3(256), 0, a.count, nb, a.tiles, a.nsplit, \
                (double)a.beta, scale, a.partial, t)
    if (F == 1) DOBB_MX4_NARROW(1);
    else if (F == 2) DOBB_MX4_NARROW(2);
    else if (F == 3) DOBB_MX4_NARROW(3);
    else if (F == 4) DOBB_MX4_NARROW(4);
#undef DOBB_MX4_NARROW
    else if (F <= 8) e = launch_wide<4, 4, 1>(a, t, grid, F, nwg, scale, s);
    else if (F <= 12) e = launch_wide<4, 6, 2>(a, t, grid, F, nwg, scale, s);
    else if (F <= 14) e = launch_wide<4, 7, 2>(a, t, grid, F, nwg, scale, s);
    else if (F <= 16) e = launch_wide<4, 8, 2>(a, t, grid, F, nwg, scale, s);
    else e = launch_wide<2, 8, 4>(a, t, grid, F, nwg, scale, s);
    if (e == hipSuccess) e = hipGetLastError();
    if (e != hipSuccess || a.nsplit == 1) return e;
    DOBB_LAUNCH("moment_mx4_reduce", s, k_moment_mx4_reduce, dim3((unsigned)(blocks * chunks)), dim3(256), 0, a.count, nb, a.nsplit,
                (int)chunks, (double)a.beta, scale, a.partial, t);
    return hipGetLastError();
}

}  // namespace dobb
