// Second moments from captures in MXFP4:  A_b <- beta A_b + (1 - beta)/N sum_t x_t x_t^T  with the
// products on the scaled fp4 matrix instruction (mfma_scale_f32_32x32x64_f8f6f4).
//
// The capture's layout (dobb_ops.h) is the instruction's operand layout: 32 consecutive columns of one
// group are 512 contiguous bytes, one 16-byte piece a lane, so operands go from HBM straight to
// registers and both sides of a product are the same kind of fragment.  A workgroup owns one pair of
// 128-column tiles of one block (a block of up to 128 columns is one pair, read once); its four waves
// take every fourth pair of token tiles and keep the whole pair's sums in registers, and add them up
// through LDS at the end.  Of a diagonal pair only the fragments on or below the diagonal are formed.
// The two half-waves of an instruction take the same group of two neighbouring token tiles: the scale
// bytes of a tile's four groups are then one 4-byte load for four instructions.
// Rounding: fp32 sums of at most 4096 tokens a wave (64 instructions), four of those in fp32, and the
// token splits in fp64 (k_moment_mx4_reduce).
#include "ops_internal.h"

namespace dobb {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 128;                     // columns of a tile
constexpr int64_t kSplitTokens = 16384;        // most tokens of one split: 4 waves x 4096

struct MomentTable {
    const uint4 *codes[kMaxMats];
    const uint32_t *scales[kMaxMats];
    float *A[kMaxMats];
};

__device__ __forceinline__ i32x8 operand(const uint4 &v) {
    return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// beta A + (1 - beta)/N times the sum, rounded to fp32 once
__device__ __forceinline__ float moment_out(double beta, double scale, float A, double sum) {
    return (float)(beta > 0.0 ? beta * (double)A + scale * sum : scale * sum);
}

template <int G>
__device__ __forceinline__ f32x16 mfma_fp4(const uint4 &a, const uint4 &b, f32x16 c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, G, (int)sa, G, (int)sb);
}

// fragments: FI of the row tile, FJ of the column tile (DIAG: the same FI fragments, pairs fj <= fi)
template <int FI, int FJ, bool DIAG>
struct Frags {
    static constexpr int NB = DIAG ? 0 : FJ;
    static constexpr int PAIRS = DIAG ? FI * (FI + 1) / 2 : FI * FJ;
    uint4 a[FI], b[NB > 0 ? NB : 1];
};

constexpr int kPairPad = 33;                   // row pitch of a 32x32 pair in LDS: rows and columns are read

// grid: (splits of every pair of every block of every matrix); lower pairs I >= J of ntile tiles
template <int FI, int FJ, bool DIAG>
__global__ void __launch_bounds__(256, 1) k_moment_mx4(int64_t n, int nb, int nblk, int64_t tiles, int nsplit, int ntile, int pair0,
                                                       int npair, double beta, double scale, float *partial, MomentTable t) {
    constexpr int PAIRS = Frags<FI, FJ, DIAG>::PAIRS;
    __shared__ float sm[PAIRS][32][kPairPad];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    int id = xcd_remap(blockIdx.x, gridDim.x);
    const int pr = pair0 + id % npair; id /= npair;
    const int split = id % nsplit; id /= nsplit;
    const int blk = id % nblk, mat = id / nblk;
    int I = 0, J = 0;                           // DIAG: tile pr; otherwise pair pr of the strict lower triangle
    if (DIAG) I = J = pr;
    else { I = 1; int p = pr; while (p >= I) { p -= I; ++I; } J = p; }
    // token tiles of this split, in pairs
    const int64_t tp = (tiles + 1) / 2;
    const int64_t per = (tp + nsplit - 1) / nsplit;
    const int64_t p0 = per * split, p1 = p0 + per < tp ? p0 + per : tp;
    const uint4 *codes = t.codes[mat];
    const uint32_t *scales = t.scales[mat];
    // columns past the block repeat its last one: they fill rows and columns that are not written
    const int64_t cb = (int64_t)blk * nb;
    uint32_t ci[FI], cj[FJ];
#pragma unroll
    for (int f = 0; f < FI; ++f) { const int c = I * kTile + 32 * f + col; ci[f] = (uint32_t)(cb + (c < nb ? c : nb - 1)); }
#pragma unroll
    for (int f = 0; f < FJ; ++f) { const int c = J * kTile + 32 * f + col; cj[f] = (uint32_t)(cb + (c < nb ? c : nb - 1)); }
    f32x16 acc[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) acc[p] = f32x16{};

    for (int64_t p = p0 + wave; p < p1; p += 4) {
        const int64_t tl = 2 * p + half;
        const bool in = tl < tiles;             // an odd last tile: the other half's scales become 2^-127,
        const int64_t tt = in ? tl : tiles - 1; // whose products vanish in fp32
        const uint4 *cp = codes + tt * 4 * n;
        const uint32_t *sp = scales + tt * n;
        uint32_t sa[FI], sb[FJ];
#pragma unroll
        for (int f = 0; f < FI; ++f) sa[f] = in ? sp[ci[f]] : 0u;
        if (!DIAG)
#pragma unroll
            for (int f = 0; f < FJ; ++f) sb[f] = in ? sp[cj[f]] : 0u;
        uint4 a[4][FI], b[4][FJ];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int f = 0; f < FI; ++f) a[g][f] = cp[g * n + ci[f]];
            if (!DIAG)
#pragma unroll
                for (int f = 0; f < FJ; ++f) b[g][f] = cp[g * n + cj[f]];
        }
#define DOBB_MX4_GROUP(g)                                                                              \
        {                                                                                              \
            int q = 0;                                                                                 \
            _Pragma("unroll") for (int i = 0; i < FI; ++i)                                             \
                _Pragma("unroll") for (int j = 0; j < (DIAG ? i + 1 : FJ); ++j, ++q)                   \
                    acc[q] = DIAG ? mfma_fp4<g>(a[g][i], a[g][j], acc[q], sa[i], sa[j])                \
                                  : mfma_fp4<g>(a[g][i], b[g][j], acc[q], sa[i], sb[j]);               \
        }
        DOBB_MX4_GROUP(0) DOBB_MX4_GROUP(1) DOBB_MX4_GROUP(2) DOBB_MX4_GROUP(3)
#undef DOBB_MX4_GROUP
    }

    // the waves' sums, in wave order
    for (int w = 0; w < 4; ++w) {
        if (wave == w) {
#pragma unroll
            for (int p = 0; p < PAIRS; ++p)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float *o = &sm[p][acc_row(r, lane)][col];
                    *o = w == 0 ? acc[p][r] : *o + acc[p][r];
                }
        }
        __syncthreads();
    }
    // out: the split's partial sums, or A with both its triangles
    const int64_t nbb = (int64_t)nb * nb;
    float *out = nsplit > 1 ? partial + ((int64_t)(mat * nblk + blk) * nsplit + split) * nbb : t.A[mat] + blk * nbb;
    int q = 0;
    for (int fi = 0; fi < FI; ++fi)
        for (int fj = 0; fj < (DIAG ? fi + 1 : FJ); ++fj, ++q) {
            const int r0 = I * kTile + 32 * fi, c0 = J * kTile + 32 * fj;
            for (int e = threadIdx.x; e < 1024; e += 256) {
                const int r = e >> 5, c = e & 31;
                const int i = r0 + r, j = c0 + c;
                if (i >= nb || j > i) continue;
                const int64_t at = (int64_t)i * nb + j;
                if (nsplit > 1) { out[at] = sm[q][r][c]; continue; }
                const float v = moment_out(beta, scale, beta > 0.0 ? out[at] : 0.f, (double)sm[q][r][c]);
                sm[q][r][c] = v;                // the mirrored entries below take what was written here
                out[at] = v;
            }
        }
    if (nsplit > 1) return;
    __syncthreads();
    q = 0;
    for (int fi = 0; fi < FI; ++fi)
        for (int fj = 0; fj < (DIAG ? fi + 1 : FJ); ++fj, ++q) {
            const int r0 = I * kTile + 32 * fi, c0 = J * kTile + 32 * fj;
            for (int e = threadIdx.x; e < 1024; e += 256) {
                const int c = e >> 5, r = e & 31;
                const int i = r0 + r, j = c0 + c;
                if (i < nb && j < i) out[(int64_t)j * nb + i] = sm[q][r][c];
            }
        }
}

// one thread per entry on or below the diagonal: the splits' sums in fp64, in split order
__global__ void __launch_bounds__(256) k_moment_mx4_reduce(int nb, int nblk, int nsplit, int chunks, double beta, double scale,
                                                           const float *partial, MomentTable t) {
    const int64_t nbb = (int64_t)nb * nb;
    const int64_t b = blockIdx.x / chunks;      // block of the launch
    const int64_t at = (int64_t)(blockIdx.x % chunks) * 256 + threadIdx.x;
    if (at >= nbb) return;
    const int i = (int)(at / nb), j = (int)(at % nb);
    if (j > i) return;
    const float *p = partial + b * nsplit * nbb + at;
    double s = 0.0;
    for (int k = 0; k < nsplit; ++k) s += (double)p[k * nbb];
    float *A = t.A[b / nblk] + (b % nblk) * nbb;
    const float v = moment_out(beta, scale, beta > 0.0 ? A[at] : 0.f, s);
    A[at] = v;
    if (i != j) A[(int64_t)j * nb + i] = v;
}

}  // namespace

// Enough workgroups to give every CU one or two (a wave holds a pair's sums in registers, so a CU runs
// one), no split shorter than one pair of token tiles a wave, none longer than kSplitTokens
int moment_mx4_splits(int64_t n, int64_t nb, int count, int64_t tiles) {
    const int64_t nt = (nb + kTile - 1) / kTile;
    const int64_t units = (int64_t)count * (n / nb) * (nt * (nt + 1) / 2);
    const int64_t tp = (tiles + 1) / 2;
    int64_t ns = (512 + units - 1) / units;
    if (ns > (tp + 3) / 4) ns = (tp + 3) / 4;
    const int64_t least = (tiles * kMx4Tile + kSplitTokens - 1) / kSplitTokens;
    if (ns < least) ns = least;
    const int64_t per = (tp + ns - 1) / ns;       // no empty split
    return (int)((tp + per - 1) / per);
}

size_t moment_mx4_ws(int64_t n, int64_t nb, int count, int64_t tiles) {
    const int ns = moment_mx4_splits(n, nb, count, tiles);
    return ns > 1 ? (size_t)count * (size_t)n * (size_t)nb * 4 * (size_t)ns : 0;
}

hipError_t launch_moment_mx4(const MomentMx4Args &a, hipStream_t s) {
    if (a.count < 1 || a.count > kMaxMats) return hipErrorInvalidValue;
    MomentTable t{};
    for (int i = 0; i < a.count; ++i) {
        t.codes[i] = (const uint4 *)a.codes[i];
        t.scales[i] = (const uint32_t *)a.scales[i];
        t.A[i] = a.A[i];
    }
    const int nb = (int)a.nb, nblk = (int)(a.n / a.nb), nt = (nb + kTile - 1) / kTile;
    const int64_t units = (int64_t)a.count * nblk * a.nsplit;
    const int offs = nt * (nt - 1) / 2;
    if (units * (nt > offs ? nt : offs) > 0x7fffffff) return hipErrorInvalidValue;
    const double scale = (1.0 - (double)a.beta) / (double)a.N;
    const int f = (nb + 31) / 32;
#define DOBB_MX4_LAUNCH(FI, FJ, DIAG, pair0, npair)                                                                       \
    DOBB_LAUNCH(DIAG ? "moment_mx4_diag" : "moment_mx4_off", s, (k_moment_mx4<FI, FJ, DIAG>), dim3((unsigned)(units * (npair))), \
                dim3(256), 0, a.n, nb, nblk, a.tiles, a.nsplit, nt, pair0, npair, (double)a.beta, scale, a.partial, t)
    if (f == 1) DOBB_MX4_LAUNCH(1, 1, true, 0, nt);
    else if (f == 2) DOBB_MX4_LAUNCH(2, 2, true, 0, nt);
    else if (f == 3) DOBB_MX4_LAUNCH(3, 3, true, 0, nt);
    else DOBB_MX4_LAUNCH(4, 4, true, 0, nt);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (offs > 0) {
        DOBB_MX4_LAUNCH(4, 4, false, 0, offs);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
#undef DOBB_MX4_LAUNCH
    if (a.nsplit > 1) {
        const int64_t blocks = (int64_t)a.count * nblk, chunks = (a.nb * a.nb + 255) / 256;
        if (blocks * chunks > 0x7fffffff) return hipErrorInvalidValue;
        DOBB_LAUNCH("moment_mx4_reduce", s, k_moment_mx4_reduce, dim3((unsigned)(blocks * chunks)), dim3(256), 0, nb, nblk,
                    a.nsplit, (int)chunks, (double)a.beta, scale, a.partial, t);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace dobb
