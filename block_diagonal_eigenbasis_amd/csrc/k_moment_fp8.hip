// Second moments from captures held as FP8 operands along their columns:
// A_b <- beta A_b + (1 - beta)/N sum_t x_t x_t^T.  Codes become bf16 on the way to v_mfma_f32_32x32x16_bf16: the
// instructions that multiply FP8 cut small products (fp8_tile.h), the moments are fp32.
//
// k_moment_fp8_narrow (nb <= 128): a workgroup owns one block.  Its four waves take every fourth tile, read a
//   block's codes once, straight into registers (the layout is the instruction's), convert each code once, keep all
//   fragment pairs on or below the diagonal and hand each other their sums through LDS at the end.
// k_moment_fp8_wide (128 < nb <= 1024): a workgroup computes 128 x 128 entries on or below the diagonal of a block as
//   a product of the operand with itself (fp8_tile.h), and leaves out fragment pairs above it or past the block.
// Rounding: fp32 sums of at most 4096 tokens in the accumulators (four of those added in fp32 by a narrow workgroup), token
// splits in fp64 (k_moment_reduce).  The matrix instruction cuts what lies below its accumulator's last bits, and a sum of
// squares only grows: with activations whose tokens differ in size, 16384 tokens in one sum left a block of 400 up to 1.4e-6
// too small (2-norm), 4096 at most 5.5e-7, where fp32 products of 1024 tokens added in fp64 are 3e-7 off.
#include <algorithm>

#include "fp8_tile.h"

namespace dobb {
namespace {

constexpr int kNarrow = 128;                   // widest block of the narrow kernel
// most tiles of one split, of which a narrow workgroup's waves take a quarter each: 4096 tokens a sum
constexpr int64_t kNarrowTiles = 128, kWideTiles = 32;

inline __host__ __device__ int tile_pairs(int64_t nb) {
    const int t = (int)((nb + 127) / 128);
    return t * (t + 1) / 2;
}

// F = ceil(nb / 32) fragments
template <int F, int FMT>
__global__ void __launch_bounds__(256, F < 4 ? 2 : 1) k_moment_fp8_narrow(int cnt, int nb, int64_t tiles, int whole, int nsplit_, double beta,
                                                                         double scale, float *partial, MomentTable t) {
    constexpr int PAIRS = F * (F + 1) / 2;
    __shared__ PairSums<F> sm;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    const Place pl = place(whole, nsplit_, 1);
    const int blk = pl.blk, mat = find_matrix(t, cnt, blk);
    const int64_t n = t.n[mat], pitch = (n + 3) / 4 * 4;
    const int64_t per = (tiles + pl.nsplit - 1) / pl.nsplit;
    const int64_t t0 = per * pl.split, t1 = t0 + per < tiles ? t0 + per : tiles;
    const int64_t cb = (int64_t)(blk - t.first[mat]) * nb;
    const char *codes = (const char *)t.codes[mat] + cb * 16, *scales = (const char *)t.scales[mat] + cb;
    // this lane's columns (past the block its last one: they fill rows and columns that are not written), its half's pieces
    uint32_t ci[F], at[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        ci[f] = (uint32_t)(32 * f + col < nb ? 32 * f + col : nb - 1);
        at[f] = (ci[f] + (uint32_t)(half ? n : 0)) * 16;
    }
    f32x16 acc[PAIRS];
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) acc[p] = f32x16{};

    // A wave's codes are one tile ahead: once a piece of 16 tokens a lane is converted, its registers take the next
    // tile's, so loads are in flight all the time.  (Of blocks of 97 to 128 columns the accumulators leave room for one wave
    // a SIMD: 576 blocks of 100, 16384 tokens, 249 us; two waves with half a tile ahead 245, one with two tiles 273; blocks
    // of 96 take 165.)
    i32x4 x[4][F];
    uint32_t e[F], en[F];
    auto load = [&](int64_t tile, int s) {
        const char *p = codes + (tile * 8 + 2 * s) * n * 16;
#pragma unroll
        for (int f = 0; f < F; ++f) x[s][f] = __builtin_nontemporal_load((const i32x4 *)(p + at[f]));
    };
    auto load_scales = [&](int64_t tile) {
#pragma unroll
        for (int f = 0; f < F; ++f) en[f] = *(const uint8_t *)(scales + tile * pitch + ci[f]);
    };
    auto products = [&](const bf16x8 (&v)[F]) {
        int q = 0;
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j <= i; ++j, ++q) acc[q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[i], v[j], acc[q], 0, 0, 0);
    };
    auto convert = [&](bf16x8 (&v)[F], int s, int u) {
#pragma unroll
        for (int f = 0; f < F; ++f) v[f] = fp8_to_bf16<FMT>(x[s][f][2 * u], x[s][f][2 * u + 1], __uint_as_float(e[f] << 23));
    };
    const int64_t mine = t0 + wave;
    if (mine < t1) {
        load_scales(mine);
#pragma unroll
        for (int s = 0; s < 4; ++s) load(mine, s);
        batch();
        bf16x8 v[2][F];
        for (int64_t tile = mine; tile < t1; tile += 4) {
            const int64_t next = tile + 4 < t1 ? tile + 4 : tile;   // (the last tile's codes again: no branches)
#pragma unroll
            for (int f = 0; f < F; ++f) e[f] = en[f];
            load_scales(next);
            convert(v[0], 0, 0);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                convert(v[1], s, 1);
                batch();
                load(next, s);
                products(v[0]);
                batch();
                if (s < 3) convert(v[0], s + 1, 0);
                products(v[1]);
                batch();
            }
        }
    }
    const int64_t nbb = (int64_t)nb * nb;
    const bool part = pl.nsplit > 1;
    float *out = part ? partial + ((int64_t)(blk - whole) * pl.nsplit + pl.split) * nbb : t.A[mat] + (blk - t.first[mat]) * nbb;
    finish_pairs<F>(acc, sm, out, nb, part, beta, scale);
}

template <int F>
__global__ void __launch_bounds__(256, 2) k_moment_fp8_wide(int cnt, int nb, int nwg, int64_t tiles, int whole, int nsplit_, double beta,
                                                            double scale, float *partial, MomentTable t) {
    using T = Fp8Tile<128, 128, 3, F, F, true, true>;
    __shared__ __align__(16) uint8_t b0[T::kSlot], b1[T::kSlot], b2[T::kSlot];
    uint8_t *const bufs[3] = {b0, b1, b2};
    const Place pl = place(whole, nsplit_, nwg);
    const int blk = pl.blk, mat = find_matrix(t, cnt, blk);
    const int64_t per = (tiles + pl.nsplit - 1) / pl.nsplit;
    const int64_t t0 = per * pl.split, t1 = t0 + per < tiles ? t0 + per : tiles;
    int ti = 0, tj = pl.wg;
    while (tj > ti) tj -= ++ti;
    const uint32_t n = (uint32_t)t.n[mat], cb = (uint32_t)(blk - t.first[mat]) * nb;
    // columns of the pair on the A side, rows on the B side: the accumulators' rows are B's
    Fp8Side a{(const uint8_t *)t.codes[mat], (const uint8_t *)t.scales[mat], n, (n + 3) / 4 * 4, cb + 128 * tj, cb + nb}, b = a;
    b.row0 = cb + 128 * ti;
    T m(a, b);
    m.part = (m.wave + blockIdx.x) & 3;          // quarters that have less to do on another SIMD in each workgroup
    const int i0 = 128 * ti + (m.part & 1) * T::kWN, j0 = 128 * tj + (m.part >> 1) * T::kWM;
    m.pairs = 0;
    f32x16 acc[T::kFM][T::kFN];
#pragma unroll
    for (int i = 0; i < T::kFM; ++i)
#pragma unroll
        for (int j = 0; j < T::kFN; ++j) {
            acc[i][j] = f32x16{};
            if (i0 + 32 * j < nb && j0 + 32 * i <= i0 + 32 * j) m.pairs |= 1u << (T::kFN * i + j);
        }
    m.run(2 * t0, 2 * t1, bufs, acc);

    const int64_t nbb = (int64_t)nb * nb;
    const bool part = pl.nsplit > 1, old = !part && beta > 0.0;
    float *out = part ? partial + ((int64_t)(blk - whole) * pl.nsplit + pl.split) * nbb : t.A[mat] + (blk - t.first[mat]) * nbb;
#pragma unroll
    for (int i = 0; i < T::kFM; ++i)
#pragma unroll
        for (int j = 0; j < T::kFN; ++j) {
            if (!(m.pairs >> (T::kFN * i + j) & 1)) continue;
            float av[16];
            if (old) read_pair(out, nb, i0 + 32 * j, j0 + 32 * i, av);
            store_pair(out, nb, i0 + 32 * j, j0 + 32 * i, acc[i][j], av, part, beta, scale);
        }
}

}  // namespace

// How a launch splits its tokens (moment_plan).  A tile takes a narrow workgroup 0.12 us a fragment (four at once; 1.8 us
// at 128 columns where all slots read at the memory's rate), a wide one 1.2 us alone on its CU and 2 us beside two others.
// Wide blocks are split all or none: workgroups of a second round begin as those of the first end, so that no round of
// whole blocks ends at once (16384 tokens, 192 blocks of 400: none split 724 us, all in four, as kWideTiles asks for, 750, in
// eight 820; 16 blocks: 149 whole, 107 in two, 78 in four, 77 in eight, 89 in sixteen; 32 blocks of 128: 63 whole, 28 in four,
// 27 in eight, 37 in sixteen).
MomentPlan moment_fp8_plan(int64_t nb, int64_t blocks, int64_t tiles) {
    const bool narrow = nb <= kNarrow;
    const int64_t nwg = narrow ? 1 : tile_pairs(nb), slots = narrow ? (nb <= 96 ? 512 : 256) : 768;
    auto run = [&](int64_t wgs, int64_t units) {
        double t = 0.0;
        for (; wgs > 0; wgs -= std::min(wgs, slots)) {
            const double now = (double)std::min(wgs, slots), w = 1.8 / 512 * (double)nb / 128;
            t += narrow ? std::max(0.12 * (double)((nb + 31) / 32) * (double)((units + 3) / 4 * 4), now * w * (double)units)
                        : std::max(1.17, 0.75 + 0.42 / 256 * now) * (double)units;
            if (wgs > 64 * slots) return t * (double)wgs / now;
        }
        return t;
    };
    return moment_plan(blocks, nwg, slots, tiles, narrow ? kNarrowTiles : kWideTiles, (double)nb * (double)nb * (narrow ? 8 : 4) / 5e6, run, narrow);
}

size_t moment_fp8_ws(int64_t nb, int64_t blocks, int64_t tiles) {
    const MomentPlan p = moment_fp8_plan(nb, blocks, tiles);
    return (size_t)(blocks - p.whole) * (size_t)nb * (size_t)nb * 4 * (size_t)p.nsplit;
}

hipError_t launch_moment_fp8(const MomentArgs &a, bool e5m2, hipStream_t s) {
    if (a.count < 1 || a.count > kMomentMats) return hipErrorInvalidValue;
    int64_t blocks;
    const MomentTable t = moment_table(a, &blocks);
    const int nwg = a.nb <= kNarrow ? 1 : tile_pairs(a.nb), F = (int)(a.nb + 31) / 32;
    const int64_t rest = blocks - a.plan.whole;
    const int64_t wgs = (a.plan.whole + rest * a.plan.nsplit) * nwg;
    if (a.plan.whole < 0 || rest < 0 || wgs > kMaxWorkgroups || rest * F * (F + 1) / 2 > 0x7fffffff) return hipErrorInvalidValue;
    const double scale = (1.0 - (double)a.beta) / (double)a.N;
    const dim3 grid((unsigned)wgs);
#define DOBB_FP8_NARROW(F, FMT)                                                                                            \
    DOBB_LAUNCH("moment_fp8_narrow", s, (k_moment_fp8_narrow<F, FMT>), grid, dim3(256), 0, a.count, (int)a.nb, a.tiles,         \
                a.plan.whole, a.plan.nsplit, (double)a.beta, scale, a.partial, t)
#define DOBB_FP8_MOMENT(FMT)                                                                                              \
    do {                                                                                                                  \
        if (F == 1) DOBB_FP8_NARROW(1, FMT);                                                                              \
        else if (F == 2) DOBB_FP8_NARROW(2, FMT);                                                                         \
        else if (F == 3) DOBB_FP8_NARROW(3, FMT);                                                                         \
        else if (F == 4) DOBB_FP8_NARROW(4, FMT);                                                                         \
        else DOBB_LAUNCH("moment_fp8_wide", s, k_moment_fp8_wide<FMT>, grid, dim3(256), 0, a.count, (int)a.nb, nwg, a.tiles, \
                         a.plan.whole, a.plan.nsplit, (double)a.beta, scale, a.partial, t);                               \
    } while (0)
    if (e5m2) DOBB_FP8_MOMENT(DOBB_E5M2);
    else DOBB_FP8_MOMENT(DOBB_E4M3);
#undef DOBB_FP8_MOMENT
#undef DOBB_FP8_NARROW
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || rest == 0 ? e : launch_moment_reduce("moment_fp8_reduce", a, t, blocks, s);
}

}  // namespace dobb
