// Second moments from captures held as FP8 operands along their columns:
// A_b <- beta A_b + (1 - beta)/N sum_t x_t x_t^T, a product of the operand with itself (fp8_tile.h) of which only
// tiles of 128 x 128 on or below the diagonal of a block are computed.
// Rounding: fp32 sums of at most 16384 tokens in the accumulators, token splits in fp64 (k_moment_reduce).
#include <algorithm>

#include "fp8_tile.h"

namespace dobb {
namespace {

constexpr int64_t kSplitTiles = 128;           // most tiles of one split: 16384 tokens

inline __host__ __device__ int tile_pairs(int64_t nb) {
    const int t = (int)((nb + 127) / 128);
    return t * (t + 1) / 2;
}

template <int F>
__global__ void __launch_bounds__(256, 2) k_moment_fp8(int cnt, int nb, int nwg, int64_t tiles, int whole, int nsplit_, double beta,
                                                       double scale, float *partial, MomentTable t) {
    using T = Fp8Tile<128, 128, 3, F, F, true>;
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
    const T m(a, b);
    f32x16 acc[T::kFM][T::kFN];
#pragma unroll
    for (int i = 0; i < T::kFM; ++i)
#pragma unroll
        for (int j = 0; j < T::kFN; ++j) acc[i][j] = f32x16{};
    m.run(2 * t0, 2 * t1, bufs, acc);

    const int64_t nbb = (int64_t)nb * nb;
    const bool part = pl.nsplit > 1, old = !part && beta > 0.0;
    float *out = part ? partial + ((int64_t)(blk - whole) * pl.nsplit + pl.split) * nbb : t.A[mat] + (blk - t.first[mat]) * nbb;
#pragma unroll
    for (int i = 0; i < T::kFM; ++i)
#pragma unroll
        for (int j = 0; j < T::kFN; ++j) {
            const int i0 = 128 * ti + (m.wave & 1) * T::kWN + 32 * j, j0 = 128 * tj + (m.wave >> 1) * T::kWM + 32 * i;
            if (i0 >= nb || j0 > i0) continue;
            float av[16];
            if (old) read_pair(out, nb, i0, j0, av);
            store_pair(out, nb, i0, j0, acc[i][j], av, part, beta, scale);
        }
}

}  // namespace

// How a launch splits its tokens: no more than kSplitTiles in one go, and enough splits for the chip's 512 slots
// (two workgroups a CU), none with less than 8 tiles for that.
MomentPlan moment_fp8_plan(int64_t nb, int64_t blocks, int64_t tiles) {
    const int64_t wgs = blocks * tile_pairs(nb);
    const int64_t least = (tiles + kSplitTiles - 1) / kSplitTiles;
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(512 / wgs, tiles / 8));
    const int64_t ns = std::max(least, want), per = (tiles + ns - 1) / ns, n = (tiles + per - 1) / per;
    return n > 1 ? MomentPlan{0, (int)n} : MomentPlan{(int)blocks, 1};
}

size_t moment_fp8_ws(int64_t nb, int64_t blocks, int64_t tiles) {
    const MomentPlan p = moment_fp8_plan(nb, blocks, tiles);
    return (size_t)(blocks - p.whole) * (size_t)nb * (size_t)nb * 4 * (size_t)p.nsplit;
}

hipError_t launch_moment_fp8(const MomentArgs &a, bool e5m2, hipStream_t s) {
    if (a.count < 1 || a.count > kMomentMats) return hipErrorInvalidValue;
    int64_t blocks;
    const MomentTable t = moment_table(a, &blocks);
    const int nwg = tile_pairs(a.nb);
    const int64_t F = (a.nb + 31) / 32, rest = blocks - a.plan.whole;
    const int64_t wgs = (a.plan.whole + rest * a.plan.nsplit) * nwg;
    if (a.plan.whole < 0 || rest < 0 || wgs > 0x7fffffff || rest * F * (F + 1) / 2 > 0x7fffffff) return hipErrorInvalidValue;
    const double scale = (1.0 - (double)a.beta) / (double)a.N;
#define DOBB_FP8_MOMENT(F)                                                                                              \
    DOBB_LAUNCH("moment_fp8", s, k_moment_fp8<F>, dim3((unsigned)wgs), dim3(256), 0, a.count, (int)a.nb, nwg, a.tiles, a.plan.whole, \
                a.plan.nsplit, (double)a.beta, scale, a.partial, t)
    if (e5m2) DOBB_FP8_MOMENT(DOBB_E5M2);
    else DOBB_FP8_MOMENT(DOBB_E4M3);
#undef DOBB_FP8_MOMENT
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || rest == 0 ? e : launch_moment_reduce(a, t, blocks, s);
}

}  // namespace dobb
