// out = A B^T (+ bias) (+ out) for two FP8 operands (dobb_layers.h).
#include "fp8_tile.h"

namespace dobb {
namespace {

struct Epilogue {
    void *out;
    const void *bias;
    int64_t ldo;
    bool bf16, bias_bf16, accumulate;
};

// four neighbouring entries n .. n + 3 of row m
__device__ __forceinline__ void store4(const Epilogue &e, int64_t m, int64_t n, int64_t N, f32x4 v) {
    if (n >= N) return;
    const bool whole = n + 4 <= N;
    if (e.bias)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] += load1(e.bias, min(n + k, N - 1), e.bias_bf16);
    char *o = (char *)e.out + (m * e.ldo + n) * (e.bf16 ? 2 : 4);
    if (e.accumulate)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n + k < N) v[k] += load1(o, k, e.bf16);
    if (e.bf16) {
        if (whole) {
            struct __attribute__((packed, aligned(2))) Four { uint32_t w[2]; };
            *(Four *)o = Four{{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}};
        } else
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (n + k < N) ((uint16_t *)o)[k] = f32_to_bf16(v[k]);
    } else if (whole) {
        struct __attribute__((packed, aligned(4))) Four { float w[4]; };
        *(Four *)o = Four{{v[0], v[1], v[2], v[3]}};
    } else
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (n + k < N) ((float *)o)[k] = v[k];
}

template <int TM, int TN, int FA, int FB, bool EXACT>
__global__ void __launch_bounds__(256, 2) k_fp8_matmul(Fp8Side a, Fp8Side b, int64_t halves, int tilesN, Epilogue e) {
    using T = Fp8Tile<TM, TN, 3, FA, FB, EXACT>;
    __shared__ __align__(16) uint8_t b0[T::kSlot], b1[T::kSlot], b2[T::kSlot];
    uint8_t *const bufs[3] = {b0, b1, b2};
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    a.row0 = (uint32_t)(id / tilesN) * TM;
    b.row0 = (uint32_t)(id % tilesN) * TN;
    const T t(a, b);
    f32x16 acc[T::kFM][T::kFN];
#pragma unroll
    for (int i = 0; i < T::kFM; ++i)
#pragma unroll
        for (int j = 0; j < T::kFN; ++j) acc[i][j] = f32x16{};
    t.run(0, halves, bufs, acc);
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < T::kFM; ++i) {
        const int64_t m = a.row0 + (t.wave >> 1) * T::kWM + 32 * i + (lane & 31);
        if (m >= a.rows) continue;
#pragma unroll
        for (int j = 0; j < T::kFN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                store4(e, m, (int64_t)b.row0 + (t.wave & 1) * T::kWN + 32 * j + 8 * q + 4 * (lane >> 5), b.rows,
                       f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
    }
}

}  // namespace

size_t fp8_matmul_ws(int64_t M, int64_t N, int64_t k) { return 0; }

hipError_t launch_fp8_matmul(const dobb_fp8_operand &A, const dobb_fp8_operand &B, const void *bias, bool bias_bf16, bool accumulate,
                             void *out, bool out_bf16, int64_t ldo, float *ws, hipStream_t s) {
    auto side = [](const dobb_fp8_operand &o) {
        return Fp8Side{(const uint8_t *)o.codes, (const uint8_t *)o.scales, (uint32_t)o.rows, (uint32_t)fp8_pitch(o.rows), 0, (uint32_t)o.rows};
    };
    const Fp8Side a = side(A), b = side(B);
    const Epilogue e{out, bias, ldo, out_bf16, bias_bf16, accumulate};
    const int64_t halves = 2 * fp8_tiles(A.k);
#define DOBB_FP8_MM_(TM, TN, FA, FB, EX)                                                                                \
    do {                                                                                                               \
        const int64_t tm = (A.rows + TM - 1) / TM, tn = (B.rows + TN - 1) / TN;                                        \
        if (tm > 0x7fffffff / tn) return hipErrorInvalidValue;                                                         \
        DOBB_LAUNCH("fp8_matmul", s, (k_fp8_matmul<TM, TN, FA, FB, EX>), dim3((unsigned)(tm * tn)), dim3(256), 0, a, b, halves, (int)tn, e); \
    } while (0)
#define DOBB_FP8_MM(TM, TN, FA, FB)                                                                                    \
    do {                                                                                                               \
        if (out_bf16) DOBB_FP8_MM_(TM, TN, FA, FB, false);                                                             \
        else DOBB_FP8_MM_(TM, TN, FA, FB, true);                                                                       \
    } while (0)
#define DOBB_FP8_MM_F(TM, TN)                                                                 \
    do {                                                                                      \
        if (A.format == DOBB_E4M3 && B.format == DOBB_E4M3) DOBB_FP8_MM(TM, TN, 0, 0);        \
        else if (A.format == DOBB_E4M3) DOBB_FP8_MM(TM, TN, 0, 1);                            \
        else if (B.format == DOBB_E4M3) DOBB_FP8_MM(TM, TN, 1, 0);                            \
        else DOBB_FP8_MM(TM, TN, 1, 1);                                                       \
    } while (0)
    if (A.rows <= 128) DOBB_FP8_MM_F(128, 128);
    else DOBB_FP8_MM_F(256, 128);
#undef DOBB_FP8_MM_F
#undef DOBB_FP8_MM
#undef DOBB_FP8_MM_
    return hipGetLastError();
}

}  // namespace dobb
