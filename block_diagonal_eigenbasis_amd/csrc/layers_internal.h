// Internal definitions of the operators of dobb_layers.h (not installed).
#pragma once

#include "../../include/dobb_layers.h"
#include "ops_internal.h"

namespace dobb {

constexpr int64_t kFp8Tile = 128;
inline int64_t fp8_tiles(int64_t k) { return k / kFp8Tile + (k % kFp8Tile != 0); }
constexpr int64_t kMaxWorkgroups = ((int64_t)1 << 24) - 1;   // of 256 threads: a launch holds fewer than 2^32
inline int64_t fp8_pitch(int64_t rows) { return (rows + 3) / 4 * 4; }   // bytes of a tile's scales

// What normalises a matrix while it is quantised (mean == nullptr: nothing)
struct NormArgs {
    const float *mean, *rstd;
    const void *w, *b;
    bool w_bf16;
};

hipError_t launch_layer_norm(int64_t N, int64_t n, const void *X, bool x_bf16, int64_t ldx, const void *w, const void *b,
                             bool w_bf16, float eps, void *Y, bool y_bf16, int64_t ldy, float *mean, float *rstd, hipStream_t s);
struct NormGradArgs {
    int64_t N, n;
    const void *dY;
    bool dy_bf16;
    int64_t lddy;
    const void *X;
    bool x_bf16;
    int64_t ldx;
    const float *mean, *rstd;
    const void *w;
    bool w_bf16;
    void *dX;
    bool dx_bf16;
    int64_t lddx;
    void *dw, *db;
    bool g_bf16;
    float *part;                      // row groups x 2 x n
};
int64_t norm_grad_groups(int64_t N, int64_t n);
hipError_t launch_layer_norm_backward(const NormGradArgs &a, hipStream_t s);

hipError_t launch_fp8_quantize(int64_t N, int64_t n, const void *X, bool bf16, int64_t ldx, bool square, const NormArgs &norm,
                               const dobb_fp8_operand *rows, const dobb_fp8_operand *cols, hipStream_t s);
// workgroups of a read-back: 32 rows of a tile each, or with `transpose` 128 rows of half a tile
inline int64_t fp8_read_rows(int64_t rows, bool transpose) { return transpose ? (rows + 127) / 128 : (rows + 31) / 32; }
inline int64_t fp8_read_tiles(int64_t k, bool transpose) { return fp8_tiles(k) * (transpose ? 2 : 1); }
hipError_t launch_fp8_dequantize(const dobb_fp8_operand &op, bool transpose, void *out, bool bf16, int64_t ldo, hipStream_t s);

size_t fp8_matmul_ws(int64_t M, int64_t N, int64_t k);
hipError_t launch_fp8_matmul(const dobb_fp8_operand &A, const dobb_fp8_operand &B, const void *bias, bool bias_bf16, bool accumulate,
                             void *out, bool out_bf16, int64_t ldo, float *ws, hipStream_t s);

// second moments from FP8 captures of one format: MomentArgs with the operands' codes and scales
MomentPlan moment_fp8_plan(int64_t nb, int64_t blocks, int64_t tiles);
size_t moment_fp8_ws(int64_t nb, int64_t blocks, int64_t tiles);
hipError_t launch_moment_fp8(const MomentArgs &a, bool e5m2, hipStream_t s);

}  // namespace dobb
