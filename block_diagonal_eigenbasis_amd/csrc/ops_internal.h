// Internal definitions of the operators of dobb_ops.h (not installed).
#pragma once

#include "../../include/dobb_ops.h"
#include "dobb_internal.h"

namespace dobb {

struct GradArgs {
    int count;
    const int64_t *numel;
    const void *const *G;
    const dobb_dtype *g_dtypes;
    void *const *out;                 // clipping only
    const dobb_dtype *out_dtypes;
};
int64_t grad_norm_chunks(int count, const int64_t *numel, const dobb_dtype *dt);   // fp64 partial sums of a call
hipError_t launch_grad_norm(const GradArgs &a, float *norms, float *total, double *part, hipStream_t s);
hipError_t launch_grad_clip(const GradArgs &a, const float *total, float max_norm, hipStream_t s);

// MXFP4 captures: tiles of 128 tokens
constexpr int64_t kMx4Tile = 128;
hipError_t launch_mx4_quantize(int64_t N, int64_t n, const void *X, bool bf16, int64_t ldx, void *codes, void *scales,
                               hipStream_t s);
hipError_t launch_mx4_dequantize(int64_t N, int64_t n, const void *codes, const void *scales, void *out, bool bf16,
                                 int64_t ldo, hipStream_t s);

constexpr int kMomentMats = 96;       // matrices of one launch
struct MomentPlan {
    int whole, nsplit;                // blocks 0 .. whole - 1 unsplit, the others in nsplit token splits
};
struct MomentArgs {
    int count;                        // matrices with blocks of one width; at most kMomentMats
    int64_t nb, tiles, N;
    const int64_t *n;                 // columns of each matrix
    const void *const *codes;
    const void *const *scales;
    float *const *A;
    float beta;
    MomentPlan plan;
    float *partial;                   // (blocks - whole) x nsplit x nb x nb
};
MomentPlan moment_mx4_plan(int64_t nb, int64_t blocks, int64_t tiles);
size_t moment_mx4_ws(int64_t nb, int64_t blocks, int64_t tiles);
hipError_t launch_moment_mx4(const MomentArgs &a, hipStream_t s);

}  // namespace dobb
