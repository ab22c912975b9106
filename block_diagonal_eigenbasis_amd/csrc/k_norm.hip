// Layer norm over the columns of every row, forward and backward (formulas: dobb_layers.h).
//
// A row stays in the registers of the threads that read it (64 to 1024 of them, up to 16 entries each), so
// X is read once: mean, the squares around it, and the output follow from there.  Weight, bias and, in
// the backward pass, the sums of their gradients stay in the same threads' registers over all rows that they
// take, and the next row is on its way while one is worked on.  Wider rows are read again for each step.
// The mean is taken twice (the second time of what is left after the first), so that rows far from
// zero lose nothing to its rounding.  Column sums: fp32 over a workgroup's rows, fp64 over those (k_norm_columns),
// in a fixed order.  HBM bounds both directions.
#include <algorithm>

#include "layers_common.h"

namespace dobb {
namespace {

// Sums over the TPR threads of a row, of K values at once.  `sm` holds them wave by wave, twice by turns of `turn`; where
// a row has several waves, every thread of the workgroup takes part.
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&x)[K], float *sm, int &turn) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = TPR == 16 ? sum16(x[k]) : wave_sum(x[k]);
    if constexpr (TPR > 64) {
        constexpr int W = TPR / 64;
        float *s = sm + (turn ^= 1) * 32 * K;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) s[wave * K + k] = x[k];
        __syncthreads();
        s += wave / W * W * K;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = s[k];
#pragma unroll
            for (int w = 1; w < W; ++w) x[k] += s[w * K + k];
        }
    }
}

// TH threads a workgroup, TPR a row: TH / TPR rows at a time, and workgroup g of `gridDim` takes every gridDim-th such lot
template <bool XB, int TPR, int CH, int TH>
__global__ void __launch_bounds__(TH) k_norm(int64_t N, int64_t n, const void *X, int64_t ldx, const void *w, const void *b,
                                             bool w_bf16, float eps, void *Y, bool y_bf16, int64_t ldy, float *mean_out, float *rstd_out) {
    __shared__ float sm[128];
    constexpr int RW = TH / TPR;
    const int at = threadIdx.x % TPR, sub = TPR < 64 ? threadIdx.x / TPR : __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    const int64_t stride = (int64_t)gridDim.x * RW;
    int turn = 0;
    float wv[CH][8], bv[CH][8];
    if (Y)
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            affine8(w, (k * TPR + at) * 8, n, w_bf16, 1.f, wv[k]);
            affine8(b, (k * TPR + at) * 8, n, w_bf16, 0.f, bv[k]);
        }
    Raw8<XB> raw[CH];
    auto fetch = [&](int64_t row) {              // (rows past the last: that one)
#pragma unroll
        for (int k = 0; k < CH; ++k) raw[k] = load8<XB>((const char *)X + min(row, N - 1) * ldx * (XB ? 2 : 4), (k * TPR + at) * 8, n);
    };
    const float inv = 1.f / (float)n;
    fetch((int64_t)blockIdx.x * RW + sub);
    for (int64_t r0 = (int64_t)blockIdx.x * RW; r0 < N; r0 += stride) {
        const int64_t r = r0 + sub;
        float x[CH][8];
#pragma unroll
        for (int k = 0; k < CH; ++k) unpack8<XB>(raw[k], x[k]);
        if (r0 + stride < N) fetch(r + stride);
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += x[k][j];
        row_sums<TPR>(s, sm, turn);
        const float m0 = s[0] * inv;
        float dq[2] = {0.f, 0.f};                // entries past n are left out
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = (k * TPR + at) * 8 + j < n ? x[k][j] - m0 : 0.f;
                dq[0] += u;
                dq[1] = fmaf(u, u, dq[1]);
            }
        row_sums<TPR>(dq, sm + 64, turn);
        const float d = dq[0] * inv, q = dq[1] * inv;
        const float mean = m0 + d, rstd = 1.f / sqrtf(fmaxf(q - d * d, q * 0.f) + eps);   // (q * 0: NaN stays NaN)
        if (r >= N) continue;
        if (at == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        if (Y) {
            char *row = (char *)Y + r * ldy * (y_bf16 ? 2 : 4);
#pragma unroll
            for (int k = 0; k < CH; ++k) {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = norm_value(x[k][j], mean, rstd, wv[k][j], bv[k][j]);
                store8(row, (k * TPR + at) * 8, n, y, y_bf16);
            }
        }
    }
}

// rows that do not fit the registers: a workgroup of 1024 a row, read three times
template <bool XB>
__global__ void __launch_bounds__(1024) k_norm_long(int64_t N, int64_t n, const void *X, int64_t ldx, const void *w, const void *b,
                                                    bool w_bf16, float eps, void *Y, bool y_bf16, int64_t ldy, float *mean_out,
                                                    float *rstd_out) {
    __shared__ float sm[128];
    int turn = 0;
    const float inv = 1.f / (float)n;
    for (int64_t r = blockIdx.x; r < N; r += gridDim.x) {
        const char *xr = (const char *)X + r * ldx * (XB ? 2 : 4);
        float s[1] = {0.f}, dq[2] = {0.f, 0.f}, x[8];
        for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
            unpack8<XB>(load8<XB>(xr, c, n), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += x[j];
        }
        row_sums<1024>(s, sm, turn);
        const float m0 = s[0] * inv;
        for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
            unpack8<XB>(load8<XB>(xr, c, n), x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = c + j < n ? x[j] - m0 : 0.f;
                dq[0] += u;
                dq[1] = fmaf(u, u, dq[1]);
            }
        }
        row_sums<1024>(dq, sm + 64, turn);
        const float d = dq[0] * inv, q = dq[1] * inv;
        const float mean = m0 + d, rstd = 1.f / sqrtf(fmaxf(q - d * d, q * 0.f) + eps);
        if (threadIdx.x == 0) {
            if (mean_out) mean_out[r] = mean;
            if (rstd_out) rstd_out[r] = rstd;
        }
        if (!Y) continue;
        char *row = (char *)Y + r * ldy * (y_bf16 ? 2 : 4);
        for (int64_t c = threadIdx.x * 8; c < n; c += 8192) {
            unpack8<XB>(load8<XB>(xr, c, n), x);
            float y[8], wv[8], bv[8];
            affine8(w, c, n, w_bf16, 1.f, wv);
            affine8(b, c, n, w_bf16, 0.f, bv);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = norm_value(x[j], mean, rstd, wv[j], bv[j]);
            store8(row, c, n, y, y_bf16);
        }
    }
}

// ---- backward ------------------------------------------------------------------------------------
struct GradPtrs {
    const void *dY, *X, *w;
    const float *mean, *rstd;
    void *dX;
    int64_t lddy, ldx, lddx;
    bool w_bf16, dx_bf16;
};

template <bool DB, bool XB, int TPR, int CH, int TH>
__global__ void __launch_bounds__(TH) k_norm_grad(int64_t N, int64_t n, GradPtrs p, float *part) {
    __shared__ float sm[128];
    constexpr int RW = TH / TPR;
    const int at = threadIdx.x % TPR, sub = TPR < 64 ? threadIdx.x / TPR : __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    const int64_t stride = (int64_t)gridDim.x * RW;
    int turn = 0;
    float wv[CH][8], dw[CH][8], db[CH][8];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        affine8(p.w, (k * TPR + at) * 8, n, p.w_bf16, 1.f, wv[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.f;
    }
    Raw8<XB> rx[CH];
    Raw8<DB> rd[CH];
    float mean, rstd;
    auto fetch = [&](int64_t row) {              // (rows past the last: that one)
        row = min(row, N - 1);
        mean = p.mean[row];
        rstd = p.rstd[row];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            rx[k] = load8<XB>((const char *)p.X + row * p.ldx * (XB ? 2 : 4), (k * TPR + at) * 8, n);
            rd[k] = load8<DB>((const char *)p.dY + row * p.lddy * (DB ? 2 : 4), (k * TPR + at) * 8, n);
        }
    };
    const float inv = 1.f / (float)n;
    fetch((int64_t)blockIdx.x * RW + sub);
    for (int64_t r0 = (int64_t)blockIdx.x * RW; r0 < N; r0 += stride) {
        const int64_t r = r0 + sub;
        const float rs = rstd;
        float h[CH][8], g[CH][8], ac[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            float x[8], dy[8];
            unpack8<XB>(rx[k], x);
            unpack8<DB>(rd[k], dy);
#pragma unroll
            for (int j = 0; j < 8; ++j) {        // dy is zero past n, and so are the terms there
                h[k][j] = (x[j] - mean) * rstd;
                if (r < N) {
                    dw[k][j] = fmaf(dy[j], h[k][j], dw[k][j]);
                    db[k][j] += dy[j];
                }
                g[k][j] = dy[j] * wv[k][j];
                ac[0] += g[k][j];
                ac[1] = fmaf(g[k][j], h[k][j], ac[1]);
            }
        }
        if (r0 + stride < N) fetch(r + stride);
        row_sums<TPR>(ac, sm, turn);
        if (r >= N) continue;
        const float a = ac[0] * inv, c = ac[1] * inv;
        char *row = (char *)p.dX + r * p.lddx * (p.dx_bf16 ? 2 : 4);
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[j] = rs * (g[k][j] - a - h[k][j] * c);
            store8(row, (k * TPR + at) * 8, n, dx, p.dx_bf16);
        }
    }
    if (!part) return;
    // this workgroup's sums: its rows' threads in order
    float *out = part + (int64_t)blockIdx.x * 2 * n;
    if constexpr (RW > 1) {
        __shared__ float acc[RW - 1][2][8][TPR];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
            __syncthreads();
            if (sub > 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[sub - 1][0][j][at] = dw[k][j];
                    acc[sub - 1][1][j][at] = db[k][j];
                }
            __syncthreads();
            if (sub == 0)
#pragma unroll 1
                for (int q = 0; q < RW - 1; ++q)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dw[k][j] += acc[q][0][j][at];
                        db[k][j] += acc[q][1][j][at];
                    }
        }
        if (sub) return;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        store8(out, (k * TPR + at) * 8, n, dw[k], false);
        store8(out + n, (k * TPR + at) * 8, n, db[k], false);
    }
}

// rows that do not fit the registers: dx by rows, read twice,
template <bool DB, bool XB>
__global__ void __launch_bounds__(1024) k_norm_grad_long(int64_t N, int64_t n, GradPtrs p) {
    __shared__ float sm[128];
    int turn = 0;
    const float inv = 1.f / (float)n;
    for (int64_t r = blockIdx.x; r < N; r += gridDim.x) {
        const char *xr = (const char *)p.X + r * p.ldx * (XB ? 2 : 4), *dr = (const char *)p.dY + r * p.lddy * (DB ? 2 : 4);
        const float mean = p.mean[r], rstd = p.rstd[r];
        float ac[2] = {0.f, 0.f};
        auto eight = [&](int64_t e, float (&g)[8], float (&h)[8]) {
            float x[8], dy[8], wv[8];
            unpack8<XB>(load8<XB>(xr, e, n), x);
            unpack8<DB>(load8<DB>(dr, e, n), dy);
            affine8(p.w, e, n, p.w_bf16, 1.f, wv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[j] = e + j < n ? (x[j] - mean) * rstd : 0.f;
                g[j] = dy[j] * wv[j];
            }
        };
        float g[8], h[8];
        for (int64_t e = threadIdx.x * 8; e < n; e += 8192) {
            eight(e, g, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ac[0] += g[j];
                ac[1] = fmaf(g[j], h[j], ac[1]);
            }
        }
        row_sums<1024>(ac, sm, turn);
        const float a = ac[0] * inv, c = ac[1] * inv;
        char *row = (char *)p.dX + r * p.lddx * (p.dx_bf16 ? 2 : 4);
        for (int64_t e = threadIdx.x * 8; e < n; e += 8192) {
            eight(e, g, h);
            float dx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) dx[j] = rstd * (g[j] - a - h[j] * c);
            store8(row, e, n, dx, p.dx_bf16);
        }
    }
}

// and before that the column sums by strips of 2048 columns and groups of rows (group g takes rows g, g + groups, ..)
template <bool DB, bool XB>
__global__ void __launch_bounds__(256) k_norm_grad_strips(int64_t N, int64_t n, int64_t groups, GradPtrs p, float *part) {
    const int64_t strips = (n + 2047) / 2048, g = blockIdx.x / strips;
    const int64_t e = (blockIdx.x % strips) * 2048 + threadIdx.x * 8;
    float dw[8] = {0.f}, db[8] = {0.f};
    for (int64_t r = g; r < N; r += groups) {
        float x[8], dy[8];
        unpack8<XB>(load8<XB>((const char *)p.X + r * p.ldx * (XB ? 2 : 4), e, n), x);
        unpack8<DB>(load8<DB>((const char *)p.dY + r * p.lddy * (DB ? 2 : 4), e, n), dy);
        const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = fmaf(dy[j], (x[j] - mean) * rstd, dw[j]);
            db[j] += dy[j];
        }
    }
    float *out = part + g * 2 * n;
    store8(out, e, n, dw, false);
    store8(out + n, e, n, db, false);
}

// the groups' sums in fp64, in a fixed order: 32 columns a workgroup, 32 threads a column
__global__ void __launch_bounds__(1024) k_norm_columns(int64_t n, int64_t groups, const float *part, void *dw, void *db, bool g_bf16) {
    __shared__ double sm[32][33];
    const int64_t blocks = (n + 31) / 32;
    const bool second = blockIdx.x >= blocks;
    const int64_t c0 = (blockIdx.x - (second ? blocks : 0)) * 32;
    const int col = threadIdx.x & 31, q = threadIdx.x >> 5;
    void *out = second ? db : dw;
    if (!out) return;                            // (the whole workgroup)
    const float *p = part + (second ? n : 0) + min(c0 + col, n - 1);
    double s = 0.0;
    int64_t g = q;
    for (; g + 224 < groups; g += 256) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = p[(g + 32 * k) * 2 * n];
#pragma unroll
        for (int k = 0; k < 8; ++k) s += (double)v[k];
    }
    for (; g < groups; g += 32) s += (double)p[g * 2 * n];
    sm[q][col] = s;
    __syncthreads();
    // 32 threads a column again, each with one of its sums
    s = sm[col][q];
#pragma unroll
    for (int k = 1; k < 32; k *= 2) s += __shfl_xor(s, k);
    const int64_t c = c0 + q;
    if (col || c >= n) return;
    if (g_bf16) ((uint16_t *)out)[c] = f32_to_bf16((float)s);
    else ((float *)out)[c] = (float)s;
}

constexpr int64_t kInRegs = 16384;              // widest rows that stay in registers in the forward pass

}  // namespace

hipError_t launch_layer_norm(int64_t N, int64_t n, const void *X, bool x_bf16, int64_t ldx, const void *w, const void *b,
                             bool w_bf16, float eps, void *Y, bool y_bf16, int64_t ldy, float *mean, float *rstd, hipStream_t s) {
    if (n > kInRegs) {
        const dim3 grid((unsigned)std::min<int64_t>(N, 512));
        if (x_bf16) DOBB_LAUNCH("layer_norm", s, k_norm_long<true>, grid, dim3(1024), 0, N, n, X, ldx, w, b, w_bf16, eps, Y, y_bf16, ldy, mean, rstd);
        else DOBB_LAUNCH("layer_norm", s, k_norm_long<false>, grid, dim3(1024), 0, N, n, X, ldx, w, b, w_bf16, eps, Y, y_bf16, ldy, mean, rstd);
        return hipGetLastError();
    }
#define DOBB_NORM_(B, TPR, CH, TH, WGS)                                                                                 \
    DOBB_LAUNCH("layer_norm", s, (k_norm<B, TPR, CH, TH>), dim3((unsigned)std::min<int64_t>((N + (TH) / (TPR) - 1) / ((TH) / (TPR)), WGS)), \
                dim3(TH), 0, N, n, X, ldx, w, b, w_bf16, eps, Y, y_bf16, ldy, mean, rstd)
#define DOBB_NORM(TPR, CH, TH, WGS)                   \
    else if (n <= 8 * (TPR) * (CH)) {                 \
        if (x_bf16) DOBB_NORM_(true, TPR, CH, TH, WGS); \
        else DOBB_NORM_(false, TPR, CH, TH, WGS);     \
    }
    if (n < 1) return hipErrorInvalidValue;
    DOBB_NORM(16, 1, 256, 2048) DOBB_NORM(64, 1, 256, 2048) DOBB_NORM(64, 2, 256, 2048) DOBB_NORM(128, 2, 256, 2048) DOBB_NORM(256, 2, 256, 2048)
    DOBB_NORM(512, 2, 512, 1024) DOBB_NORM(1024, 2, 1024, 512)
#undef DOBB_NORM
#undef DOBB_NORM_
    return hipGetLastError();
}

// How a width is taken: threads a row, chunks of 8 entries a thread, threads a workgroup, and the workgroups that are
// resident on the chip together (two a CU, one where a thread holds two chunks), each of which leaves its sums.
// Measured, us: 16384 x 1600 in bf16 with 256 threads a row and 512 workgroups 44, 256 workgroups 66, with 128 threads a
// row 53; 4096 x 4096 with 512 workgroups of two chunks 27, with 256 23; 16384 x 768 with 64 threads and two chunks 27,
// with 128 and one 22.
struct GradShape {
    int tpr, ch, th;
    int64_t groups;
};
static GradShape grad_shape(int64_t n) {
    if (n <= 128) return {16, 1, 512, 512};
    if (n <= 512) return {64, 1, 512, 512};
    if (n <= 1024) return {128, 1, 512, 512};
    if (n <= 2048) return {256, 1, 512, 512};
    if (n <= 4096) return {256, 2, 512, 256};
    if (n <= 8192) return {512, 2, 512, 256};
    return {1024, 0, 1024, 64};                  // in two passes
}

// Row groups of the column sums: with two lots of rows each where there are as many, and never more than 1024 rows
// (fp32 sums)
int64_t norm_grad_groups(int64_t N, int64_t n) {
    const GradShape g = grad_shape(n);
    const int64_t at = g.th / g.tpr;
    return std::max<int64_t>(std::min<int64_t>((N + 2 * at - 1) / (2 * at), g.groups), (N + 1023) / 1024);
}

hipError_t launch_layer_norm_backward(const NormGradArgs &a, hipStream_t s) {
    const int64_t groups = norm_grad_groups(a.N, a.n), n = a.n;
    const GradShape shape = grad_shape(n);
    const GradPtrs p{a.dY, a.X, a.w, a.mean, a.rstd, a.dX, a.lddy, a.ldx, a.lddx, a.w_bf16, a.dx_bf16};
    float *part = a.dw || a.db ? a.part : nullptr;
    if (n < 1 || groups > 0x7fffffff) return hipErrorInvalidValue;
#define DOBB_GRAD_T(L)                                    \
    do {                                                  \
        if (a.dy_bf16 && a.x_bf16) { L(true, true); }     \
        else if (a.dy_bf16) { L(true, false); }           \
        else if (a.x_bf16) { L(false, true); }            \
        else { L(false, false); }                         \
    } while (0)
#define DOBB_GRAD(TPR, CH, TH)                                        \
    else if (shape.tpr == (TPR) && shape.ch == (CH)) {                \
        constexpr int T = TPR, C = CH, H = TH;                        \
        DOBB_GRAD_T(DOBB_GRAD_L);                                     \
    }
#define DOBB_GRAD_L(D, B) DOBB_LAUNCH("layer_norm_grad", s, (k_norm_grad<D, B, T, C, H>), dim3((unsigned)groups), dim3(H), 0, a.N, n, p, part)
    if (shape.ch == 0) {                         // the sums first: dX may be dY itself
        const dim3 grid((unsigned)std::min<int64_t>(a.N, 512));
        const int64_t strips = (n + 2047) / 2048;
        if (strips > kMaxWorkgroups / groups) return hipErrorInvalidValue;
#define DOBB_GRAD_STRIPS(D, B) \
    DOBB_LAUNCH("layer_norm_grad_strips", s, (k_norm_grad_strips<D, B>), dim3((unsigned)(strips * groups)), dim3(256), 0, a.N, n, groups, p, part)
        if (part) DOBB_GRAD_T(DOBB_GRAD_STRIPS);
#define DOBB_GRAD_LONG(D, B) DOBB_LAUNCH("layer_norm_grad", s, (k_norm_grad_long<D, B>), grid, dim3(1024), 0, a.N, n, p)
        DOBB_GRAD_T(DOBB_GRAD_LONG);
    }
    DOBB_GRAD(16, 1, 512) DOBB_GRAD(64, 1, 512) DOBB_GRAD(128, 1, 512) DOBB_GRAD(256, 1, 512) DOBB_GRAD(256, 2, 512) DOBB_GRAD(512, 2, 512)
#undef DOBB_GRAD
#undef DOBB_GRAD_L
#undef DOBB_GRAD_LONG
#undef DOBB_GRAD_STRIPS
#undef DOBB_GRAD_T
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !part) return e;
    const int64_t blocks = (n + 31) / 32;
    DOBB_LAUNCH("layer_norm_columns", s, k_norm_columns, dim3((unsigned)(2 * blocks)), dim3(1024), 0, n, groups, part, a.dw, a.db, a.g_bf16);
    return hipGetLastError();
}

}  // namespace dobb
