// FP8 operands (OCP e4m3 and e5m2, one e8m0 scale per 128 entries of a row or per 128 x 128): quantising,
// with a layer norm on the way or without, and reading back.  Layout: dobb_layers.h.
//
// A workgroup takes one 128 x 128 tile of X and writes its piece of both operands from one read.  A thread
// holds 8 x 8 entries: a row's magnitudes then meet over 16 neighbouring lanes (four lane swaps), a column's over
// the four groups of a wave and the four waves.  Codes go through LDS, so that each operand leaves in runs of
// 2 KB; the paddings below make every LDS access of a wave fall in distinct banks.  HBM bounds it.
// The conversions are gfx950's scaled ones (v_cvt_scalef32_pk_fp8_f32 and .._bf8_f32): nearest, ties to
// even.  The scale is chosen so that nothing saturates.
// Both operands of 16384 x 1600 in bf16 take 25 us (4.2 TB/s), of 16384 x 6400 82 (5.1), one operand 17 and 57; with a
// layer norm on the way 28 and 97: with mean, rstd and the weights a thread needs 134 registers, so that three workgroups
// share a CU and not four (four: 5 registers spilled, 1 us more).  Each row is read once more than by a kernel
// that held whole rows, which would have to hold 128 of them.
#include "layers_common.h"

namespace dobb {
namespace {

constexpr int kRowPitch = 128 * 16 + 16;        // LDS bytes of 16 columns of all rows
constexpr int kColPitch = 8 * 17 * 16;          // of 16 rows of all columns: column 8 x + j at piece 17 j + x

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block from its largest magnitude's bits: the exponent field less the format's largest
// exponent, one more where the mantissa is above 1.75 (448 = 1.75 2^8, 57344 = 1.75 2^15); 255 if not finite
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7f800000u) return 255u;
    const int e = (int)(top >> 23) - (FMT == DOBB_E4M3 ? 8 : 15) + ((top & 0x7fffffu) > 0x600000u);
    return e > 0 ? (uint32_t)e : 0u;
}
// the scale as the conversions take it: its byte is the exponent field, 0 stands for 2^-127
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// four values to four codes
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float scale) {
    s16x2 p = {0, 0};
    if constexpr (FMT == DOBB_E4M3) {
        p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, a, b, scale, false);
        p = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(p, c, d, scale, true);
    } else {
        p = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(p, a, b, scale, false);
        p = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(p, c, d, scale, true);
    }
    return __builtin_bit_cast(uint32_t, p);
}

struct Operands {
    uint4 *rc;
    uint8_t *rs;
    uint4 *cc;
    uint8_t *cs;
};

template <bool BF16, int FMT, bool SQUARE, bool NORM>
__global__ void __launch_bounds__(256, NORM ? 3 : 4) k_fp8_quantize(int64_t N, int64_t n, int64_t ldx, unsigned colblocks, const void *X,
                                                      NormArgs norm, Operands o) {
    __shared__ __align__(16) uint8_t rl[8 * kRowPitch], cl[8 * kColPitch];
    __shared__ uint32_t top[4][128];
    __shared__ __align__(4) uint8_t rsc[128], csc[128];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, wave = tid >> 6;
    const int64_t tr = blockIdx.x / colblocks, tc = blockIdx.x % colblocks;
    const int64_t r0 = tr * 128 + 8 * ty, c0 = tc * 128 + 8 * tx;
    constexpr int ES = BF16 ? 2 : 4;
    [[maybe_unused]] __shared__ float2 stat[NORM ? 128 : 1];
    [[maybe_unused]] float2 own;
    if constexpr (NORM)                         // a row's statistics, asked for before X
        if (tid < 128) {
            const int64_t r = tr * 128 + tid < N ? tr * 128 + tid : N - 1;
            own = float2{norm.mean[r], norm.rstd[r]};
        }
    Raw8<BF16> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {               // rows past the last repeat it; zeros below
        const int64_t r = r0 + i < N ? r0 + i : N - 1;
        raw[i] = load8<BF16>((const char *)X + r * ldx * ES, c0, n);
    }
    if constexpr (NORM) {
        if (tid < 128) stat[tid] = own;
        __syncthreads();
    }
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (!NORM) unpack8<BF16>(raw[i], v[i]);
    if constexpr (NORM) {
        float w[8], b[8];
        affine8(norm.w, c0, n, norm.w_bf16, 1.f, w);
        affine8(norm.b, c0, n, norm.w_bf16, 0.f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            __builtin_amdgcn_sched_barrier(0);   // (a row at a time: 161 registers without)
            unpack8<BF16>(raw[i], v[i]);
            const float mean = stat[8 * ty + i].x, rstd = stat[8 * ty + i].y;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                v[i][j] = norm_value(v[i][j], mean, rstd, w[j], b[j]);
                v[i][j + 1] = norm_value(v[i][j + 1], mean, rstd, w[j + 1], b[j + 1]);
                if (BF16) {
                    const uint32_t y = pack_bf16(v[i][j], v[i][j + 1]);
                    v[i][j] = __uint_as_float(y << 16);
                    v[i][j + 1] = __uint_as_float(y & 0xffff0000u);
                }
            }
        }
        if (tc * 128 + 128 > n)                  // a tile that ends past the last column: zeros there
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c0 + j >= n)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i][j] = 0.f;
    }
    if (r0 + 8 > N)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r0 + i >= N)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;

    auto mag = [&](int i, int j) { return __float_as_uint(v[i][j]) & 0x7fffffffu; };
    uint32_t re[8], ce[8];
    if (SQUARE || o.rc) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, mag(i, j));
            re[i] = max16(m);
        }
    }
    if constexpr (SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, re[i]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if ((tid & 63) == 0) top[wave][0] = m;
        __syncthreads();
        const uint32_t e = scale_byte<FMT>(max(max(top[0][0], top[1][0]), max(top[2][0], top[3][0])));
#pragma unroll
        for (int i = 0; i < 8; ++i) re[i] = ce[i] = e;
    } else {
        if (o.cc) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, mag(i, j));
                m = max(m, (uint32_t)__shfl_xor((int)m, 16));
                ce[j] = max(m, (uint32_t)__shfl_xor((int)m, 32));
            }
            if ((tid & 63) < 16)
#pragma unroll
                for (int j = 0; j < 8; ++j) top[wave][8 * tx + j] = ce[j];
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j)
                ce[j] = scale_byte<FMT>(max(max(top[0][8 * tx + j], top[1][8 * tx + j]), max(top[2][8 * tx + j], top[3][8 * tx + j])));
        }
        if (o.rc)
#pragma unroll
            for (int i = 0; i < 8; ++i) re[i] = scale_byte<FMT>(re[i]);
    }
    if (o.rc) {                                  // a thread's 8 columns of a row: half a piece
        uint8_t *at = rl + (tx >> 1) * kRowPitch + 8 * ty * 16 + (tx & 1) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = scale_of(re[i]);
            uint2 q = {codes4<FMT>(v[i][0], v[i][1], v[i][2], v[i][3], s), codes4<FMT>(v[i][4], v[i][5], v[i][6], v[i][7], s)};
            if (re[i] == 255u) q = uint2{0x7f7f7f7fu, 0x7f7f7f7fu};   // a block that is not finite holds NaN
            *(uint2 *)(at + i * 16) = q;
        }
        if (tx == 0)
#pragma unroll
            for (int i = 0; i < 8; ++i) rsc[8 * ty + i] = r0 + i < N ? (uint8_t)re[i] : (uint8_t)0;
    }
    if (o.cc) {
        uint8_t *at = cl + (ty >> 1) * kColPitch + tx * 16 + (ty & 1) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = scale_of(ce[j]);
            uint2 q = {codes4<FMT>(v[0][j], v[1][j], v[2][j], v[3][j], s), codes4<FMT>(v[4][j], v[5][j], v[6][j], v[7][j], s)};
            if (ce[j] == 255u) q = uint2{0x7f7f7f7fu, 0x7f7f7f7fu};
            *(uint2 *)(at + j * 17 * 16) = q;
        }
        if (ty == 0)
#pragma unroll
            for (int j = 0; j < 8; ++j) csc[8 * tx + j] = c0 + j < n ? (uint8_t)ce[j] : (uint8_t)0;
    }
    __syncthreads();
    if (o.rc) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = tid + 256 * k, h = p >> 7, r = p & 127;
            if (tr * 128 + r < N) o.rc[(tc * 8 + h) * N + tr * 128 + r] = *(const uint4 *)(rl + h * kRowPitch + r * 16);
        }
        const int64_t pitch = (N + 3) / 4 * 4;
        if (tid < 32 && tr * 128 + 4 * tid < pitch) *(uint32_t *)(o.rs + tc * pitch + tr * 128 + 4 * tid) = *(const uint32_t *)(rsc + 4 * tid);
    }
    if (o.cc) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = tid + 256 * k, h = p >> 7, c = p & 127;
            if (tc * 128 + c < n)
                o.cc[(tr * 8 + h) * n + tc * 128 + c] = *(const uint4 *)(cl + h * kColPitch + ((c & 7) * 17 + (c >> 3)) * 16);
        }
        const int64_t pitch = (n + 3) / 4 * 4;
        const int t = tid - 32;
        if (t >= 0 && t < 32 && tc * 128 + 4 * t < pitch) *(uint32_t *)(o.cs + tr * pitch + tc * 128 + 4 * t) = *(const uint32_t *)(csc + 4 * t);
    }
}

// 16 codes to values
template <int FMT>
__device__ __forceinline__ void values16(const uint4 &q, uint32_t byte, float (&v)[16]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    const float s = scale_of(byte), nan = __builtin_nanf("");
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f32x2 lo, hi;
        if constexpr (FMT == DOBB_E4M3) {
            lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[k], s, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w[k], s, true);
        } else {
            lo = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w[k], s, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w[k], s, true);
        }
        v[4 * k] = lo[0]; v[4 * k + 1] = lo[1]; v[4 * k + 2] = hi[0]; v[4 * k + 3] = hi[1];
    }
    if (byte == 255u)
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = nan;
}

// rows x k: a workgroup takes 32 rows of a tile, 8 lanes a row, 32 or 64 bytes a lane
template <int FMT>
__global__ void __launch_bounds__(256) k_fp8_dequantize(int64_t R, int64_t K, unsigned rowblocks, const uint4 *codes,
                                                        const uint8_t *scales, void *out, bool bf16, int64_t ldo) {
    const int64_t t = blockIdx.x / rowblocks, rb = blockIdx.x % rowblocks;
    const int h = threadIdx.x & 7;
    const int64_t pitch = (R + 3) / 4 * 4, c = t * 128 + 16 * h, r = rb * 32 + (threadIdx.x >> 3);
    if (r >= R) return;
    float v[16];
    values16<FMT>(codes[(t * 8 + h) * R + r], scales[t * pitch + r], v);
    char *row = (char *)out + r * ldo * (bf16 ? 2 : 4);
    const float lo[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]}, hi[8] = {v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]};
    store8(row, c, K, lo, bf16);
    store8(row, c + 8, K, hi, bf16);
}

struct __attribute__((packed, aligned(2))) PairBf16 { uint32_t w; };
struct __attribute__((packed, aligned(4))) PairF32 { float a, b; };

// k x rows: a workgroup takes 128 rows of half a tile, two neighbouring ones a lane, a wave one of the 16-entry groups
template <int FMT>
__global__ void __launch_bounds__(256) k_fp8_dequantize_t(int64_t R, int64_t K, unsigned rowblocks, const uint4 *codes,
                                                          const uint8_t *scales, void *out, bool bf16, int64_t ldo) {
    const int64_t t = blockIdx.x / rowblocks / 2, rb = blockIdx.x % rowblocks;
    const int64_t r = rb * 128 + 2 * (threadIdx.x & 63), pitch = (R + 3) / 4 * 4;
    const int h = (threadIdx.x >> 6) + 4 * (blockIdx.x / rowblocks & 1);
    if (r >= R) return;
    const bool two = r + 1 < R;
    const uint32_t ea = scales[t * pitch + r], eb = two ? scales[t * pitch + r + 1] : 0;
    const uint4 *p = codes + (t * 8 + h) * R + r;
    const uint4 qa = p[0], qb = two ? p[1] : uint4{0, 0, 0, 0};
    float a[16], b[16];
    values16<FMT>(qa, ea, a);
    values16<FMT>(qb, eb, b);
    const int64_t k0 = t * 128 + 16 * h;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        if (k0 + k >= K) break;
        if (bf16) {
            uint16_t *x = (uint16_t *)out + (k0 + k) * ldo + r;
            if (two) ((PairBf16 *)x)->w = pack_bf16(a[k], b[k]);
            else *x = f32_to_bf16(a[k]);
        } else {
            float *x = (float *)out + (k0 + k) * ldo + r;
            if (two) *(PairF32 *)x = PairF32{a[k], b[k]};
            else *x = a[k];
        }
    }
}

}  // namespace

hipError_t launch_fp8_quantize(int64_t N, int64_t n, const void *X, bool bf16, int64_t ldx, bool square, const NormArgs &norm,
                               const dobb_fp8_operand *rows, const dobb_fp8_operand *cols, hipStream_t s) {
    const int64_t tr = fp8_tiles(N), tc = fp8_tiles(n);
    if (tr > kMaxWorkgroups / tc) return hipErrorInvalidValue;
    const Operands o{rows ? (uint4 *)rows->codes : nullptr, rows ? (uint8_t *)rows->scales : nullptr,
                     cols ? (uint4 *)cols->codes : nullptr, cols ? (uint8_t *)cols->scales : nullptr};
    const bool e5 = (rows ? rows : cols)->format == DOBB_E5M2;
#define DOBB_FP8_QUANT(B, F, SQ, NM)                                                                                   \
    DOBB_LAUNCH("fp8_quantize", s, (k_fp8_quantize<B, F, SQ, NM>), dim3((unsigned)(tr * tc)), dim3(256), 0, N, n, ldx, (unsigned)tc, X, norm, o)
#define DOBB_FP8_QUANT_F(B, SQ, NM)                          \
    do {                                                     \
        if (e5) DOBB_FP8_QUANT(B, DOBB_E5M2, SQ, NM);         \
        else DOBB_FP8_QUANT(B, DOBB_E4M3, SQ, NM);            \
    } while (0)
    if (norm.mean) {
        if (bf16) DOBB_FP8_QUANT_F(true, false, true);
        else DOBB_FP8_QUANT_F(false, false, true);
    } else if (square) {
        if (bf16) DOBB_FP8_QUANT_F(true, true, false);
        else DOBB_FP8_QUANT_F(false, true, false);
    } else {
        if (bf16) DOBB_FP8_QUANT_F(true, false, false);
        else DOBB_FP8_QUANT_F(false, false, false);
    }
#undef DOBB_FP8_QUANT_F
#undef DOBB_FP8_QUANT
    return hipGetLastError();
}

hipError_t launch_fp8_dequantize(const dobb_fp8_operand &op, bool transpose, void *out, bool bf16, int64_t ldo, hipStream_t s) {
    const int64_t rb = fp8_read_rows(op.rows, transpose), T = fp8_read_tiles(op.k, transpose);
    if (T > kMaxWorkgroups / rb) return hipErrorInvalidValue;
    const dim3 grid((unsigned)(T * rb));
#define DOBB_FP8_READ(K, F)                                                                                            \
    DOBB_LAUNCH("fp8_dequantize", s, (K<F>), grid, dim3(256), 0, op.rows, op.k, (unsigned)rb, (const uint4 *)op.codes,    \
                (const uint8_t *)op.scales, out, bf16, ldo)
    if (transpose) {
        if (op.format == DOBB_E5M2) DOBB_FP8_READ(k_fp8_dequantize_t, DOBB_E5M2);
        else DOBB_FP8_READ(k_fp8_dequantize_t, DOBB_E4M3);
    } else {
        if (op.format == DOBB_E5M2) DOBB_FP8_READ(k_fp8_dequantize, DOBB_E5M2);
        else DOBB_FP8_READ(k_fp8_dequantize, DOBB_E4M3);
    }
#undef DOBB_FP8_READ
    return hipGetLastError();
}

}  // namespace dobb
