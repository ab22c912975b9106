// Device helpers of the layer operators (not installed).
#pragma once

#include "layers_internal.h"

namespace dobb {

// eight neighbouring entries of a row, aligned to their entries only
template <bool BF16>
struct __attribute__((packed, aligned(2))) Raw8 { uint32_t w[BF16 ? 4 : 8]; };

template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw8<BF16> &r, float (&v)[8]) {
    if constexpr (BF16) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(r.w[k] << 16);
            v[2 * k + 1] = __uint_as_float(r.w[k] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.w[k]);
    }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    return BF16 ? bf16_to_f32(((const uint16_t *)p)[i]) : ((const float *)p)[i];
}
__device__ __forceinline__ float load1(const void *p, int64_t i, bool bf16) { return bf16 ? load1<true>(p, i) : load1<false>(p, i); }

// entries c .. c + 7 of a row, zeros from n on
template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8(const void *row, int64_t c, int64_t n) {
    constexpr int ES = BF16 ? 2 : 4;
    if (c + 8 <= n) return *(const Raw8<BF16> *)((const char *)row + c * ES);
    Raw8<BF16> r;
#pragma unroll
    for (int k = 0; k < (BF16 ? 4 : 8); ++k) r.w[k] = 0;
    if (c < n) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < n) {
                if (BF16) r.w[k / 2] |= (uint32_t)((const uint16_t *)row)[c + k] << (16 * (k & 1));
                else r.w[BF16 ? 0 : k] = ((const uint32_t *)row)[c + k];
            }
    }
    return r;
}

// to nearest, ties to even (v_cvt_pk_bf16_f32)
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) { return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b}); }

__device__ __forceinline__ void store8(void *row, int64_t c, int64_t n, const float (&v)[8], bool bf16) {
    if (bf16) {
        if (c + 8 <= n) {
            Raw8<true> r;
#pragma unroll
            for (int k = 0; k < 4; ++k) r.w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
            *(Raw8<true> *)((char *)row + c * 2) = r;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (c + k < n) ((uint16_t *)row)[c + k] = f32_to_bf16(v[k]);
        }
    } else if (c + 8 <= n) {
        Raw8<false> r;
#pragma unroll
        for (int k = 0; k < 8; ++k) r.w[k] = __float_as_uint(v[k]);
        *(Raw8<false> *)((char *)row + c * 4) = r;
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (c + k < n) ((float *)row)[c + k] = v[k];
    }
}

// entries c .. c + 7 of a weight or bias (zeros from n on), `missing` where there is none
__device__ __forceinline__ void affine8(const void *p, int64_t c, int64_t n, bool bf16, float missing, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = missing;
    } else if (bf16) unpack8<true>(load8<true>(p, c, n), v);
    else unpack8<false>(load8<false>(p, c, n), v);
}

// What each of a group of 16 lanes receives from a lane of it: exchanges with the lane whose number differs
// in bit 0, in bit 1, then the mirrored one of 8 and of 16: after the four, a butterfly over 16 lanes.
template <int STEP>
__device__ __forceinline__ uint32_t lane16(uint32_t x) {
    constexpr int ctrl = STEP == 0 ? 0xB1 : STEP == 1 ? 0x4E : STEP == 2 ? 0x141 : 0x140;
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t max16(uint32_t x) {
    x = max(x, lane16<0>(x));
    x = max(x, lane16<1>(x));
    x = max(x, lane16<2>(x));
    return max(x, lane16<3>(x));
}
__device__ __forceinline__ float sum16(float x) {
    x += __uint_as_float(lane16<0>(__float_as_uint(x)));
    x += __uint_as_float(lane16<1>(__float_as_uint(x)));
    x += __uint_as_float(lane16<2>(__float_as_uint(x)));
    return x + __uint_as_float(lane16<3>(__float_as_uint(x)));
}
__device__ __forceinline__ float wave_sum(float x) {
    x = sum16(x);
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// A normalised entry; one function, so that the norm and the quantiser that normalises agree bit for bit
__device__ __forceinline__ float norm_value(float x, float mean, float rstd, float w, float b) { return fmaf((x - mean) * rstd, w, b); }

}  // namespace dobb
