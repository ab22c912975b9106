// Captures in MXFP4 (OCP Microscaling Formats: e2m1 elements, one e8m0 scale per 32 tokens of a
// column): quantising and reading back.  Layout: dobb_ops.h.
//
// One wave takes one group (32 tokens) of 128 columns, two neighbouring columns a lane: 32 row reads of
// 256 (bf16) or 512 (fp32) contiguous bytes, all in flight, no exchange between lanes for the largest
// magnitude, and 32 contiguous bytes of codes a lane.  The four waves of a workgroup take the four
// groups of a tile, whose scale bytes leave together through LDS.  HBM bounds both directions: 16384 x 6400 in
// bf16 (210 MB, 56 MB of codes and scales) quantises in 46 us (5.8 TB/s) and reads back in 43 (6.2 TB/s).
// The conversions are gfx950's scaled ones (v_cvt_scalef32_pk_fp4_f32, .._bf16 and back): nearest, ties to
// even, saturating at 6, exact for every scale from 2^-127 (checked against the definition on the card).
#include "ops_internal.h"

namespace dobb {
namespace {

constexpr int kCols = 128;   // columns per workgroup

typedef uint32_t __attribute__((aligned(2))) packed_u32;
template <bool BF16>
struct __attribute__((packed, aligned(2))) Pair { uint32_t w[BF16 ? 1 : 2]; };

// The scale byte of a group from its largest magnitude's exponent field: two below it, 255 if not finite
__device__ __forceinline__ uint32_t scale_byte(uint32_t field) { return field == 255 ? 255u : field < 2 ? 0u : field - 2; }
// the scale as the conversions take it: its byte is the exponent field, 0 stands for 2^-127
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// 32 tokens of two neighbouring columns: scale bytes and codes.  The largest magnitudes are found as
// integers (a NaN's bits are above an infinity's).  In bf16 both columns' at once in packed 16-bit
// integers, and one byte permute pairs two tokens of a column for the conversion from bf16: about half the
// vector instructions of going through fp32.
template <bool BF16>
__device__ __forceinline__ void quantize_pair(const Pair<BF16> (&v)[32], uint32_t &ea, uint32_t &eb, uint32_t (&qa)[4], uint32_t (&qb)[4]) {
    if constexpr (BF16) {
        u16x2 m = {0, 0};
#pragma unroll
        for (int k = 0; k < 32; ++k) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[k].w[0] & 0x7fff7fffu));
        ea = scale_byte((uint32_t)m[0] >> 7);
        eb = scale_byte((uint32_t)m[1] >> 7);
        const float sa = scale_of(ea), sb = scale_of(eb);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t p = 0, q = 0;
#define DOBB_MX4_PAIR(k)                                                                                             \
            p = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(                                                            \
                p, __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(v[8 * w + 2 * k + 1].w[0], v[8 * w + 2 * k].w[0], 0x05040100u)), sa, k); \
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(                                                            \
                q, __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(v[8 * w + 2 * k + 1].w[0], v[8 * w + 2 * k].w[0], 0x07060302u)), sb, k);
            DOBB_MX4_PAIR(0) DOBB_MX4_PAIR(1) DOBB_MX4_PAIR(2) DOBB_MX4_PAIR(3)
#undef DOBB_MX4_PAIR
            qa[w] = p;
            qb[w] = q;
        }
    } else {
        uint32_t ma = 0, mb = 0;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            ma = max(ma, v[k].w[0] & 0x7fffffffu);
            mb = max(mb, v[k].w[BF16 ? 0 : 1] & 0x7fffffffu);
        }
        ea = scale_byte(ma >> 23);
        eb = scale_byte(mb >> 23);
        const float sa = scale_of(ea), sb = scale_of(eb);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t p = 0, q = 0;
#define DOBB_MX4_AT(t, c) __uint_as_float(v[8 * w + (t)].w[BF16 ? 0 : (c)])
#define DOBB_MX4_PAIR(k)                                                                                             \
            p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, DOBB_MX4_AT(2 * k, 0), DOBB_MX4_AT(2 * k + 1, 0), sa, k);  \
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, DOBB_MX4_AT(2 * k, 1), DOBB_MX4_AT(2 * k + 1, 1), sb, k);
            DOBB_MX4_PAIR(0) DOBB_MX4_PAIR(1) DOBB_MX4_PAIR(2) DOBB_MX4_PAIR(3)
#undef DOBB_MX4_PAIR
#undef DOBB_MX4_AT
            qa[w] = p;
            qb[w] = q;
        }
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) {                           // a group that is not finite holds zeros
        if (ea == 255) qa[w] = 0;
        if (eb == 255) qb[w] = 0;
    }
}

template <bool BF16>
__global__ void __launch_bounds__(256) k_mx4_quantize(int64_t N, int64_t n, int64_t ldx, unsigned colblocks, const void *X,
                                                      uint4 *codes, uint32_t *scales) {
    __shared__ uint8_t sc[kCols][4];
    const int64_t tile = blockIdx.x / colblocks;
    const int64_t c0 = (int64_t)(blockIdx.x % colblocks) * kCols;
    const int g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t c = c0 + 2 * lane;
    const int64_t t0 = tile * kMx4Tile + 32 * g;
    const int rows = N - t0 < 0 ? 0 : N - t0 < 32 ? (int)(N - t0) : 32;
    // Every load is in bounds and unconditional (a condition would wait for each in turn): rows past the
    // last token repeat it and become zeros below, a pair past the last column moves to the last two.
    constexpr int ES = BF16 ? 2 : 4;
    const uint32_t xc = (uint32_t)(c + 1 < n ? c : n > 1 ? n - 2 : 0) * ES;
    const char *x = (const char *)X + (t0 < N ? t0 : 0) * ldx * ES;
    const int last = rows > 0 ? rows - 1 : 0;
    Pair<BF16> v[32];
    if (n > 1) {
#pragma unroll
        for (int k = 0; k < 32; ++k) {                      // read once: past the caches (16384 x 6400 in bf16:
            const uint32_t *r = (const uint32_t *)(x + min(k, last) * ldx * ES + xc);   // 62 -> 49 us)
            v[k].w[0] = __builtin_nontemporal_load((const packed_u32 *)r);
            if (!BF16) v[k].w[BF16 ? 0 : 1] = __builtin_nontemporal_load((const packed_u32 *)r + 1);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const char *r = x + min(k, last) * ldx * ES + xc;
            v[k].w[0] = BF16 ? *(const uint16_t *)r : *(const uint32_t *)r;
            if (!BF16) v[k].w[BF16 ? 0 : 1] = 0;
        }
    }
    if (n > 1 && c + 1 >= n)                                // the pair's second column is this lane's first
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k].w[0] = BF16 ? v[k].w[0] >> 16 : v[k].w[BF16 ? 0 : 1];
    if (rows < 32)
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (k >= rows) v[k].w[0] = v[k].w[BF16 ? 0 : 1] = 0;
    uint32_t qa[4], qb[4], ea, eb;
    quantize_pair<BF16>(v, ea, eb, qa, qb);
    uint4 *o = codes + (tile * 4 + g) * n + c;
    if (c < n) o[0] = uint4{qa[0], qa[1], qa[2], qa[3]};
    if (c + 1 < n) o[1] = uint4{qb[0], qb[1], qb[2], qb[3]};
    sc[2 * lane][g] = (uint8_t)ea;
    sc[2 * lane + 1][g] = (uint8_t)eb;
    __syncthreads();
    if (threadIdx.x < kCols && c0 + threadIdx.x < n) scales[tile * n + c0 + threadIdx.x] = *(const uint32_t *)sc[threadIdx.x];
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

template <bool BF16>
__global__ void __launch_bounds__(256) k_mx4_dequantize(int64_t N, int64_t n, int64_t ldo, unsigned colblocks, const uint4 *codes,
                                                        const uint8_t *scales, void *out) {
    const int64_t tile = blockIdx.x / colblocks;
    const int64_t c0 = (int64_t)(blockIdx.x % colblocks) * kCols;
    const int g = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t c = c0 + 2 * lane;
    const int64_t t0 = tile * kMx4Tile + 32 * g;
    if (c >= n || t0 >= N) return;
    const int rows = N - t0 < 32 ? (int)(N - t0) : 32;
    const bool two = c + 1 < n;
    const uint4 *p = codes + (tile * 4 + g) * n + c;
    const uint4 ca = p[0], cb = two ? p[1] : uint4{0, 0, 0, 0};
    const uint8_t *s = scales + (tile * n + c) * 4 + g;
    const uint32_t ea = s[0], eb = two ? s[4] : 0;
    const float sa = scale_of(ea), sb = scale_of(eb);
    const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
    constexpr int ES = BF16 ? 2 : 4;
    char *o = (char *)out + t0 * ldo * ES;
    const uint32_t oc = (uint32_t)c * ES;
    float a[32], b[32];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f32x2 x;
#define DOBB_MX4_PAIR(k)                                                     \
        x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(wa[w], sa, k);          \
        a[8 * w + 2 * k] = x[0]; a[8 * w + 2 * k + 1] = x[1];                \
        x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(wb[w], sb, k);          \
        b[8 * w + 2 * k] = x[0]; b[8 * w + 2 * k + 1] = x[1];
        DOBB_MX4_PAIR(0) DOBB_MX4_PAIR(1) DOBB_MX4_PAIR(2) DOBB_MX4_PAIR(3)
#undef DOBB_MX4_PAIR
    }
    const float nan = __builtin_nanf("");
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        if (ea == 255) a[k] = nan;
        if (eb == 255) b[k] = nan;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        if (k >= rows) break;
        char *r = o + k * ldo * ES + oc;
        if (two) {
            Pair<BF16> v;
            if (BF16) v.w[0] = (uint32_t)f32_to_bf16(a[k]) | ((uint32_t)f32_to_bf16(b[k]) << 16);
            else { v.w[0] = __float_as_uint(a[k]); v.w[BF16 ? 0 : 1] = __float_as_uint(b[k]); }
            *(Pair<BF16> *)r = v;
        } else if (BF16) *(uint16_t *)r = f32_to_bf16(a[k]);
        else *(float *)r = a[k];
    }
}

// workgroups of a capture, 0 if a grid cannot hold them
unsigned mx4_grid(int64_t N, int64_t n, unsigned *colblocks) {
    *colblocks = (unsigned)((n + kCols - 1) / kCols);
    const int64_t tiles = N / kMx4Tile + (N % kMx4Tile != 0);
    if (tiles > 0x7fffffff / *colblocks) return 0;
    return (unsigned)(tiles * *colblocks);
}

}  // namespace

hipError_t launch_mx4_quantize(int64_t N, int64_t n, const void *X, bool bf16, int64_t ldx, void *codes, void *scales,
                               hipStream_t s) {
    unsigned cb;
    const unsigned grid = mx4_grid(N, n, &cb);
    if (!grid) return hipErrorInvalidValue;
    if (bf16) DOBB_LAUNCH("mx4_quantize", s, k_mx4_quantize<true>, dim3(grid), dim3(256), 0, N, n, ldx, cb, X, (uint4 *)codes, (uint32_t *)scales);
    else DOBB_LAUNCH("mx4_quantize", s, k_mx4_quantize<false>, dim3(grid), dim3(256), 0, N, n, ldx, cb, X, (uint4 *)codes, (uint32_t *)scales);
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(int64_t N, int64_t n, const void *codes, const void *scales, void *out, bool bf16,
                                 int64_t ldo, hipStream_t s) {
    unsigned cb;
    const unsigned grid = mx4_grid(N, n, &cb);
    if (!grid) return hipErrorInvalidValue;
    if (bf16) DOBB_LAUNCH("mx4_dequantize", s, k_mx4_dequantize<true>, dim3(grid), dim3(256), 0, N, n, ldo, cb, (const uint4 *)codes, (const uint8_t *)scales, out);
    else DOBB_LAUNCH("mx4_dequantize", s, k_mx4_dequantize<false>, dim3(grid), dim3(256), 0, N, n, ldo, cb, (const uint4 *)codes, (const uint8_t *)scales, out);
    return hipGetLastError();
}

}  // namespace dobb
