// One tile of a product of two FP8 operands (layout: dobb_layers.h) on the matrix cores.
//
// Two ways to multiply, by what the result is worth:
// * v_mfma_scale_f32_32x32x64_f8f6f4 on the codes, with the operands' own scale bytes.  The instruction adds its 64
//   products in groups of eight, and cuts each at 2^-13 of the power of two of the group's largest (found with a
//   large product and a small one: bits below that are dropped inside a group of eight, and none across groups or
//   against the accumulator).  Normal entries: 1.4e-5 of the result (2-norm).  For results in bf16, whose
//   rounding is a hundred times that.
// * EXACT: codes to bf16 by v_cvt_scalef32_pk_bf16_.. (exact from 2^-126 up) and v_mfma_f32_32x32x16_bf16, sums
//   in fp32 at half the rate.  For results in fp32.
// The operands' layout is the instructions', read 16 bytes a lane (the order of the contraction is free as
// long as both sides agree).  A workgroup of four waves computes TM x TN entries, a wave a quarter of them.
// Half a tile of k (64 entries) of both operands is a slot of TM + TN pieces of 64 bytes and their scales,
// which the memory engine writes straight into LDS; of NS slots one is multiplied while the others are on
// their way.  What orders loads and reads is the wait and barrier at the end of each half: all but the last NS - 2 halves'
// loads done, on every wave, before the next half is read.
// Rows past an operand's last and slots past the last are loaded from past the end of the buffer, as zeros.
#pragma once

#include "layers_common.h"
#include "moment_common.h"

namespace dobb {

typedef __attribute__((address_space(3))) void *lds_void;

constexpr unsigned kFp8Off = 0xffffffffu;      // buffer offset past the end: the load returns zeros

// rows row0 .. end - 1 of an operand of `rows` rows
struct Fp8Side {
    const uint8_t *codes, *scales;
    uint32_t rows, pitch;
    uint32_t row0, end;
};

// `bytes` of every lane from offset `off` of a buffer into LDS at dst + bytes * lane
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t r, void *dst, unsigned off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void)dst, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void lds_load4(__amdgpu_buffer_rsrc_t r, void *dst, unsigned off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void)dst, 4, off, 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void fp8_vm_wait() {
    static_assert(N >= 0 && N < 64, "vmcnt immediate");
    __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}
__device__ __forceinline__ void fp8_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// eight codes to bf16
template <int F>
__device__ __forceinline__ bf16x8 fp8_to_bf16(int lo, int hi, float scale) {
    bf16x2 p[4];
    if constexpr (F == DOBB_E4M3) {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    } else {
        p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
        p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
        p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
        p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
    }
    return bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// FA, FB: formats of the operands; acc[i][j]: rows 32 i .. of the wave's A side, 32 j .. of its B side
// SQUARE: both sides are one operand (TM = TN), of which each wave multiplies the pairs of `pairs` (bit kFN i + j)
template <int TM, int TN, int NS, int FA, int FB, bool EXACT, bool SQUARE = false>
struct Fp8Tile {
    static constexpr int kWM = TM / 2, kWN = TN / 2;             // of a wave
    static constexpr int kFM = kWM / 32, kFN = kWN / 32;
    static constexpr int kPieces = (TM + TN) * 64, kScales = 512;
    static constexpr int kSlot = kPieces + kScales;
    static constexpr int kLoads = (TM + TN) / 64 + 1;            // of a wave and slot
    static constexpr int kB = TM * 64;                           // of B's pieces in a slot
    uint32_t offA[TM / 64], offB[TN / 64], offS;
    Fp8Side a, b;
    bool scale_of_b;
    int wave, part;                   // part: the quarter that this wave multiplies
    uint32_t pairs = ~0u;
    bool same = false;                // the sides are the same rows: B's are not loaded again

    // Codes are read from row0, scales, which come by fours, from the word that holds row0's.
    __device__ __forceinline__ Fp8Tile(const Fp8Side &a_, const Fp8Side &b_) : a(a_), b(b_) {
        const int lane = threadIdx.x & 63;
        part = wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        same = SQUARE && a.row0 == b.row0;
#pragma unroll
        for (int k = 0; k < TM / 64; ++k) {
            const uint32_t r = a.row0 + 64 * k + lane;
            offA[k] = r < a.end ? ((uint32_t)wave * a.rows + r) * 16 : kFp8Off;
        }
#pragma unroll
        for (int k = 0; k < TN / 64; ++k) {
            const uint32_t r = b.row0 + 64 * k + lane;
            offB[k] = r < b.end && !same ? ((uint32_t)wave * b.rows + r) * 16 : kFp8Off;
        }
        // scales: 64 words from the word that holds row0's, by waves 0 and 2 of A, 1 and 3 of B
        scale_of_b = wave & 1;
        const Fp8Side &s = scale_of_b ? b : a;
        const uint32_t w = (s.row0 & ~3u) + 4 * lane;
        offS = w < s.pitch ? w : kFp8Off;
    }
    // half tile hs of H into buf (zeros past the last)
    __device__ __forceinline__ void issue(int64_t hs, int64_t end, uint8_t *buf) const {
        const bool in = hs < end;
        const int64_t at = in ? hs : 0;
        const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(a.codes) + at * 64 * a.rows, (short)0,
                                                                            in ? (int)(64 * a.rows) : 0, 0x00020000);
        const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(b.codes) + at * 64 * b.rows, (short)0,
                                                                            in ? (int)(64 * b.rows) : 0, 0x00020000);
        const uint8_t *sc = scale_of_b ? b.scales + (at >> 1) * b.pitch : a.scales + (at >> 1) * a.pitch;
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(sc), (short)0,
                                                                            in ? (int)(scale_of_b ? b.pitch : a.pitch) : 0, 0x00020000);
        lds_load4(rs, buf + kPieces + (scale_of_b ? 256 : 0), offS);
#pragma unroll
        for (int k = 0; k < TM / 64; ++k) lds_load16(ra, buf + (wave * TM + 64 * k) * 16, offA[k]);
#pragma unroll
        for (int k = 0; k < TN / 64; ++k) lds_load16(rb, buf + kB + (wave * TN + 64 * k) * 16, offB[k]);
    }
    struct Frags {                               // a wave's operands of half a tile, and their scales
        i32x8 x[kFM], y[kFN];
        uint32_t ea[kFM], eb[kFN];
    };
    __device__ __forceinline__ void read(const uint8_t *buf, Frags &f) const {
        const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
        const int ra = (part >> 1) * kWM + col, rb = (part & 1) * kWN + col;
        const uint8_t *sa = buf + kPieces + (a.row0 & 3u), *sb = buf + kPieces + 256 + (b.row0 & 3u);
        const uint8_t *bb = buf + (SQUARE && same ? 0 : kB);
#pragma unroll
        for (int i = 0; i < kFM; ++i) {
            const i32x4 lo = *(const i32x4 *)(buf + (half * TM + ra + 32 * i) * 16), hi = *(const i32x4 *)(buf + ((half + 2) * TM + ra + 32 * i) * 16);
            f.x[i] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            f.ea[i] = sa[ra + 32 * i];
        }
#pragma unroll
        for (int j = 0; j < kFN; ++j) {
            const i32x4 lo = *(const i32x4 *)(bb + (half * TN + rb + 32 * j) * 16), hi = *(const i32x4 *)(bb + ((half + 2) * TN + rb + 32 * j) * 16);
            f.y[j] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            f.eb[j] = sb[rb + 32 * j];
        }
    }
    __device__ __forceinline__ void multiply(const Frags &f, f32x16 (&acc)[kFM][kFN]) const {
        const auto &x = f.x;
        const auto &y = f.y;
        const auto &ea = f.ea;
        const auto &eb = f.eb;
        // B's rows are the accumulator's rows: a lane then holds four neighbouring columns of the output at a time
        if constexpr (EXACT) {
            float fa[kFM], fb[kFN];
#pragma unroll
            for (int i = 0; i < kFM; ++i) fa[i] = __uint_as_float(ea[i] << 23);
#pragma unroll
            for (int j = 0; j < kFN; ++j) fb[j] = __uint_as_float(eb[j] << 23);
            if constexpr (SQUARE) {
                if (!pairs) return;
                bf16x8 p[kFM][4], q[kFN][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int i = 0; i < kFM; ++i) p[i][k] = fp8_to_bf16<FA>(x[i][2 * k], x[i][2 * k + 1], fa[i]);
#pragma unroll
                    for (int j = 0; j < kFN; ++j) q[j][k] = fp8_to_bf16<FB>(y[j][2 * k], y[j][2 * k + 1], fb[j]);
                }
#pragma unroll
                for (int i = 0; i < kFM; ++i)
#pragma unroll
                    for (int j = 0; j < kFN; ++j)
                        if (pairs >> (kFN * i + j) & 1)
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[j][k], p[i][k], acc[i][j], 0, 0, 0);
                return;
            }
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
                bf16x8 p[kFM], q[kFN];
#pragma unroll
                for (int i = 0; i < kFM; ++i) p[i] = fp8_to_bf16<FA>(x[i][k], x[i][k + 1], fa[i]);
#pragma unroll
                for (int j = 0; j < kFN; ++j) q[j] = fp8_to_bf16<FB>(y[j][k], y[j][k + 1], fb[j]);
#pragma unroll
                for (int i = 0; i < kFM; ++i)
#pragma unroll
                    for (int j = 0; j < kFN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q[j], p[i], acc[i][j], 0, 0, 0);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < kFM; ++i)
#pragma unroll
            for (int j = 0; j < kFN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(y[j], x[i], acc[i][j], FB, FA, 0, (int)eb[j], 0, (int)ea[i]);
    }
    // acc += the products over half tiles h0 .. h1 - 1.  On return no load is in flight and every wave is done with LDS.
    // (Reading the next half's operands while this one's are multiplied measured no faster: two or three workgroups on
    // each CU cover the reads, and the registers cost one of three.)
    __device__ __forceinline__ void run(int64_t h0, int64_t h1, uint8_t *const (&buf)[NS], f32x16 (&acc)[kFM][kFN]) const {
#pragma unroll
        for (int k = 0; k < NS - 1; ++k) issue(h0 + k, h1, buf[k]);
        fp8_vm_wait<(NS - 2) * kLoads>();
        fp8_barrier();
        for (int64_t h = h0; h < h1; h += 2 * NS) {
#pragma unroll
            for (int k = 0; k < 2 * NS; ++k) {
                if (h + k >= h1) break;
                issue(h + k + NS - 1, h1, buf[(k + NS - 1) % NS]);
                Frags f;
                read(buf[k % NS], f);
                multiply(f, acc);
                fp8_vm_wait<(NS - 2) * kLoads>();
                fp8_barrier();
            }
        }
        fp8_vm_wait<0>();
    }
};

}  // namespace dobb
