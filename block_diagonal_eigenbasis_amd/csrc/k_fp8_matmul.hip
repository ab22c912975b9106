// out_ij = sum_t 2^(ea_it + eb_jt) sum_k a_itk b_jtk (+ bias_j) (+ out_ij) for two FP8 operands (dobb_layers.h), t over
// tiles of 128 entries: the scaled matrix instructions take the exponents with the codes, so nothing is left for the
// vector units but the epilogue.  Their sums drop what is 2^-13 below the largest of eight products (1.4e-5 of a result
// of normal data), a hundredth of what rounding to bf16 costs; results in fp32 take codes converted to bf16 (exactly) and
// that type's instruction, which drops nothing, at half the rate.  Sums are fp32, parts of k are added in their order.
//
// Three kernels (matmul_plan): up to 32 rows on one side stream the other operand (HBM bounds it: 11008 x 4096 of 45 MB
// in 10.3 us); tiles of 64 x 64 or 128 x 128, over parts of k where there are few of them; persistent 256 x 256 tiles.
// Large products: the scaled instruction alone runs 3.67 PFLOP/s on random codes (4.95 on zeros: power sets the clock;
// the 16x16x128 one 4.29), the bf16 one 1.67 (2.46).  8192^3: 2.70 to 2.82 PFLOP/s to bf16, 1.49 to 1.52 to fp32.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fp8_tile.h"
#include "load_stream.h"

namespace dobb {
namespace {

struct Epilogue {
    void *out;
    const void *bias;
    int64_t ldo;
    bool bf16, bias_bf16, accumulate;
};

__device__ __forceinline__ void store1(const Epilogue &e, int64_t m, int64_t n, float v) {
    if (e.bias) v += load1(e.bias, n, e.bias_bf16);
    const int64_t at = m * e.ldo + n;
    if (e.accumulate) v += load1(e.out, at, e.bf16);
    if (e.bf16) ((uint16_t *)e.out)[at] = f32_to_bf16(v);
    else ((float *)e.out)[at] = v;
}

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

// ---- few tiles -------------------------------------------------------------------------------------
// TM x TN entries a workgroup, over one of nsplit parts of k: the result, or with more than one part a partial
// product (parts x M x N in fp32) for k_fp8_join.
template <int TM, int TN, int NS, int FA, int FB, bool EXACT>
__global__ void __launch_bounds__(256, 2) k_fp8_matmul(Fp8Side a, Fp8Side b, int64_t tiles, int tilesN, int nsplit, Epilogue e, float *part) {
    using T = Fp8Tile<TM, TN, NS, FA, FB, EXACT>;
    __shared__ __align__(16) uint8_t ring[NS][T::kSlot];
    uint8_t *bufs[NS];
#pragma unroll
    for (int k = 0; k < NS; ++k) bufs[k] = ring[k];
    const int id = xcd_remap(blockIdx.x, gridDim.x);
    const int split = id % nsplit, tile = id / nsplit;
    const int64_t per = (tiles + nsplit - 1) / nsplit, t0 = per * split, t1 = min(t0 + per, tiles);
    a.row0 = (uint32_t)(tile / tilesN) * TM;
    b.row0 = (uint32_t)(tile % tilesN) * TN;
    const T t(a, b);
    f32x16 acc[T::kFM][T::kFN];
#pragma unroll
    for (int i = 0; i < T::kFM; ++i)
#pragma unroll
        for (int j = 0; j < T::kFN; ++j) acc[i][j] = f32x16{};
    t.run(2 * t0, 2 * t1, bufs, acc);
    const int lane = threadIdx.x & 63;
    if (nsplit > 1) e = Epilogue{part + (int64_t)split * a.rows * b.rows, nullptr, (int64_t)b.rows, false, false, false};
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

// the parts' sums, in order, four neighbouring entries a thread
__global__ void __launch_bounds__(256) k_fp8_join(int64_t M, int64_t N, int nsplit, const float *part, Epilogue e) {
    const int64_t quads = (N + 3) / 4, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= M * quads) return;
    const int64_t m = at / quads, n = at % quads * 4;
    const float *p = part + m * N + n;
    f32x4 s{};
    if (n + 4 <= N) {
        for (int k = 0; k < nsplit; ++k) s += *(const f32x4u *)(p + k * M * N);
    } else
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (n + r < N)
                for (int k = 0; k < nsplit; ++k) s[r] += p[k * M * N + r];
    store4(e, m, n, N, s);
}

// ---- few rows --------------------------------------------------------------------------------------
// An operand b of many rows against one, a, of at most 32: b is read once, straight into the instruction's
// registers.  A workgroup takes 32 rows of b, its W waves every W-th tile of k, some tiles' loads in flight, and adds
// their sums up in the order of the waves through LDS.  `turned`: b is the product's A, so the output is transposed.
template <int FA, int FB, bool EXACT>
__global__ void __launch_bounds__(256) k_fp8_matmul_thin(Fp8Side a, Fp8Side b, int64_t tiles, bool turned, Epilogue e) {
    constexpr int kAhead = 4;
    extern __shared__ float sums[];              // W x 32 x 32
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
    const int col = lane & 31, half = lane >> 5;
    const uint32_t n0 = (uint32_t)xcd_remap(blockIdx.x, gridDim.x) * 32;
    const uint32_t rb = min(n0 + col, b.rows - 1), ra = min((uint32_t)col, a.rows - 1);
    f32x16 acc{};
    for (int64_t t = wave; t < tiles; t += kAhead * W) {
        i32x4 x[kAhead][4], y[kAhead][4];        // a half-wave's pieces of a tile: every other one
        uint32_t ea[kAhead], eb[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t tt = min(t + k * W, tiles - 1);
            const i32x4 *pa = (const i32x4 *)a.codes + (tt * 8 + half) * a.rows + ra, *pb = (const i32x4 *)b.codes + (tt * 8 + half) * b.rows + rb;
            ea[k] = a.scales[tt * a.pitch + ra];
            eb[k] = b.scales[tt * b.pitch + rb];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                y[k][h] = pb[(uint64_t)(2 * h) * b.rows];
                x[k][h] = pa[(uint64_t)(2 * h) * a.rows];
            }
        }
        batch();
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (t + k * W >= tiles) break;
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                if constexpr (EXACT) {
                    const float fa = __uint_as_float(ea[k] << 23), fb = __uint_as_float(eb[k] << 23);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const i32x4 &p = x[k][h + (u >> 1)], &q = y[k][h + (u >> 1)];
                        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp8_to_bf16<FB>(q[2 * (u & 1)], q[2 * (u & 1) + 1], fb),
                                                                     fp8_to_bf16<FA>(p[2 * (u & 1)], p[2 * (u & 1) + 1], fa), acc, 0, 0, 0);
                    }
                } else {
                    const i32x4 &p0 = x[k][h], &p1 = x[k][h + 1], &q0 = y[k][h], &q1 = y[k][h + 1];
                    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(i32x8{q0[0], q0[1], q0[2], q0[3], q1[0], q1[1], q1[2], q1[3]},
                                                                          i32x8{p0[0], p0[1], p0[2], p0[3], p1[0], p1[1], p1[2], p1[3]}, acc, FB, FA, 0,
                                                                          (int)eb[k], 0, (int)ea[k]);
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)                  // [wave][row of a][row of b]
        *(f32x4 *)(sums + (wave * 32 + col) * 32 + 8 * q + 4 * half) = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    __syncthreads();
    for (uint32_t at = threadIdx.x; at < 32 * a.rows; at += blockDim.x) {
        float s = sums[at];
        for (int w = 1; w < W; ++w) s += sums[w * 1024 + at];
        const uint32_t m = at >> 5, n = n0 + (at & 31);
        if (n < b.rows) store1(e, turned ? n : m, turned ? m : n, s);
    }
}

// ---- large products --------------------------------------------------------------------------------
// A workgroup of four waves a CU, 256 x 256 entries at a time, a wave a quarter of them in 256 accumulators: the LDS
// then serves 1.33 times the bytes that the matrix cores leave it time for (at 128 x 64 a wave, 0.89).  With one
// wave a SIMD nothing else covers a wait, so everything is one stream: half tiles of k, tile after tile, go
// through a ring of four slots; a wave's operands of the next half are read while this one is multiplied, the slot
// that it has left is loaded again behind the barrier, three halves ahead, and a tile's results leave while the
// next one's first slots are on their way.  The loads into LDS are written in assembly (they have no register to
// return to): the compiler would wait for all of them before each read of LDS.
constexpr int kBig = 256;
constexpr int kBigPieces = 2 * kBig * 64, kBigSlot = kBigPieces + 2 * kBig;

// m0, which takes the LDS address, is put back: it cannot be named as overwritten, and the compiler may hold a value of
// its own there.  One block for two loads, so that this is two scalar moves for both (0.5 to 1 % of a product to fp32, less
// of one to bf16).
__device__ __forceinline__ void dma16(const i32x4 &ra, uint32_t la, uint32_t oa, const i32x4 &rb, uint32_t lb, uint32_t ob) {
    uint32_t held;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds\n\t"
                 "s_mov_b32 m0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %5, %6, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(held) : "s"(la), "v"(oa), "s"(ra), "s"(lb), "v"(ob), "s"(rb));
}
__device__ __forceinline__ void dma4(const i32x4 &rsrc, uint32_t lds, uint32_t off) {
    uint32_t held;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
                 : "=&s"(held) : "s"(lds), "v"(off), "s"(rsrc));
}
__device__ __forceinline__ i32x4 buffer_of(const uint8_t *p, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)p;
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xffffu)),
                 __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
// all but the last N memory operations of this wave done (all but the last M where `more`), its LDS reads too, and
// every wave here
template <int N, int M>
__device__ __forceinline__ void wait_all_but(int more) {
    asm volatile("s_cmp_lg_u32 %2, 0\n\ts_cbranch_scc1 1f\n\ts_waitcnt vmcnt(%0)\n\ts_branch 2f\n1:\ts_waitcnt vmcnt(%1)\n2:\ts_waitcnt lgkmcnt(0)\n\ts_barrier"
                 ::"n"(N), "n"(M), "s"(__builtin_amdgcn_readfirstlane(more)) : "memory", "scc");
}
template <int N>
__device__ __forceinline__ void wait_all_but() {
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_waitcnt lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
// An accumulator's entry, fetched where it is used: the compiler moves all 256 into registers of the other kind at once,
// more than there are, and each one that it has to fetch back from memory then waits for the stores in flight.
__device__ __forceinline__ float acc_read(float a) {
    float v;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
    return v;
}
// what an instruction written in assembly has to leave between a matrix instruction and its read (19 at most)
__device__ __forceinline__ void acc_wait() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
// keeps the order in which the source interleaves products, reads and loads
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

// Tile t of a round-robin over the chip: workgroup ids go round the XCDs, whose 32 workgroups then take
// 32 neighbouring tiles, 8 rows of tiles by 4 columns: an XCD's L2 reads 12 strips for 32 tiles' 64.
struct TileAt {
    uint32_t m, n;
};
__device__ __forceinline__ TileAt tile_at(uint32_t t, uint32_t tm, uint32_t tn) {
    constexpr uint32_t G = 8;
    const uint32_t group = t / (G * tn), r = t - group * (G * tn);
    const uint32_t rows = min(G, tm - group * G);
    return {group * G + r % rows, r / rows};
}

using No = std::false_type;
using Yes = std::true_type;

#define DOBB_INLINE __attribute__((always_inline))

struct BigArgs {
    Fp8Side a, b;
    uint32_t tm, tn;
    int halves;
    Epilogue e;
};

// A wave's results leave through a patch of LDS in rows of 128 bytes, as the L2 takes them (stored as they lie in the
// registers, 32 bytes of 32 rows at a time: 16384 x 4800 x 1600 in 148 us instead of 139); those that are
// added to an output in bf16 entry by entry.
constexpr int kPatchRow = 128 + 16;              // bytes; the padding spreads rows over the banks
constexpr int kPatch = kPatchRow / 4;
typedef int i32x4u __attribute__((ext_vector_type(4), aligned(2)));

template <int FA, int FB, bool EXACT>
__global__ void __launch_bounds__(256, 1) k_fp8_matmul_big(BigArgs g) {
    __shared__ __align__(16) uint8_t ring[kRing * kBigSlot];
    __shared__ __align__(16) uint8_t patch[4][32 * kPatchRow];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, half = lane >> 5;
    const uint32_t tiles = g.tm * g.tn, stride = gridDim.x;
    const uint32_t first = (uint32_t)xcd_remap(blockIdx.x, gridDim.x);
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ring;
    const int H = g.halves;

    // the stream of loads: slot `is`, half ih of tile `it`
    uint32_t it = first, offA[4], offB[4], offS = kFp8Off;
    int ih = 0, is = 0;
    const bool of_b = wave & 1;
    const uint8_t *pa, *pb, *ps;
    const uint32_t pitch = of_b ? g.b.pitch : g.a.pitch;
    auto aim = [&]() DOBB_INLINE {                           // at tile `it` (past the last: at nothing)
        const bool in = it < tiles;
        const TileAt t = tile_at(in ? it : 0, g.tm, g.tn);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t r = t.m * kBig + 64 * k + lane, q = t.n * kBig + 64 * k + lane;
            offA[k] = in && r < g.a.rows ? ((uint32_t)wave * g.a.rows + r) * 16 : kFp8Off;
            offB[k] = in && q < g.b.rows ? ((uint32_t)wave * g.b.rows + q) * 16 : kFp8Off;
        }
        const uint32_t w = (of_b ? t.n : t.m) * kBig + 4 * lane;
        offS = in && w < pitch ? w : kFp8Off;
        pa = g.a.codes;
        pb = g.b.codes;
        ps = of_b ? g.b.scales : g.a.scales;
    };
    // part 0..3 of a half: a load of A, one of B (and the scales of a tile of k with its first half)
    auto issue = [&](int part, bool scales) DOBB_INLINE {
        const uint32_t slot = base + (uint32_t)is * kBigSlot;
        if (scales) {
            dma4(buffer_of(ps, pitch), slot + kBigPieces + (of_b ? kBig : 0), offS);
            ps += pitch;
        }
        const uint32_t to = slot + (wave * kBig + 64 * part) * 16;
        dma16(buffer_of(pa, 64 * g.a.rows), to, offA[part], buffer_of(pb, 64 * g.b.rows), to + kBig * 64, offB[part]);
        if (part == 3) {
            pa += (uint64_t)64 * g.a.rows;
            pb += (uint64_t)64 * g.b.rows;
            is = (is + 1) & (kRing - 1);
            ++ih;
        }
    };
    auto step_tile = [&]() DOBB_INLINE {                     // before two halves
        if (ih == H) {
            ih = 0;
            it += stride;
            aim();
        }
    };

    // a wave's operands of one half: fragments 0..3 of A, 4..7 of B
    const int ra = (wave >> 1) * 128 + col, rb = (wave & 1) * 128 + col;
    const uint32_t at[2] = {(uint32_t)(half * kBig + ra) * 16, (uint32_t)(kBig * 64 + (half * kBig + rb) * 16)};
    auto read = [&](i32x8 (&f)[8], int k, int s) DOBB_INLINE {
        const uint8_t *p = ring + s * kBigSlot + at[k >> 2] + 512 * (k & 3);
        const i32x4 lo = *(const i32x4 *)p, hi = *(const i32x4 *)(p + 2 * kBig * 16);
        f[k] = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    auto read_scale = [&](uint32_t (&e)[8], int k, int s) DOBB_INLINE {
        e[k] = ring[s * kBigSlot + kBigPieces + (k < 4 ? ra + 32 * k : kBig + rb + 32 * (k - 4))];
    };
    f32x16 acc[4][4];
    i32x8 f0[8], f1[8];
    uint32_t e0[8], e1[8];
    int c[2][8][4];                              // EXACT: eight entries of every fragment in bf16, this step's and the next one's
    // two of the four words: entries 8 q + 4 w .. + 3 of fragment k
    auto convert = [&](int to, int k, int w, int src, uint32_t e) DOBB_INLINE {
        const float scale = __uint_as_float(e << 23);
        bf16x2 lo, hi;
        if ((k < 4 ? FA : FB) == DOBB_E4M3) {
            lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(src, scale, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(src, scale, true);
        } else {
            lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(src, scale, false);
            hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(src, scale, true);
        }
        c[to][k][2 * w] = __builtin_bit_cast(int, lo);
        c[to][k][2 * w + 1] = __builtin_bit_cast(int, hi);
    };
    auto wide = [](const int (&c)[4]) DOBB_INLINE { return __builtin_bit_cast(bf16x8, i32x4{c[0], c[1], c[2], c[3]}); };

    // One half: the products of f, and between them the reads of the next half's operands (and scales, where `scales`
    // the tile of k is the next one) and the loads of the half three ahead.
    auto body = [&](auto fresh, const i32x8 (&f)[8], const uint32_t (&e)[8], i32x8 (&nf)[8], uint32_t (&ne)[8], auto odd, int s) DOBB_INLINE {
        constexpr bool FRESH = decltype(fresh)::value, ODD = decltype(odd)::value;
        const f32x16 zero{};
        if constexpr (!EXACT) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f[4 + j], f[i], FRESH ? zero : acc[i][j], FB, FA, 0,
                                                                                (int)e[4 + j], 0, (int)e[i]);
                    pin();
                    const int k = 4 * i + j;
                    if (k < 8) read(nf, k, s);
                    else if (k < 12) issue(k - 8, !ODD && k == 8);
                    else if (ODD) {
                        read_scale(ne, 2 * (k - 12), s);
                        read_scale(ne, 2 * (k - 12) + 1, s);
                    }
                    pin();
                }
        } else {
            auto step = [&](auto nq) DOBB_INLINE {           // entries 8 q .. + 7 of a lane, and the conversion of the next eight
                constexpr int q = decltype(nq)::value;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wide(c[q & 1][4 + j]), wide(c[q & 1][i]), FRESH && q == 0 ? zero : acc[i][j], 0, 0, 0);
                        pin();
                        const int k = 4 * i + j;
                        if constexpr (q < 3) convert((q + 1) & 1, k >> 1, k & 1, f[k >> 1][2 * (q + 1) + (k & 1)], e[k >> 1]);
                        else if constexpr (ODD) convert(0, k >> 1, k & 1, nf[k >> 1][k & 1], ne[k >> 1]);
                        else convert(0, k >> 1, k & 1, nf[k >> 1][k & 1], e[k >> 1]);
                        if constexpr (q == 0) {
                            if (k < 8) read(nf, k, s);
                            else if (ODD && k < 12) {
                                read_scale(ne, 2 * (k - 8), s);
                                read_scale(ne, 2 * (k - 8) + 1, s);
                            }
                        } else if constexpr (q == 1) {
                            if ((k & 3) == 0) issue(k >> 2, !ODD && k == 0);
                        }
                        pin();
                    }
            };
            step(std::integral_constant<int, 0>());
            step(std::integral_constant<int, 1>());
            step(std::integral_constant<int, 2>());
            step(std::integral_constant<int, 3>());
        }
    };

    aim();
#pragma unroll
    for (int k = 0; k < kRing; ++k) {
        if (!(k & 1)) step_tile();
#pragma unroll
        for (int part = 0; part < 4; ++part) issue(part, !(k & 1) && part == 0);
    }
    wait_all_but<kStartLeft>();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        read(f0, k, 0);
        read_scale(e0, k, 0);
    }
    if constexpr (EXACT)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            convert(0, k, 0, f0[k][0], e0[k]);
            convert(0, k, 1, f0[k][1], e0[k]);
        }
    int s = 0;                                   // slot of the half that is multiplied
    // Three halves of the next tile are on their way when a tile's results leave: the waits for them, and no others, leave
    // out the stores behind them (load_stream.h: 32 in bf16, 46 of the 64 in fp32).
    StreamWaits waits;
    constexpr int kLeft = stream_left(EXACT);
    for (uint32_t tile = first; tile < tiles; tile += stride) {
        auto pair = [&](auto fresh) DOBB_INLINE {
            step_tile();                         // (a branch behind the products would let the compiler move them past it)
            wait_all_but<kBehind, kLeft>(waits.next());
            body(fresh, f0, e0, f1, e1, No(), (s + 1) & 3);
            wait_all_but<kBehind, kLeft>(waits.next());
            body(No(), f1, e0, f0, e1, Yes(), (s + 2) & 3);
#pragma unroll
            for (int k = 0; k < 8; ++k) e0[k] = e1[k];
            s = (s + 2) & 3;
        };
        pair(Yes());
        for (int h = 2; h < H; h += 2) pair(No());
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));   // they stay where they are
        acc_wait();
        const TileAt t = tile_at(tile, g.tm, g.tn);
        const int64_t m0 = (int64_t)t.m * kBig + (wave >> 1) * 128, n0 = (int64_t)t.n * kBig + (wave & 1) * 128;
        if (EXACT || !g.e.accumulate) {
            // by 32 rows of 128 bytes: registers to LDS as they lie, LDS to memory in rows, 16 bytes a lane
            constexpr int JS = EXACT ? 1 : 2, ES = EXACT ? 4 : 2;   // fragments side by side, bytes of an entry
            const bool whole = (t.m + 1) * kBig <= g.a.rows && (t.n + 1) * kBig <= g.b.rows;
            const bool stored = whole && !g.e.accumulate;
            waits.stored(stored);
            uint8_t *mine = patch[wave];
            uint8_t *put = mine + col * kPatchRow + (EXACT ? 16 : 8) * half;
            const uint8_t *get = mine + (lane >> 3) * kPatchRow + (lane & 7) * 16;
            char *out = (char *)g.e.out + ((m0 + (lane >> 3)) * g.e.ldo + n0) * ES + (lane & 7) * 16;
            const int64_t row8 = 8 * g.e.ldo * ES;
#pragma unroll
            for (int j = 0; j < 4; j += JS) {
                f32x4 bias[JS][4];
#pragma unroll
                for (int u = 0; u < JS; ++u)
#pragma unroll
                    for (int q = 0; q < 4; ++q) bias[u][q] = f32x4{};
                if (g.e.bias)
#pragma unroll
                    for (int u = 0; u < JS; ++u)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int64_t n = n0 + 32 * (j + u) + 8 * q + 4 * half;
                            if (whole && !g.e.bias_bf16) bias[u][q] = *(const f32x4u *)((const float *)g.e.bias + n);
                            else
#pragma unroll
                                for (int r = 0; r < 4; ++r) bias[u][q][r] = load1(g.e.bias, min<int64_t>(n + r, (int64_t)g.b.rows - 1), g.e.bias_bf16);
                        }
                // this lane's columns of the output
                const int64_t n = n0 + 32 * j + (lane & 7) * (16 / ES);
                const int cols = n >= g.b.rows ? 0 : (int)min<int64_t>(g.b.rows - n, 16 / ES);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int u = 0; u < JS; ++u)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f32x16 &c = acc[i][j + u];
                            const f32x4 v = f32x4{acc_read(c[4 * q]), acc_read(c[4 * q + 1]), acc_read(c[4 * q + 2]), acc_read(c[4 * q + 3])} + bias[u][q];
                            if constexpr (EXACT) *(f32x4 *)(put + 32 * q) = v;
                            else *(uint2 *)(put + 64 * u + 16 * q) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                        }
                    pin();
                    i32x4 w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = *(const i32x4 *)(get + 8 * k * kPatchRow);
                    char *o = out + 4 * i * row8 + 128 * (j / JS);
                    if (stored) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) *(i32x4u *)(o + k * row8) = w[k];
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (m0 + 32 * i + 8 * k + (lane >> 3) >= g.a.rows) continue;
                            char *at = o + k * row8;
                            if constexpr (EXACT) {
                                f32x4 v = __builtin_bit_cast(f32x4, w[k]);
                                if (cols == 4) {
                                    if (g.e.accumulate) v += *(const f32x4u *)at;
                                    *(f32x4u *)at = v;
                                } else
#pragma unroll
                                    for (int r = 0; r < 3; ++r)
                                        if (r < cols) ((float *)at)[r] = g.e.accumulate ? v[r] + ((float *)at)[r] : v[r];
                            } else if (cols == 8) *(i32x4u *)at = w[k];
                            else
#pragma unroll
                                for (int r = 0; r < 7; ++r)
                                    if (r < cols) ((uint16_t *)at)[r] = (uint16_t)((uint32_t)w[k][r >> 1] >> (16 * (r & 1)));
                        }
                    }
                    pin();
                }
            }
        } else {
            waits.stored(false);
            float *mine = (float *)patch[wave];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (m0 + 32 * i >= g.a.rows || n0 + 32 * j >= g.b.rows) continue;
#pragma unroll
                    for (int r = 0; r < 16; ++r) mine[col * kPatch + acc_row(r, lane)] = acc_read(acc[i][j][r]);
                    __builtin_amdgcn_wave_barrier();
#pragma unroll 1
                    for (int r = 0; r < 16; ++r) {
                        const int64_t m = m0 + 32 * i + 2 * r + half, n = n0 + 32 * j + col;
                        if (m < g.a.rows && n < g.b.rows) store1(g.e, m, n, mine[(2 * r + half) * kPatch + col]);
                    }
                    __builtin_amdgcn_wave_barrier();
                }
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace

// Which kernel a product takes, and in how many parts of k: the one that an estimate of the time makes fastest.  Half
// a tile of k takes a workgroup of 64 x 64 entries 0.17 us and the chip 0.155 us for every 256 of them (to fp32 0.31
// and 0.2), one of 128 x 128 0.32 and 0.32 (0.6 and 0.53), one of 256 x 256, alone on its CU, 0.58 (1.08); the smaller
// ones' results cost 1 us for 2.5 million, results in parts a second launch and their bytes twice.  Measured, us, 64 / 128 / 256 entries a side: 768 x 768 x 768
// 6.0 / 8.8 / 13.1; 1024 x 1600 x 1600 10.8 / 13.0 / 17.6; 1024 x 4096 x 4096 42 / 27 / 42; 4800 x 1600 x 4096 79 / 42
// / 50; 4096 x 4096 x 256 23.5 / 18.4 / 12.5.  In parts: 128 x 4096 x 4096 15.0 in one, 12.8 in two; 300 x 300 x 11008
// 25 in one, 12.5 in eight; 1600 x 1600 x 16384 83 in one, 60 in two.  Up to 32 rows on one side: 1 x 11008 x 4096
// 10.3 thin (four waves), 13.7 tiled; 33 rows: 16.1 thin, 14.4 tiled.
struct MatmulPlan {
    enum Kind { kThin, kTile64, kTile128, kLarge } kind;
    int nsplit;                       // parts of k; waves of a thin workgroup
};
static MatmulPlan matmul_plan(int64_t M, int64_t N, int64_t k, bool exact) {
    const int64_t T = fp8_tiles(k);
    if (std::min(M, N) <= 32) return {MatmulPlan::kThin, T >= 4 ? 4 : T >= 2 ? 2 : 1};
    auto tiles = [&](int64_t tm) { return ((M + tm - 1) / tm) * ((N + tm - 1) / tm); };
    const double H = 2.0 * (double)T, big = std::ceil((double)tiles(kBig) / 256);
    MatmulPlan best{MatmulPlan::kLarge, 1};
    double cost = 6 + big * (exact ? 4 + 1.08 * H : 3 + 0.58 * H);
    for (const MatmulPlan::Kind kind : {MatmulPlan::kTile64, MatmulPlan::kTile128}) {
        const bool small = kind == MatmulPlan::kTile64;
        const double wgs = (double)tiles(small ? 64 : 128) / 256;
        const double one = small ? (exact ? 0.31 : 0.17) : exact ? 0.6 : 0.32, all = small ? (exact ? 0.2 : 0.155) : exact ? 0.53 : 0.32;
        for (int64_t ns = 1; ns <= 32 && ns <= T; ++ns) {
            const int64_t per = (T + ns - 1) / ns;
            if ((T + per - 1) / per != ns) continue;
            const double c = 4 + (double)M * (double)N / 2.5e6 + 2.0 * (double)per * std::max(one, all * wgs * (double)ns) +
                             (ns > 1 ? 3 + (double)ns * (double)M * (double)N / 0.75e6 : 0.0);
            if (c < cost) { best = {kind, (int)ns}; cost = c; }
        }
    }
    return best;
}

size_t fp8_matmul_ws(int64_t M, int64_t N, int64_t k) {
    size_t need = 0;                  // for a result of either type
    for (const bool exact : {false, true}) {
        const MatmulPlan p = matmul_plan(M, N, k, exact);
        if (p.kind != MatmulPlan::kThin && p.nsplit > 1) need = std::max(need, (size_t)p.nsplit * (size_t)M * (size_t)N * 4);
    }
    return need;
}

hipError_t launch_fp8_matmul(const dobb_fp8_operand &A, const dobb_fp8_operand &B, const void *bias, bool bias_bf16, bool accumulate,
                             void *out, bool out_bf16, int64_t ldo, float *ws, hipStream_t s) {
    auto side = [](const dobb_fp8_operand &o) {
        return Fp8Side{(const uint8_t *)o.codes, (const uint8_t *)o.scales, (uint32_t)o.rows, (uint32_t)fp8_pitch(o.rows), 0, (uint32_t)o.rows};
    };
    const Fp8Side a = side(A), b = side(B);
    const Epilogue e{out, bias, ldo, out_bf16, bias_bf16, accumulate};
    const int64_t T = fp8_tiles(A.k);
    const MatmulPlan p = matmul_plan(A.rows, B.rows, A.k, !out_bf16);
    auto tiles = [](int64_t rows, int64_t tm) { return (rows + tm - 1) / tm; };
// L(format of A, of B, exact) for the call's
#define DOBB_FP8_BY(L)                                                                        \
    do {                                                                                      \
        const int f = 2 * (A.format == DOBB_E5M2) + (B.format == DOBB_E5M2);                  \
        if (out_bf16) {                                                                       \
            if (f == 0) L(0, 0, false); else if (f == 1) L(0, 1, false); else if (f == 2) L(1, 0, false); else L(1, 1, false); \
        } else {                                                                              \
            if (f == 0) L(0, 0, true); else if (f == 1) L(0, 1, true); else if (f == 2) L(1, 0, true); else L(1, 1, true);     \
        }                                                                                     \
    } while (0)
    if (p.kind == MatmulPlan::kThin) {
        const bool turned = A.rows > B.rows;
        const Fp8Side &few = turned ? b : a, &many = turned ? a : b;
        const dim3 grid((unsigned)tiles(many.rows, 32)), block(64u * p.nsplit);
#define DOBB_FP8_THIN(F, G, EX)                                                                                                              \
    do {                                                                                                                                    \
        if (!turned) DOBB_LAUNCH("fp8_matmul_thin", s, (k_fp8_matmul_thin<F, G, EX>), grid, block, 4096u * p.nsplit, few, many, T, turned, e); \
        else DOBB_LAUNCH("fp8_matmul_thin", s, (k_fp8_matmul_thin<G, F, EX>), grid, block, 4096u * p.nsplit, few, many, T, turned, e);         \
    } while (0)
        DOBB_FP8_BY(DOBB_FP8_THIN);
#undef DOBB_FP8_THIN
        return hipGetLastError();
    }
    if (p.kind == MatmulPlan::kLarge) {
        const int64_t tm = tiles(A.rows, kBig), tn = tiles(B.rows, kBig);
        if (tm * tn >= 0x7fffffff - 256 || 2 * T > 0x7ffffff0) return hipErrorInvalidValue;
        const BigArgs g{a, b, (uint32_t)tm, (uint32_t)tn, (int)(2 * T), e};
        const dim3 grid((unsigned)std::min<int64_t>(tm * tn, 256));
#define DOBB_FP8_BIG(F, G, EX) DOBB_LAUNCH("fp8_matmul_large", s, (k_fp8_matmul_big<F, G, EX>), grid, dim3(256), 0, g)
        DOBB_FP8_BY(DOBB_FP8_BIG);
#undef DOBB_FP8_BIG
        return hipGetLastError();
    }
    const int64_t size = p.kind == MatmulPlan::kTile64 ? 64 : 128, tn = tiles(B.rows, size), wgs = tiles(A.rows, size) * tn * p.nsplit;
    const int64_t quads = A.rows * ((B.rows + 3) / 4);
    if (wgs > kMaxWorkgroups || (p.nsplit > 1 && quads / 256 >= kMaxWorkgroups)) return hipErrorInvalidValue;
#define DOBB_FP8_TILE(F, G, EX)                                                                                                        \
    do {                                                                                                                              \
        if (size == 64) DOBB_LAUNCH("fp8_matmul", s, (k_fp8_matmul<64, 64, 6, F, G, EX>), dim3((unsigned)wgs), dim3(256), 0, a, b, T, (int)tn, p.nsplit, e, ws); \
        else DOBB_LAUNCH("fp8_matmul", s, (k_fp8_matmul<128, 128, 4, F, G, EX>), dim3((unsigned)wgs), dim3(256), 0, a, b, T, (int)tn, p.nsplit, e, ws);          \
    } while (0)
    DOBB_FP8_BY(DOBB_FP8_TILE);
#undef DOBB_FP8_TILE
#undef DOBB_FP8_BY
    const hipError_t r = hipGetLastError();
    if (r != hipSuccess || p.nsplit == 1) return r;
    DOBB_LAUNCH("fp8_join", s, k_fp8_join, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, A.rows, B.rows, p.nsplit, ws, e);
    return hipGetLastError();
}

}  // namespace dobb
