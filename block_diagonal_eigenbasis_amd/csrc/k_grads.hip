// Global gradient norm over many tensors, and clipping.
//   sum_i sum_k g^2 in fp64;   out = g * min(1, max_norm / (sqrt(sum) + 1e-6))
// Both passes stream their tensors once and do a handful of operations an entry: HBM bounds them (2.95 GB of
// bf16 gradients: sums 514 us, 5.7 TB/s; clipped into buffers of their own 994 us, 5.9 TB/s), and for small
// lists the launches and their latency do (one 768 x 768 gradient: 3.5 + 2.8 us).  A list is cut into
// chunks of whole 16-byte vectors, one workgroup each, so tensors of any size share one launch; the
// chunk's tensor is looked up in the table that arrives with the kernel's arguments.  Vectors are
// loaded with the alignment of an entry (gradients are views into buckets); what is behind the last
// whole vector of a tensor is read entry by entry.  Squares are formed and added in fp64: fp32 would overflow
// from 1.8e19 on and lose what is below 1e-19, and at the memory's rate the vector units are idle anyway.
#include <math.h>

#include "ops_internal.h"

namespace dobb {
namespace {

constexpr int kNormMats = 192;   // tensors per launch: the tables fit the 4 KB of kernel arguments
constexpr int kClipMats = 128;
constexpr int kFinishMats = 900;
constexpr int kUnroll = 4;       // 16-byte vectors in flight per thread
constexpr int kThreads = 256;
constexpr int64_t kStep = (int64_t)kThreads * kUnroll;   // vectors a workgroup reads at a time
// Clipping: one workgroup for every step of 8 KB.  Workgroups of four steps of 16 KB took 1.62 ms for the call
// on the GPT-2 XL set in bf16, of one such step 1.51, of one of 8 KB 1.50 (4 KB: 1.53).
constexpr int kClipUnroll = 2;
constexpr int64_t kClipStep = (int64_t)kThreads * kClipUnroll;

struct NormTable {
    const void *g[kNormMats];
    int64_t numel[kNormMats];
    uint32_t first[kNormMats + 1];          // first chunk of each tensor, counted from this launch's
    uint32_t bf16[(kNormMats + 31) / 32];
};

struct FinishTable {
    uint32_t first[kFinishMats + 1];        // counted from the first table's
};

struct ClipTable {
    const void *g[kClipMats];
    void *out[kClipMats];
    int64_t numel[kClipMats];
    uint32_t first[kClipMats + 1];
    uint32_t bf16[kClipMats / 32], out_bf16[kClipMats / 32];
};

// 16 bytes at the alignment of one entry
struct __attribute__((packed, aligned(2))) Vec16 { uint32_t w[4]; };

// the tensor of a chunk: how many of the ascending first[0 .. cnt - 1] are at most chunk, less one.  One
// read a lane and a ballot for every 64 (bisecting was a chain of eight dependent reads)
template <int MATS>
__device__ __forceinline__ int find_tensor(const uint32_t *first, int cnt, uint32_t chunk) {
    const int lane = threadIdx.x & 63;
    bool le[(MATS + 63) / 64];
#pragma unroll
    for (int k = 0; k < (MATS + 63) / 64; ++k) {
        const int i = 64 * k + lane;
        le[k] = first[i < MATS ? i : MATS] <= chunk && i < cnt;
    }
    int n = 0;
#pragma unroll
    for (int k = 0; k < (MATS + 63) / 64; ++k) n += __popcll(__ballot(le[k]));
    return __builtin_amdgcn_readfirstlane(n - 1);
}

__device__ __forceinline__ double sq(float v) { return (double)v * (double)v; }
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// entries per 16-byte vector: 4 (fp32) or 8 (bf16)
template <bool BF16>
__device__ __forceinline__ double sumsq_chunk(const char *g, int64_t numel, int64_t v0, int64_t nv) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t whole = numel / E;                    // vectors that lie inside the tensor
    const int64_t end = v0 + nv < whole ? v0 + nv : whole;
    double s0 = 0.0, s1 = 0.0;
    auto add = [&](const Vec16 &x) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (BF16) { s0 += sq(lo_bf16(x.w[c])); s1 += sq(hi_bf16(x.w[c])); }
            else if (c & 1) s1 += sq(__uint_as_float(x.w[c]));
            else s0 += sq(__uint_as_float(x.w[c]));
        }
    };
    int64_t b = v0;
    for (; b + kStep <= end; b += kStep) {              // whole steps: no bounds to check
        Vec16 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) x[u] = *(const Vec16 *)(g + (b + u * kThreads + threadIdx.x) * 16);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) add(x[u]);
    }
    if (b < end) {
        Vec16 x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {             // places past the end repeat the last vector
            const int64_t p = b + u * kThreads + threadIdx.x;
            x[u] = *(const Vec16 *)(g + (p < end ? p : end - 1) * 16);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (b + u * kThreads + threadIdx.x < end) add(x[u]);
    }
    if (whole >= v0 && whole < v0 + nv) {               // the entries behind the last whole vector
        const int64_t e = whole * E + threadIdx.x;
        if ((int)threadIdx.x < E && e < numel) s0 += sq(BF16 ? bf16_to_f32(((const uint16_t *)g)[e]) : ((const float *)g)[e]);
    }
    return s0 + s1;
}

// sum over the workgroup in a fixed order; valid in thread 0
__device__ __forceinline__ double block_sum(double s, double *sm) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_down(s, o);
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
    if (threadIdx.x == 0)
        for (unsigned w = 0; w < blockDim.x / 64; ++w) s += sm[w];
    return s;
}

// one workgroup per chunk of nv vectors; part: this launch's chunks
__global__ void __launch_bounds__(kThreads) k_grad_sumsq(int cnt, int64_t nv, double *part, NormTable t) {
    __shared__ double sm[kThreads / 64];
    const uint32_t chunk = blockIdx.x;
    const int i = find_tensor<kNormMats>(t.first, cnt, chunk);
    const int64_t v0 = (int64_t)(chunk - t.first[i]) * nv;
    const bool bf = (t.bf16[i >> 5] >> (i & 31)) & 1;
    const double s = block_sum(bf ? sumsq_chunk<true>((const char *)t.g[i], t.numel[i], v0, nv)
                                  : sumsq_chunk<false>((const char *)t.g[i], t.numel[i], v0, nv), sm);
    if (threadIdx.x == 0) part[chunk] = s;
}

// workgroup i < cnt: norms[i] from its tensor's chunks of part; workgroup cnt (where there is one): the
// norm of all `all` chunks of the call
__global__ void __launch_bounds__(512) k_grad_norms(int cnt, const double *part, uint32_t all, float *norms, float *total,
                                                    FinishTable t) {
    __shared__ double sm[8];
    const int i = blockIdx.x;
    const uint32_t k0 = i < cnt ? t.first[i] : 0, k1 = i < cnt ? t.first[i + 1] : all;
    double s = 0.0;
    for (uint32_t b = k0; b < k1; b += 8 * 512) {
        double x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t k = b + u * 512 + threadIdx.x;
            x[u] = part[k < k1 ? k : k1 - 1];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (b + u * 512 + threadIdx.x < k1) s += x[u];
    }
    s = block_sum(s, sm);
    if (threadIdx.x == 0) *(i < cnt ? norms + i : total) = (float)sqrt(s);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    return (uint32_t)f32_to_bf16(a) | ((uint32_t)f32_to_bf16(b) << 16);
}

// vectors are of the input's 16 bytes; the output takes 8, 16 or 32 bytes for each
template <bool IBF, bool OBF>
__device__ __forceinline__ void scale_chunk(const char *g, char *o, int64_t numel, int64_t v0, int64_t nv, float c) {
    constexpr int E = IBF ? 8 : 4;
    constexpr int OB = E * (OBF ? 2 : 4);
    const int64_t whole = numel / E;
    const int64_t end = v0 + nv < whole ? v0 + nv : whole;
    auto put = [&](int64_t p, const Vec16 &x) {
        float f[E];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (IBF) { f[2 * k] = lo_bf16(x.w[k]) * c; f[2 * k + 1] = hi_bf16(x.w[k]) * c; }
            else f[k] = __uint_as_float(x.w[k]) * c;
        }
        struct __attribute__((packed, aligned(2))) Out { uint32_t w[OB / 4]; } r;
#pragma unroll
        for (int k = 0; k < OB / 4; ++k) r.w[k] = OBF ? pack_bf16(f[2 * k], f[2 * k + 1]) : __float_as_uint(f[k]);
        *(Out *)(o + p * OB) = r;
    };
    int64_t b = v0;
    for (; b + kClipStep <= end; b += kClipStep) {              // whole steps: no bounds to check
        Vec16 x[kClipUnroll];
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) x[u] = *(const Vec16 *)(g + (b + u * kThreads + threadIdx.x) * 16);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) put(b + u * kThreads + threadIdx.x, x[u]);
    }
    if (b < end) {
        Vec16 x[kClipUnroll];
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) {             // places past the end read the last vector, for nothing
            const int64_t p = b + u * kThreads + threadIdx.x;
            x[u] = *(const Vec16 *)(g + (p < end ? p : end - 1) * 16);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < kClipUnroll; ++u) {
            const int64_t p = b + u * kThreads + threadIdx.x;
            if (p < end) put(p, x[u]);
        }
    }
    if (whole >= v0 && whole < v0 + nv) {
        const int64_t e = whole * E + threadIdx.x;
        if ((int)threadIdx.x < E && e < numel) {
            const float f = c * (IBF ? bf16_to_f32(((const uint16_t *)g)[e]) : ((const float *)g)[e]);
            if (OBF) ((uint16_t *)o)[e] = f32_to_bf16(f);
            else ((float *)o)[e] = f;
        }
    }
}

__global__ void __launch_bounds__(kThreads) k_grad_clip(int cnt, int64_t nv, const float *total, float max_norm, ClipTable t) {
    const float norm = *total;
    const float q = max_norm / (norm + 1e-6f);
    // a NaN stays one, but for inf / inf: no limit on an infinite norm
    const float c = q > 1.f || (max_norm == INFINITY && norm == INFINITY) ? 1.f : q;
    const uint32_t chunk = blockIdx.x;
    const int i = find_tensor<kClipMats>(t.first, cnt, chunk);
    const char *g = (const char *)t.g[i];
    char *o = (char *)t.out[i];
    if (c == 1.f && (const char *)o == g) return;
    const int64_t v0 = (int64_t)(chunk - t.first[i]) * nv;
    const bool ib = (t.bf16[i >> 5] >> (i & 31)) & 1, ob = (t.out_bf16[i >> 5] >> (i & 31)) & 1;
    if (ib && ob) scale_chunk<true, true>(g, o, t.numel[i], v0, nv, c);
    else if (ib) scale_chunk<true, false>(g, o, t.numel[i], v0, nv, c);
    else if (ob) scale_chunk<false, true>(g, o, t.numel[i], v0, nv, c);
    else scale_chunk<false, false>(g, o, t.numel[i], v0, nv, c);
}

int64_t vectors(int64_t numel, dobb_dtype dt) {
    const int sh = dt == DOBB_BF16 ? 3 : 2;
    return (numel + (1 << sh) - 1) >> sh;
}

constexpr int64_t kMostChunks = 8192;

}  // namespace

// Vectors per chunk of the norm: one step of a workgroup, or as many as keep the list's partial sums
// near kMostChunks (they are added by one workgroup)
int64_t grad_norm_chunk(int count, const int64_t *numel, const dobb_dtype *dt) {
    int64_t all = 0;
    for (int i = 0; i < count; ++i) all += vectors(numel[i], dt[i]);
    const int64_t steps = (all + kStep * kMostChunks - 1) / (kStep * kMostChunks);
    return (steps < 1 ? 1 : steps) * kStep;
}

int64_t grad_norm_chunks(int count, const int64_t *numel, const dobb_dtype *dt) {
    const int64_t nv = grad_norm_chunk(count, numel, dt);
    int64_t n = 0;
    for (int i = 0; i < count; ++i) n += (vectors(numel[i], dt[i]) + nv - 1) / nv;
    return n;
}

hipError_t launch_grad_norm(const GradArgs &a, float *norms, float *total, double *part, hipStream_t s) {
    const int64_t nv = grad_norm_chunk(a.count, a.numel, a.g_dtypes);
    auto chunks_of = [&](int i) { return (vectors(a.numel[i], a.g_dtypes[i]) + nv - 1) / nv; };
    int64_t all = 0;
    for (int i = 0; i < a.count; ++i) all += chunks_of(i);
    if (all > 0x7fffffff) return hipErrorInvalidValue;
    double *p = part;
    for (int i0 = 0; i0 < a.count; i0 += kNormMats) {
        const int cnt = a.count - i0 < kNormMats ? a.count - i0 : kNormMats;
        NormTable t{};
        int64_t chunks = 0;
        for (int i = 0; i < cnt; ++i) {
            t.g[i] = a.G[i0 + i];
            t.numel[i] = a.numel[i0 + i];
            t.first[i] = (uint32_t)chunks;
            chunks += chunks_of(i0 + i);
            if (a.g_dtypes[i0 + i] == DOBB_BF16) t.bf16[i >> 5] |= 1u << (i & 31);
        }
        if (chunks == 0) continue;
        DOBB_LAUNCH("grad_sumsq", s, k_grad_sumsq, dim3((unsigned)chunks), dim3(kThreads), 0, cnt, nv, p, t);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p += chunks;
    }
    int64_t at = 0;
    for (int i0 = 0; i0 < a.count; i0 += kFinishMats) {
        const int cnt = a.count - i0 < kFinishMats ? a.count - i0 : kFinishMats;
        const bool last = i0 + cnt == a.count;
        if (!norms && !last) continue;
        FinishTable t{};
        if (norms) {
            for (int i = 0; i < cnt; ++i) { t.first[i] = (uint32_t)at; at += chunks_of(i0 + i); }
            t.first[cnt] = (uint32_t)at;
        }
        const int nn = norms ? cnt : 0;
        DOBB_LAUNCH("grad_norms", s, k_grad_norms, dim3((unsigned)(nn + (last ? 1 : 0))), dim3(512), 0, nn, part, (uint32_t)all,
                    norms ? norms + i0 : nullptr, total, t);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_grad_clip(const GradArgs &a, const float *total, float max_norm, hipStream_t s) {
    const int64_t nv = kClipStep;
    for (int i0 = 0; i0 < a.count;) {
        ClipTable t{};
        int64_t chunks = 0;
        int cnt = 0;
        for (; i0 + cnt < a.count && cnt < kClipMats; ++cnt) {
            const int i = i0 + cnt;
            const int64_t c = (vectors(a.numel[i], a.g_dtypes[i]) + nv - 1) / nv;
            if (chunks + c > 0x7fffffff) break;
            t.g[cnt] = a.G[i];
            t.out[cnt] = a.out[i];
            t.numel[cnt] = a.numel[i];
            t.first[cnt] = (uint32_t)chunks;
            chunks += c;
            if (a.g_dtypes[i] == DOBB_BF16) t.bf16[cnt >> 5] |= 1u << (cnt & 31);
            if (a.out_dtypes[i] == DOBB_BF16) t.out_bf16[cnt >> 5] |= 1u << (cnt & 31);
        }
        if (cnt == 0) return hipErrorInvalidValue;
        if (chunks > 0)
            DOBB_LAUNCH("grad_clip", s, k_grad_clip, dim3((unsigned)chunks), dim3(kThreads), 0, cnt, nv, total, max_norm, t);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        i0 += cnt;
    }
    return hipSuccess;
}

}  // namespace dobb
