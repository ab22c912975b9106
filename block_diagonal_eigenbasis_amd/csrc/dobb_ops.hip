// C ABI of dobb_ops.h: host-side validation and workspace sizing.  Every computation is done by the
// kernels in k_grads.hip, k_mx4.hip and k_moment_mx4.hip.
#include <algorithm>
#include <new>
#include <vector>

#include "ops_internal.h"

using namespace dobb;

namespace {

constexpr int64_t kMaxNb = 1024;
constexpr int64_t kMaxN = (int64_t)1 << 24;       // the product's column offsets are 32-bit
constexpr int64_t kMaxTokens = (int64_t)1 << 40;

// nothing thrown inside (host memory for the lists) leaves a C entry
template <typename F>
dobb_status guarded(F f) {
    try {
        return f();
    } catch (...) {
        return DOBB_ERR_INVALID_ARG;
    }
}

bool dtype_ok(dobb_dtype d) { return d == DOBB_F32 || d == DOBB_BF16; }
int64_t size_of(dobb_dtype d) { return d == DOBB_BF16 ? 2 : 4; }
inline size_t al256(size_t x) { return (x + 255) / 256 * 256; }
dobb_status hip_status(hipError_t e) { return e == hipSuccess ? DOBB_OK : DOBB_ERR_HIP; }

dobb_status check_ws(void *ws, size_t ws_bytes, size_t need) {
    if (need == 0) return DOBB_OK;
    if (!ws || ((uintptr_t)ws & 255u) != 0 || ws_bytes < need) return DOBB_ERR_WORKSPACE;
    return DOBB_OK;
}

// a list of tensors: dtypes, sizes, pointers aligned to their entries
dobb_status check_list(int count, const int64_t *numel, const void *const *p, const dobb_dtype *dt) {
    if (count < 1 || !numel || !p || !dt) return DOBB_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        if (!dtype_ok(dt[i])) return DOBB_ERR_DTYPE;
        if (numel[i] < 0 || numel[i] > ((int64_t)1 << 44)) return DOBB_ERR_SHAPE;
        if (numel[i] > 0 && !p[i]) return DOBB_ERR_INVALID_ARG;
        if ((uintptr_t)p[i] & (uintptr_t)(size_of(dt[i]) - 1)) return DOBB_ERR_INVALID_ARG;
    }
    return DOBB_OK;
}

struct Span {
    uintptr_t lo, hi;
    bool out;
};

// Whether no written span of v overlaps any other.  Lists mostly come as a few buckets, each laid out in
// order: spans are first put into runs of neighbours (at most 1 MB apart), and if those are few and lie
// apart there is nothing to sort (331 tensors in two buckets: 3 us of host time instead of 11).
bool apart(std::vector<Span> &v) {
    constexpr int kRuns = 8;
    Span run[kRuns];
    int runs = 0;
    bool few = true;
    for (const Span &s : v) {
        int k = 0;
        while (k < runs && !(run[k].out == s.out && s.lo >= run[k].hi && s.lo - run[k].hi <= ((uintptr_t)1 << 20))) ++k;
        if (k < runs) run[k].hi = s.hi;
        else if (runs < kRuns) run[runs++] = s;
        else { few = false; break; }
    }
    for (int i = 0; few && i < runs; ++i)
        for (int k = 0; few && k < i; ++k)
            few = !(run[i].out || run[k].out) || run[i].hi <= run[k].lo || run[k].hi <= run[i].lo;
    if (few) return true;
    std::sort(v.begin(), v.end(), [](const Span &x, const Span &y) { return x.lo < y.lo; });
    uintptr_t out_end = 0, in_end = 0;
    for (const Span &s : v) {
        if (s.lo < out_end || (s.out && s.lo < in_end)) return false;
        uintptr_t &end = s.out ? out_end : in_end;
        if (s.hi > end) end = s.hi;
    }
    return true;
}

// Every buffer written is the tensor it is made from (same type) or apart from everything else in the
// list: a chunk of one is then read and written by one workgroup only.
// norms, total: written too where `sums` (read, total, where not); ws_bytes of ws likewise.
dobb_status check_outputs(const GradArgs &a, const float *norms, const float *total, bool sums, const void *ws, size_t ws_bytes) {
    std::vector<Span> v;
    v.reserve(2 * (size_t)a.count + 3);
    auto add = [&](const void *p, size_t bytes, bool out) {
        if (p && bytes) v.push_back({(uintptr_t)p, (uintptr_t)p + bytes, out});
    };
    for (int i = 0; i < a.count; ++i) {
        if (a.numel[i] == 0) continue;
        if (!a.out) {
            add(a.G[i], (size_t)(a.numel[i] * size_of(a.g_dtypes[i])), false);
            continue;
        }
        const uintptr_t g = (uintptr_t)a.G[i], o = (uintptr_t)a.out[i];
        if (g != o || a.g_dtypes[i] != a.out_dtypes[i]) v.push_back({g, g + (uintptr_t)(a.numel[i] * size_of(a.g_dtypes[i])), false});
        v.push_back({o, o + (uintptr_t)(a.numel[i] * size_of(a.out_dtypes[i])), true});
    }
    add(norms, 4 * (size_t)a.count, sums);
    add(total, 4, sums);
    add(ws, ws_bytes, true);
    return apart(v) ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

dobb_status check_clip(const GradArgs &a, const float *total, float max_norm) {
    dobb_status st = check_list(a.count, a.numel, a.G, a.g_dtypes);
    if (st != DOBB_OK) return st;
    st = check_list(a.count, a.numel, (const void *const *)a.out, a.out_dtypes);
    if (st != DOBB_OK) return st;
    return total && max_norm >= 0.f ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

size_t norm_ws(int count, const int64_t *numel, const dobb_dtype *dt) {
    return al256((size_t)grad_norm_chunks(count, numel, dt) * 8 + 8);
}

dobb_status check_capture(int64_t N, int64_t n, const void *p, dobb_dtype dt, int64_t ld, const void *codes, const void *scales) {
    if (!p || !codes || !scales) return DOBB_ERR_INVALID_ARG;
    if (!dtype_ok(dt)) return DOBB_ERR_DTYPE;
    if (N < 1) return DOBB_ERR_INVALID_ARG;
    if (N > kMaxTokens || n < 1 || n > kMaxN || ld < n) return DOBB_ERR_SHAPE;
    if ((N / kMx4Tile + 1) * ((n + 127) / 128) > 0x7fffffff) return DOBB_ERR_SHAPE;
    if (((uintptr_t)codes & 15u) || ((uintptr_t)scales & 3u) || ((uintptr_t)p & (uintptr_t)(size_of(dt) - 1)))
        return DOBB_ERR_INVALID_ARG;
    // values, codes and scales are three buffers, whichever of them is written
    auto span = [](const void *q, uintptr_t bytes) { return Span{(uintptr_t)q, (uintptr_t)q + bytes, true}; };
    const uintptr_t cells = (uintptr_t)((N + kMx4Tile - 1) / kMx4Tile) * (uintptr_t)n;
    std::vector<Span> v{span(p, ((uintptr_t)(N - 1) * (uintptr_t)ld + (uintptr_t)n) * (uintptr_t)size_of(dt)), span(codes, 64 * cells),
                        span(scales, 4 * cells)};
    return apart(v) ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

dobb_status check_moment_shape(const dobb_shape &s) {
    if (s.n < 1 || s.n > kMaxN || s.nb < 1 || s.nb > kMaxNb || s.n % s.nb != 0) return DOBB_ERR_SHAPE;
    return DOBB_OK;
}

// One launch of a grouped call: matrices with blocks of one width, as many as the table and a grid hold
struct MomentLaunch {
    std::vector<int> idx;
    int64_t nb, blocks;
};

std::vector<MomentLaunch> moment_launches(int count, const dobb_shape *shapes) {
    std::vector<MomentLaunch> out, open;
    for (int i = 0; i < count; ++i) {
        const int64_t nb = shapes[i].nb, blocks = shapes[i].n / nb;
        const int64_t most = 0x3fffffff / std::max<int64_t>(64, (nb * nb + 255) / 256);
        size_t k = 0;
        while (k < open.size() && open[k].nb != nb) ++k;
        if (k == open.size()) open.push_back({{}, nb, 0});
        if (!open[k].idx.empty() && ((int)open[k].idx.size() == kMomentMats || open[k].blocks + blocks > most)) {
            out.push_back(open[k]);
            open[k] = {{}, nb, 0};
        }
        open[k].idx.push_back(i);
        open[k].blocks += blocks;
    }
    out.insert(out.end(), open.begin(), open.end());
    return out;
}

size_t moment_ws(const std::vector<MomentLaunch> &launches, int64_t tiles) {
    size_t need = 0;
    for (const MomentLaunch &l : launches) need = std::max(need, al256(moment_mx4_ws(l.nb, l.blocks, tiles)));
    return need;
}

dobb_status moment_grouped(int count, const dobb_shape *shapes, const void *const *codes, const void *const *scales,
                           int64_t tiles, int64_t N, float beta, float *const *A, void *ws, size_t ws_bytes,
                           hipStream_t stream) {
    if (count < 1 || !shapes || !codes || !scales || !A) return DOBB_ERR_INVALID_ARG;
    if (tiles < 1 || N < 1 || N / kMx4Tile + (N % kMx4Tile != 0) > tiles || !(beta >= 0.f && beta < 1.f)) return DOBB_ERR_INVALID_ARG;
    if (tiles > kMaxTokens / kMx4Tile) return DOBB_ERR_SHAPE;
    for (int i = 0; i < count; ++i) {
        const dobb_status st = check_moment_shape(shapes[i]);
        if (st != DOBB_OK) return st;
        if (!codes[i] || !scales[i] || !A[i] || ((uintptr_t)codes[i] & 15u) || ((uintptr_t)scales[i] & 3u) || ((uintptr_t)A[i] & 3u))
            return DOBB_ERR_INVALID_ARG;
    }
    const std::vector<MomentLaunch> launches = moment_launches(count, shapes);
    const size_t need = moment_ws(launches, tiles);
    // moments and the workspace are written: no two the same, and none over a capture (captures may be shared)
    std::vector<Span> spans;
    spans.reserve(3 * (size_t)count + 1);
    for (int i = 0; i < count; ++i) {
        auto add = [&](const void *p, int64_t bytes, bool out) { spans.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, out}); };
        add(A[i], 4 * shapes[i].n * shapes[i].nb, true);
        add(codes[i], 64 * tiles * shapes[i].n, false);
        add(scales[i], 4 * tiles * shapes[i].n, false);
    }
    if (ws && need) spans.push_back({(uintptr_t)ws, (uintptr_t)ws + need, true});
    if (!apart(spans)) return DOBB_ERR_INVALID_ARG;
    const dobb_status st = check_ws(ws, ws_bytes, need);
    if (st != DOBB_OK) return st;
    for (const MomentLaunch &l : launches) {
        const void *cs[kMomentMats], *ss[kMomentMats];
        float *as[kMomentMats];
        int64_t ns[kMomentMats];
        MomentMx4Args a{};
        a.count = (int)l.idx.size();
        for (int k = 0; k < a.count; ++k) {
            const int i = l.idx[k];
            cs[k] = codes[i]; ss[k] = scales[i]; as[k] = A[i]; ns[k] = shapes[i].n;
        }
        a.nb = l.nb;
        a.tiles = tiles;
        a.N = N;
        a.n = ns;
        a.codes = cs;
        a.scales = ss;
        a.A = as;
        a.beta = beta;
        a.plan = moment_mx4_plan(l.nb, l.blocks, tiles);
        a.partial = (float *)ws;
        const dobb_status r = hip_status(launch_moment_mx4(a, stream));
        if (r != DOBB_OK) return r;
    }
    return DOBB_OK;
}

}  // namespace

extern "C" {

size_t dobb_grad_norm_workspace_size(int count, const int64_t *numel, const dobb_dtype *g_dtypes) {
    if (count < 1 || !numel || !g_dtypes) return 0;
    for (int i = 0; i < count; ++i)
        if (!dtype_ok(g_dtypes[i]) || numel[i] < 0 || numel[i] > ((int64_t)1 << 44)) return 0;
    return norm_ws(count, numel, g_dtypes);
}

dobb_status dobb_grad_norm_grouped(int count, const int64_t *numel, const void *const *G, const dobb_dtype *g_dtypes,
                                   float *norms, float *total, void *ws, size_t ws_bytes, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_list(count, numel, G, g_dtypes);
        if (st != DOBB_OK) return st;
        if (!total) return DOBB_ERR_INVALID_ARG;
        const GradArgs a{count, numel, G, g_dtypes, nullptr, nullptr};
        const size_t need = norm_ws(count, numel, g_dtypes);
        st = check_outputs(a, norms, total, true, ws, need);
        if (st != DOBB_OK) return st;
        st = check_ws(ws, ws_bytes, need);
        if (st != DOBB_OK) return st;
        return hip_status(launch_grad_norm(a, norms, total, (double *)ws, (hipStream_t)stream));
    });
}

dobb_status dobb_clip_grads_grouped(int count, const int64_t *numel, const void *const *G, const dobb_dtype *g_dtypes,
                                    void *const *out, const dobb_dtype *out_dtypes, const float *total, float max_norm,
                                    dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        const GradArgs a{count, numel, G, g_dtypes, out, out_dtypes};
        dobb_status st = check_clip(a, total, max_norm);
        if (st == DOBB_OK) st = check_outputs(a, nullptr, total, false, nullptr, 0);
        if (st != DOBB_OK) return st;
        return hip_status(launch_grad_clip(a, total, max_norm, (hipStream_t)stream));
    });
}

dobb_status dobb_clip_grad_norm_grouped(int count, const int64_t *numel, const void *const *G, const dobb_dtype *g_dtypes,
                                        void *const *out, const dobb_dtype *out_dtypes, float max_norm, float *norms,
                                        float *total, void *ws, size_t ws_bytes, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        const GradArgs a{count, numel, G, g_dtypes, out, out_dtypes};
        dobb_status st = check_clip(a, total, max_norm);
        if (st != DOBB_OK) return st;
        const size_t need = norm_ws(count, numel, g_dtypes);
        st = check_outputs(a, norms, total, true, ws, need);
        if (st != DOBB_OK) return st;
        st = check_ws(ws, ws_bytes, need);
        if (st != DOBB_OK) return st;
        st = hip_status(launch_grad_norm(a, norms, total, (double *)ws, (hipStream_t)stream));
        if (st != DOBB_OK) return st;
        return hip_status(launch_grad_clip(a, total, max_norm, (hipStream_t)stream));
    });
}

dobb_status dobb_mx4_quantize(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, void *codes, void *scales,
                              dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        const dobb_status st = check_capture(N, n, X, x_dtype, ldx, codes, scales);
        if (st != DOBB_OK) return st;
        return hip_status(launch_mx4_quantize(N, n, X, x_dtype == DOBB_BF16, ldx, codes, scales, (hipStream_t)stream));
    });
}

dobb_status dobb_mx4_dequantize(int64_t N, int64_t n, const void *codes, const void *scales, void *out, dobb_dtype out_dtype,
                                int64_t ldo, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        const dobb_status st = check_capture(N, n, out, out_dtype, ldo, codes, scales);
        if (st != DOBB_OK) return st;
        return hip_status(launch_mx4_dequantize(N, n, codes, scales, out, out_dtype == DOBB_BF16, ldo, (hipStream_t)stream));
    });
}

size_t dobb_moment_mx4_workspace_size(int count, const dobb_shape *shapes, int64_t tiles) {
    if (count < 1 || !shapes || tiles < 1 || tiles > kMaxTokens / kMx4Tile) return 0;
    for (int i = 0; i < count; ++i)
        if (check_moment_shape(shapes[i]) != DOBB_OK) return 0;
    try {
        return moment_ws(moment_launches(count, shapes), tiles);
    } catch (...) {
        return 0;
    }
}

dobb_status dobb_accumulate_moment_mx4_grouped(int count, const dobb_shape *shapes, const void *const *codes,
                                               const void *const *scales, int64_t tiles, int64_t N, float beta,
                                               float *const *A, void *ws, size_t ws_bytes, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        return moment_grouped(count, shapes, codes, scales, tiles, N, beta, A, ws, ws_bytes, (hipStream_t)stream);
    });
}

dobb_status dobb_accumulate_moment_mx4(const dobb_shape *s, const void *codes, const void *scales, int64_t tiles, int64_t N,
                                       float beta, float *A, void *ws, size_t ws_bytes, dobb_stream_t stream) {
    if (!s) return DOBB_ERR_INVALID_ARG;
    return dobb_accumulate_moment_mx4_grouped(1, s, &codes, &scales, tiles, N, beta, &A, ws, ws_bytes, stream);
}

}  // extern "C"
