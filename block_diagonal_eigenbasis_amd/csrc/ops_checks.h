// Host-side checks that the C entry points of dobb_ops.h and dobb_layers.h share (not installed).
#pragma once

#include <algorithm>
#include <vector>

#include "ops_internal.h"

namespace dobb {

constexpr int64_t kMaxNb = 1024;
constexpr int64_t kMaxN = (int64_t)1 << 24;       // the products' row and column offsets are 32-bit
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

inline bool dtype_ok(dobb_dtype d) { return d == DOBB_F32 || d == DOBB_BF16; }
inline int64_t size_of(dobb_dtype d) { return d == DOBB_BF16 ? 2 : 4; }
inline size_t al256(size_t x) { return (x + 255) / 256 * 256; }
inline dobb_status hip_status(hipError_t e) { return e == hipSuccess ? DOBB_OK : DOBB_ERR_HIP; }

inline dobb_status check_ws(void *ws, size_t ws_bytes, size_t need) {
    if (need == 0) return DOBB_OK;
    if (!ws || ((uintptr_t)ws & 255u) != 0 || ws_bytes < need) return DOBB_ERR_WORKSPACE;
    return DOBB_OK;
}

struct Span {
    uintptr_t lo, hi;
    bool out;
};

// Whether no written span of v overlaps any other.  Lists mostly come as a few buckets, each laid out in
// order: spans are first put into runs of neighbours (at most 1 MB apart), and if those are few and lie
// apart there is nothing to sort (331 tensors in two buckets: 3 us of host time instead of 11).
inline bool apart(std::vector<Span> &v) {
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

// ---- second moments from captures held in few bits ------------------------------------------------
inline dobb_status check_moment_shape(const dobb_shape &s) {
    if (s.n < 1 || s.n > kMaxN || s.nb < 1 || s.nb > kMaxNb || s.n % s.nb != 0) return DOBB_ERR_SHAPE;
    return DOBB_OK;
}

// One launch of a grouped call: matrices with blocks of one width, as many as the table and a grid hold
struct MomentLaunch {
    std::vector<int> idx;
    int64_t nb, blocks;
};

inline std::vector<MomentLaunch> moment_launches(int count, const dobb_shape *shapes) {
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

}  // namespace dobb
