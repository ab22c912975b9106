// C ABI of dobb_layers.h: host-side validation and workspace sizing.  Every computation is done by the
// kernels in k_norm.hip, k_fp8.hip, k_fp8_matmul.hip and k_moment_fp8.hip.
#include <cmath>

#include "layers_internal.h"
#include "ops_checks.h"

using namespace dobb;

namespace {

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// N x n with rows of stride ld
dobb_status check_matrix(const void *p, int64_t N, int64_t n, dobb_dtype dt, int64_t ld) {
    if (!p) return DOBB_ERR_INVALID_ARG;
    if (!dtype_ok(dt)) return DOBB_ERR_DTYPE;
    if (N < 1) return DOBB_ERR_INVALID_ARG;
    if (n < 1 || n > kMaxN || ld < n || N > kMaxTokens || ld > (((int64_t)1 << 60) / N)) return DOBB_ERR_SHAPE;   // bytes in 64 bits
    return aligned(p, (uintptr_t)size_of(dt)) ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

// weight, bias and their like: n entries or nothing
dobb_status check_vector(const void *p, dobb_dtype dt) {
    if (!p) return DOBB_OK;
    if (!dtype_ok(dt)) return DOBB_ERR_DTYPE;
    return aligned(p, (uintptr_t)size_of(dt)) ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

dobb_status check_operand(const dobb_fp8_operand *op) {
    if (!op || !op->codes || !op->scales) return DOBB_ERR_INVALID_ARG;
    if (op->format != DOBB_E4M3 && op->format != DOBB_E5M2) return DOBB_ERR_DTYPE;
    if (op->rows < 1 || op->rows > kMaxN || op->k < 1 || op->k > kMaxTokens) return DOBB_ERR_SHAPE;
    return aligned(op->codes, 16) && aligned(op->scales, 4) ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

struct Spans {
    std::vector<Span> v;
    void add(const void *p, uintptr_t bytes, bool out) {
        if (p && bytes) v.push_back({(uintptr_t)p, (uintptr_t)p + bytes, out});
    }
    void matrix(const void *p, int64_t N, int64_t n, dobb_dtype dt, int64_t ld, bool out) {
        add(p, ((uintptr_t)(N - 1) * (uintptr_t)ld + (uintptr_t)n) * (uintptr_t)size_of(dt), out);
    }
    void vector(const void *p, int64_t n, dobb_dtype dt, bool out) { add(p, (uintptr_t)n * (uintptr_t)size_of(dt), out); }
    void operand(const dobb_fp8_operand &op, bool out) {
        add(op.codes, 128 * (uintptr_t)fp8_tiles(op.k) * (uintptr_t)op.rows, out);
        add(op.scales, (uintptr_t)fp8_tiles(op.k) * (uintptr_t)fp8_pitch(op.rows), out);
    }
    dobb_status check() { return apart(v) ? DOBB_OK : DOBB_ERR_INVALID_ARG; }
};

// the arguments that dobb_layer_norm and dobb_layer_norm_fp8 share
dobb_status check_norm(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, const void *weight, const void *bias,
                       dobb_dtype w_dtype, float eps) {
    dobb_status st = check_matrix(X, N, n, x_dtype, ldx);
    if (st == DOBB_OK) st = check_vector(weight, w_dtype);
    if (st == DOBB_OK) st = check_vector(bias, w_dtype);
    if (st != DOBB_OK) return st;
    if (N > kMaxN) return DOBB_ERR_SHAPE;
    return eps >= 0.f && std::isfinite(eps) ? DOBB_OK : DOBB_ERR_INVALID_ARG;
}

// the operands that a quantising call writes: of X's sizes, and of one format
dobb_status check_made(int64_t N, int64_t n, const dobb_fp8_operand *rows, const dobb_fp8_operand *cols) {
    if (!rows && !cols) return DOBB_ERR_INVALID_ARG;
    for (const dobb_fp8_operand *op : {rows, cols}) {
        if (!op) continue;
        const dobb_status st = check_operand(op);
        if (st != DOBB_OK) return st;
        if (op->rows != (op == rows ? N : n) || op->k != (op == rows ? n : N)) return DOBB_ERR_SHAPE;
    }
    if (rows && cols && rows->format != cols->format) return DOBB_ERR_DTYPE;
    return fp8_tiles(N) <= kMaxWorkgroups / fp8_tiles(n) ? DOBB_OK : DOBB_ERR_SHAPE;
}

size_t grad_ws(int64_t N, int64_t n) { return al256((size_t)norm_grad_groups(N, n) * 2 * (size_t)n * 4); }

size_t moment_ws(const std::vector<MomentLaunch> &launches, int64_t tiles) {
    size_t need = 0;
    for (const MomentLaunch &l : launches) need = std::max(need, al256(moment_fp8_ws(l.nb, l.blocks, tiles)));
    return need;
}

dobb_status moment_grouped(int count, const dobb_shape *shapes, const dobb_fp8_operand *ops, int64_t N, float beta, float *const *A,
                           void *ws, size_t ws_bytes, hipStream_t stream) {
    if (count < 1 || !shapes || !ops || !A || !(beta >= 0.f && beta < 1.f)) return DOBB_ERR_INVALID_ARG;
    Spans spans;
    for (int i = 0; i < count; ++i) {
        dobb_status st = check_moment_shape(shapes[i]);
        if (st == DOBB_OK) st = check_operand(&ops[i]);
        if (st != DOBB_OK) return st;
        if (ops[i].rows != shapes[i].n) return DOBB_ERR_SHAPE;
        if (ops[i].format != ops[0].format) return DOBB_ERR_DTYPE;
        if (fp8_tiles(ops[i].k) != fp8_tiles(ops[0].k) || !A[i] || !aligned(A[i], 4)) return DOBB_ERR_INVALID_ARG;
        spans.add(A[i], 4 * (uintptr_t)shapes[i].n * (uintptr_t)shapes[i].nb, true);
        spans.operand(ops[i], false);
    }
    const int64_t tiles = fp8_tiles(ops[0].k);
    if (N < 1 || fp8_tiles(N) > tiles) return DOBB_ERR_INVALID_ARG;
    const std::vector<MomentLaunch> launches = moment_launches(count, shapes);
    const size_t need = moment_ws(launches, tiles);
    if (need) spans.add(ws, need, true);
    dobb_status st = spans.check();
    if (st == DOBB_OK) st = check_ws(ws, ws_bytes, need);
    if (st != DOBB_OK) return st;
    for (const MomentLaunch &l : launches) {
        const void *cs[kMomentMats], *ss[kMomentMats];
        float *as[kMomentMats];
        int64_t ns[kMomentMats];
        MomentArgs a{};
        a.count = (int)l.idx.size();
        for (int k = 0; k < a.count; ++k) {
            const int i = l.idx[k];
            cs[k] = ops[i].codes; ss[k] = ops[i].scales; as[k] = A[i]; ns[k] = shapes[i].n;
        }
        a.nb = l.nb;
        a.tiles = tiles;
        a.N = N;
        a.n = ns;
        a.codes = cs;
        a.scales = ss;
        a.A = as;
        a.beta = beta;
        a.plan = moment_fp8_plan(l.nb, l.blocks, tiles);
        a.partial = (float *)ws;
        st = hip_status(launch_moment_fp8(a, ops[0].format == DOBB_E5M2, stream));
        if (st != DOBB_OK) return st;
    }
    return DOBB_OK;
}

}  // namespace

extern "C" {

dobb_status dobb_layer_norm(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, const void *weight,
                            const void *bias, dobb_dtype w_dtype, float eps, void *Y, dobb_dtype y_dtype, int64_t ldy, float *mean,
                            float *rstd, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_norm(N, n, X, x_dtype, ldx, weight, bias, w_dtype, eps);
        if (st == DOBB_OK) st = check_matrix(Y, N, n, y_dtype, ldy);
        if (st != DOBB_OK) return st;
        if (!aligned(mean, 4) || !aligned(rstd, 4)) return DOBB_ERR_INVALID_ARG;
        Spans s;
        if (!(X == Y && x_dtype == y_dtype && ldx == ldy)) s.matrix(X, N, n, x_dtype, ldx, false);   // in place: a row is read whole first
        s.matrix(Y, N, n, y_dtype, ldy, true);
        s.vector(weight, n, w_dtype, false);
        s.vector(bias, n, w_dtype, false);
        s.vector(mean, N, DOBB_F32, true);
        s.vector(rstd, N, DOBB_F32, true);
        st = s.check();
        if (st != DOBB_OK) return st;
        return hip_status(launch_layer_norm(N, n, X, x_dtype == DOBB_BF16, ldx, weight, bias, w_dtype == DOBB_BF16, eps, Y,
                                            y_dtype == DOBB_BF16, ldy, mean, rstd, (hipStream_t)stream));
    });
}

size_t dobb_layer_norm_backward_workspace_size(int64_t N, int64_t n) {
    return N < 1 || N > kMaxN || n < 1 || n > kMaxN ? 0 : grad_ws(N, n);
}

dobb_status dobb_layer_norm_backward(int64_t N, int64_t n, const void *dY, dobb_dtype dy_dtype, int64_t lddy, const void *X,
                                     dobb_dtype x_dtype, int64_t ldx, const float *mean, const float *rstd, const void *weight,
                                     dobb_dtype w_dtype, void *dX, dobb_dtype dx_dtype, int64_t lddx, void *dweight, void *dbias,
                                     dobb_dtype g_dtype, void *ws, size_t ws_bytes, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_matrix(dY, N, n, dy_dtype, lddy);
        if (st == DOBB_OK) st = check_matrix(X, N, n, x_dtype, ldx);
        if (st == DOBB_OK) st = check_matrix(dX, N, n, dx_dtype, lddx);
        if (st == DOBB_OK) st = check_vector(weight, w_dtype);
        if (st == DOBB_OK) st = check_vector(dweight, g_dtype);
        if (st == DOBB_OK) st = check_vector(dbias, g_dtype);
        if (st != DOBB_OK) return st;
        if (N > kMaxN) return DOBB_ERR_SHAPE;
        if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return DOBB_ERR_INVALID_ARG;
        const size_t need = dweight || dbias ? grad_ws(N, n) : 0;
        Spans s;
        if (!(dY == dX && dy_dtype == dx_dtype && lddy == lddx)) s.matrix(dY, N, n, dy_dtype, lddy, false);
        s.matrix(X, N, n, x_dtype, ldx, false);
        s.matrix(dX, N, n, dx_dtype, lddx, true);
        s.vector(mean, N, DOBB_F32, false);
        s.vector(rstd, N, DOBB_F32, false);
        s.vector(weight, n, w_dtype, false);
        s.vector(dweight, n, g_dtype, true);
        s.vector(dbias, n, g_dtype, true);
        if (need) s.add(ws, need, true);
        st = s.check();
        if (st == DOBB_OK) st = check_ws(ws, ws_bytes, need);
        if (st != DOBB_OK) return st;
        NormGradArgs a{};
        a.N = N; a.n = n;
        a.dY = dY; a.dy_bf16 = dy_dtype == DOBB_BF16; a.lddy = lddy;
        a.X = X; a.x_bf16 = x_dtype == DOBB_BF16; a.ldx = ldx;
        a.mean = mean; a.rstd = rstd;
        a.w = weight; a.w_bf16 = w_dtype == DOBB_BF16;
        a.dX = dX; a.dx_bf16 = dx_dtype == DOBB_BF16; a.lddx = lddx;
        a.dw = dweight; a.db = dbias; a.g_bf16 = g_dtype == DOBB_BF16;
        a.part = (float *)ws;
        return hip_status(launch_layer_norm_backward(a, (hipStream_t)stream));
    });
}

dobb_status dobb_fp8_quantize(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, int32_t square,
                              const dobb_fp8_operand *along_rows, const dobb_fp8_operand *along_cols, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_matrix(X, N, n, x_dtype, ldx);
        if (st == DOBB_OK) st = check_made(N, n, along_rows, along_cols);
        if (st != DOBB_OK) return st;
        Spans s;
        s.matrix(X, N, n, x_dtype, ldx, false);
        if (along_rows) s.operand(*along_rows, true);
        if (along_cols) s.operand(*along_cols, true);
        st = s.check();
        if (st != DOBB_OK) return st;
        return hip_status(launch_fp8_quantize(N, n, X, x_dtype == DOBB_BF16, ldx, square != 0, NormArgs{}, along_rows, along_cols,
                                              (hipStream_t)stream));
    });
}

dobb_status dobb_layer_norm_fp8(int64_t N, int64_t n, const void *X, dobb_dtype x_dtype, int64_t ldx, const void *weight,
                                const void *bias, dobb_dtype w_dtype, float eps, float *mean, float *rstd,
                                const dobb_fp8_operand *along_rows, const dobb_fp8_operand *along_cols, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_norm(N, n, X, x_dtype, ldx, weight, bias, w_dtype, eps);
        if (st == DOBB_OK) st = check_made(N, n, along_rows, along_cols);
        if (st != DOBB_OK) return st;
        if (!mean || !rstd || !aligned(mean, 4) || !aligned(rstd, 4)) return DOBB_ERR_INVALID_ARG;
        Spans s;
        s.matrix(X, N, n, x_dtype, ldx, false);
        s.vector(weight, n, w_dtype, false);
        s.vector(bias, n, w_dtype, false);
        s.vector(mean, N, DOBB_F32, true);
        s.vector(rstd, N, DOBB_F32, true);
        if (along_rows) s.operand(*along_rows, true);
        if (along_cols) s.operand(*along_cols, true);
        st = s.check();
        if (st != DOBB_OK) return st;
        st = hip_status(launch_layer_norm(N, n, X, x_dtype == DOBB_BF16, ldx, nullptr, nullptr, false, eps, nullptr, false, n, mean,
                                          rstd, (hipStream_t)stream));
        if (st != DOBB_OK) return st;
        const NormArgs a{mean, rstd, weight, bias, w_dtype == DOBB_BF16};
        return hip_status(launch_fp8_quantize(N, n, X, x_dtype == DOBB_BF16, ldx, false, a, along_rows, along_cols, (hipStream_t)stream));
    });
}

dobb_status dobb_fp8_dequantize(const dobb_fp8_operand *op, int32_t transpose, void *out, dobb_dtype out_dtype, int64_t ldo,
                                dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_operand(op);
        if (st != DOBB_OK) return st;
        const int64_t R = transpose ? op->k : op->rows, C = transpose ? op->rows : op->k;
        st = check_matrix(out, R, C, out_dtype, ldo);
        if (st != DOBB_OK) return st;
        if (fp8_read_tiles(op->k, transpose) > kMaxWorkgroups / fp8_read_rows(op->rows, transpose)) return DOBB_ERR_SHAPE;
        Spans s;
        s.operand(*op, false);
        s.matrix(out, R, C, out_dtype, ldo, true);
        st = s.check();
        if (st != DOBB_OK) return st;
        return hip_status(launch_fp8_dequantize(*op, transpose != 0, out, out_dtype == DOBB_BF16, ldo, (hipStream_t)stream));
    });
}

size_t dobb_fp8_matmul_workspace_size(int64_t M, int64_t N, int64_t k) {
    if (M < 1 || M > kMaxN || N < 1 || N > kMaxN || k < 1 || k > kMaxTokens) return 0;
    return al256(fp8_matmul_ws(M, N, k));
}

dobb_status dobb_fp8_matmul(const dobb_fp8_operand *A, const dobb_fp8_operand *B, const void *bias, dobb_dtype bias_dtype,
                            int32_t accumulate, void *out, dobb_dtype out_dtype, int64_t ldo, void *ws, size_t ws_bytes,
                            dobb_stream_t stream) {
    return guarded([&]() -> dobb_status {
        dobb_status st = check_operand(A);
        if (st == DOBB_OK) st = check_operand(B);
        if (st != DOBB_OK) return st;
        if (A->k != B->k) return DOBB_ERR_SHAPE;
        st = check_matrix(out, A->rows, B->rows, out_dtype, ldo);
        if (st == DOBB_OK) st = check_vector(bias, bias_dtype);
        if (st != DOBB_OK) return st;
        const size_t need = al256(fp8_matmul_ws(A->rows, B->rows, A->k));
        Spans s;
        s.operand(*A, false);
        s.operand(*B, false);
        s.vector(bias, B->rows, bias_dtype, false);
        s.matrix(out, A->rows, B->rows, out_dtype, ldo, true);
        if (need) s.add(ws, need, true);
        st = s.check();
        if (st == DOBB_OK) st = check_ws(ws, ws_bytes, need);
        if (st != DOBB_OK) return st;
        return hip_status(launch_fp8_matmul(*A, *B, bias, bias_dtype == DOBB_BF16, accumulate != 0, out, out_dtype == DOBB_BF16, ldo,
                                            (float *)ws, (hipStream_t)stream));
    });
}

size_t dobb_moment_fp8_workspace_size(int count, const dobb_shape *shapes, int64_t tiles) {
    if (count < 1 || !shapes || tiles < 1 || tiles > kMaxTokens / kFp8Tile) return 0;
    for (int i = 0; i < count; ++i)
        if (check_moment_shape(shapes[i]) != DOBB_OK) return 0;
    try {
        return moment_ws(moment_launches(count, shapes), tiles);
    } catch (...) {
        return 0;
    }
}

dobb_status dobb_accumulate_moment_fp8_grouped(int count, const dobb_shape *shapes, const dobb_fp8_operand *ops, int64_t N, float beta,
                                               float *const *A, void *ws, size_t ws_bytes, dobb_stream_t stream) {
    return guarded([&]() -> dobb_status { return moment_grouped(count, shapes, ops, N, beta, A, ws, ws_bytes, (hipStream_t)stream); });
}

dobb_status dobb_accumulate_moment_fp8(const dobb_shape *s, const dobb_fp8_operand *op, int64_t N, float beta, float *A, void *ws,
                                       size_t ws_bytes, dobb_stream_t stream) {
    if (!s || !op) return DOBB_ERR_INVALID_ARG;
    return dobb_accumulate_moment_fp8_grouped(1, s, op, N, beta, &A, ws, ws_bytes, stream);
}

}  // extern "C"
