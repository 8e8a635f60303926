// fk_head.cu -- the extern "C" boundary of the embedding-head operators: argument checks,
// workspace sizes and launches of layer_norm.cu, linear.cu and balance.cu.
#include <cmath>

#include "head.cuh"

using namespace fk;

namespace {

struct Span {
    const void *p;
    size_t bytes;
};

bool overlaps(const Span &a, const Span &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    return pa < pb + b.bytes && pb < pa + a.bytes;
}

// Every output against every input and every other output.  An output that starts where
// its `same` input starts may be that input (in place).
template <int NO, int NI>
bool clash(const Span (&out)[NO], const Span (&in)[NI], int out_same = -1, int in_same = -1) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlaps(out[o], in[i]) &&
                !(o == out_same && i == in_same && out[o].p == in[i].p))
                return true;
        for (int q = o + 1; q < NO; ++q)
            if (overlaps(out[o], out[q])) return true;
    }
    return false;
}

fk_status check_dtype(fk_dtype dtype) {
    return dtype == FK_F32 || dtype == FK_BF16 ? FK_OK : FK_ERR_UNSUPPORTED;
}

size_t elem(fk_dtype dtype) { return dtype == FK_F32 ? 4 : 2; }

// N rows of d elements, few enough that byte counts and sums of them fit 64 bits.
bool rows_ok(int64_t N, int64_t d) {
    return N >= 0 && N < (int64_t(1) << 31) && d >= 1 && d < (int64_t(1) << 31) &&
           N * d <= (int64_t(1) << 46);
}
bool linear_ok(int64_t N, int d, int m) { return m >= 1 && rows_ok(N, d) && rows_ok(N, m) && rows_ok(m, d); }

fk_status check_space(const void *ws, size_t ws_bytes, size_t need) {
    if (!ws || !aligned(ws, 256) || ws_bytes < need) return FK_ERR_WORKSPACE;
    if (injected_fault() == kFaultWorkspace) return FK_ERR_WORKSPACE;
    return FK_OK;
}

fk_status ready() {
    const fk_status s = check_device();
    if (s != FK_OK) return s;
    return injected_fault() == kFaultLaunch ? FK_ERR_CUDA : FK_OK;
}

fk_status done(cudaError_t e) { return e == cudaSuccess ? FK_OK : FK_ERR_CUDA; }

size_t layer_norm_ws(int64_t N, int d) {
    return 256 + sizeof(float) * 2 * static_cast<size_t>(layer_norm_parts(N, d)) * d;
}

size_t balance_ws(int64_t N, int K) {
    return 256 + sizeof(double) * static_cast<size_t>(balance_parts(N, K));
}

}  // namespace

extern "C" {

FK_API fk_status fk_layer_norm(const void *X, fk_dtype dtype, int64_t N, int d,
                               const float *gamma, const float *beta, float eps, void *Y,
                               float *mean, float *rstd, fk_stream_t stream) {
    if (!rows_ok(N, d) || !(eps >= 0.f) || std::isinf(eps)) return FK_ERR_INVALID_ARG;
    fk_status s = check_dtype(dtype);
    if (s != FK_OK) return s;
    if (N == 0) return FK_OK;
    if (!X || !Y) return FK_ERR_INVALID_ARG;
    const size_t e = elem(dtype), x = e * N * d, v = sizeof(float) * d, n = sizeof(float) * N;
    if (clash({{Y, x}, {mean, n}, {rstd, n}}, {{X, x}, {gamma, v}, {beta, v}}, 0, 0))
        return FK_ERR_INVALID_ARG;
    if (!aligned(X, e) || !aligned(Y, e) || !aligned(gamma, 4) || !aligned(beta, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return FK_ERR_UNSUPPORTED;
    if ((s = ready()) != FK_OK) return s;
    LayerNormArgs a{};
    a.X = X;
    a.dtype = dtype;
    a.N = N;
    a.d = d;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.Y = Y;
    a.mean = mean;
    a.rstd = rstd;
    return done(launch_layer_norm(a, stream));
}

FK_API fk_status fk_layer_norm_backward_workspace_size(int64_t N, int d, fk_dtype dtype,
                                                       size_t *bytes) {
    if (!rows_ok(N, d) || !bytes) return FK_ERR_INVALID_ARG;
    const fk_status s = check_dtype(dtype);
    if (s == FK_OK) *bytes = layer_norm_ws(N, d);
    return s;
}

FK_API fk_status fk_layer_norm_backward(const void *dY, const void *X, fk_dtype dtype, int64_t N,
                                        int d, const float *gamma, const float *mean,
                                        const float *rstd, void *dX, float *dgamma, float *dbeta,
                                        void *ws, size_t ws_bytes, fk_stream_t stream) {
    if (!rows_ok(N, d)) return FK_ERR_INVALID_ARG;
    fk_status s = check_dtype(dtype);
    if (s != FK_OK) return s;
    if (N > 0 && (!dY || !X || !mean || !rstd)) return FK_ERR_INVALID_ARG;
    const size_t e = elem(dtype), x = e * N * d, v = sizeof(float) * d, n = sizeof(float) * N;
    if (clash({{dX, x}, {dgamma, v}, {dbeta, v}, {ws, ws_bytes}},
              {{dY, x}, {X, x}, {gamma, v}, {mean, n}, {rstd, n}}, 0, 0))
        return FK_ERR_INVALID_ARG;
    if (!aligned(dY, e) || !aligned(X, e) || !aligned(dX, e) || !aligned(gamma, 4) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
        return FK_ERR_UNSUPPORTED;
    if ((s = check_space(ws, ws_bytes, layer_norm_ws(N, d))) != FK_OK) return s;
    if ((s = ready()) != FK_OK) return s;
    LayerNormArgs a{};
    a.X = X;
    a.dY = dY;
    a.dtype = dtype;
    a.N = N;
    a.d = d;
    a.gamma = gamma;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.Y = dX;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = ws_ptr<float>(ws, 256);
    a.parts = layer_norm_parts(N, d);
    a.err = ws_ptr<uint32_t>(ws, 0);
    return done(launch_layer_norm_backward(a, stream));
}

FK_API fk_status fk_linear_workspace_size(int64_t N, int d, int m, fk_dtype dtype,
                                          size_t *bytes) {
    if (!linear_ok(N, d, m) || !bytes) return FK_ERR_INVALID_ARG;
    const fk_status s = check_dtype(dtype);
    if (s == FK_OK) *bytes = linear_ws_bytes(N, d, m, dtype);
    return s;
}

FK_API fk_status fk_linear_backward_workspace_size(int64_t N, int d, int m, fk_dtype dtype,
                                                   size_t *bytes) {
    if (!linear_ok(N, d, m) || !bytes) return FK_ERR_INVALID_ARG;
    const fk_status s = check_dtype(dtype);
    if (s == FK_OK) *bytes = linear_backward_ws_bytes(N, d, m, dtype);
    return s;
}

FK_API fk_status fk_linear(const void *X, fk_dtype dtype, int64_t N, int d, const void *W, int m,
                           const float *bias, fk_activation act, const void *residual, void *Y,
                           void *Z, void *ws, size_t ws_bytes, fk_stream_t stream) {
    if (!linear_ok(N, d, m)) return FK_ERR_INVALID_ARG;
    fk_status s = check_dtype(dtype);
    if (s != FK_OK) return s;
    if (act < FK_ACT_NONE || act > FK_ACT_SILU) return FK_ERR_INVALID_ARG;
    if (N == 0) return FK_OK;
    if (!X || !W || !Y) return FK_ERR_INVALID_ARG;
    const size_t e = elem(dtype), x = e * N * d, w = e * m * d, y = e * N * m,
                 b = sizeof(float) * m;
    if (clash({{Y, y}, {Z, y}, {ws, ws_bytes}}, {{residual, y}, {X, x}, {W, w}, {bias, b}}, 0, 0))
        return FK_ERR_INVALID_ARG;
    if (!aligned(X, e) || !aligned(W, e) || !aligned(Y, e) || !aligned(Z, e) ||
        !aligned(residual, e) || !aligned(bias, 4))
        return FK_ERR_UNSUPPORTED;
    if ((s = check_space(ws, ws_bytes, linear_ws_bytes(N, d, m, dtype))) != FK_OK) return s;
    if ((s = ready()) != FK_OK) return s;
    LinearArgs a{};
    a.dtype = dtype;
    a.N = N;
    a.d = d;
    a.m = m;
    a.X = X;
    a.W = W;
    a.bias = bias;
    a.act = act;
    a.R = residual;
    a.Y = Y;
    a.Z = Z;
    return done(launch_linear(a, ws, stream));
}

FK_API fk_status fk_linear_backward(const void *dY, const void *X, fk_dtype dtype, int64_t N,
                                    int d, const void *W, int m, fk_activation act,
                                    const void *Z, void *dX, void *dW, float *dbias, void *ws,
                                    size_t ws_bytes, fk_stream_t stream) {
    if (!linear_ok(N, d, m)) return FK_ERR_INVALID_ARG;
    fk_status s = check_dtype(dtype);
    if (s != FK_OK) return s;
    if (act < FK_ACT_NONE || act > FK_ACT_SILU) return FK_ERR_INVALID_ARG;
    if (N > 0 && (!dY || (dW && !X) || (dX && !W) || (act != FK_ACT_NONE && !Z)))
        return FK_ERR_INVALID_ARG;
    const size_t e = elem(dtype), x = e * N * d, w = e * m * d, y = e * N * m,
                 b = sizeof(float) * m;
    if (clash({{dX, x}, {dW, w}, {dbias, b}, {ws, ws_bytes}}, {{dY, y}, {Z, y}, {X, x}, {W, w}}))
        return FK_ERR_INVALID_ARG;
    if (!aligned(dY, e) || !aligned(X, e) || !aligned(W, e) || !aligned(Z, e) ||
        !aligned(dX, e) || !aligned(dW, e) || !aligned(dbias, 4))
        return FK_ERR_UNSUPPORTED;
    if ((s = check_space(ws, ws_bytes, linear_backward_ws_bytes(N, d, m, dtype))) != FK_OK)
        return s;
    if ((s = ready()) != FK_OK) return s;
    LinearArgs a{};
    a.dtype = dtype;
    a.N = N;
    a.d = d;
    a.m = m;
    a.X = X;
    a.W = W;
    a.act = act;
    a.dY = dY;
    a.Zin = Z;
    a.dX = dX;
    a.dW = dW;
    a.db = dbias;
    return done(launch_linear_backward(a, ws, stream));
}

FK_API fk_status fk_balance_counts(const int32_t *labels, int64_t N, int top, int K,
                                   int32_t *counts, int32_t *rows, fk_stream_t stream) {
    if (!rows_ok(N, K) || top < 1 || N * top >= (int64_t(1) << 31) || !counts || !rows ||
        (N > 0 && !labels))
        return FK_ERR_INVALID_ARG;
    if (clash({{counts, sizeof(int32_t) * K}, {rows, sizeof(int32_t)}},
              {{labels, sizeof(int32_t) * N * top}}))
        return FK_ERR_INVALID_ARG;
    if (!aligned(labels, 4) || !aligned(counts, 4) || !aligned(rows, 4))
        return FK_ERR_UNSUPPORTED;
    const fk_status s = ready();
    if (s != FK_OK) return s;
    return done(launch_balance_counts(labels, N, top, K, counts, rows, stream));
}

FK_API fk_status fk_balance_workspace_size(int64_t N, int K, fk_dtype dtype, size_t *bytes) {
    if (!rows_ok(N, K) || !bytes) return FK_ERR_INVALID_ARG;
    const fk_status s = check_dtype(dtype);
    if (s == FK_OK) *bytes = balance_ws(N, K);
    return s;
}

FK_API fk_status fk_balance_loss(const void *S, fk_dtype dtype, int64_t N, int K,
                                 const int32_t *labels, int top, const int32_t *counts,
                                 const int32_t *rows, float scale, float coef, float *loss,
                                 void *dS, void *ws, size_t ws_bytes, fk_stream_t stream) {
    if (!rows_ok(N, K) || top < 1 || N * top >= (int64_t(1) << 31)) return FK_ERR_INVALID_ARG;
    fk_status s = check_dtype(dtype);
    if (s != FK_OK) return s;
    if (!(scale > 0.f && scale <= 1e37f) || !std::isfinite(coef) ||
        std::fabs(static_cast<double>(coef)) * scale * K > 1e38)
        return FK_ERR_INVALID_ARG;
    if (!counts || !rows || !loss || (N > 0 && (!S || !labels))) return FK_ERR_INVALID_ARG;
    const size_t e = elem(dtype), x = e * N * K;
    if (clash({{dS, x}, {loss, 4}, {ws, ws_bytes}},
              {{S, x}, {labels, sizeof(int32_t) * N * top}, {counts, sizeof(int32_t) * K},
               {rows, 4}},
              0, 0))
        return FK_ERR_INVALID_ARG;
    if (!aligned(S, e) || !aligned(dS, e) || !aligned(labels, 4) || !aligned(counts, 4) ||
        !aligned(rows, 4) || !aligned(loss, 4))
        return FK_ERR_UNSUPPORTED;
    if ((s = check_space(ws, ws_bytes, balance_ws(N, K))) != FK_OK) return s;
    if ((s = ready()) != FK_OK) return s;
    BalanceArgs a{};
    a.S = S;
    a.dtype = dtype;
    a.N = N;
    a.K = K;
    a.labels = labels;
    a.top = top;
    a.counts = counts;
    a.rows = rows;
    a.scale = scale;
    a.coef = coef;
    a.loss = loss;
    a.dS = dS;
    a.part = ws_ptr<double>(ws, 256);
    a.parts = balance_parts(N, K);
    a.err = ws_ptr<uint32_t>(ws, 0);
    return done(launch_balance_loss(a, stream));
}

}  // extern "C"
