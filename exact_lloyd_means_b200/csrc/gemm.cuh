// gemm.cuh -- the tensor-core product behind fk_linear: C = A B^T over a depth, with the
// epilogue act(C + bias) + R, or fp32 partial products of a part of the depth.
#pragma once

#include "head.cuh"

namespace fk {

// One bf16 operand: element (i, k) of plane p, i the row of A (or of B, a column of C).
// K-major: base[p][i][k], rows of ld; MN-major: base[p][k][i], rows of ld.  ld % 8 == 0 and
// base 16-byte aligned, as TMA asks.  One plane, or the three pieces of fp32 values.
struct GemmOperand {
    const uint16_t *base;
    int64_t ld;
    bool mn_major;
};

// How a product is cut: tiles of 128 * cg rows by bn columns (cg CTAs each), the depth in
// `splits` parts whose partial products are joined afterwards.
struct GemmPlan {
    int cg, bn, splits;
};

struct GemmArgs {
    fk_dtype dtype;  // of R, C and Z
    GemmOperand A, B;
    int planes;  // 1, or 3 with the six products that keep fp32 accuracy
    int64_t rows;
    int64_t cols, depth;
    const float *bias;
    int act;
    const void *R;
    void *C, *Z;
    float *part;  // [splits][rows][round_up(cols, 4)] when splits > 1
    uint32_t *err;
};

GemmPlan gemm_plan(int64_t rows, int64_t cols, int64_t depth, int planes);
inline size_t gemm_part_bytes(int64_t rows, int64_t cols, const GemmPlan &p) {
    return p.splits > 1 ? sizeof(float) * p.splits * rows * round_up(cols, 4) : 0;
}
cudaError_t launch_gemm(const GemmArgs &a, const GemmPlan &p, cudaStream_t st);

// ----------------------------------------------------------------- epilogue
template <int V>
__device__ __forceinline__ void act_values(float (&z)[V], int act) {
    if (act == FK_ACT_NONE) return;
    if (act == FK_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = act_value(z[j], FK_ACT_RELU);
    } else if (act == FK_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = act_value(z[j], FK_ACT_GELU);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = act_value(z[j], FK_ACT_SILU);
    }
}

struct Epilogue {
    const float *bias;
    const void *R;
    void *C, *Z;
    int64_t cols;
    int act;
    int vec;  // rows of C, Z and R start on 16-byte boundaries
};

// The residual of V columns, read before anything of the row is written (C may be R).
template <typename T>
__device__ __forceinline__ uint4 epilogue_residual(const Epilogue &e, int64_t row, int64_t col) {
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (e.R == nullptr) return u;
    const T *r = static_cast<const T *>(e.R) + row * e.cols + col;
    if (e.vec) return *reinterpret_cast<const uint4 *>(r);
    T *t = reinterpret_cast<T *>(&u);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
        if (col + j < e.cols) t[j] = r[j];
    return u;
}

template <typename T>
__device__ __forceinline__ void epilogue_bias(const Epilogue &e, int64_t col,
                                              float (&b)[kVec<T>]) {
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
        b[j] = e.bias != nullptr && col + j < e.cols ? e.bias[col + j] : 0.f;
}

template <typename T>
__device__ __forceinline__ void epilogue_put(T *row, int64_t col, int64_t cols, int vec,
                                             const uint4 &u) {
    if (vec) {
        *reinterpret_cast<uint4 *>(row + col) = u;
        return;
    }
    const T *t = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int j = 0; j < kVec<T>; ++j)
        if (col + j < cols) row[col + j] = t[j];
}

// z: products without the bias.  Each output is rounded once from fp32 (the additions are kept
// apart from the activation's products, so that the bits do not depend on which outputs are
// asked for).
template <typename T>
__device__ __forceinline__ void epilogue_store(const Epilogue &e, int64_t row, int64_t col,
                                               float (&z)[kVec<T>],
                                               const float (&b)[kVec<T>], const uint4 &r) {
    constexpr int V = kVec<T>;
#pragma unroll
    for (int j = 0; j < V; ++j) z[j] = __fadd_rn(z[j], b[j]);
    if (e.Z != nullptr)
        epilogue_put(static_cast<T *>(e.Z) + row * e.cols, col, e.cols, e.vec, pack16(z));
    act_values(z, e.act);
    if (e.R != nullptr) {
        float rv[V];
        unpack16(r, rv);
#pragma unroll
        for (int j = 0; j < V; ++j) z[j] = __fadd_rn(z[j], rv[j]);
    }
    epilogue_put(static_cast<T *>(e.C) + row * e.cols, col, e.cols, e.vec, pack16(z));
}

}  // namespace fk
