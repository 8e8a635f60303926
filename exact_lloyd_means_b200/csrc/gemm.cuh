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

// How a product is cut: tiles of 128 * cg rows by bn columns (cg CTAs each).  The first `full`
// tiles take the whole depth; that of the others, which would leave most of the GPU idle, is
// cut into `splits` parts, whose partial products are joined afterwards.
struct GemmPlan {
    int cg, bn, splits;
    int64_t full, tail;
    int64_t tile() const { return int64_t(128) * cg * bn; }
};

struct GemmArgs {
    fk_dtype dtype;  // of R, C and Z; FK_F32: operands of three planes
    GemmOperand A, B;
    int64_t rows;
    int64_t cols, depth;
    const float *bias;
    int act;
    const void *R;
    void *C, *Z;
    float *part;  // [tail tile][split][row][column] of whole tiles, when splits > 1
    uint32_t *err;
};

// Up to two products of the same type run in one launch, with tiles of one shape.
constexpr int kMaxProducts = 2;
struct GemmSize {
    int64_t rows, cols, depth;
};
void gemm_plan(const GemmSize *sizes, int n, fk_dtype dtype, GemmPlan *plans);
inline size_t gemm_part_bytes(const GemmPlan &p) {
    return p.splits > 1 ? sizeof(float) * p.tail * p.splits * p.tile() : 0;
}
cudaError_t launch_gemm(const GemmArgs *args, const GemmPlan *plans, int n, cudaStream_t st);

// ----------------------------------------------------------------- epilogue
// One branch for all the values, which keeps their chains of dependent instructions side by
// side.
template <int P, int V>
__device__ __forceinline__ void act_values(float (&z)[P][V], int act) {
    static_assert(P * V % 2 == 0 || P * V == 1, "pairs");
    auto all = [&](int which) {
        if constexpr (P * V == 1) {
            z[0][0] = act_value(z[0][0], which);
        } else {
#pragma unroll
            for (int i = 0; i < P * V; i += 2) {
                float &lo = z[i / V][i % V], &hi = z[(i + 1) / V][(i + 1) % V];
                split(act_value2(f2(lo, hi), which), lo, hi);
            }
        }
    };
    if (act == FK_ACT_NONE) return;
    if (act == FK_ACT_RELU)
        all(FK_ACT_RELU);
    else if (act == FK_ACT_GELU)
        all(FK_ACT_GELU);
    else
        all(FK_ACT_SILU);
}

struct Epilogue {
    const float *bias;
    const void *R;
    void *C, *Z;
    int64_t cols;
    int act;
};

// P pieces of V consecutive columns of the output: piece p starts at element at + p * step of the
// output, in column col + p * cstep; it exists if bit p of `in` is set (or ALL of them do).
struct Pieces {
    int64_t at, step, col;
    int cstep;
    uint32_t in;
};

// z: their products without the bias.  Each output is rounded once from fp32.  The residual
// is read before anything of the pieces is written (C may be R).  The additions
// are kept apart from the activation's products, so that the bits do not depend on which
// outputs are asked for.
template <typename T, int V, bool ALL, int P>
__device__ __forceinline__ void epilogue_pieces(const Epilogue &e, const Pieces &o, int bvec,
                                                float (&z)[P][V]) {
    Raw<T, V> res[P];
    if (e.R != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            res[p].zero();
            if (ALL || (o.in >> p & 1u)) res[p].load(static_cast<const T *>(e.R) + o.at + p * o.step);
        }
    }
    if (e.bias != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (ALL || (o.in >> p & 1u)) {
                float b[V];
                load_params<V>(e.bias + o.col + p * o.cstep, bvec, b);
#pragma unroll
                for (int j = 0; j < V; ++j) z[p][j] = __fadd_rn(z[p][j], b[j]);
            }
        }
    }
    if (e.Z != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (ALL || (o.in >> p & 1u)) Raw<T, V>::put(static_cast<T *>(e.Z) + o.at + p * o.step, z[p]);
    }
    act_values(z, e.act);
    if (e.R != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float r[V];
            res[p].get(r);
#pragma unroll
            for (int j = 0; j < V; ++j) z[p][j] = __fadd_rn(z[p][j], r[j]);
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
        if (ALL || (o.in >> p & 1u)) Raw<T, V>::put(static_cast<T *>(e.C) + o.at + p * o.step, z[p]);
}

}  // namespace fk
