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

// Column sums to be finished: db = the sum of the parts, each of `cols`.
struct ColSums {
    const float *part;
    float *db;
    int parts, cols;
};

// `sums`: finished by the launch that joins cut products, so only where there is one (or NULL
// db: none).
cudaError_t launch_gemm(const GemmArgs *args, const GemmPlan *plans, int n, const ColSums &sums,
                        cudaStream_t st);

// Columns 32 b .. 32 b + 31 of the sums by T threads: 32 runs of parts side by side, then the
// runs in a tree, whatever T is.
template <int T>
__device__ __forceinline__ void join_columns(const ColSums &s, int b, float (&red)[32][33]) {
    const int x = threadIdx.x & 31;
    const int64_t c = static_cast<int64_t>(b) * 32 + x;
    constexpr int Y = 32 * 32 / T, H = T / 32;  // runs of a thread: y, y + H, ...
    const int y0 = threadIdx.x >> 5;
    float v[Y] = {};
    if (c < s.cols) {
        const float *part = s.part + c;
        const auto at = [&](int p) { return static_cast<int64_t>(p) * s.cols; };
        const int whole = s.parts / 32 * 32;
#pragma unroll(8 / Y)
        for (int p = y0; p < whole; p += 32)
#pragma unroll
            for (int i = 0; i < Y; ++i) v[i] += part[at(p + i * H)];
#pragma unroll
        for (int i = 0; i < Y; ++i) {
            const int p = whole + y0 + i * H;
            if (p < s.parts) v[i] += part[at(p)];
        }
    }
#pragma unroll
    for (int i = 0; i < Y; ++i) red[y0 + i * H][x] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < Y; ++i) {
        const int y = y0 + i * H;
        const float t = warp_sum_f(red[x][y]);  // the runs of column y
        const int64_t o = static_cast<int64_t>(b) * 32 + y;
        if (x == 0 && o < s.cols) s.db[o] = t;
    }
}

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

// ----------------------------------------------------------------- epilogue of an fp32 warp
// A warp that holds 32 columns of 32 fp32 rows, a row a thread, in P pieces of R words (16 or 32
// bytes).  turn() exchanges them within groups of four threads: thread i of a group then holds,
// at position r of each run of four pieces, piece i of the group's row r; and back.  What a group
// reads or writes at one position is then a run of 64 or 128 bytes of a row, where a thread's
// own pieces touch 32 rows at once.  65536 x 128 of depth 1024: 162 us, 173 us with each
// thread's own pieces; 54531 x 80 of depth 1544 with Z 230 and 245.  In bf16, whose 32 columns are
// 64 bytes, the exchange costs more than it saves: 63 against 49 us.
template <int P, int R>
__device__ __forceinline__ void turn(uint32_t (&w)[P][R], int lane) {
    static_assert(P % 4 == 0, "whole groups");
#pragma unroll
    for (int s = 1; s < 4; s *= 2) {
        const bool up = (lane & s) != 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if ((p & s) == 0) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const uint32_t give = up ? w[p][k] : w[p | s][k];
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, s);
                    if (up)
                        w[p][k] = got;
                    else
                        w[p | s][k] = got;
                }
            }
        }
    }
}

// Rows r0 .. r0 + 31 (those below `rows`), columns col .. col + 31 (those below e.cols, a multiple
// of V): v holds the products of row r0 + lane without the bias.  Called by the whole warp; the
// same arithmetic as epilogue_pieces.
template <int V>
__device__ __forceinline__ void epilogue_warp_f32(const Epilogue &e, int64_t r0, int64_t rows,
                                                  int64_t col, int bvec, int lane,
                                                  float (&v)[32]) {
    constexpr int P = 32 / V;
    const int mate = lane & 3;
    const int64_t left = e.cols - col;  // columns from col on
    // at position p: row r0 + lane - mate + p % 4, piece p - p % 4 + mate
    const int64_t at = (r0 + lane - mate) * e.cols + col + mate * V;
    const auto offset = [&](int p) { return at + (p % 4) * e.cols + (p - p % 4) * V; };
    const auto has = [&](int p) {
        return r0 + lane - mate + p % 4 < rows && (p - p % 4 + mate) * V < left;
    };
    uint32_t w[P][V];
    if (e.bias != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (p * V < left) {
                float b[V];
                load_params<V>(e.bias + col + p * V, bvec, b);
#pragma unroll
                for (int j = 0; j < V; ++j) v[p * V + j] = __fadd_rn(v[p * V + j], b[j]);
            }
        }
    }
    const auto out = [&](void *base) {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j / V][j % V] = __float_as_uint(v[j]);
        turn(w, lane);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float f[V];
#pragma unroll
            for (int k = 0; k < V; ++k) f[k] = __uint_as_float(w[p][k]);
            if (has(p)) Raw<float, V>::put(static_cast<float *>(base) + offset(p), f);
        }
    };
    if (e.Z != nullptr) out(e.Z);
    float(&one)[1][32] = reinterpret_cast<float(&)[1][32]>(v);
    act_values(one, e.act);
    if (e.R != nullptr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (has(p)) {  // (of a piece that does not exist nothing is stored either)
                Raw<float, V> r;
                r.load(static_cast<const float *>(e.R) + offset(p));
                float f[V];
                r.get(f);
#pragma unroll
                for (int k = 0; k < V; ++k) w[p][k] = __float_as_uint(f[k]);
            }
        }
        turn(w, lane);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __fadd_rn(v[j], __uint_as_float(w[j / V][j % V]));
    }
    out(e.C);
}

}  // namespace fk
