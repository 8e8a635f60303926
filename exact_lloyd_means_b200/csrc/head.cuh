// head.cuh -- shared declarations of the embedding-head operators (layer norm, linear,
// balance loss): element access for the two point types, workspace layouts, launchers.
#pragma once

#include "fk_common.cuh"
#include "prep_row.cuh"

namespace fk {

__device__ __forceinline__ float head_load(const float *p) { return *p; }
__device__ __forceinline__ float head_load(const uint16_t *p) { return bf16_val(*p); }
__device__ __forceinline__ void head_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void head_store(uint16_t *p, float v) { *p = bf16_bits(v); }

// ----------------------------------------------------------------- 16-byte vectors
// Elements of 16 bytes of a point type.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ void unpack16(const uint4 &u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack16(const uint4 &u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}
__device__ __forceinline__ uint4 pack16(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                      pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
}

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// N consecutive elements as they lie in memory: 16 bytes, or one element where rows are not
// multiples of 16 bytes.
template <typename T, int N>
struct Raw;
template <typename T>
struct Raw<T, kVec<T>> {
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void zero() { u = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void lowest() {  // -inf
        const uint32_t w = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
        u = make_uint4(w, w, w, w);
    }
    __device__ __forceinline__ void get(float (&v)[kVec<T>]) const { unpack16(u, v); }
    static __device__ __forceinline__ void put(T *p, const float (&v)[kVec<T>]) {
        *reinterpret_cast<uint4 *>(p) = pack16(v);
    }
};
// 32 bytes: one whole sector of memory for each thread of a warp that walks down rows.
template <typename T>
struct Raw<T, 2 * kVec<T>> {
    uint4 u[2];
    __device__ __forceinline__ void load(const T *p) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(u[0].x), "=r"(u[0].y), "=r"(u[0].z), "=r"(u[0].w), "=r"(u[1].x),
                       "=r"(u[1].y), "=r"(u[1].z), "=r"(u[1].w)
                     : "l"(p)
                     : "memory");
    }
    __device__ __forceinline__ void zero() { u[0] = u[1] = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&v)[2 * kVec<T>]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t[kVec<T>];
            unpack16(u[h], t);
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) v[h * kVec<T> + j] = t[j];
        }
    }
    static __device__ __forceinline__ void put(T *p, const float (&v)[2 * kVec<T>]) {
        uint4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t[kVec<T>];
#pragma unroll
            for (int j = 0; j < kVec<T>; ++j) t[j] = v[h * kVec<T> + j];
            w[h] = pack16(t);
        }
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                     "r"(w[0].x), "r"(w[0].y), "r"(w[0].z), "r"(w[0].w), "r"(w[1].x),
                     "r"(w[1].y), "r"(w[1].z), "r"(w[1].w)
                     : "memory");
    }
};
template <typename T>
struct Raw<T, 1> {
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ void zero() { u = T(0); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = head_load(&u); }
    static __device__ __forceinline__ void put(T *p, const float (&v)[1]) { head_store(p, v[0]); }
};

// V fp32 parameters (any 4-byte alignment; `vec`: 16-byte aligned).
template <int V>
__device__ __forceinline__ void load_params(const float *p, int vec, float (&v)[V]) {
    if constexpr (V % 4 == 0) {
        if (vec) {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(p + j);
                v[j] = f.x;
                v[j + 1] = f.y;
                v[j + 2] = f.z;
                v[j + 3] = f.w;
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = p[j];
}

// Two fp32 operations an instruction.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(F2 a, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ float sum2(F2 a) {
    float lo, hi;
    split(a, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
// 16 bytes of points as pairs.
__device__ __forceinline__ void unpack2(const uint4 &u, F2 (&v)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack2(const uint4 &u, F2 (&v)[2]) {
    v[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 pack2(const F2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(v[i], lo, hi);
        w[i] = pack_bf16(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack2(const F2 (&v)[2]) {
    float a, b, c, d;
    split(v[0], a, b);
    split(v[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c),
                      __float_as_uint(d));
}

// ----------------------------------------------------------------- layer norm
struct LayerNormArgs {
    const void *X, *dY;
    fk_dtype dtype;
    int64_t N;
    int d;
    const float *gamma, *beta;
    float eps;
    void *Y;  // forward: Y; backward: dX (optional)
    float *mean, *rstd;
    float *dgamma, *dbeta;  // backward, optional
    float *part;            // backward: [parts][2][d] partial column sums
    int64_t parts;
    uint32_t *err;          // backward: the workspace's error word
};
// Row groups whose column sums of the backward pass are formed apart and then joined in
// order (the workspace holds two rows of d floats for each).
int64_t layer_norm_parts(int64_t N, int d);
cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st);
cudaError_t launch_layer_norm_backward(const LayerNormArgs &a, cudaStream_t st);

// ----------------------------------------------------------------- balance loss
struct BalanceArgs {
    const void *S;
    fk_dtype dtype;
    int64_t N;
    int K;
    const int32_t *labels;
    int top;
    const int32_t *counts, *rows;
    float scale, coef;
    float *loss;
    void *dS;  // optional
    double *part;
    int64_t parts;
    uint32_t *err;  // the workspace's error word
};
int64_t balance_parts(int64_t N, int K);
cudaError_t launch_balance_counts(const int32_t *labels, int64_t N, int top, int K,
                                  int32_t *counts, int32_t *rows, cudaStream_t st);
cudaError_t launch_balance_loss(const BalanceArgs &a, cudaStream_t st);

// ----------------------------------------------------------------- linear
// Forward  Z = X W^T + b, Y = act(Z) + R; backward G = dY act'(Z), dX = G W, dW = G^T X,
// db = column sums of G.
struct LinearArgs {
    fk_dtype dtype;
    int64_t N;
    int d, m;
    const void *X, *W;
    const float *bias;
    fk_activation act;
    const void *R;
    void *Y, *Z;        // forward outputs (Z optional)
    const void *dY, *Zin;  // backward inputs
    void *dX, *dW;      // backward outputs, optional
    float *db;
};
size_t linear_ws_bytes(int64_t N, int d, int m, fk_dtype dtype);
size_t linear_backward_ws_bytes(int64_t N, int d, int m, fk_dtype dtype);
cudaError_t launch_linear(const LinearArgs &a, void *ws, cudaStream_t st);
cudaError_t launch_linear_backward(const LinearArgs &a, void *ws, cudaStream_t st);

// 1 / x and 2^x by the special function unit, subnormal results flushed: a few units of 2^-24,
// one instruction each (the forms that keep subnormals take several more).
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Half the complementary error function at |z| / sqrt(2), so that the normal distribution
// function Phi(z) is 1 - h for z > 0 and h otherwise, and e = exp(-z^2 / 2).  Abramowitz and
// Stegun 7.1.26: erf within 1.5e-7, so Phi within 0.75e-7 (1.3 units of 2^-24), in two special
// function calls and about ten products; with CUDA's erff, several times the instructions,
// the epilogue of a 768-deep product is bound by its arithmetic.
__device__ __forceinline__ F2 half_erfc2(F2 z, F2 a, F2 *e) {
    float lo, hi;
    split(fma2(a, f2(0.23164190f, 0.23164190f), f2(1.f, 1.f)), lo, hi);  // 0.3275911 / sqrt(2)
    const F2 t = f2(rcp_fast(lo), rcp_fast(hi));
    const auto twice = [](float c) { return f2(c, c); };
    F2 p = fma2(twice(0.5f * 1.061405429f), t, twice(-0.5f * 1.453152027f));
    p = fma2(p, t, twice(0.5f * 1.421413741f));
    p = fma2(p, t, twice(-0.5f * 0.284496736f));
    p = fma2(p, t, twice(0.5f * 0.254829592f));
    split(mul2(mul2(z, z), twice(-0.72134752f)), lo, hi);
    *e = f2(exp2_fast(lo), exp2_fast(hi));
    return mul2(mul2(p, t), *e);
}

__device__ __forceinline__ F2 abs2(F2 z) {
    F2 r;
    r.v = z.v & 0x7fffffff7fffffffull;
    return r;
}

// act(z) of a pair: relu max(z, 0); GELU z Phi(z) with the normal distribution function Phi
// (the erf form), as max(z, 0) - |z| h (h is 0 long before |z| = 32); SiLU z / (1 + exp(-z)).
// NaN stays NaN; at infinity, the limits of GELU, and for SiLU what its formula gives.
__device__ __forceinline__ F2 act_value2(F2 z, int act) {
    float lo, hi;
    if (act == FK_ACT_RELU) {
        split(z, lo, hi);
        return f2(lo > 0.f ? lo : (lo == lo ? 0.f : lo), hi > 0.f ? hi : (hi == hi ? 0.f : hi));
    }
    if (act == FK_ACT_GELU) {
        F2 e;
        const F2 a = abs2(z), h = half_erfc2(z, a, &e);
        float al, ah;
        split(z, lo, hi);
        split(a, al, ah);
        return fma2(f2(-fminf(al, 32.f), -fminf(ah, 32.f)), h, f2(fmaxf(lo, 0.f), fmaxf(hi, 0.f)));
    }
    if (act == FK_ACT_SILU) {
        split(mul2(z, f2(-1.44269504f, -1.44269504f)), lo, hi);
        split(add2(f2(exp2_fast(lo), exp2_fast(hi)), f2(1.f, 1.f)), lo, hi);
        return mul2(z, f2(rcp_fast(lo), rcp_fast(hi)));
    }
    return z;
}
// act'(z) of a pair; the slope of relu at 0 is 0.
__device__ __forceinline__ F2 act_slope2(F2 z, int act) {
    float lo, hi;
    if (act == FK_ACT_RELU) {
        split(z, lo, hi);
        return f2(lo > 0.f ? 1.f : (lo == lo ? 0.f : lo), hi > 0.f ? 1.f : (hi == hi ? 0.f : hi));
    }
    if (act == FK_ACT_GELU) {  // Phi + z phi, Phi = 1/2 + sign(z) (1/2 - h)
        F2 e;
        const F2 h = half_erfc2(z, abs2(z), &e);
        F2 u = fma2(h, f2(-1.f, -1.f), f2(0.5f, 0.5f));
        u.v ^= z.v & 0x8000000080000000ull;
        return fma2(mul2(z, f2(0.39894228f, 0.39894228f)), e, add2(u, f2(0.5f, 0.5f)));
    }
    if (act == FK_ACT_SILU) {  // s + z s (1 - s)
        split(mul2(z, f2(-1.44269504f, -1.44269504f)), lo, hi);
        split(add2(f2(exp2_fast(lo), exp2_fast(hi)), f2(1.f, 1.f)), lo, hi);
        const F2 s = f2(rcp_fast(lo), rcp_fast(hi));
        return fma2(mul2(z, s), fma2(s, f2(-1.f, -1.f), f2(1.f, 1.f)), s);
    }
    return f2(1.f, 1.f);
}
__device__ __forceinline__ float act_value(float z, int act) {
    float lo, hi;
    split(act_value2(f2(z, z), act), lo, hi);
    return lo;
}

}  // namespace fk
