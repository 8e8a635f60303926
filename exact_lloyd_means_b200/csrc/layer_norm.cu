// layer_norm.cu -- layer norm over the rows of N x d points, forward and backward.
//
// mean_i = sum_j x_ij / d, rstd_i = 1 / sqrt(sum_j (x_ij - mean_i)^2 / d + eps),
// y = (x - mean) rstd gamma + beta.  With h = (x - mean) rstd and w = dy gamma:
//   dx = rstd (w - mean_j(w) - h mean_j(w h)),  dgamma = sum_i dy h,  dbeta = sum_i dy.
// All statistics and sums are fp32; each output is rounded once.
//
// Both passes are bound by memory: the forward pass reads and writes each element once, the
// backward pass reads two and writes one.  So a row is read once and kept in registers, by a
// group of TPR threads that hold NV vectors of V elements each (V: 16 bytes, or one element
// where rows are not multiples of 16 bytes); statistics are sums over the group.  Rows that
// do not fit the registers of a block are read again for each sum.
#include "head.cuh"

namespace fk {
namespace {

constexpr int kThreads = 256;

// Sum of v over the TPR threads of a row group; red: a block's scratch, [2][warps][2], one of
// whose halves (`slot`) this row uses, so that one barrier a row is enough.
template <int TPR>
__device__ __forceinline__ void group_sum2(float &a, float &b, float (*red)[kThreads / 32][2],
                                           int slot) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TPR > 32) {
        static_assert(TPR == kThreads, "one row a block");
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) {
            red[slot][warp][0] = a;
            red[slot][warp][1] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            a += red[slot][w][0];
            b += red[slot][w][1];
        }
    }
}

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(kThreads)
    layer_norm_kernel(const T *X, int64_t N, int d, const float *__restrict__ gamma,
                      const float *__restrict__ beta, int pvec, float eps, T *Y,
                      float *__restrict__ mean, float *__restrict__ rstd) {
    __shared__ float red[2][kThreads / 32][2];
    pdl_wait();
    pdl_trigger();
    constexpr int G = kThreads / TPR;
    const int t = threadIdx.x % TPR;
    const float inv = 1.f / static_cast<float>(d);
    int slot = 0;
    // every thread of a block takes the same number of turns (the groups meet in shuffles)
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * G; i0 < N;
         i0 += static_cast<int64_t>(gridDim.x) * G) {
        const int64_t i = i0 + threadIdx.x / TPR;
        const bool row = i < N;
        Raw<T, V> x[NV];
        float s = 0.f, q = 0.f, unused = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
            if (row && j < d)
                x[n].load(X + i * d + j);
            else
                x[n].zero();
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float v[V];
            x[n].get(v);
#pragma unroll
            for (int k = 0; k < V; ++k) s += v[k];
        }
        group_sum2<TPR>(s, unused, red, slot);
        slot ^= 1;
        const float mu = s * inv;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if ((n * TPR + t) * V < d) {
                float v[V];
                x[n].get(v);
#pragma unroll
                for (int k = 0; k < V; ++k) q += (v[k] - mu) * (v[k] - mu);
            }
        }
        group_sum2<TPR>(q, unused, red, slot);
        slot ^= 1;
        const float r = 1.f / sqrtf(q * inv + eps);
        if (!row) continue;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
            if (j < d) {
                float v[V], g[V], b[V];
                x[n].get(v);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    g[k] = 1.f;
                    b[k] = 0.f;
                }
                if (gamma) load_params<V>(gamma + j, pvec, g);
                if (beta) load_params<V>(beta + j, pvec, b);
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] = (v[k] - mu) * r * g[k] + b[k];
                Raw<T, V>::put(Y + i * d + j, v);
            }
        }
        if (t == 0) {
            if (mean) mean[i] = mu;
            if (rstd) rstd[i] = r;
        }
    }
}

// Rows longer than a block's registers: one block a row, read again for each sum.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_long_kernel(const T *X, int64_t N, int d, const float *__restrict__ gamma,
                           const float *__restrict__ beta, float eps, T *Y,
                           float *__restrict__ mean, float *__restrict__ rstd) {
    __shared__ float red[2][kThreads / 32][2];
    pdl_wait();
    pdl_trigger();
    for (int64_t i = blockIdx.x; i < N; i += gridDim.x) {
        const T *x = X + i * d;
        float s = 0.f, q = 0.f, unused = 0.f;
        for (int64_t j = threadIdx.x; j < d; j += kThreads) s += head_load(x + j);
        group_sum2<kThreads>(s, unused, red, 0);
        const float mu = s / static_cast<float>(d);
        for (int64_t j = threadIdx.x; j < d; j += kThreads) {
            const float c = head_load(x + j) - mu;
            q += c * c;
        }
        group_sum2<kThreads>(q, unused, red, 1);
        const float r = 1.f / sqrtf(q / static_cast<float>(d) + eps);
        for (int64_t j = threadIdx.x; j < d; j += kThreads) {
            const float h = (head_load(x + j) - mu) * r;
            head_store(Y + i * d + j, h * (gamma ? gamma[j] : 1.f) + (beta ? beta[j] : 0.f));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[i] = mu;
            if (rstd) rstd[i] = r;
        }
    }
}

// Backward: dX row by row, and the block's column sums of its rows in registers; the groups
// of a block are joined in shared memory, the blocks by layer_norm_join_kernel.  The next
// row is loaded before this row's sums are formed.
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(kThreads)
    layer_norm_backward_kernel(const T *dY, const T *__restrict__ X, int64_t N, int d,
                               const float *__restrict__ gamma, int pvec,
                               const float *__restrict__ mean, const float *__restrict__ rstd,
                               T *dX, float *__restrict__ part) {
    constexpr int G = kThreads / TPR;
    __shared__ float red[2][kThreads / 32][2];
    __shared__ float sums[G > 1 ? kThreads * 2 : 2];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const float inv = 1.f / static_cast<float>(d);
    float sg[NV][V], sb[NV][V];
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int k = 0; k < V; ++k) sg[n][k] = sb[n][k] = 0.f;
    Raw<T, V> x[NV], y[NV];
    float mu = 0.f, r = 0.f;
    auto fetch = [&](int64_t i) {
        if (i < N) {
            mu = mean[i];
            r = rstd[i];
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
            if (i < N && j < d) {
                x[n].load(X + i * d + j);
                y[n].load(dY + i * d + j);
            } else {
                x[n].zero();
                y[n].zero();
            }
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    int64_t i0 = static_cast<int64_t>(blockIdx.x) * G;
    if (i0 < N) fetch(i0 + grp);
    int slot = 0;
    for (; i0 < N; i0 += step) {
        const int64_t i = i0 + grp;
        float h[NV][V], w[NV][V];
        float a = 0.f, b = 0.f;
        const float rr = r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
            float xv[V], yv[V], g[V];
            x[n].get(xv);
            y[n].get(yv);
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] = 1.f;
            if (gamma && j < d) load_params<V>(gamma + j, pvec, g);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                h[n][k] = j < d && i < N ? (xv[k] - mu) * r : 0.f;
                w[n][k] = yv[k] * g[k];
                a += w[n][k];
                b += w[n][k] * h[n][k];
                sg[n][k] += yv[k] * h[n][k];
                sb[n][k] += yv[k];
            }
        }
        if (i0 + step < N) fetch(i0 + step + grp);
        group_sum2<TPR>(a, b, red, slot);
        slot ^= 1;
        a *= inv;
        b *= inv;
        if (dX != nullptr && i < N) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int j = (n * TPR + t) * V;
                if (j < d) {
                    float v[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) v[k] = rr * (w[n][k] - a - h[n][k] * b);
                    Raw<T, V>::put(dX + i * d + j, v);
                }
            }
        }
    }
    if (part == nullptr) return;
    float *out = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int j = (n * TPR + t) * V + k;
            float g = sg[n][k], b = sb[n][k];
            if constexpr (G > 1) {
                sums[threadIdx.x] = g;
                sums[kThreads + threadIdx.x] = b;
                __syncthreads();
                if (grp == 0) {
                    for (int o = 1; o < G; ++o) {
                        g += sums[o * TPR + t];
                        b += sums[kThreads + o * TPR + t];
                    }
                }
                __syncthreads();
            }
            if (grp == 0 && j < d) {
                out[j] = g;
                out[d + j] = b;
            }
        }
    }
}

// The same for rows longer than a block's registers: dX, one block a row ...
template <typename T>
__global__ void __launch_bounds__(kThreads)
    layer_norm_long_dx_kernel(const T *dY, const T *__restrict__ X, int64_t N, int d,
                              const float *__restrict__ gamma, const float *__restrict__ mean,
                              const float *__restrict__ rstd, T *dX) {
    __shared__ float red[2][kThreads / 32][2];
    pdl_wait();
    pdl_trigger();
    int slot = 0;
    for (int64_t i = blockIdx.x; i < N; i += gridDim.x) {
        const T *x = X + i * d, *g = dY + i * d;
        const float mu = mean[i], r = rstd[i];
        float a = 0.f, b = 0.f;
        for (int64_t j = threadIdx.x; j < d; j += kThreads) {
            const float w = head_load(g + j) * (gamma ? gamma[j] : 1.f);
            a += w;
            b += w * ((head_load(x + j) - mu) * r);
        }
        group_sum2<kThreads>(a, b, red, slot);
        slot ^= 1;
        a /= static_cast<float>(d);
        b /= static_cast<float>(d);
        for (int64_t j = threadIdx.x; j < d; j += kThreads) {
            const float w = head_load(g + j) * (gamma ? gamma[j] : 1.f);
            const float h = (head_load(x + j) - mu) * r;
            head_store(dX + i * d + j, r * (w - a - h * b));
        }
    }
}

// ... and the column sums of row run blockIdx.y, one thread a column.
template <typename T>
__global__ void __launch_bounds__(128)
    layer_norm_long_cols_kernel(const T *__restrict__ dY, const T *__restrict__ X, int64_t N,
                                int d, const float *__restrict__ mean,
                                const float *__restrict__ rstd, float *__restrict__ part) {
    pdl_wait();
    pdl_trigger();
    const int64_t j = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (j >= d) return;
    const int64_t p = blockIdx.y, parts = gridDim.y;
    float sg = 0.f, sb = 0.f;
    for (int64_t i = N * p / parts; i < N * (p + 1) / parts; ++i) {
        const float g = head_load(dY + i * d + j);
        sg += g * ((head_load(X + i * d + j) - mean[i]) * rstd[i]);
        sb += g;
    }
    part[(p * 2) * d + j] = sg;
    part[(p * 2 + 1) * d + j] = sb;
}

// dgamma and dbeta: the sums of the parts.  32 columns a block (of 2 d: dgamma's, then
// dbeta's), 8 runs of parts side by side.
__global__ void __launch_bounds__(kThreads)
    layer_norm_join_kernel(const float *__restrict__ part, int parts, int64_t d,
                           float *__restrict__ dgamma, float *__restrict__ dbeta) {
    __shared__ float red[8][33];
    pdl_wait();
    pdl_trigger();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float s = 0.f;
    if (c < 2 * d) {
#pragma unroll 4
        for (int p = y; p < parts; p += 8) s += part[static_cast<int64_t>(p) * 2 * d + c];
    }
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && c < 2 * d) {
        for (int t = 1; t < 8; ++t) s += red[t][x];
        float *o = c < d ? dgamma : dbeta;
        if (o) o[c < d ? c : c - d] = s;
    }
}

int block_grid(int64_t rows, int groups, int per_sm) {
    const int64_t g = ceil_div(rows, groups),
                  cap = static_cast<int64_t>(device_sm_count()) * per_sm;
    return static_cast<int>(g < cap ? g : cap);
}

// Blocks of the backward pass, and so parts of the column sums: at most four an SM.
constexpr int64_t kMaxParts = 148 * 4;

template <typename T, int V, int NV, int TPR>
cudaError_t forward_cfg(const LayerNormArgs &a, cudaStream_t st) {
    const int pvec = aligned(a.gamma, 16) && aligned(a.beta, 16);
    const cudaError_t e = launch_pdl(
        layer_norm_kernel<T, V, NV, TPR>, dim3(block_grid(a.N, kThreads / TPR, 16)),
        dim3(kThreads), 0, st, static_cast<const T *>(a.X), a.N, a.d, a.gamma, a.beta, pvec, a.eps,
        static_cast<T *>(a.Y), a.mean, a.rstd);
    if (e == cudaSuccess) note_launch();
    return e;
}

// A warp a row up to 16 vectors a lane, a block a row up to 16 vectors a thread.
template <typename T, int V>
cudaError_t forward_v(const LayerNormArgs &a, cudaStream_t st) {
    const int64_t nv = ceil_div(a.d, V);
    if (nv <= 32) return forward_cfg<T, V, 1, 32>(a, st);
    if (nv <= 64) return forward_cfg<T, V, 2, 32>(a, st);
    if (nv <= 128) return forward_cfg<T, V, 4, 32>(a, st);
    if (nv <= 256) return forward_cfg<T, V, 8, 32>(a, st);
    if (nv <= 512) return forward_cfg<T, V, 16, 32>(a, st);
    if (nv <= 1024) return forward_cfg<T, V, 4, kThreads>(a, st);
    if (nv <= 2048) return forward_cfg<T, V, 8, kThreads>(a, st);
    if (nv <= 4096) return forward_cfg<T, V, 16, kThreads>(a, st);
    const cudaError_t e = launch_pdl(
        layer_norm_long_kernel<T>, dim3(block_grid(a.N, 1, 8)), dim3(kThreads), 0, st,
        static_cast<const T *>(a.X), a.N, a.d, a.gamma, a.beta, a.eps, static_cast<T *>(a.Y),
        a.mean, a.rstd);
    if (e == cudaSuccess) note_launch();
    return e;
}

template <typename T, int V, int NV, int TPR>
cudaError_t backward_cfg(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    const int64_t g = ceil_div(a.N, kThreads / TPR);
    *parts = static_cast<int>(g < a.parts ? g : a.parts);
    const cudaError_t e = launch_pdl(
        layer_norm_backward_kernel<T, V, NV, TPR>, dim3(*parts), dim3(kThreads), 0, st,
        static_cast<const T *>(a.dY), static_cast<const T *>(a.X), a.N, a.d, a.gamma,
        static_cast<int>(aligned(a.gamma, 16)), static_cast<const float *>(a.mean),
        static_cast<const float *>(a.rstd), static_cast<T *>(a.Y),
        a.dgamma || a.dbeta ? a.part : nullptr);
    if (e == cudaSuccess) note_launch();
    return e;
}

template <typename T>
cudaError_t backward_long(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    cudaError_t e = cudaSuccess;
    if (a.dgamma || a.dbeta) {
        int64_t p = ceil_div(a.N, 64);
        if (p > a.parts) p = a.parts;
        *parts = static_cast<int>(p);
        e = launch_pdl(layer_norm_long_cols_kernel<T>,
                       dim3(static_cast<unsigned>(ceil_div(a.d, 128)), *parts), dim3(128), 0, st,
                       static_cast<const T *>(a.dY), static_cast<const T *>(a.X), a.N, a.d,
                       static_cast<const float *>(a.mean), static_cast<const float *>(a.rstd),
                       a.part);
        if (e != cudaSuccess) return e;
        note_launch();
    }
    if (a.Y) {
        e = launch_pdl(layer_norm_long_dx_kernel<T>, dim3(block_grid(a.N, 1, 8)), dim3(kThreads),
                       0, st, static_cast<const T *>(a.dY), static_cast<const T *>(a.X), a.N, a.d,
                       a.gamma, static_cast<const float *>(a.mean),
                       static_cast<const float *>(a.rstd), static_cast<T *>(a.Y));
        if (e == cudaSuccess) note_launch();
    }
    return e;
}

// At most 16 columns a thread up to a block a row, then 32 (their sums take two registers
// each).
template <typename T, int V>
cudaError_t backward_v(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    constexpr int C16 = 16 / V;  // vectors of 16 columns
    if (a.d <= 8 * V) return backward_cfg<T, V, 1, 8>(a, st, parts);
    if (a.d <= 32 * V) return backward_cfg<T, V, 1, 32>(a, st, parts);
    if (a.d <= 32 * 16) return backward_cfg<T, V, C16, 32>(a, st, parts);
    if (a.d <= kThreads * V) return backward_cfg<T, V, 1, kThreads>(a, st, parts);
    if (a.d <= kThreads * 16) return backward_cfg<T, V, C16, kThreads>(a, st, parts);
    if (a.d <= kThreads * 32) return backward_cfg<T, V, 2 * C16, kThreads>(a, st, parts);
    return backward_long<T>(a, st, parts);
}

template <typename T>
bool rows_in_vectors(const LayerNormArgs &a) {
    return a.d % kVec<T> == 0 && aligned(a.X, 16) && aligned(a.Y, 16) && aligned(a.dY, 16);
}

template <typename T>
cudaError_t forward_t(const LayerNormArgs &a, cudaStream_t st) {
    return rows_in_vectors<T>(a) ? forward_v<T, kVec<T>>(a, st) : forward_v<T, 1>(a, st);
}

template <typename T>
cudaError_t backward_t(const LayerNormArgs &a, cudaStream_t st) {
    int parts = 0;
    cudaError_t e = cudaSuccess;
    if (a.N > 0 && (a.Y || a.dgamma || a.dbeta))
        e = rows_in_vectors<T>(a) ? backward_v<T, kVec<T>>(a, st, &parts)
                                  : backward_v<T, 1>(a, st, &parts);
    if (e != cudaSuccess || (!a.dgamma && !a.dbeta)) return e;
    e = launch_pdl(layer_norm_join_kernel,
                   dim3(static_cast<unsigned>(ceil_div(2 * static_cast<int64_t>(a.d), 32))),
                   dim3(kThreads), 0, st, static_cast<const float *>(a.part), parts,
                   static_cast<int64_t>(a.d), a.dgamma, a.dbeta);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace

int64_t layer_norm_parts(int64_t N, int d) {
    (void)d;
    return N < 1 ? 1 : (N < kMaxParts ? N : kMaxParts);
}

cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st) {
    return a.dtype == FK_F32 ? forward_t<float>(a, st) : forward_t<uint16_t>(a, st);
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs &a, cudaStream_t st) {
    return a.dtype == FK_F32 ? backward_t<float>(a, st) : backward_t<uint16_t>(a, st);
}

}  // namespace fk
