// balance.cu -- the balance loss over K cells (or experts): counts of a selection, and the
// loss of the scores with its gradient.
//
// labels[i][t] is the t-th cell selected by row i; an entry outside [0, K) selects nothing,
// and a row without any selection is padding.  counts_k = #{(i, t): labels[i][t] = k}, n =
// rows that are not padding, f_k = counts_k / (n top), p_i = softmax(scale s_i):
//   loss = coef K sum_k f_k (1/n) sum_i p_ik = (coef K / n) sum_i t_i, t_i = sum_k f_k p_ik,
//   dS_ij = (coef scale K / n) p_ij (f_j - t_i)     (f is a constant, as the counts are).
// The second form of the loss needs only the counts before the pass over S, so loss and
// gradient take one pass, bound by reading S and writing dS.  A row is read once and kept in
// registers by a group of TPR threads: each forms the maximum m, sum z = sum exp(x - m) and
// weighted sum sum f exp(x - m) of its own columns, and the group joins them (rescaled to
// the common maximum).  A row whose scores are all -inf has p = 0.
#include "head.cuh"

namespace fk {
namespace {

constexpr int kThreads = 256;
constexpr int kOneBlockLabels = 1 << 15;  // counted by one block in one launch
constexpr int kSharedCells = 12288;       // counters kept in shared memory (48 KB)

// Counts of one run of labels: in shared memory, then (several blocks) added to the zeroed
// totals.  Integer atomics: the order does not change the sums.
template <bool ONE>
__global__ void __launch_bounds__(1024)
    balance_counts_kernel(const int32_t *__restrict__ labels, int64_t N, int top, int K,
                          int32_t *__restrict__ counts, int32_t *__restrict__ rows) {
    extern __shared__ int32_t hist[];
    __shared__ int32_t srows;
    pdl_wait();
    pdl_trigger();
    const bool local = K <= kSharedCells;
    if (local)
        for (int k = threadIdx.x; k < K; k += blockDim.x) hist[k] = 0;
    if (threadIdx.x == 0) srows = 0;
    __syncthreads();
    int32_t *h = local ? hist : counts;
    int mine = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < N;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        bool any = false;
        for (int t = 0; t < top; ++t) {
            const int32_t l = labels[i * top + t];
            if (l >= 0 && l < K) {
                any = true;
                atomicAdd(h + l, 1);
            }
        }
        mine += any;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0 && mine) atomicAdd(&srows, mine);
    __syncthreads();
    if (ONE) {
        for (int k = threadIdx.x; k < K; k += blockDim.x) counts[k] = hist[k];
        if (threadIdx.x == 0) *rows = srows;
    } else {
        if (local)
            for (int k = threadIdx.x; k < K; k += blockDim.x)
                if (hist[k]) atomicAdd(counts + k, hist[k]);
        if (threadIdx.x == 0 && srows) atomicAdd(rows, srows);
    }
}

__global__ void balance_zero_kernel(int32_t *__restrict__ counts, int K,
                                    int32_t *__restrict__ rows) {
    pdl_wait();
    pdl_trigger();
    for (int k = blockIdx.x * blockDim.x + threadIdx.x; k < K; k += gridDim.x * blockDim.x)
        counts[k] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *rows = 0;
}

struct LossArgs {
    int64_t N;
    int K, top;
    const int32_t *labels, *counts, *rows;
    float scale, coef;
    int cvec;  // counts start on a 16-byte boundary
    float *loss;
    double *part;
};

// n, 1 / (n top) and coef scale K / n.
struct LossScales {
    float n, unit, gc;
    __device__ __forceinline__ explicit LossScales(const LossArgs &a) {
        const int32_t r = *a.rows;
        n = static_cast<float>(r > 0 ? r : 1);
        unit = 1.f / (n * static_cast<float>(a.top));
        gc = a.coef * a.scale * static_cast<float>(a.K) / n;
    }
};

__device__ __forceinline__ bool row_selects(const LossArgs &a, int64_t i) {
    for (int t = 0; t < a.top; ++t) {
        const int32_t l = a.labels[i * a.top + t];
        if (l >= 0 && l < a.K) return true;
    }
    return false;
}

// The running softmax sums of some columns: maximum, sum of exp(x - m), and that sum
// weighted by f.  m = -inf (with zero sums) where there is nothing but -inf; NaN anywhere
// makes all NaN.
struct Soft {
    float m, z, t;
    __device__ __forceinline__ void join(float m2, float z2, float t2) {
        const float mm = fmaxf(m, m2);
        const float a = mm == -INFINITY ? 0.f : __expf(m - mm);
        const float b = mm == -INFINITY ? 0.f : __expf(m2 - mm);
        z = z * a + z2 * b;
        t = t * a + t2 * b;
        m = mm;
    }
};

template <int W>
__device__ __forceinline__ void join_lanes(Soft &s) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        s.join(__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.z, o),
               __shfl_xor_sync(0xffffffffu, s.t, o));
}

template <int TPR>
__device__ __forceinline__ void join_group(Soft &s, Soft (*red)[kThreads / 32], int slot) {
    join_lanes<(TPR < 32 ? TPR : 32)>(s);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[slot][warp] = s;
        __syncthreads();
        const int w0 = warp / W * W;
        s = red[slot][w0];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const Soft o = red[slot][w0 + w];
            s.join(o.m, o.z, o.t);
        }
    }
}

// part[block] = the block's sum of t_i (its rows in order, its groups in order); a single
// block writes the loss itself.
__device__ __forceinline__ void finish_block(const LossArgs &a, const LossScales &c,
                                             double total, bool lead, double *sums) {
    __syncthreads();
    if (threadIdx.x < kThreads) sums[threadIdx.x] = lead ? total : 0.0;
    __syncthreads();
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int w = threadIdx.x; w < kThreads; w += 32) s += sums[w];
        s = warp_sum_d(s);
        if (threadIdx.x == 0) {
            if (gridDim.x == 1)
                *a.loss = static_cast<float>(s * a.coef * a.K / c.n);
            else
                a.part[blockIdx.x] = s;
        }
    }
}

template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(kThreads)
    balance_loss_kernel(const T *S, T *dS, const LossArgs a) {
    __shared__ Soft red[2][kThreads / 32];
    __shared__ double sums[kThreads];
    pdl_wait();
    pdl_trigger();
    constexpr int G = kThreads / TPR;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const LossScales c(a);
    double total = 0.0;
    int slot = 0;
    Raw<T, V> x[NV];
    bool keep = false;
    // padding rows are read like the others (their values are not used)
    auto fetch = [&](int64_t i) {
        keep = i < a.N && row_selects(a, i);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
            if (i < a.N && j < a.K) x[n].load(S + i * a.K + j);
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    int64_t i0 = static_cast<int64_t>(blockIdx.x) * G;
    if (i0 < a.N) fetch(i0 + grp);
    for (; i0 < a.N; i0 += step) {
        const int64_t i = i0 + grp;
        const bool on = keep;
        float e[NV][V];
        Soft s{-INFINITY, 0.f, 0.f};
        float mine = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const bool in = on && (n * TPR + t) * V < a.K;
            x[n].get(e[n]);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                e[n][k] = in ? a.scale * e[n][k] : -INFINITY;
                nan |= e[n][k] != e[n][k];
                mine = fmaxf(mine, e[n][k]);
            }
        }
        if (nan) mine = NAN;
        if (i0 + step < a.N) fetch(i0 + step + grp);
        float f[NV][V];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
#pragma unroll
            for (int k = 0; k < V; ++k) f[n][k] = 0.f;
            if (j < a.K) {
                int32_t q[V];
                if (V % 4 == 0 && a.cvec) {
#pragma unroll
                    for (int k = 0; k < V; k += 4) {
                        const int4 u = *reinterpret_cast<const int4 *>(a.counts + j + k);
                        q[k] = u.x;
                        if constexpr (V > 1) {
                            q[k + 1] = u.y;
                            q[k + 2] = u.z;
                            q[k + 3] = u.w;
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < V; ++k) q[k] = a.counts[j + k];
                }
#pragma unroll
                for (int k = 0; k < V; ++k) f[n][k] = static_cast<float>(q[k]) * c.unit;
            }
            if (mine != -INFINITY) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    e[n][k] = __expf(e[n][k] - mine);
                    s.z += e[n][k];
                    s.t += e[n][k] * f[n][k];
                }
            }
        }
        s.m = mine;
        join_group<TPR>(s, red, slot);
        slot ^= 1;
        const bool none = s.m == -INFINITY;
        const float inv = none ? 0.f : 1.f / s.z;
        const float ti = s.t * inv;
        if (t == 0 && on) total += ti;
        if (dS != nullptr && i < a.N) {
            const float own = none || mine == -INFINITY ? 0.f : __expf(mine - s.m) * inv;
            const float gp = c.gc * own;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int j = (n * TPR + t) * V;
                if (j < a.K) {
                    float v[V];
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        v[k] = own == 0.f ? 0.f : gp * e[n][k] * (f[n][k] - ti);
                    Raw<T, V>::put(dS + i * a.K + j, v);
                }
            }
        }
    }
    finish_block(a, c, total, t == 0, sums);
}

// Rows longer than a block's registers: one block a row, read twice.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    balance_long_kernel(const T *S, T *dS, const LossArgs a) {
    __shared__ Soft red[2][kThreads / 32];
    __shared__ double sums[kThreads];
    pdl_wait();
    pdl_trigger();
    const LossScales c(a);
    double total = 0.0;
    int slot = 0;
    for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
        const T *s = S + i * a.K;
        if (!row_selects(a, i)) {
            if (dS)
                for (int64_t j = threadIdx.x; j < a.K; j += kThreads)
                    head_store(dS + i * a.K + j, 0.f);
            continue;
        }
        Soft r{-INFINITY, 0.f, 0.f};
        for (int64_t j = threadIdx.x; j < a.K; j += kThreads) {
            const float v = a.scale * head_load(s + j);
            if (v != -INFINITY) r.join(v, 1.f, static_cast<float>(a.counts[j]) * c.unit);
        }
        join_group<kThreads>(r, red, slot);
        slot ^= 1;
        const bool none = r.m == -INFINITY;
        const float inv = none ? 0.f : 1.f / r.z;
        const float ti = r.t * inv;
        if (threadIdx.x == 0) total += ti;
        if (dS)
            for (int64_t j = threadIdx.x; j < a.K; j += kThreads) {
                const float p = none ? 0.f : __expf(a.scale * head_load(s + j) - r.m) * inv;
                head_store(dS + i * a.K + j,
                           c.gc * p * (static_cast<float>(a.counts[j]) * c.unit - ti));
            }
    }
    finish_block(a, c, total, threadIdx.x == 0, sums);
}

// loss = (coef K / n) sum of the parts, in a fixed order.
__global__ void balance_join_kernel(const double *__restrict__ part, int parts, int K,
                                    const int32_t *__restrict__ rows, float coef,
                                    float *__restrict__ loss) {
    __shared__ double warps[kThreads / 32];
    pdl_wait();
    pdl_trigger();
    double s = 0.0;
    for (int p = threadIdx.x; p < parts; p += kThreads) s += part[p];
    s = warp_sum_d(s);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) s += warps[w];
        *loss = static_cast<float>(s * coef * K / (*rows > 0 ? *rows : 1));
    }
}

template <typename T, int V, int NV, int TPR>
cudaError_t loss_cfg(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    const int64_t g = ceil_div(a.N, kThreads / TPR);
    *grid = static_cast<int>(g < b.parts ? g : b.parts);
    return launch_pdl(balance_loss_kernel<T, V, NV, TPR>, dim3(*grid), dim3(kThreads), 0, st,
                      static_cast<const T *>(b.S), static_cast<T *>(b.dS), a);
}

// About 16 columns a thread; from 32 a thread in a block on, rows are read twice.
template <typename T, int V>
cudaError_t loss_v(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    constexpr int C16 = 16 / V;
    if (a.K <= 8 * V) return loss_cfg<T, V, 1, 8>(b, a, grid, st);
    if (a.K <= 16 * V) return loss_cfg<T, V, 1, 16>(b, a, grid, st);
    if (a.K <= 32 * V) return loss_cfg<T, V, 1, 32>(b, a, grid, st);
    if (a.K <= 32 * 16) return loss_cfg<T, V, C16, 32>(b, a, grid, st);
    if (a.K <= 32 * 32) return loss_cfg<T, V, 2 * C16, 32>(b, a, grid, st);
    if (a.K <= kThreads * 16) return loss_cfg<T, V, C16, kThreads>(b, a, grid, st);
    if (a.K <= kThreads * 32) return loss_cfg<T, V, 2 * C16, kThreads>(b, a, grid, st);
    *grid = static_cast<int>(a.N < b.parts ? a.N : b.parts);
    return launch_pdl(balance_long_kernel<T>, dim3(*grid), dim3(kThreads), 0, st,
                      static_cast<const T *>(b.S), static_cast<T *>(b.dS), a);
}

template <typename T>
cudaError_t loss_t(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    const bool vec = a.K % kVec<T> == 0 && aligned(b.S, 16) && aligned(b.dS, 16);
    return vec ? loss_v<T, kVec<T>>(b, a, grid, st) : loss_v<T, 1>(b, a, grid, st);
}

}  // namespace

int64_t balance_parts(int64_t N, int K) {
    (void)K;
    return N < 1 ? 1 : (N < 148 * 8 ? N : 148 * 8);
}

cudaError_t launch_balance_counts(const int32_t *labels, int64_t N, int top, int K,
                                  int32_t *counts, int32_t *rows, cudaStream_t st) {
    const bool local = K <= kSharedCells;
    const size_t smem = local ? sizeof(int32_t) * K : 0;
    cudaError_t e;
    if (local && N * top <= kOneBlockLabels) {
        e = launch_pdl(balance_counts_kernel<true>, dim3(1), dim3(1024), smem, st, labels, N, top,
                       K, counts, rows);
        if (e == cudaSuccess) note_launch();
        return e;
    }
    const int64_t z = ceil_div(K, 1024);
    e = launch_pdl(balance_zero_kernel, dim3(static_cast<unsigned>(z < 148 ? z : 148)), dim3(1024),
                   0, st, counts, K, rows);
    if (e != cudaSuccess) return e;
    note_launch();
    if (N == 0) return e;
    const int64_t g = ceil_div(N, 1024);
    e = launch_pdl(balance_counts_kernel<false>, dim3(static_cast<unsigned>(g < 148 ? g : 148)),
                   dim3(1024), smem, st, labels, N, top, K, counts, rows);
    if (e == cudaSuccess) note_launch();
    return e;
}

cudaError_t launch_balance_loss(const BalanceArgs &b, cudaStream_t st) {
    LossArgs a{};
    a.N = b.N;
    a.K = b.K;
    a.top = b.top;
    a.labels = b.labels;
    a.counts = b.counts;
    a.rows = b.rows;
    a.scale = b.scale;
    a.coef = b.coef;
    a.cvec = aligned(b.counts, 16);
    a.loss = b.loss;
    a.part = b.part;
    int grid = 0;
    cudaError_t e = cudaSuccess;
    if (b.N > 0) {
        e = b.dtype == FK_F32 ? loss_t<float>(b, a, &grid, st) : loss_t<uint16_t>(b, a, &grid, st);
        if (e != cudaSuccess) return e;
        note_launch();
    }
    if (grid == 1) return e;  // a single block wrote the loss
    e = launch_pdl(balance_join_kernel, dim3(1), dim3(kThreads), 0, st,
                   static_cast<const double *>(b.part), grid, b.K, b.rows, b.coef, b.loss);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace fk
