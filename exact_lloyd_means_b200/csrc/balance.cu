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

// Softmax sums of some columns: the maximum score m, z = sum exp(scale (s - m)) and t = that
// sum weighted by f (the exponentials as 2^(scale log2(e) (s - m)); the difference comes
// first, so that scores at the type's lowest value do not overflow).  m = -inf (with zero
// sums) where there is nothing but -inf; a NaN anywhere makes all NaN.
struct Soft {
    float m, z, t;
};

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// What to subtract from scores below the maximum m (nothing but -inf: anything finite).
__device__ __forceinline__ float soft_base(float m) { return m == -INFINITY ? 0.f : m; }

template <int W>
__device__ __forceinline__ float lanes_max(float m) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
template <int W>
__device__ __forceinline__ void lanes_sum(float &z, float &t) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
}

// The group's sums from those of its threads: s.m is the maximum of this warp's part of the
// group already, s.z and s.t this thread's sums against it.  For a group of several warps,
// one barrier; lane l then holds warp l's sums.
template <int TPR>
__device__ __forceinline__ Soft join_group(Soft s, float scale2, Soft (*red)[kThreads / 32], int slot) {
    lanes_sum<(TPR < 32 ? TPR : 32)>(s.z, s.t);
    if constexpr (TPR > 32) {
        static_assert(TPR == kThreads, "one row a block");
        constexpr int W = kThreads / 32;
        if ((threadIdx.x & 31) == 0) red[slot][threadIdx.x >> 5] = s;
        __syncthreads();
        s = red[slot][threadIdx.x & (W - 1)];
        const float m = lanes_max<W>(s.m);
        const float c = exp2_fast(scale2 * (s.m - soft_base(m)));
        s.z *= c;
        s.t *= c;
        lanes_sum<W>(s.z, s.t);
        s.m = m;
    }
    return s;
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

// f of the thread's columns j .. j + V - 1
template <int V>
__device__ __forceinline__ void load_shares(const LossArgs &a, const LossScales &c, int j,
                                            float (&f)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = 0.f;
    if (j >= a.K) return;
    int32_t q[V];
    bool done = false;
    if constexpr (V % 4 == 0) {
        if (a.cvec) {
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                const int4 u = *reinterpret_cast<const int4 *>(a.counts + j + k);
                q[k] = u.x;
                q[k + 1] = u.y;
                q[k + 2] = u.z;
                q[k + 3] = u.w;
            }
            done = true;
        }
    }
    if (!done) {
#pragma unroll
        for (int k = 0; k < V; ++k) q[k] = a.counts[j + k];
    }
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = static_cast<float>(q[k]) * c.unit;
}

// Up to 16 columns a thread, f stays in registers for all rows of the block.
template <typename T, int V, int NV, int TPR>
__global__ void __launch_bounds__(kThreads, NV * V <= 8 ? 4 : (NV * V <= 16 ? 3 : 2))
    balance_loss_kernel(const T *S, T *dS, const LossArgs a) {
    __shared__ Soft red[2][kThreads / 32];
    __shared__ double sums[kThreads];
    pdl_wait();
    pdl_trigger();
    constexpr int G = kThreads / TPR;
    constexpr bool KEEP_F = NV * V <= 16;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const LossScales c(a);
    const float scale2 = a.scale * 1.44269504f;
    double total = 0.0;
    int slot = 0;
    Raw<T, V> x[NV];
    float f[KEEP_F ? NV : 1][V];
    if constexpr (KEEP_F) {
#pragma unroll
        for (int n = 0; n < NV; ++n) load_shares<V>(a, c, (n * TPR + t) * V, f[n]);
    }
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
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const bool in = on && (n * TPR + t) * V < a.K;
            x[n].get(e[n]);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                e[n][k] = in ? e[n][k] : -INFINITY;
                m = max_nan(m, e[n][k]);
            }
        }
        if (i0 + step < a.N) fetch(i0 + step + grp);
        m = lanes_max<(TPR < 32 ? TPR : 32)>(m);
        Soft s{m, 0.f, 0.f};
        const float base = soft_base(m);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            float g[V];
            if constexpr (!KEEP_F) load_shares<V>(a, c, (n * TPR + t) * V, g);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                e[n][k] = exp2_fast(scale2 * (e[n][k] - base));
                s.z += e[n][k];
                s.t += e[n][k] * (KEEP_F ? f[KEEP_F ? n : 0][k] : g[k]);
            }
        }
        s = join_group<TPR>(s, scale2, red, slot);
        slot ^= 1;
        const float inv = s.m == -INFINITY ? 0.f : 1.f / s.z;
        const float ti = s.t * inv;
        if (t == 0 && on) total += ti;
        if (dS != nullptr && i < a.N) {
            // this warp's exponentials against the group's maximum, over the sum
            const float gp = TPR > 32 ? c.gc * exp2_fast(scale2 * (m - soft_base(s.m))) * inv : c.gc * inv;
            const float gt = -ti * gp;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int j = (n * TPR + t) * V;
                if (j < a.K) {
                    float v[V], g[V];
                    if constexpr (!KEEP_F) load_shares<V>(a, c, j, g);
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        v[k] = e[n][k] * ((KEEP_F ? f[KEEP_F ? n : 0][k] : g[k]) * gp + gt);
                    Raw<T, V>::put(dS + i * a.K + j, v);
                }
            }
        }
    }
    finish_block(a, c, total, t == 0, sums);
}

// Rows longer than a block's registers: one block a row, read once for the maximum, once for
// the sums and once for the gradient.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    balance_long_kernel(const T *S, T *dS, const LossArgs a) {
    __shared__ Soft red[2][kThreads / 32];
    __shared__ double sums[kThreads];
    pdl_wait();
    pdl_trigger();
    const LossScales c(a);
    const float scale2 = a.scale * 1.44269504f;
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
        for (int64_t j = threadIdx.x; j < a.K; j += kThreads)
            r.m = max_nan(r.m, head_load(s + j));
        r.m = lanes_max<32>(r.m);
        for (int64_t j = threadIdx.x; j < a.K; j += kThreads) {
            const float e = exp2_fast(scale2 * (head_load(s + j) - soft_base(r.m)));
            r.z += e;
            r.t += e * (static_cast<float>(a.counts[j]) * c.unit);
        }
        r = join_group<kThreads>(r, scale2, red, slot);
        slot ^= 1;
        const float inv = r.m == -INFINITY ? 0.f : 1.f / r.z;
        const float ti = r.t * inv;
        if (threadIdx.x == 0) total += ti;
        if (dS)
            for (int64_t j = threadIdx.x; j < a.K; j += kThreads) {
                const float p = exp2_fast(scale2 * (head_load(s + j) - soft_base(r.m))) * inv;
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
