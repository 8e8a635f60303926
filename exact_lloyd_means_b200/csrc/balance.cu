// balance.cu -- the balance loss over K cells (or experts): counts of a selection, and the
// loss of the scores with its gradient.
//
// labels[i][t] is the t-th cell selected by row i; an entry outside [0, K) selects nothing,
// and a row without any selection is padding.  counts_k = #{(i, t): labels[i][t] = k}, n =
// rows that are not padding, f_k = counts_k / (n top), p_i = softmax(scale s_i):
//   loss = coef K sum_k f_k (1/n) sum_i p_ik = (coef K / n) sum_i t_i, t_i = sum_k f_k p_ik,
//   dS_ij = (coef scale K / n) p_ij (f_j - t_i)     (f is a constant, as the counts are).
// The second form of the loss needs only the counts before the pass over S, so loss and
// gradient take one pass.  A row whose scores are all -inf has p = 0.
#include "head.cuh"

namespace fk {
namespace {

__global__ void balance_counts_kernel(const int32_t *__restrict__ labels, int64_t N, int top,
                                      int K, int32_t *counts, int32_t *rows) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < N;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        bool any = false;
        for (int t = 0; t < top; ++t) {
            const int32_t l = labels[i * top + t];
            if (l >= 0 && l < K) {
                any = true;
                atomicAdd(counts + l, 1);
            }
        }
        if (any) atomicAdd(rows, 1);
    }
}

__device__ __forceinline__ bool row_selects(const int32_t *labels, int64_t i, int top, int K,
                                            int lane) {
    bool any = false;
    for (int t = lane; t < top; t += 32) {
        const int32_t l = labels[i * top + t];
        any |= l >= 0 && l < K;
    }
    return __any_sync(0xffffffffu, any);
}

// One warp per row; part[warp] = the warp's sum of t_i.
template <typename T>
__global__ void balance_loss_kernel(const T *S, int64_t N, int K,
                                    const int32_t *__restrict__ labels, int top,
                                    const int32_t *__restrict__ counts,
                                    const int32_t *__restrict__ rows, float scale, float coef,
                                    T *dS, double *__restrict__ part) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    const float n = static_cast<float>(*rows > 0 ? *rows : 1);
    const float unit = 1.f / (n * top);
    const float gc = coef * scale * static_cast<float>(K) / n;
    double total = 0.0;
    for (int64_t i = warp; i < N; i += nwarps) {
        const T *s = S + i * K;
        if (!row_selects(labels, i, top, K, lane)) {
            if (dS)
                for (int j = lane; j < K; j += 32) head_store(dS + i * K + j, 0.f);
            continue;
        }
        float mx = -INFINITY;
        bool nan = false;
        for (int j = lane; j < K; j += 32) {
            const float v = scale * head_load(s + j);
            nan |= v != v;
            mx = fmaxf(mx, v);
        }
        mx = warp_max_f(mx);
        if (__any_sync(0xffffffffu, nan)) mx = NAN;
        const bool none = mx == -INFINITY;
        float z = 0.f, t = 0.f;
        for (int j = lane; j < K; j += 32) {
            const float e = none ? 0.f : expf(scale * head_load(s + j) - mx);
            z += e;
            t += e * (counts[j] * unit);
        }
        z = warp_sum_f(z);
        t = warp_sum_f(t);
        const float inv = none ? 0.f : 1.f / z;
        t *= inv;
        total += t;
        if (dS)
            for (int j = lane; j < K; j += 32) {
                const float p = none ? 0.f : expf(scale * head_load(s + j) - mx) * inv;
                head_store(dS + i * K + j, gc * p * (counts[j] * unit - t));
            }
    }
    if (lane == 0) part[warp] = total;
}

// loss = (coef K / n) sum of the parts, in a fixed order.
__global__ void balance_join_kernel(const double *__restrict__ part, int64_t parts, int K,
                                    const int32_t *__restrict__ rows, float coef, float *loss) {
    double s = 0.0;
    for (int64_t p = threadIdx.x; p < parts; p += 32) s += part[p];
    s = warp_sum_d(s);
    if (threadIdx.x == 0)
        *loss = static_cast<float>(s * coef * K / (*rows > 0 ? *rows : 1));
}

}  // namespace

int64_t balance_parts(int64_t N, int K) {
    (void)K;
    const int64_t g = ceil_div(N, 8);
    return 8 * (g < 148 * 8 ? g : 148 * 8);
}

cudaError_t launch_balance_counts(const int32_t *labels, int64_t N, int top, int K,
                                  int32_t *counts, int32_t *rows, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * K, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(rows, 0, sizeof(int32_t), st);
    if (e != cudaSuccess || N == 0) return e;
    const int64_t g = ceil_div(N, 256);
    balance_counts_kernel<<<static_cast<int>(g < 148 * 8 ? g : 148 * 8), 256, 0, st>>>(
        labels, N, top, K, counts, rows);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_balance_loss(const BalanceArgs &a, cudaStream_t st) {
    if (a.N > 0) {
        const int grid = static_cast<int>(a.parts / 8);
        if (a.dtype == FK_F32)
            balance_loss_kernel<float><<<grid, 256, 0, st>>>(
                static_cast<const float *>(a.S), a.N, a.K, a.labels, a.top, a.counts, a.rows,
                a.scale, a.coef, static_cast<float *>(a.dS), a.part);
        else
            balance_loss_kernel<uint16_t><<<grid, 256, 0, st>>>(
                static_cast<const uint16_t *>(a.S), a.N, a.K, a.labels, a.top, a.counts, a.rows,
                a.scale, a.coef, static_cast<uint16_t *>(a.dS), a.part);
        note_launch();
    }
    balance_join_kernel<<<1, 32, 0, st>>>(a.part, a.N > 0 ? a.parts : 0, a.K, a.rows, a.coef,
                                          a.loss);
    note_launch();
    return cudaGetLastError();
}

}  // namespace fk
