// layer_norm.cu -- layer norm over the rows of N x d points, forward and backward.
//
// mean_i = sum_j x_ij / d, rstd_i = 1 / sqrt(sum_j (x_ij - mean_i)^2 / d + eps),
// y = (x - mean) rstd gamma + beta.  With h = (x - mean) rstd and w = dy gamma:
//   dx = rstd (w - mean_j(w) - h mean_j(w h)),  dgamma = sum_i dy h,  dbeta = sum_i dy.
// All statistics and sums are fp32; each output is rounded once.
#include "head.cuh"

namespace fk {
namespace {

template <typename T>
__global__ void layer_norm_kernel(const T *X, int64_t N, int d, const float *__restrict__ gamma,
                                  const float *__restrict__ beta, float eps, T *Y,
                                  float *__restrict__ mean, float *__restrict__ rstd) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t i = warp; i < N; i += nwarps) {
        const T *x = X + i * d;
        float s = 0.f;
        for (int j = lane; j < d; j += 32) s += head_load(x + j);
        const float mu = warp_sum_f(s) / d;
        float q = 0.f;
        for (int j = lane; j < d; j += 32) {
            const float c = head_load(x + j) - mu;
            q += c * c;
        }
        const float r = 1.f / sqrtf(warp_sum_f(q) / d + eps);
        T *y = Y + i * d;
        for (int j = lane; j < d; j += 32) {
            const float h = (head_load(x + j) - mu) * r;
            head_store(y + j, h * (gamma ? gamma[j] : 1.f) + (beta ? beta[j] : 0.f));
        }
        if (lane == 0) {
            if (mean) mean[i] = mu;
            if (rstd) rstd[i] = r;
        }
    }
}

template <typename T>
__global__ void layer_norm_dx_kernel(const T *dY, const T *X, int64_t N, int d,
                                     const float *__restrict__ gamma,
                                     const float *__restrict__ mean,
                                     const float *__restrict__ rstd, T *dX) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
    for (int64_t i = warp; i < N; i += nwarps) {
        const T *x = X + i * d, *g = dY + i * d;
        const float mu = mean[i], r = rstd[i];
        float a = 0.f, b = 0.f;
        for (int j = lane; j < d; j += 32) {
            const float w = head_load(g + j) * (gamma ? gamma[j] : 1.f);
            a += w;
            b += w * ((head_load(x + j) - mu) * r);
        }
        a = warp_sum_f(a) / d;
        b = warp_sum_f(b) / d;
        for (int j = lane; j < d; j += 32) {
            const float w = head_load(g + j) * (gamma ? gamma[j] : 1.f);
            const float h = (head_load(x + j) - mu) * r;
            head_store(dX + i * d + j, r * (w - a - h * b));
        }
    }
}

// Column sums of row group blockIdx.y: one thread per column.
template <typename T>
__global__ void layer_norm_cols_kernel(const T *dY, const T *X, int64_t N, int d, int64_t parts,
                                       const float *__restrict__ mean,
                                       const float *__restrict__ rstd, float *part) {
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= d) return;
    const int64_t p = blockIdx.y;
    float sg = 0.f, sb = 0.f;
    for (int64_t i = N * p / parts; i < N * (p + 1) / parts; ++i) {
        const float g = head_load(dY + i * d + j);
        sg += g * ((head_load(X + i * d + j) - mean[i]) * rstd[i]);
        sb += g;
    }
    part[(p * 2) * d + j] = sg;
    part[(p * 2 + 1) * d + j] = sb;
}

__global__ void layer_norm_join_kernel(const float *part, int64_t parts, int d, float *dgamma,
                                       float *dbeta) {
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= d) return;
    float sg = 0.f, sb = 0.f;
    for (int64_t p = 0; p < parts; ++p) {
        sg += part[(p * 2) * d + j];
        sb += part[(p * 2 + 1) * d + j];
    }
    if (dgamma) dgamma[j] = sg;
    if (dbeta) dbeta[j] = sb;
}

int row_grid(int64_t N) {
    const int64_t g = ceil_div(N, 8), cap = static_cast<int64_t>(device_sm_count()) * 16;
    return static_cast<int>(g < cap ? g : cap);
}

template <typename T>
cudaError_t backward_t(const LayerNormArgs &a, cudaStream_t st) {
    const T *dY = static_cast<const T *>(a.dY), *X = static_cast<const T *>(a.X);
    if (a.dgamma || a.dbeta) {
        const int bx = static_cast<int>(ceil_div(a.d, 128));
        layer_norm_cols_kernel<T><<<dim3(bx, static_cast<unsigned>(a.parts)), 128, 0, st>>>(
            dY, X, a.N, a.d, a.parts, a.mean, a.rstd, a.part);
        layer_norm_join_kernel<<<bx, 128, 0, st>>>(a.part, a.parts, a.d, a.dgamma, a.dbeta);
        note_launch(2);
    }
    if (a.Y && a.N > 0) {
        layer_norm_dx_kernel<T><<<row_grid(a.N), 256, 0, st>>>(dY, X, a.N, a.d, a.gamma, a.mean,
                                                               a.rstd, static_cast<T *>(a.Y));
        note_launch();
    }
    return cudaGetLastError();
}

}  // namespace

int64_t layer_norm_parts(int64_t N, int d) {
    (void)d;
    const int64_t p = ceil_div(N, 64);
    return p < 1 ? 1 : (p > 128 ? 128 : p);
}

cudaError_t launch_layer_norm(const LayerNormArgs &a, cudaStream_t st) {
    if (a.dtype == FK_F32)
        layer_norm_kernel<float><<<row_grid(a.N), 256, 0, st>>>(
            static_cast<const float *>(a.X), a.N, a.d, a.gamma, a.beta, a.eps,
            static_cast<float *>(a.Y), a.mean, a.rstd);
    else
        layer_norm_kernel<uint16_t><<<row_grid(a.N), 256, 0, st>>>(
            static_cast<const uint16_t *>(a.X), a.N, a.d, a.gamma, a.beta, a.eps,
            static_cast<uint16_t *>(a.Y), a.mean, a.rstd);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs &a, cudaStream_t st) {
    return a.dtype == FK_F32 ? backward_t<float>(a, st) : backward_t<uint16_t>(a, st);
}

}  // namespace fk
