// linear.cu -- Y = act(X W^T + b) + R and its gradients, the embedding head's matrix
// products: X N x d, W m x d (rows, like centroids), Y N x m.
#include "head.cuh"

namespace fk {
namespace {

// C[i][j] = sum_k A(i, k) B(j, k) over a 64 x 64 tile; A(i, k) = A[i * ar + k * ak] and
// likewise B, so that the three products of the two passes share one kernel.
template <typename TA, typename TB, typename TC>
__global__ void __launch_bounds__(256)
    tile_kernel(const TA *__restrict__ A, int64_t ar, int64_t ak, const TB *__restrict__ B,
                int64_t br, int64_t bk, int64_t rows, int cols, int64_t depth,
                const float *__restrict__ bias, int act, const TC *R, TC *C, TC *Z) {
    __shared__ float sa[16][65], sb[16][65];
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 64;
    const int c0 = blockIdx.y * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < depth; k0 += 16) {
        for (int t = threadIdx.x; t < 1024; t += 256) {
            const int k = ak == 1 ? t & 15 : t >> 6, i = ak == 1 ? t >> 4 : t & 63;
            const bool ok = r0 + i < rows && k0 + k < depth;
            sa[k][i] = ok ? head_load(A + (r0 + i) * ar + (k0 + k) * ak) : 0.f;
        }
        for (int t = threadIdx.x; t < 1024; t += 256) {
            const int k = bk == 1 ? t & 15 : t >> 6, j = bk == 1 ? t >> 4 : t & 63;
            const bool ok = c0 + j < cols && k0 + k < depth;
            sb[k][j] = ok ? head_load(B + (c0 + j) * br + (k0 + k) * bk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty + 16 * i;
            const int c = c0 + tx + 16 * j;
            if (r >= rows || c >= cols) continue;
            const float z = acc[i][j] + (bias ? bias[c] : 0.f);
            if (Z) head_store(Z + r * cols + c, z);
            float y = act_value(z, act);
            if (R) y += head_load(R + r * cols + c);
            head_store(C + r * cols + c, y);
        }
}

template <typename T>
__global__ void slope_kernel(const T *__restrict__ dY, const T *__restrict__ Z, int64_t n,
                             int act, float *__restrict__ G) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const float g = head_load(dY + i);
        G[i] = act == FK_ACT_NONE ? g : g * act_slope(head_load(Z + i), act);
    }
}

__global__ void col_sum_kernel(const float *__restrict__ G, int64_t N, int m, int64_t parts,
                               float *__restrict__ part) {
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= m) return;
    const int64_t p = blockIdx.y;
    float s = 0.f;
    for (int64_t i = N * p / parts; i < N * (p + 1) / parts; ++i) s += G[i * m + j];
    part[p * m + j] = s;
}

__global__ void col_join_kernel(const float *__restrict__ part, int64_t parts, int m,
                                float *__restrict__ db) {
    const int j = blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= m) return;
    float s = 0.f;
    for (int64_t p = 0; p < parts; ++p) s += part[p * m + j];
    db[j] = s;
}

constexpr int64_t kColParts = 128;

template <typename T>
cudaError_t linear_t(const LinearArgs &a, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(ceil_div(a.N, 64)),
                    static_cast<unsigned>(ceil_div(a.m, 64)));
    tile_kernel<T, T, T><<<grid, 256, 0, st>>>(
        static_cast<const T *>(a.X), a.d, 1, static_cast<const T *>(a.W), a.d, 1, a.N, a.m, a.d,
        a.bias, a.act, static_cast<const T *>(a.R), static_cast<T *>(a.Y),
        static_cast<T *>(a.Z));
    note_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t linear_backward_t(const LinearArgs &a, void *ws, cudaStream_t st) {
    float *G = ws_ptr<float>(ws, 256);
    float *part = G + a.N * a.m;
    const T *X = static_cast<const T *>(a.X), *W = static_cast<const T *>(a.W);
    if (a.N > 0) {
        slope_kernel<T><<<148 * 8, 256, 0, st>>>(static_cast<const T *>(a.dY),
                                                 static_cast<const T *>(a.Zin), a.N * a.m, a.act,
                                                 G);
        note_launch();
    }
    if (a.db) {
        const unsigned bx = static_cast<unsigned>(ceil_div(a.m, 128));
        col_sum_kernel<<<dim3(bx, kColParts), 128, 0, st>>>(G, a.N, a.m, kColParts, part);
        col_join_kernel<<<bx, 128, 0, st>>>(part, kColParts, a.m, a.db);
        note_launch(2);
    }
    if (a.dX && a.N > 0) {
        const dim3 grid(static_cast<unsigned>(ceil_div(a.N, 64)),
                        static_cast<unsigned>(ceil_div(a.d, 64)));
        tile_kernel<float, T, T><<<grid, 256, 0, st>>>(G, a.m, 1, W, 1, a.d, a.N, a.d, a.m,
                                                       nullptr, FK_ACT_NONE, nullptr,
                                                       static_cast<T *>(a.dX), nullptr);
        note_launch();
    }
    if (a.dW) {
        const dim3 grid(static_cast<unsigned>(ceil_div(a.m, 64)),
                        static_cast<unsigned>(ceil_div(a.d, 64)));
        tile_kernel<float, T, T><<<grid, 256, 0, st>>>(G, 1, a.m, X, 1, a.d, a.m, a.d, a.N,
                                                       nullptr, FK_ACT_NONE, nullptr,
                                                       static_cast<T *>(a.dW), nullptr);
        note_launch();
    }
    return cudaGetLastError();
}

}  // namespace

size_t linear_ws_bytes(int64_t, int, int, fk_dtype) { return 256; }
size_t linear_backward_ws_bytes(int64_t N, int, int m, fk_dtype) {
    return 256 + 4 * (static_cast<size_t>(N) * m + static_cast<size_t>(kColParts) * m);
}

cudaError_t launch_linear(const LinearArgs &a, void *, cudaStream_t st) {
    return a.dtype == FK_F32 ? linear_t<float>(a, st) : linear_t<uint16_t>(a, st);
}

cudaError_t launch_linear_backward(const LinearArgs &a, void *ws, cudaStream_t st) {
    return a.dtype == FK_F32 ? linear_backward_t<float>(a, ws, st)
                             : linear_backward_t<uint16_t>(a, ws, st);
}

}  // namespace fk
