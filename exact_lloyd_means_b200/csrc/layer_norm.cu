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
#include "ptx_sm100.cuh"

namespace fk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxStages = 8;   // slots of the backward pass's ring of rows
constexpr int kRingBytes = 96 << 10;  // its size: two blocks an SM

// Sums of a and b over the TPR threads of a row group; red: a block's scratch, of which `slot`
// picks the half this row uses, so that one barrier a row is enough (every group of the block
// takes part in it).
template <int TPR>
__device__ __forceinline__ void group_sum2(float &a, float &b, float (*red)[kThreads / 32][2],
                                           int slot) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) {
            red[slot][warp][0] = a;
            red[slot][warp][1] = b;
        }
        __syncthreads();
        a = b = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += red[slot][warp / W * W + w][0];
            b += red[slot][warp / W * W + w][1];
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

// Forward, bf16 rows in 16-byte vectors.  At two bytes an element the instructions hold the loop
// above back, and its reads of gamma and beta from L1.  Here a thread has the same columns of
// every row it works on: it keeps their gamma and beta in registers, works on two columns an
// instruction, and brings its vectors of the S rows ahead into shared memory of its own by
// asynchronous copies (nobody else reads them, so they take no barrier).  65536 rows: of 768 35
// us (56 in the loop above), of 4096 174 (360; 6.2 TB/s), of 8192 352 (550).  fp32 rows, with
// half the elements a byte, are no faster so: of 768 71 us against 65, of 1024 89 and 85.
template <typename T, int NV, int TPR, int S>
__global__ void __launch_bounds__(kThreads)
    layer_norm_ahead_kernel(const T *X, int64_t N, int d, const float *__restrict__ gamma,
                            const float *__restrict__ beta, int pvec, float eps, T *Y,
                            float *__restrict__ mean, float *__restrict__ rstd) {
    constexpr int V = kVec<T>, H = V / 2, G = kThreads / TPR;
    __shared__ float red[2][kThreads / 32][2];
    __shared__ uint4 ring[S][NV][kThreads];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * G;
    auto bring = [&](int64_t i, int s) {  // a group of copies for each row, also an empty one
        if (i < N) {
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int j = (n * TPR + t) * V;
                if (j < d) ptx::copy16_async(&ring[s][n][threadIdx.x], X + i * d + j);
            }
        }
        ptx::copies_commit();
    };
#pragma unroll
    for (int s = 0; s < S; ++s) bring(first + grp + s * step, s);
    F2 gm[NV][H], bt[NV][H];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int j = (n * TPR + t) * V;
        float g[V], b[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            g[k] = 1.f;
            b[k] = 0.f;
        }
        if (gamma && j < d) load_params<V>(gamma + j, pvec, g);
        if (beta && j < d) load_params<V>(beta + j, pvec, b);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            gm[n][k] = f2(g[2 * k], g[2 * k + 1]);
            bt[n][k] = f2(b[2 * k], b[2 * k + 1]);
        }
    }
    const float inv = 1.f / static_cast<float>(d);
    int slot = 0, s = 0;
    // every thread of a block takes the same number of turns (the groups meet in the sums)
    for (int64_t i0 = first; i0 < N; i0 += step) {
        const int64_t i = i0 + grp;
        const bool row = i < N;
        ptx::copies_wait<S - 1>();
        F2 h[NV][H];
        F2 a2 = f2(0.f, 0.f);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (row && (n * TPR + t) * V < d) u = ring[s][n][threadIdx.x];
            unpack2(u, h[n]);
#pragma unroll
            for (int k = 0; k < H; ++k) a2 = add2(a2, h[n][k]);
        }
        float a = sum2(a2), unused = 0.f;
        group_sum2<TPR>(a, unused, red, slot);
        slot ^= 1;
        bring(i + S * step, s);  // (the row is in registers)
        if (++s == S) s = 0;
        const float mu = a * inv;
        const F2 off = f2(-mu, -mu);
        F2 q2 = f2(0.f, 0.f);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if ((n * TPR + t) * V < d) {
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    h[n][k] = add2(h[n][k], off);
                    q2 = fma2(h[n][k], h[n][k], q2);
                }
            }
        }
        float q = sum2(q2);
        group_sum2<TPR>(q, unused, red, slot);
        slot ^= 1;
        const float r = 1.f / sqrtf(q * inv + eps);
        if (!row) continue;
        const F2 rr = f2(r, r);
        T *o = Y + i * d + t * V;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if ((n * TPR + t) * V < d) {
                F2 v[H];
#pragma unroll
                for (int k = 0; k < H; ++k) v[k] = fma2(mul2(h[n][k], rr), gm[n][k], bt[n][k]);
                *reinterpret_cast<uint4 *>(o + n * TPR * V) = pack2(v);
            }
        }
        if (t == 0) {
            if (mean) mean[i] = mu;
            if (rstd) rstd[i] = r;
        }
    }
}

// The block's column sums, joined over its row groups in shared memory.
template <int V, int NV, int TPR>
__device__ __forceinline__ void write_part(const float (&sg)[NV][V], const float (&sb)[NV][V],
                                           int d, float *sums, float *part) {
    constexpr int G = kThreads / TPR;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
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

// Backward, rows in 16-byte vectors: dX row by row, and the block's column sums of its rows in
// registers; the groups of a block are joined in shared memory, the blocks by
// layer_norm_join_kernel.  The G rows a block takes at once lie one behind the other, so one
// bulk copy a tensor brings them into a ring of `stages` slots, several turns ahead: with the
// sums in registers there is no room there for enough loads in flight.
template <typename T, int NV, int TPR>
__global__ void __launch_bounds__(kThreads)
    layer_norm_backward_ring_kernel(const T *dY, const T *__restrict__ X, int64_t N, int d,
                                    const float *__restrict__ gamma, int pvec,
                                    const float *__restrict__ mean,
                                    const float *__restrict__ rstd, T *dX,
                                    float *__restrict__ part, int stages,
                                    uint32_t *__restrict__ err, uint64_t wait_ns) {
    constexpr int V = kVec<T>, H = V / 2, G = kThreads / TPR;
    __shared__ float red[2][kThreads / 32][2];
    __shared__ float sums[G > 1 ? kThreads * 2 : 2];
    __shared__ uint64_t full[kMaxStages];
    __shared__ uint32_t abort_flag;
    extern __shared__ __align__(128) uint8_t ring[];
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
        abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const uint32_t row_bytes = static_cast<uint32_t>(d * sizeof(T));
    const uint32_t half = G * row_bytes;  // a slot: G rows of X, then G rows of dY
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * G;
    auto bring = [&](int64_t i0, int s) {
        if (i0 >= N) return;
        const uint32_t rows = static_cast<uint32_t>(N - i0 < G ? N - i0 : G);
        ptx::mbar_arrive_expect_tx(&full[s], 2 * rows * row_bytes);
        uint8_t *p = ring + static_cast<size_t>(s) * 2 * half;
        ptx::bulk_load(p, X + i0 * d, rows * row_bytes, &full[s]);
        ptx::bulk_load(p + half, dY + i0 * d, rows * row_bytes, &full[s]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < stages; ++s) bring(first + s * step, s);
    F2 sg[NV][H], sb[NV][H], gm[NV][H];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int j = (n * TPR + t) * V;
        float g[V];
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = j < d ? 1.f : 0.f;
        if (gamma && j < d) load_params<V>(gamma + j, pvec, g);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            sg[n][k] = sb[n][k] = f2(0.f, 0.f);
            gm[n][k] = f2(g[2 * k], g[2 * k + 1]);
        }
    }
    const float inv = 1.f / static_cast<float>(d);
    float mu1 = 0.f, r1 = 0.f;  // of the next row
    if (first + grp < N) {
        mu1 = mean[first + grp];
        r1 = rstd[first + grp];
    }
    int slot = 0, s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t i0 = first; i0 < N; i0 += step) {
        const int64_t i = i0 + grp;
        const bool row = i < N;
        const float mu = mu1, r = r1;
        if (i + step < N) {
            mu1 = mean[i + step];
            r1 = rstd[i + step];
        }
        // a wait that runs out is recorded, and the pass runs to its end without its data; nothing
        // more is brought then, as the slot's last copy may still be on its way
        if (!ptx::mbar_wait(&full[s], phase, &abort_flag, wait_ns)) {
            ok = false;
            *const_cast<volatile uint32_t *>(&abort_flag) = 1u;
            err[0] = kErrTimeout;
        }
        const T *x = reinterpret_cast<const T *>(ring + static_cast<size_t>(s) * 2 * half +
                                                 grp * row_bytes);
        const T *y = reinterpret_cast<const T *>(reinterpret_cast<const uint8_t *>(x) + half);
        F2 h[NV][H], w[NV][H];
        F2 a2 = f2(0.f, 0.f), b2 = a2;
        const F2 rr = f2(r, r), off = f2(-mu, -mu);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = (n * TPR + t) * V;
            F2 yv[H];
            uint4 ux = make_uint4(0u, 0u, 0u, 0u), uy = ux;
            if (row && j < d) {
                ux = *reinterpret_cast<const uint4 *>(x + j);
                uy = *reinterpret_cast<const uint4 *>(y + j);
            }
            unpack2(ux, h[n]);
            unpack2(uy, yv);  // (nothing where there is no column or no row)
#pragma unroll
            for (int k = 0; k < H; ++k) {
                h[n][k] = mul2(add2(h[n][k], off), rr);  // (x r - mu r would cancel)
                w[n][k] = mul2(yv[k], gm[n][k]);
                a2 = add2(a2, w[n][k]);
                b2 = fma2(w[n][k], h[n][k], b2);
                sg[n][k] = fma2(yv[k], h[n][k], sg[n][k]);
                sb[n][k] = add2(sb[n][k], yv[k]);
            }
        }
        float a = sum2(a2), b = sum2(b2);
        group_sum2<TPR>(a, b, red, slot);
        if constexpr (TPR <= 32) __syncthreads();
        slot ^= 1;
        // every thread has the slot's rows in registers now
        if (threadIdx.x == 0 && ok) bring(i0 + stages * step, s);
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
        if (dX != nullptr && row) {
            // (as the formula has it: r w - r mean(w) would round r w first.  Where all w of a
            // row are the same, w - mean(w) is what the mean's sum and its division by d round: 0
            // for d a power of two, a few units of 2^-24 |w| otherwise)
            const float na = -a * inv, nb = -b * inv;
            const F2 na2 = f2(na, na), nb2 = f2(nb, nb);
            T *o = dX + i * d + t * V;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                if ((n * TPR + t) * V < d) {
                    F2 v[H];
#pragma unroll
                    for (int k = 0; k < H; ++k)
                        v[k] = mul2(rr, fma2(nb2, h[n][k], add2(w[n][k], na2)));
                    *reinterpret_cast<uint4 *>(o + n * TPR * V) = pack2(v);
                }
            }
        }
    }
    if (part != nullptr) {
        float g[NV][V], b[NV][V];
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int k = 0; k < H; ++k) {
                split(sg[n][k], g[n][2 * k], g[n][2 * k + 1]);
                split(sb[n][k], b[n][2 * k], b[n][2 * k + 1]);
            }
        write_part<V, NV, TPR>(g, b, d, sums, part);
    }
    if (abort_flag) {  // give copies already in flight a moment to land (bounded)
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 200000ull) {
        }
    }
}

// The same for rows that are not in 16-byte vectors, element by element; the next row is
// loaded before this row's sums are formed.
template <typename T, int NV, int TPR>
__global__ void __launch_bounds__(kThreads)
    layer_norm_backward_kernel(const T *dY, const T *__restrict__ X, int64_t N, int d,
                               const float *__restrict__ gamma, const float *__restrict__ mean,
                               const float *__restrict__ rstd, T *dX, float *__restrict__ part) {
    constexpr int G = kThreads / TPR;
    __shared__ float red[2][kThreads / 32][2];
    __shared__ float sums[G > 1 ? kThreads * 2 : 2];
    pdl_wait();
    pdl_trigger();
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const float inv = 1.f / static_cast<float>(d);
    float sg[NV][1], sb[NV][1];
#pragma unroll
    for (int n = 0; n < NV; ++n) sg[n][0] = sb[n][0] = 0.f;
    T x[NV], y[NV];
    float mu = 0.f, r = 0.f;
    auto fetch = [&](int64_t i) {
        if (i < N) {
            mu = mean[i];
            r = rstd[i];
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = n * TPR + t;
            const bool in = i < N && j < d;
            x[n] = in ? X[i * d + j] : T(0);
            y[n] = in ? dY[i * d + j] : T(0);
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    int64_t i0 = static_cast<int64_t>(blockIdx.x) * G;
    if (i0 < N) fetch(i0 + grp);
    int slot = 0;
    for (; i0 < N; i0 += step) {
        const int64_t i = i0 + grp;
        float h[NV], w[NV];
        float a = 0.f, b = 0.f;
        const float rr = r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = n * TPR + t;
            const bool in = j < d && i < N;
            const float yv = head_load(&y[n]);
            h[n] = in ? (head_load(&x[n]) - mu) * r : 0.f;
            w[n] = in && gamma ? yv * gamma[j] : yv;
            a += w[n];
            b += w[n] * h[n];
            sg[n][0] += yv * h[n];
            sb[n][0] += yv;
        }
        if (i0 + step < N) fetch(i0 + step + grp);
        group_sum2<TPR>(a, b, red, slot);
        slot ^= 1;
        if (dX != nullptr && i < N) {
            const float ma = a * inv, mb = b * inv;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int j = n * TPR + t;
                if (j < d) head_store(dX + i * d + j, rr * (__fsub_rn(w[n], ma) - mb * h[n]));
            }
        }
    }
    if (part != nullptr) write_part<1, NV, TPR>(sg, sb, d, sums, part);
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
// dbeta's), 32 runs of parts side by side.
__global__ void __launch_bounds__(1024)
    layer_norm_join_kernel(const float *__restrict__ part, int parts, int64_t d,
                           float *__restrict__ dgamma, float *__restrict__ dbeta) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + x;
    float s = 0.f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int p = y; p < parts; p += 32) s += part[static_cast<int64_t>(p) * 2 * d + c];
    }
    red[y][x] = s;
    __syncthreads();
    // warp y sums the runs of column y
    s = warp_sum_f(red[x][y]);
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 32 + y;
    if (x == 0 && o < 2 * d) {
        float *out = o < d ? dgamma : dbeta;
        if (out) out[o < d ? o : o - d] = s;
    }
}

int block_grid(int64_t rows, int groups, int per_sm) {
    const int64_t g = ceil_div(rows, groups),
                  cap = static_cast<int64_t>(device_sm_count()) * per_sm;
    return static_cast<int>(g < cap ? g : cap);
}

// Blocks of the backward pass, and so parts of the column sums: at most two an SM.
constexpr int64_t kMaxParts = 148 * 2;

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

// (32 KB a block for the rows ahead, four blocks an SM)
template <typename T, int NV, int TPR>
cudaError_t forward_ahead(const LayerNormArgs &a, cudaStream_t st) {
    const int pvec = aligned(a.gamma, 16) && aligned(a.beta, 16);
    const cudaError_t e = launch_pdl(
        layer_norm_ahead_kernel<T, NV, TPR, 8 / NV>, dim3(block_grid(a.N, kThreads / TPR, 4)),
        dim3(kThreads), 0, st, static_cast<const T *>(a.X), a.N, a.d, a.gamma, a.beta, pvec, a.eps,
        static_cast<T *>(a.Y), a.mean, a.rstd);
    if (e == cudaSuccess) note_launch();
    return e;
}

// bf16 rows in vectors: up to 32 columns a thread and as few threads a row as that allows (16
// columns a thread and twice the threads: 57 us at 768 columns for 34, 56 at 1024 for 45).
// Other rows: a warp a row up to 16 vectors a lane, a block a row up to 16 vectors a thread (a
// block a row of 1024 or 2048 fp32 columns too: 132 us for 84 and 207 for 168, 65,536 rows).
template <typename T, int V>
cudaError_t forward_v(const LayerNormArgs &a, cudaStream_t st) {
    const int64_t nv = ceil_div(a.d, V);
    if constexpr (sizeof(T) == 2 && V > 1) {
        if (nv <= 32) return forward_ahead<T, 1, 32>(a, st);
        if (nv <= 64) return forward_ahead<T, 2, 32>(a, st);
        if (nv <= 96) return forward_ahead<T, 3, 32>(a, st);
        if (nv <= 128) return forward_ahead<T, 4, 32>(a, st);
        if (nv <= 256) return forward_ahead<T, 4, 64>(a, st);
        if (nv <= 512) return forward_ahead<T, 4, 128>(a, st);
        if (nv <= 1024) return forward_ahead<T, 4, kThreads>(a, st);
    } else {
        if (nv <= 32) return forward_cfg<T, V, 1, 32>(a, st);
        if (nv <= 64) return forward_cfg<T, V, 2, 32>(a, st);
        if (nv <= 128) return forward_cfg<T, V, 4, 32>(a, st);
        if (nv <= 256) return forward_cfg<T, V, 8, 32>(a, st);
        if (nv <= 512) return forward_cfg<T, V, 16, 32>(a, st);
        if (nv <= 1024) return forward_cfg<T, V, 4, kThreads>(a, st);
    }
    if (nv <= 2048) return forward_cfg<T, V, 8, kThreads>(a, st);
    if (nv <= 4096) return forward_cfg<T, V, 16, kThreads>(a, st);
    const cudaError_t e = launch_pdl(
        layer_norm_long_kernel<T>, dim3(block_grid(a.N, 1, 8)), dim3(kThreads), 0, st,
        static_cast<const T *>(a.X), a.N, a.d, a.gamma, a.beta, a.eps, static_cast<T *>(a.Y),
        a.mean, a.rstd);
    if (e == cudaSuccess) note_launch();
    return e;
}

int backward_grid(const LayerNormArgs &a, int groups) {
    const int64_t g = ceil_div(a.N, groups);
    return static_cast<int>(g < a.parts ? g : a.parts);
}

template <typename T, int NV, int TPR>
cudaError_t backward_ring(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    auto kernel = layer_norm_backward_ring_kernel<T, NV, TPR>;
    const int slot = 2 * (kThreads / TPR) * a.d * static_cast<int>(sizeof(T));
    int stages = kRingBytes / slot;
    if (stages < 2) stages = 2;
    if (stages > kMaxStages) stages = kMaxStages;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = smem_opt_in(kernel, 160 << 10, smem_set);
    if (e != cudaSuccess) return e;
    *parts = backward_grid(a, kThreads / TPR);
    e = launch_pdl(kernel, dim3(*parts), dim3(kThreads), static_cast<size_t>(stages) * slot, st,
                   static_cast<const T *>(a.dY), static_cast<const T *>(a.X), a.N, a.d, a.gamma,
                   static_cast<int>(aligned(a.gamma, 16)), static_cast<const float *>(a.mean),
                   static_cast<const float *>(a.rstd), static_cast<T *>(a.Y),
                   a.dgamma || a.dbeta ? a.part : nullptr, stages, a.err, kDefaultWaitNs);
    if (e == cudaSuccess) note_launch();
    return e;
}

template <typename T, int NV, int TPR>
cudaError_t backward_elements(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    *parts = backward_grid(a, kThreads / TPR);
    const cudaError_t e = launch_pdl(
        layer_norm_backward_kernel<T, NV, TPR>, dim3(*parts), dim3(kThreads), 0, st,
        static_cast<const T *>(a.dY), static_cast<const T *>(a.X), a.N, a.d, a.gamma,
        static_cast<const float *>(a.mean), static_cast<const float *>(a.rstd),
        static_cast<T *>(a.Y), a.dgamma || a.dbeta ? a.part : nullptr);
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

// Up to 16 columns a thread (their sums and values take four registers each), and as few
// threads a row as that allows.  65,536 rows with twice the threads: of 512 bf16 columns 49 us
// for 40, of 768 102 for 61, of 2048 175 for 128; of 512 fp32 columns 67 for 68, of 768 101 for
// 98; of 1024 121 for 133 and of 2048 235 for 259, so there they are used.
template <typename T>
cudaError_t backward_vectors(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    constexpr int V = kVec<T>, C16 = 16 / V;
    if (a.d <= 8 * V) return backward_ring<T, 1, 8>(a, st, parts);
    if (a.d <= 32 * V) return backward_ring<T, 1, 32>(a, st, parts);
    if (a.d <= 32 * 16) return backward_ring<T, C16, 32>(a, st, parts);
    if constexpr (C16 == 4) {
        if (a.d <= 64 * 12) return backward_ring<T, 3, 64>(a, st, parts);
        if (a.d <= 128 * 8) return backward_ring<T, 2, 128>(a, st, parts);
        if (a.d <= 256 * 8) return backward_ring<T, 2, 256>(a, st, parts);
    } else {
        if (a.d <= 64 * 16) return backward_ring<T, C16, 64>(a, st, parts);
        if (a.d <= 128 * 16) return backward_ring<T, C16, 128>(a, st, parts);
    }
    if (a.d <= 256 * 16) return backward_ring<T, C16, 256>(a, st, parts);
    if (a.d <= 256 * 32) return backward_ring<T, 2 * C16, 256>(a, st, parts);
    return backward_long<T>(a, st, parts);
}

template <typename T>
cudaError_t backward_scalars(const LayerNormArgs &a, cudaStream_t st, int *parts) {
    if (a.d <= 8) return backward_elements<T, 1, 8>(a, st, parts);
    if (a.d <= 32) return backward_elements<T, 1, 32>(a, st, parts);
    if (a.d <= 32 * 4) return backward_elements<T, 4, 32>(a, st, parts);
    if (a.d <= 32 * 8) return backward_elements<T, 8, 32>(a, st, parts);
    if (a.d <= 32 * 16) return backward_elements<T, 16, 32>(a, st, parts);
    if (a.d <= 64 * 16) return backward_elements<T, 16, 64>(a, st, parts);
    if (a.d <= 128 * 16) return backward_elements<T, 16, 128>(a, st, parts);
    if (a.d <= 256 * 16) return backward_elements<T, 16, 256>(a, st, parts);
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
        e = rows_in_vectors<T>(a) ? backward_vectors<T>(a, st, &parts)
                                  : backward_scalars<T>(a, st, &parts);
    if (e != cudaSuccess || (!a.dgamma && !a.dbeta)) return e;
    e = launch_pdl(layer_norm_join_kernel,
                   dim3(static_cast<unsigned>(ceil_div(2 * static_cast<int64_t>(a.d), 32))),
                   dim3(1024), 0, st, static_cast<const float *>(a.part), parts,
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
