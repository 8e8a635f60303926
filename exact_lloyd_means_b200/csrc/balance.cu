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
#include "ptx_sm100.cuh"

namespace fk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxStages = 8;         // slots of the ring of rows
constexpr int kRingBytes = 48 << 10;  // its size: three blocks an SM
// Labels counted by one block in one launch (8192 of 64 cells 3.0 us against 3.3 in two
// launches, 16,384 4.9 against 3.8; but a launch costs the host more than 2).
constexpr int kOneBlockLabels = 1 << 14;
constexpr int kSharedCells = 12256;       // counters kept in shared memory (under 48 KB in all)

// Counts of one run of rows: in shared memory, in `copies` histograms (warp w adds to copy w
// mod copies, so that warps meet less often on a popular cell), which are then added to the
// zeroed totals; with more cells than fit there (copies = 0), in the totals at once, equal
// labels of a warp together.  Integer atomics: the order does not change the sums.
template <bool ONE>
__global__ void __launch_bounds__(1024)
    balance_counts_kernel(const int32_t *__restrict__ labels, int64_t N, int top, int K,
                          int copies, int32_t *__restrict__ counts, int32_t *__restrict__ rows) {
    extern __shared__ int32_t hist[];
    __shared__ int32_t srows;
    pdl_wait();
    pdl_trigger();
    for (int k = threadIdx.x; k < copies * K; k += blockDim.x) hist[k] = 0;
    if (threadIdx.x == 0) srows = 0;
    __syncthreads();
    const int64_t i0 = N * blockIdx.x / gridDim.x, i1 = N * (blockIdx.x + 1) / gridDim.x;
    int32_t *mine = copies > 0 ? hist + (threadIdx.x >> 5) % copies * K : nullptr;
    // every selection, four loads ahead
    const int64_t e = i1 * top, stride = blockDim.x;
    int kept = 0;  // rows with any selection
    for (int64_t j0 = i0 * top; j0 < e; j0 += 4 * stride) {
        int32_t l[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t j = j0 + u * stride + threadIdx.x;
            l[u] = j < e ? labels[j] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const bool in = l[u] >= 0 && l[u] < K;
            kept += top == 1 && in;
            if (copies > 0) {
                if (in) atomicAdd(mine + l[u], 1);
            } else {
                const uint32_t same = __match_any_sync(0xffffffffu, in ? l[u] : -1);
                if (in && (threadIdx.x & 31) == __ffs(same) - 1)
                    atomicAdd(counts + l[u], __popc(same));
            }
        }
    }
    for (int64_t r0 = i0; top > 1 && r0 < i1; r0 += 4 * stride) {
        int32_t l[4];  // most rows show it in their first selection
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = r0 + u * stride + threadIdx.x;
            l[u] = i < i1 ? labels[i * top] : -1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = r0 + u * stride + threadIdx.x;
            bool any = l[u] >= 0 && l[u] < K;
            for (int t = 1; t < top && !any && i < i1; ++t) {
                const int32_t o = labels[i * top + t];
                any = o >= 0 && o < K;
            }
            kept += any;
        }
    }
    kept = __reduce_add_sync(0xffffffffu, kept);
    if ((threadIdx.x & 31) == 0 && kept) atomicAdd(&srows, kept);
    __syncthreads();
    for (int k = threadIdx.x; k < K && copies > 0; k += blockDim.x) {
        int32_t s = 0;
        for (int c = 0; c < copies; ++c) s += hist[c * K + k];
        if (ONE)
            counts[k] = s;
        else if (s)
            atomicAdd(counts + k, s);
    }
    if (threadIdx.x == 0) {
        if (ONE)
            *rows = srows;
        else if (srows)
            atomicAdd(rows, srows);
    }
}

__global__ void balance_zero_kernel(int32_t *__restrict__ counts, int K,
                                    int32_t *__restrict__ rows) {
    pdl_wait();
    pdl_trigger();
    for (int64_t k = blockIdx.x * blockDim.x + threadIdx.x; k < K; k += gridDim.x * blockDim.x)
        counts[k] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *rows = 0;
}

struct LossArgs {
    int64_t N;
    int K, top;
    const int32_t *labels, *counts, *rows;
    float scale, coef;
    float *loss;
    double *part;
};

// n, 1 / (n top) and coef scale K / n (at most 1e38, so that the gradients of rows without
// probabilities are 0 times a number); and the least count.  A share f_k is worked with as its
// distance from the least one, (counts_k - least) / (n top), exact before its one rounding:
// f_j - t_i is then formed from numbers no larger than f_j and t_i, and is 0 where all counts
// are the same.  t_i is the weighted mean of these plus the least share, as p sums to 1.
// Called by the whole block.
struct LossScales {
    float n, unit, gc;
    int32_t least;
    __device__ __forceinline__ LossScales(const LossArgs &a, int32_t *warps) {
        const int32_t r = *a.rows;
        n = static_cast<float>(r > 0 ? r : 1);
        unit = 1.f / (n * static_cast<float>(a.top));
        gc = static_cast<float>(static_cast<double>(a.coef) * a.scale * a.K / n);
        least = 0x7fffffff;
        for (int64_t k = threadIdx.x; k < a.K; k += kThreads) least = min(least, a.counts[k]);
        least = __reduce_min_sync(0xffffffffu, least);
        if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = least;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) least = min(least, warps[w]);
    }
    __device__ __forceinline__ float share(int32_t count) const {
        return static_cast<float>(count - least) * unit;
    }
    // t_i from its part t and whether the row has any finite score
    __device__ __forceinline__ float whole(float t, bool some) const {
        return some ? t + static_cast<float>(least) * unit : 0.f;
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
    if constexpr (W == 32) {
        // (volatile: a meeting of the warp's lanes must stay where it stands)
        asm volatile("redux.sync.max.NaN.f32 %0, %0, 0xffffffff;" : "+f"(m));
    } else {
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    return m;
}
// Both sums in one chain: even lanes go on with z, odd lanes with t.
template <int W>
__device__ __forceinline__ void lanes_sum(float &z, float &t) {
    const bool odd = (threadIdx.x & 1) != 0;
    float v = odd ? t : z;
    const float w = odd ? z : t;
    v += __shfl_xor_sync(0xffffffffu, w, 1);
#pragma unroll
    for (int o = W / 2; o > 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const float u = __shfl_xor_sync(0xffffffffu, v, 1);
    z = odd ? u : v;
    t = odd ? v : u;
}

// The group's sums from those of its threads: s.m is the maximum of this warp's part of the
// group already, s.z and s.t this thread's sums against it.  For a group of several warps,
// one barrier of the block; lane l then holds the sums of the group's warp l.
template <int TPR>
__device__ __forceinline__ Soft join_group(Soft s, float scale2, Soft (*red)[kThreads / 32],
                                           int slot) {
    lanes_sum<(TPR < 32 ? TPR : 32)>(s.z, s.t);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) red[slot][warp] = s;
        __syncthreads();
        s = red[slot][warp / W * W + (threadIdx.x & (W - 1))];
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

// max of pairs of scores that keeps a NaN (of bf16, before they are widened)
__device__ __forceinline__ float vec_max(const uint4 *u, int n, float) {
    float m = -INFINITY;
    for (int i = 0; i < n; ++i)
        m = max_nan(max_nan(max_nan(m, __uint_as_float(u[i].x)), __uint_as_float(u[i].y)),
                    max_nan(__uint_as_float(u[i].z), __uint_as_float(u[i].w)));
    return m;
}
__device__ __forceinline__ uint32_t max_pairs(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float vec_max(const uint4 *u, int n, uint16_t) {
    uint32_t m = 0xff80ff80u;
    for (int i = 0; i < n; ++i)
        m = max_pairs(max_pairs(max_pairs(m, u[i].x), u[i].y), max_pairs(u[i].z, u[i].w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// Rows in 16-byte vectors.  The G rows a block takes at once lie one behind the other: one bulk
// copy brings them into a ring of `stages` slots, several turns ahead.  f is kept in shared
// memory.  The arithmetic is nearly as long as the memory access, so two columns go in one
// instruction where there is one.  An exponent takes the difference first, scale2 (s - m): one
// multiply-add scale2 s - scale2 m would leave each warp the rounding of its own scale2 m (1e-5 of
// dS at scores of 400 over several warps; infinite exponentials from 1e10 on) and is no faster
// (65,536 x 4096 bf16, the call with its counts: 197.5 us, 195.6 with the difference).
template <typename T, int NV, int TPR>
__global__ void __launch_bounds__(kThreads, 3)
    balance_ring_kernel(const T *S, T *dS, const LossArgs a, int stages,
                        uint32_t *__restrict__ err, uint64_t wait_ns) {
    constexpr int V = kVec<T>, H = V / 2, G = kThreads / TPR;
    __shared__ Soft red[2][kThreads / 32];
    __shared__ double sums[kThreads];
    __shared__ uint64_t full[kMaxStages];
    __shared__ uint32_t abort_flag;
    extern __shared__ __align__(128) uint8_t space[];
    float4 *f = reinterpret_cast<float4 *>(space);  // four columns of a thread; then TPR threads
    uint8_t *ring = space + NV * TPR * V * 4;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
        abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const uint32_t row_bytes = static_cast<uint32_t>(a.K * sizeof(T));
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * G;
    auto bring = [&](int64_t i0, int s) {
        if (i0 >= a.N) return;
        const uint32_t bytes = static_cast<uint32_t>(a.N - i0 < G ? a.N - i0 : G) * row_bytes;
        ptx::mbar_arrive_expect_tx(&full[s], bytes);
        ptx::bulk_load(ring + static_cast<size_t>(s) * G * row_bytes, S + i0 * a.K, bytes,
                       &full[s]);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < stages; ++s) bring(first + s * step, s);
    __shared__ int32_t least[kThreads / 32];
    const LossScales c(a, least);
    for (int k = threadIdx.x; k < a.K; k += kThreads) {
        const int v = k / V, q = (v / TPR * (H / 2) + k % V / 4) * TPR + v % TPR;
        reinterpret_cast<float *>(f + q)[k % 4] = c.share(a.counts[k]);
    }
    __syncthreads();
    const float scale2 = a.scale * 1.44269504f;
    const F2 scale22 = f2(scale2, scale2);
    double total = 0.0;
    int slot = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int64_t i = first + grp;
    // the first selection of the next row, read a turn ahead (the others only if it is none)
    int32_t next = i < a.N ? a.labels[i * a.top] : -1;
    T *out = dS + i * a.K + t * V;
    for (int64_t i0 = first; i0 < a.N; i0 += step, i += step, out += step * a.K) {
        const int32_t lab = next;
        if (i + step < a.N) next = a.labels[(i + step) * a.top];
        const bool on = i < a.N && ((lab >= 0 && lab < a.K) || (a.top > 1 && row_selects(a, i)));
        // a wait that runs out is recorded, and the pass runs to its end without its data; nothing
        // more is brought then, as the slot's last copy may still be on its way
        if (!ptx::mbar_wait(&full[stage], phase, &abort_flag, wait_ns)) {
            ok = false;
            *const_cast<volatile uint32_t *>(&abort_flag) = 1u;
            err[0] = kErrTimeout;
        }
        const uint8_t *x = ring + (static_cast<size_t>(stage) * G + grp) * row_bytes + t * 16;
        uint4 u[NV];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            Raw<T, V> r;
            r.lowest();
            if (on && (n * TPR + t) * V < a.K)
                r.u = *reinterpret_cast<const uint4 *>(x + n * TPR * 16);
            u[n] = r.u;
        }
        const float m = lanes_max<(TPR < 32 ? TPR : 32)>(vec_max(u, NV, T()));
        const float base = soft_base(m);
        const F2 off = f2(-base, -base);
        F2 e[NV][H];
        F2 z2 = f2(0.f, 0.f), t2 = z2;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            unpack2(u[n], e[n]);
#pragma unroll
            for (int k = 0; k < H; ++k) e[n][k] = mul2(scale22, add2(e[n][k], off));
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) {
#pragma unroll
            for (int k = 0; k < H; ++k) {
                float lo, hi;
                split(e[n][k], lo, hi);
                e[n][k] = f2(exp2_fast(lo), exp2_fast(hi));
                z2 = add2(z2, e[n][k]);
            }
            if ((n * TPR + t) * V < a.K) {
#pragma unroll
                for (int k = 0; k < H; k += 2) {
                    const float4 q = f[(n * (H / 2) + k / 2) * TPR + t];
                    t2 = fma2(e[n][k], f2(q.x, q.y), t2);
                    t2 = fma2(e[n][k + 1], f2(q.z, q.w), t2);
                }
            }
        }
        const Soft s = join_group<TPR>(Soft{m, sum2(z2), sum2(t2)}, scale2, red, slot);
        if constexpr (TPR <= 32) __syncthreads();
        slot ^= 1;
        // every thread has the slot's rows in registers now
        if (threadIdx.x == 0 && ok) bring(i0 + stages * step, stage);
        if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
        }
        const float inv = s.m == -INFINITY ? 0.f : rcp_fast(s.z);
        const float ti = s.t * inv;
        if (t == 0 && on) total += c.whole(ti, s.m != -INFINITY);
        if (dS == nullptr || i >= a.N) continue;
        // this warp's exponentials against the group's maximum, over the sum
        const float gp = TPR > 32 ? c.gc * exp2_fast(scale2 * (m - soft_base(s.m))) * inv
                                  : c.gc * inv;
        const F2 gp2 = f2(gp, gp), gt2 = f2(-ti * gp, -ti * gp);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            if ((n * TPR + t) * V < a.K) {
                F2 v[H];
#pragma unroll
                for (int k = 0; k < H; k += 2) {
                    const float4 q = f[(n * (H / 2) + k / 2) * TPR + t];
                    v[k] = mul2(e[n][k], fma2(f2(q.x, q.y), gp2, gt2));
                    v[k + 1] = mul2(e[n][k + 1], fma2(f2(q.z, q.w), gp2, gt2));
                }
                *reinterpret_cast<uint4 *>(out + n * TPR * V) = pack2(v);
            }
        }
    }
    finish_block(a, c, total, t == 0, sums);
    if (abort_flag) {  // give copies already in flight a moment to land (bounded)
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 200000ull) {
        }
    }
}

// Rows that are not in 16-byte vectors, element by element.
template <typename T, int NV, int TPR>
__global__ void __launch_bounds__(kThreads, 2)
    balance_elements_kernel(const T *S, T *dS, const LossArgs a) {
    __shared__ Soft red[2][kThreads / 32];
    __shared__ double sums[kThreads];
    pdl_wait();
    pdl_trigger();
    constexpr int G = kThreads / TPR;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    __shared__ int32_t least[kThreads / 32];
    const LossScales c(a, least);
    const float scale2 = a.scale * 1.44269504f;
    double total = 0.0;
    int slot = 0;
    T x[NV];
    bool keep = false;
    auto fetch = [&](int64_t i) {
        keep = i < a.N && row_selects(a, i);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            head_store(&x[n], -INFINITY);
            if (keep && n * TPR + t < a.K) x[n] = S[i * a.K + n * TPR + t];
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * G;
    int64_t i0 = static_cast<int64_t>(blockIdx.x) * G;
    if (i0 < a.N) fetch(i0 + grp);
    for (; i0 < a.N; i0 += step) {
        const int64_t i = i0 + grp;
        const bool on = keep;
        float e[NV];
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            e[n] = head_load(&x[n]);
            m = max_nan(m, e[n]);
        }
        if (i0 + step < a.N) fetch(i0 + step + grp);
        m = lanes_max<(TPR < 32 ? TPR : 32)>(m);
        Soft s{m, 0.f, 0.f};
        const float base = soft_base(m);
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int j = n * TPR + t;
            e[n] = exp2_fast(scale2 * (e[n] - base));
            s.z += e[n];
            if (j < a.K) s.t += e[n] * c.share(a.counts[j]);
        }
        s = join_group<TPR>(s, scale2, red, slot);
        slot ^= 1;
        const float inv = s.m == -INFINITY ? 0.f : rcp_fast(s.z);
        const float ti = s.t * inv;
        if (t == 0 && on) total += c.whole(ti, s.m != -INFINITY);
        if (dS != nullptr && i < a.N) {
            const float gp = TPR > 32 ? c.gc * exp2_fast(scale2 * (m - soft_base(s.m))) * inv
                                      : c.gc * inv;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int j = n * TPR + t;
                if (j < a.K)
                    head_store(dS + i * a.K + j,
                               e[n] * gp * (c.share(a.counts[j]) - ti));
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
    __shared__ int32_t least[kThreads / 32];
    const LossScales c(a, least);
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
            r.t += e * c.share(a.counts[j]);
        }
        r = join_group<kThreads>(r, scale2, red, slot);
        slot ^= 1;
        const float inv = r.m == -INFINITY ? 0.f : 1.f / r.z;
        const float ti = r.t * inv;
        if (threadIdx.x == 0) total += c.whole(ti, r.m != -INFINITY);
        if (dS)
            for (int64_t j = threadIdx.x; j < a.K; j += kThreads) {
                const float p = exp2_fast(scale2 * (head_load(s + j) - soft_base(r.m))) * inv;
                head_store(dS + i * a.K + j,
                           c.gc * p * (c.share(a.counts[j]) - ti));
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

int loss_grid(const BalanceArgs &b, int groups) {
    const int64_t g = ceil_div(b.N, groups);
    return static_cast<int>(g < b.parts ? g : b.parts);
}

template <typename T, int NV, int TPR>
cudaError_t loss_ring(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    auto kernel = balance_ring_kernel<T, NV, TPR>;
    const int slot = kThreads / TPR * a.K * static_cast<int>(sizeof(T));
    int stages = kRingBytes / slot;
    if (stages < 2) stages = 2;
    if (stages > kMaxStages) stages = kMaxStages;
    static std::atomic<uint64_t> smem_set{0};
    const cudaError_t e = smem_opt_in(kernel, 128 << 10, smem_set);
    if (e != cudaSuccess) return e;
    *grid = loss_grid(b, kThreads / TPR);
    return launch_pdl(kernel, dim3(*grid), dim3(kThreads),
                      NV * TPR * kVec<T> * 4 + static_cast<size_t>(stages) * slot, st,
                      static_cast<const T *>(b.S), static_cast<T *>(b.dS), a, stages, b.err,
                      kDefaultWaitNs);
}

template <typename T, int NV, int TPR>
cudaError_t loss_elements(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    *grid = loss_grid(b, kThreads / TPR);
    return launch_pdl(balance_elements_kernel<T, NV, TPR>, dim3(*grid), dim3(kThreads), 0, st,
                      static_cast<const T *>(b.S), static_cast<T *>(b.dS), a);
}

template <typename T>
cudaError_t loss_long(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    *grid = loss_grid(b, 1);
    return launch_pdl(balance_long_kernel<T>, dim3(*grid), dim3(kThreads), 0, st,
                      static_cast<const T *>(b.S), static_cast<T *>(b.dS), a);
}

// Up to 32 columns a thread (16 for one element at a time), and as few threads a row as that
// allows: the sums over the threads cost about as much as ten columns.  65,536 bf16 rows: of 1024
// 50 us (twice the threads: 63), of 2048 93 (114), of 4096 184 (203).
template <typename T>
cudaError_t loss_t(const BalanceArgs &b, const LossArgs &a, int *grid, cudaStream_t st) {
    constexpr int V = kVec<T>, C32 = 32 / V;
    const int K = a.K;
    if (K % V == 0 && aligned(b.S, 16) && aligned(b.dS, 16)) {
        if (K <= 8 * V) return loss_ring<T, 1, 8>(b, a, grid, st);
        if (K <= 16 * V) return loss_ring<T, 1, 16>(b, a, grid, st);
        if (K <= 32 * V) return loss_ring<T, 1, 32>(b, a, grid, st);
        if (K <= 32 * 16) return loss_ring<T, C32 / 2, 32>(b, a, grid, st);
        if (K <= 32 * 32) return loss_ring<T, C32, 32>(b, a, grid, st);
        if (K <= 64 * 32) return loss_ring<T, C32, 64>(b, a, grid, st);
        if (K <= 128 * 32) return loss_ring<T, C32, 128>(b, a, grid, st);
        if (K <= 256 * 32) return loss_ring<T, C32, 256>(b, a, grid, st);
        return loss_long<T>(b, a, grid, st);
    }
    if (K <= 8) return loss_elements<T, 1, 8>(b, a, grid, st);
    if (K <= 32) return loss_elements<T, 1, 32>(b, a, grid, st);
    if (K <= 32 * 4) return loss_elements<T, 4, 32>(b, a, grid, st);
    if (K <= 32 * 16) return loss_elements<T, 16, 32>(b, a, grid, st);
    if (K <= 64 * 16) return loss_elements<T, 16, 64>(b, a, grid, st);
    if (K <= 256 * 8) return loss_elements<T, 8, 256>(b, a, grid, st);
    if (K <= 256 * 16) return loss_elements<T, 16, 256>(b, a, grid, st);
    if (K <= 256 * 32) return loss_elements<T, 32, 256>(b, a, grid, st);
    return loss_long<T>(b, a, grid, st);
}

}  // namespace

int64_t balance_parts(int64_t N, int K) {
    (void)K;
    return N < 1 ? 1 : (N < 148 * 3 ? N : 148 * 3);
}

cudaError_t launch_balance_counts(const int32_t *labels, int64_t N, int top, int K,
                                  int32_t *counts, int32_t *rows, cudaStream_t st) {
    cudaError_t e;
    int copies = kSharedCells / K;
    if (copies > 32) copies = 32;
    const size_t smem = sizeof(int32_t) * copies * K;
    if (copies > 0 && N * top <= kOneBlockLabels) {
        e = launch_pdl(balance_counts_kernel<true>, dim3(1), dim3(1024), smem, st, labels, N, top,
                       K, copies, counts, rows);
        if (e == cudaSuccess) note_launch();
        return e;
    }
    const int64_t z = ceil_div(K, 1024);
    e = launch_pdl(balance_zero_kernel, dim3(static_cast<unsigned>(z < 148 ? z : 148)), dim3(1024),
                   0, st, counts, K, rows);
    if (e != cudaSuccess) return e;
    note_launch();
    if (N == 0) return e;
    int64_t g = ceil_div(N * top, 1024);
    if (g > 148) g = 148;
    e = launch_pdl(balance_counts_kernel<false>, dim3(static_cast<unsigned>(g)), dim3(1024), smem,
                   st, labels, N, top, K, copies, counts, rows);
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
