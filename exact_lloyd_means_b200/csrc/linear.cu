// linear.cu -- Y = act(X W^T + b) + R and its gradients, the embedding head's matrix
// products: X N x d, W m x d (rows, like centroids), Y N x m.
//
//   forward   Z = X W^T + b, Y = act(Z) + R          (rows N, columns m, depth d)
//   backward  G = dY act'(Z), db = column sums of G,
//             dX = G W (rows N, columns d, depth m), dW = G^T X (rows m, columns d, depth N)
//
// The products run in gemm_sm100.cu, which reads an operand along either of its sides, so
// nothing is transposed.  What this file adds is the staging of operands that TMA cannot
// read as they lie (fp32 values as three bf16 planes; bf16 rows that are not multiples of 16
// bytes), G with its column sums, and a kernel for a few rows, which only reads W.
#include <type_traits>

#include "gemm.cuh"

namespace fk {
namespace {

// ----------------------------------------------------------------- staging
// The three bf16 pieces of an fp32 value, x = p0 + p1 + p2 (8 significant bits each; each
// remainder is exact in fp32).  A value that rounds up to infinity is cut instead; an
// infinity or NaN has no remainder.
__device__ __forceinline__ void pieces(float x, uint16_t (&p)[3]) {
    uint32_t h = bf16_bits(x);
    if ((h & 0x7f80u) == 0x7f80u) {
        const uint32_t b = __float_as_uint(x);
        if ((b & 0x7f800000u) == 0x7f800000u) {  // infinity or NaN itself
            p[0] = static_cast<uint16_t>(h);
            p[1] = p[2] = 0;
            return;
        }
        h = b >> 16;
    }
    const float r = x - bf16_val(static_cast<uint16_t>(h));
    p[0] = static_cast<uint16_t>(h);
    p[1] = bf16_bits(r);
    p[2] = bf16_bits(r - bf16_val(p[1]));
}

struct StageJob {
    const void *src, *Z;  // rows x cols; Z non-null: multiply by act'(Z)
    int64_t rows;
    int cols;
    int act;
    int vec;         // src and Z in 16-byte vectors
    uint16_t *out;   // planes [P][rows][ld], or null for column sums alone
    int64_t ld;
    float *colpart;  // [parts][cols], or null
    int tx;          // threads across a row (a power of two), 8 columns each
    int gx, parts;   // blocks across the columns, runs of rows
};
constexpr int kMaxJobs = 3;  // operands staged in one launch
struct StageJobs {
    StageJob job[kMaxJobs];
    int first[kMaxJobs + 1];  // their first blocks
    int n;
};

// Eight consecutive values as they lie in memory (zero where there is no column).
template <typename T>
struct Eight {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p, int64_t left, int vec) {
        if (vec) {
#pragma unroll
            for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
                u[h] = *reinterpret_cast<const uint4 *>(p + h * kVec<T>);
        } else {
            T *t = reinterpret_cast<T *>(u);
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = j < left ? p[j] : T(0);
        }
    }
    __device__ __forceinline__ void pairs(F2 (&o)[4]) const {
        if constexpr (sizeof(T) == 2) {
            unpack2(u[0], o);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                F2 t[2];
                unpack2(u[h], t);
                o[2 * h] = t[0];
                o[2 * h + 1] = t[1];
            }
        }
    }
};

template <typename T>
__device__ __forceinline__ void stage_store(const StageJob &a, int64_t i, int64_t col,
                                            const F2 (&v)[4]) {
    uint16_t *o = a.out + i * a.ld + col;
    // A bf16 operand: G is rounded once.  With GELU, 65,536 x 768 -> 4096, that takes the gradients
    // from 1.7e-3 of their norm (their own rounding to bf16) to 2.3e-3.  G as two bf16 pieces would
    // not, but would double the products, which take 569 of the call's 1020 us at 95% tensor
    // activity, and add 1.6 GB of traffic.
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(o) = pack2(v);
    } else {
        uint16_t pc[8][3];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            split(v[j], lo, hi);
            pieces(lo, pc[2 * j]);
            pieces(hi, pc[2 * j + 1]);
        }
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            uint4 u;
            u.x = pc[0][p] | static_cast<uint32_t>(pc[1][p]) << 16;
            u.y = pc[2][p] | static_cast<uint32_t>(pc[3][p]) << 16;
            u.z = pc[4][p] | static_cast<uint32_t>(pc[5][p]) << 16;
            u.w = pc[6][p] | static_cast<uint32_t>(pc[7][p]) << 16;
            *reinterpret_cast<uint4 *>(o + p * a.rows * a.ld) = u;
        }
    }
}

// A block of a job: 8 * tx columns, one of the job's runs of rows.
template <typename T, int ACT>
__device__ __forceinline__ void stage_rows(const StageJob &a, int64_t i0, int64_t i1, int64_t col,
                                           int ty, int nty, F2 (&sum)[4]) {
    const T *src = static_cast<const T *>(a.src) + col, *Z = static_cast<const T *>(a.Z) + col;
    const int64_t left = a.cols - col;
    constexpr int B = sizeof(T) == 2 ? 4 : 2;  // rows read before any is worked on
    for (int64_t i = i0 + ty; i < i1; i += B * nty) {
        Eight<T> x[B], y[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (i + b * nty < i1) {
                x[b].load(src + (i + b * nty) * a.cols, left, a.vec);
                if constexpr (ACT != FK_ACT_NONE)
                    y[b].load(Z + (i + b * nty) * a.cols, left, a.vec);
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (i + b * nty >= i1) break;
            F2 v[4];
            x[b].pairs(v);
            if constexpr (ACT != FK_ACT_NONE) {
                F2 z[4];
                y[b].pairs(z);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], act_slope2(z[j], ACT));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], v[j]);
            if (a.out != nullptr) stage_store<T>(a, i + b * nty, col, v);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) stage_kernel(const __grid_constant__ StageJobs jobs) {
    __shared__ float red[256][9];
    pdl_wait();
    pdl_trigger();
    int which = 0;
    while (which + 1 < jobs.n && static_cast<int>(blockIdx.x) >= jobs.first[which + 1]) ++which;
    const StageJob &a = jobs.job[which];
    const int block = blockIdx.x - jobs.first[which];
    const int by = block / a.gx, bx = block - by * a.gx;
    const int tx = threadIdx.x & (a.tx - 1), ty = threadIdx.x / a.tx, nty = 256 / a.tx;
    const int64_t col = (static_cast<int64_t>(bx) * a.tx + tx) * 8;
    const int64_t i0 = a.rows * by / a.parts, i1 = a.rows * (by + 1) / a.parts;
    F2 sum[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
    if (col < a.cols) {
        const int act = a.Z != nullptr ? a.act : FK_ACT_NONE;
        if (act == FK_ACT_NONE)
            stage_rows<T, FK_ACT_NONE>(a, i0, i1, col, ty, nty, sum);
        else if (act == FK_ACT_RELU)
            stage_rows<T, FK_ACT_RELU>(a, i0, i1, col, ty, nty, sum);
        else if (act == FK_ACT_GELU)
            stage_rows<T, FK_ACT_GELU>(a, i0, i1, col, ty, nty, sum);
        else
            stage_rows<T, FK_ACT_SILU>(a, i0, i1, col, ty, nty, sum);
    }
    if (a.colpart == nullptr) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) split(sum[j], red[threadIdx.x][2 * j], red[threadIdx.x][2 * j + 1]);
    __syncthreads();
    // thread c sums column c of the block over the ty row threads, in order
    for (int c = threadIdx.x; c < 8 * a.tx; c += 256) {
        const int64_t cc = static_cast<int64_t>(bx) * a.tx * 8 + c;
        if (cc >= a.cols) continue;
        float s = 0.f;
        for (int y = 0; y < nty; ++y) s += red[y * a.tx + c / 8][c % 8];
        a.colpart[static_cast<int64_t>(by) * a.cols + cc] = s;
    }
}

// The column sums in a launch of their own.  A join of cut products takes up to kJoinParts
// parts along instead: the gradients of 1001 x 300 x 129 fp32 (126 parts) take 16.8 us so and 18.8
// with the launch, 3000 x 768 x 768 bf16 (375) 23.8 and 26.3, but 8192 x 768 x 768 (888 parts,
// which 1024 threads read faster than 256) 48.8 and 47.5.
constexpr int kJoinParts = 400;
__global__ void __launch_bounds__(1024) col_join_kernel(const ColSums s) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    join_columns<1024>(s, blockIdx.x, red);
}

// Threads across a row, 8 columns each: whole rows where they fit (memory likes long runs: at
// 4096 bf16 columns, 4 KB of a row at a time and four rows ahead take 275 us where 512 bytes
// and two rows took 447, 65,536 rows with GELU's slope, 1.6 GB).
int stage_tx(int cols) {
    int tx = 1;
    while (tx < 256 && tx * 8 < cols) tx *= 2;
    return tx;
}

// Runs of rows the staging kernel is cut into: up to about six blocks an SM with four rows or
// more a thread, or two an SM with fewer.
int stage_parts(int64_t rows, int cols) {
    const int tx = stage_tx(cols), ty = 256 / tx;
    const int64_t bx = ceil_div(cols, tx * 8);
    auto up_to = [&](int64_t blocks, int64_t per_thread) {
        const int64_t p = blocks / bx, most = ceil_div(rows, per_thread * ty);
        return p < most ? p : most;
    };
    const int64_t wide = up_to(148 * 6, 4), narrow = up_to(148 * 2, 1);
    const int64_t p = wide > narrow ? wide : narrow;
    return static_cast<int>(p < 1 ? 1 : p);
}

void add_job(StageJobs &jobs, StageJob a) {
    a.tx = stage_tx(a.cols);
    a.vec = a.cols % 8 == 0 && aligned(a.src, 16) && aligned(a.Z, 16);
    a.gx = static_cast<int>(ceil_div(a.cols, a.tx * 8));
    a.parts = stage_parts(a.rows, a.cols);
    jobs.job[jobs.n] = a;
    jobs.first[jobs.n + 1] = jobs.first[jobs.n] + a.gx * a.parts;
    ++jobs.n;
}

template <typename T>
cudaError_t launch_stage(const StageJobs &jobs, cudaStream_t st) {
    if (jobs.n == 0) return cudaSuccess;
    const cudaError_t e = launch_pdl(stage_kernel<T>,
                                     dim3(static_cast<unsigned>(jobs.first[jobs.n])), dim3(256), 0,
                                     st, jobs);
    if (e == cudaSuccess) note_launch();
    return e;
}

// ----------------------------------------------------------------- a few rows
// A few rows of X: a block reads CW rows of W once, its four warps a quarter of the depth each,
// and keeps a sum per row of X (which stays in L1) and column.  W is all the traffic.
//
// Where it is taken (us, this kernel / the tensor cores, replayed from a graph):
//   fp32, up to 16 rows: 1 x 768 x 768 1.7 / 14.6, 8 x 768 x 4096 8.1 / 23.1, 16 x 4096 x 4096
//   56 / 73 (the split of W costs the tensor cores more than its products);
//   bf16, up to 4 rows: 1 x 768 x 768 1.6 / 6.2, 4 x 4096 x 4096 12.6 / 13.7; up to 8 where W
//   has at most 2^20 elements: 8 x 768 x 768 4.1 / 6.1, but 8 x 768 x 4096 8.5 / 6.7.
bool few_rows(int64_t N, int d, int m, fk_dtype dtype) {
    if (dtype == FK_F32) return N <= 16;
    return N <= 4 || (N <= 8 && static_cast<int64_t>(m) * d <= (1 << 20));
}

// Depth after which a block joins its threads' sums: a thread adds up 1/128 of it, 8192 products,
// one after the other, and longer chains would show (fp32 sums of positive terms were 3e-7 low at
// a depth of 2^22 in one chain a thread and 2.3e-5 at 2^25).
constexpr int64_t kFewRun = 1 << 20;

// LONG: a depth of more than kFewRun.
template <typename T, int NR, int CW, bool LONG>
__global__ void __launch_bounds__(128)
    few_rows_kernel(const T *__restrict__ X, const T *__restrict__ W, int N, int d, int vec,
                    const Epilogue ep) {
    constexpr int V = kVec<T>;
    __shared__ float red[4][NR * CW];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * CW;
    // (columns past the last are formed from the last row of W and not written)
    const T *w[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) w[c] = W + (c0 + c < ep.cols ? c0 + c : ep.cols - 1) * d;
    float s[NR][CW] = {};
    auto step = [&](int64_t k, auto width) {
        constexpr int L = decltype(width)::value;
        Raw<T, L> raw[CW];
#pragma unroll
        for (int c = 0; c < CW; ++c) raw[c].load(w[c] + k);
        float a[CW][L];
#pragma unroll
        for (int c = 0; c < CW; ++c) raw[c].get(a[c]);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            if (r < N) {
                Raw<T, L> u;
                u.load(X + static_cast<int64_t>(r) * d + k);
                float x[L];
                u.get(x);
#pragma unroll
                for (int c = 0; c < CW; ++c)
#pragma unroll
                    for (int j = 0; j < L; ++j) s[r][c] += a[c][j] * x[j];
            }
        }
    };
    // the threads' sums over columns k0 .. k1 - 1, joined: thread r * CW + c has that of (r, c)
    auto run = [&](int64_t k0, int64_t k1) {
        if (vec) {
#pragma unroll 2
            for (int64_t k = k0 + threadIdx.x * V; k < k1; k += 128 * V)
                step(k, std::integral_constant<int, V>{});
        } else {
#pragma unroll 2
            for (int64_t k = k0 + threadIdx.x; k < k1; k += 128)
                step(k, std::integral_constant<int, 1>{});
        }
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                if (r < N) s[r][c] = warp_sum_f(s[r][c]);
                if (lane == 0) red[warp][r * CW + c] = s[r][c];
            }
        __syncthreads();
        float v = 0.f;
        if (static_cast<int>(threadIdx.x) < NR * CW) {
            v = red[0][threadIdx.x];
#pragma unroll
            for (int t = 1; t < 4; ++t) v += red[t][threadIdx.x];
        }
        return v;
    };
    float z = run(0, LONG ? kFewRun : d);
    if constexpr (LONG) {
        for (int64_t k0 = kFewRun; k0 < d; k0 += kFewRun) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int c = 0; c < CW; ++c) s[r][c] = 0.f;
            z += run(k0, k0 + kFewRun < d ? k0 + kFewRun : d);
        }
    }
    if (static_cast<int>(threadIdx.x) >= NR * CW) return;
    const int r = threadIdx.x / CW;
    const int64_t col = c0 + threadIdx.x % CW;
    if (r >= N || col >= ep.cols) return;
    z = __fadd_rn(z, ep.bias != nullptr ? ep.bias[col] : 0.f);
    const int64_t o = r * ep.cols + col;
    const float res = ep.R != nullptr ? head_load(static_cast<const T *>(ep.R) + o) : 0.f;
    if (ep.Z != nullptr) head_store(static_cast<T *>(ep.Z) + o, z);
    head_store(static_cast<T *>(ep.C) + o, __fadd_rn(act_value(z, ep.act), res));
}

template <typename T>
cudaError_t launch_few_rows(const LinearArgs &a, cudaStream_t st) {
    Epilogue ep{};
    ep.bias = a.bias;
    ep.R = a.R;
    ep.C = a.Y;
    ep.Z = a.Z;
    ep.cols = a.m;
    ep.act = a.act;
    const int vec = a.d % kVec<T> == 0 && aligned(a.X, 16) && aligned(a.W, 16);
    const T *X = static_cast<const T *>(a.X), *W = static_cast<const T *>(a.W);
    const int N = static_cast<int>(a.N);
    auto launch = [&](auto kernel, int columns) {
        const cudaError_t e =
            launch_pdl(kernel, dim3(static_cast<unsigned>(ceil_div(a.m, columns))), dim3(128), 0,
                       st, X, W, N, a.d, vec, ep);
        if (e == cudaSuccess) note_launch();
        return e;
    };
    // four columns a block from 1024 on (4 x 768 x 4096 bf16 5.3 against 6.3 with one), one
    // where the GPU would stay empty (8 x 4096 x 100 bf16 4.1 against 9.2) and for the deepest (4 x
    // 2^20 x 1100 fp32 1174 against 2291)
    auto rows = [&](auto columns, auto deep) {
        constexpr int CW = decltype(columns)::value;
        constexpr bool L = decltype(deep)::value;
        if (N == 1) return launch(few_rows_kernel<T, 1, CW, L>, CW);
        if (N <= 2) return launch(few_rows_kernel<T, 2, CW, L>, CW);
        if (N <= 4) return launch(few_rows_kernel<T, 4, CW, L>, CW);
        if (N <= 8 || sizeof(T) == 2) return launch(few_rows_kernel<T, 8, CW, L>, CW);
        return launch(few_rows_kernel<T, sizeof(T) == 4 ? 16 : 8, CW, L>, CW);
    };
    using One = std::integral_constant<int, 1>;
    if (a.d > kFewRun) return rows(One{}, std::true_type{});
    return a.m >= 1024 ? rows(std::integral_constant<int, 4>{}, std::false_type{})
                       : rows(One{}, std::false_type{});
}

// ----------------------------------------------------------------- unaligned bf16 operands
// C[i][j] = sum_k A(i, k) B(j, k) on the CUDA cores, for bf16 operands that start off a
// 16-byte boundary: any strides, no staging (whose space would be as large as the operand).
// Sums are added up in runs of kUnalignedRun and the runs apart: one chain of fp32 additions of
// positive products of bf16 numbers is 0.3% low after 2^22 of them and 3.5% after 2^24.
constexpr int kUnalignedRun = 4096;
__global__ void __launch_bounds__(256)
    unaligned_kernel(const uint16_t *__restrict__ A, int64_t ar, int64_t ak,
                     const uint16_t *__restrict__ B, int64_t br, int64_t bk, int64_t rows,
                     int64_t depth, const Epilogue ep) {
    __shared__ float sa[16][65], sb[16][65];
    pdl_wait();
    pdl_trigger();
    const int64_t ct = (ep.cols + 63) / 64;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) / ct * 64;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) % ct * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float sum[4][4] = {}, acc[4][4] = {};
    for (int64_t k0 = 0; k0 < depth; k0 += 16) {
        for (int t = threadIdx.x; t < 1024; t += 256) {
            const int k = ak == 1 ? t & 15 : t >> 6, i = ak == 1 ? t >> 4 : t & 63;
            const bool ok = r0 + i < rows && k0 + k < depth;
            sa[k][i] = ok ? bf16_val(A[(r0 + i) * ar + (k0 + k) * ak]) : 0.f;
        }
        for (int t = threadIdx.x; t < 1024; t += 256) {
            const int k = bk == 1 ? t & 15 : t >> 6, j = bk == 1 ? t >> 4 : t & 63;
            const bool ok = c0 + j < ep.cols && k0 + k < depth;
            sb[k][j] = ok ? bf16_val(B[(c0 + j) * br + (k0 + k) * bk]) : 0.f;
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
        if ((k0 + 16) % kUnalignedRun == 0 || k0 + 16 >= depth) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[i][j] += acc[i][j];
                    acc[i][j] = 0.f;
                }
        }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + ty + 16 * i, c = c0 + tx + 16 * j;
            if (r >= rows || c >= ep.cols) continue;
            const int64_t o = r * ep.cols + c;
            const float z = sum[i][j] + (ep.bias ? ep.bias[c] : 0.f);
            const float res = ep.R ? bf16_val(static_cast<const uint16_t *>(ep.R)[o]) : 0.f;
            if (ep.Z) static_cast<uint16_t *>(ep.Z)[o] = bf16_bits(z);
            static_cast<uint16_t *>(ep.C)[o] = bf16_bits(act_value(z, ep.act) + res);
        }
}

// ----------------------------------------------------------------- layouts
struct LinearLayout {
    size_t x = 0, w = 0, g = 0, col = 0, part = 0, part2 = 0, total = 0;
    GemmPlan plan[kMaxProducts] = {};  // forward; or dX and dW
    int64_t ldd = 0, ldm = 0;  // staged row lengths
    int planes = 1;
    bool stage_x = false, stage_m = false;  // X and W; G and dY
};

LinearLayout linear_layout(int64_t N, int d, int m, fk_dtype dtype, bool backward) {
    LinearLayout L;
    L.planes = dtype == FK_F32 ? 3 : 1;
    L.ldd = round_up(d, 8);
    L.ldm = round_up(m, 8);
    L.stage_x = dtype == FK_F32 || d % 8 != 0;
    L.stage_m = dtype == FK_F32 || m % 8 != 0;
    size_t o = 256;  // the error words
    auto take = [&](int64_t bytes) {
        const size_t at = o;
        o += static_cast<size_t>(round_up(bytes, 256));
        return at;
    };
    const bool few = !backward && few_rows(N, d, m, dtype);
    L.x = take(L.stage_x && !few ? 2 * L.planes * N * L.ldd : 0);
    L.w = take(L.stage_x && !few ? 2 * L.planes * m * L.ldd : 0);
    if (backward) {
        L.g = take(2 * L.planes * N * L.ldm);
        L.col = take(sizeof(float) * static_cast<int64_t>(stage_parts(N, m)) * m);
        const GemmSize sizes[2] = {{N, d, m}, {m, d, N}};
        if (N > 0) gemm_plan(sizes, 2, dtype, L.plan);
    } else if (!few) {
        const GemmSize size{N, m, d};
        gemm_plan(&size, 1, dtype, L.plan);
    }
    L.part = take(static_cast<int64_t>(gemm_part_bytes(L.plan[0])));
    L.part2 = take(static_cast<int64_t>(gemm_part_bytes(L.plan[1])));
    L.total = o;
    return L;
}

// An operand of `rows` x `cols` as the tensor cores can read it: staged into `space` where
// its type or row length asks for it.
GemmOperand operand(StageJobs &jobs, const void *src, int64_t rows, int cols, bool stage,
                    uint16_t *space, bool mn_major) {
    if (!stage) return GemmOperand{static_cast<const uint16_t *>(src), cols, mn_major};
    StageJob s{};
    s.src = src;
    s.rows = rows;
    s.cols = cols;
    s.out = space;
    s.ld = round_up(cols, 8);
    add_job(jobs, s);
    return GemmOperand{space, s.ld, mn_major};
}

// Products in one launch on the tensor cores; each whose bf16 operands lie off 16-byte boundaries
// without them.  Either way a product's bits are its own: they do not depend on the other.
bool on_tensor_cores(const GemmArgs &a) { return aligned(a.A.base, 16) && aligned(a.B.base, 16); }
cudaError_t unaligned_product(const GemmArgs &a, cudaStream_t st) {
    Epilogue ep{};
    ep.bias = a.bias;
    ep.R = a.R;
    ep.C = a.C;
    ep.Z = a.Z;
    ep.cols = a.cols;
    ep.act = a.act;
    const int64_t tiles = ceil_div(a.rows, 64) * ceil_div(a.cols, 64);
    if (tiles > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_pdl(
        unaligned_kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, st, a.A.base,
        a.A.mn_major ? 1 : a.A.ld, a.A.mn_major ? a.A.ld : 1, a.B.base, a.B.mn_major ? 1 : a.B.ld,
        a.B.mn_major ? a.B.ld : 1, a.rows, a.depth, ep);
    if (e == cudaSuccess) note_launch();
    return e;
}
// `sums` are finished by the launch that joins cut products, where there is one, or else by one of
// their own.
cudaError_t products(const GemmArgs *args, const GemmPlan *plans, int n, ColSums sums,
                     cudaStream_t st) {
    GemmArgs on[kMaxProducts];
    GemmPlan plan[kMaxProducts];
    int count = 0;
    bool cut = false;
    for (int i = 0; i < n; ++i) {
        if (!on_tensor_cores(args[i])) continue;
        on[count] = args[i];
        plan[count++] = plans[i];
        cut = cut || plans[i].splits > 1;
    }
    if (sums.db != nullptr && !(cut && sums.parts <= kJoinParts)) {
        const cudaError_t e = launch_pdl(col_join_kernel,
                                         dim3(static_cast<unsigned>(ceil_div(sums.cols, 32))),
                                         dim3(1024), 0, st, sums);
        if (e != cudaSuccess) return e;
        note_launch();
        sums.db = nullptr;
    }
    if (count > 0) {
        const cudaError_t e = launch_gemm(on, plan, count, sums, st);
        if (e != cudaSuccess) return e;
    }
    for (int i = 0; i < n; ++i) {
        if (on_tensor_cores(args[i])) continue;
        const cudaError_t e = unaligned_product(args[i], st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t linear_t(const LinearArgs &a, void *ws, cudaStream_t st) {
    if (few_rows(a.N, a.d, a.m, a.dtype)) return launch_few_rows<T>(a, st);
    const LinearLayout L = linear_layout(a.N, a.d, a.m, a.dtype, false);
    GemmArgs g{};
    StageJobs jobs{};
    g.A = operand(jobs, a.X, a.N, a.d, L.stage_x, ws_ptr<uint16_t>(ws, L.x), false);
    g.B = operand(jobs, a.W, a.m, a.d, L.stage_x, ws_ptr<uint16_t>(ws, L.w), false);
    const cudaError_t e = launch_stage<T>(jobs, st);
    if (e != cudaSuccess) return e;
    g.dtype = a.dtype;
    g.rows = a.N;
    g.cols = a.m;
    g.depth = a.d;
    g.bias = a.bias;
    g.act = a.act;
    g.R = a.R;
    g.C = a.Y;
    g.Z = a.Z;
    g.part = ws_ptr<float>(ws, L.part);
    g.err = ws_ptr<uint32_t>(ws, 0);
    return products(&g, L.plan, 1, ColSums{}, st);
}

template <typename T>
cudaError_t linear_backward_t(const LinearArgs &a, void *ws, cudaStream_t st) {
    const LinearLayout L = linear_layout(a.N, a.d, a.m, a.dtype, true);
    if (a.N == 0) {
        cudaError_t e = cudaSuccess;
        if (a.dW) e = cudaMemsetAsync(a.dW, 0, sizeof(T) * a.m * static_cast<int64_t>(a.d), st);
        if (e == cudaSuccess && a.db) e = cudaMemsetAsync(a.db, 0, sizeof(float) * a.m, st);
        return e;
    }
    // G, with its column sums from the values before they are rounded to an operand, and the
    // other operands: one launch
    StageJobs jobs{};
    const bool any = a.dX != nullptr || a.dW != nullptr;
    const bool write = any && (L.stage_m || a.act != FK_ACT_NONE);
    ColSums sums{};
    if (write || a.db) {
        StageJob s{};
        s.src = a.dY;
        s.Z = a.act != FK_ACT_NONE ? a.Zin : nullptr;
        s.rows = a.N;
        s.cols = a.m;
        s.act = a.act;
        s.out = write ? ws_ptr<uint16_t>(ws, L.g) : nullptr;
        s.ld = L.ldm;
        // a single run of rows has the sums themselves
        const int parts = stage_parts(a.N, a.m);
        s.colpart = a.db;
        if (a.db && parts > 1) {
            s.colpart = ws_ptr<float>(ws, L.col);
            sums = ColSums{s.colpart, a.db, parts, a.m};
        }
        add_job(jobs, s);
    }
    GemmOperand W{}, X{};
    if (a.dX) W = operand(jobs, a.W, a.m, a.d, L.stage_x, ws_ptr<uint16_t>(ws, L.w), true);
    if (a.dW) X = operand(jobs, a.X, a.N, a.d, L.stage_x, ws_ptr<uint16_t>(ws, L.x), true);
    cudaError_t e = launch_stage<T>(jobs, st);
    if (e != cudaSuccess) return e;
    // dX and dW in one launch (each cut the same way when asked for alone)
    GemmArgs args[2] = {};
    GemmPlan plans[2];
    int n = 0;
    auto add = [&](const GemmOperand &A, const GemmOperand &B, int64_t rows, int64_t depth,
                   void *C, int which, size_t part) {
        GemmArgs &g = args[n];
        g.dtype = a.dtype;
        g.A = A;
        g.B = B;
        g.rows = rows;
        g.cols = a.d;
        g.depth = depth;
        g.act = FK_ACT_NONE;
        g.C = C;
        g.part = ws_ptr<float>(ws, part);
        g.err = ws_ptr<uint32_t>(ws, 0);
        plans[n++] = L.plan[which];
    };
    GemmOperand G{write ? ws_ptr<uint16_t>(ws, L.g) : static_cast<const uint16_t *>(a.dY),
                  write ? L.ldm : a.m, false};
    if (a.dX) add(G, W, a.N, a.m, a.dX, 0, L.part);
    G.mn_major = true;
    if (a.dW) add(G, X, a.m, a.N, a.dW, 1, L.part2);
    return products(args, plans, n, sums, st);
}

}  // namespace

size_t linear_ws_bytes(int64_t N, int d, int m, fk_dtype dtype) {
    return linear_layout(N, d, m, dtype, false).total;
}
size_t linear_backward_ws_bytes(int64_t N, int d, int m, fk_dtype dtype) {
    return linear_layout(N, d, m, dtype, true).total;
}

cudaError_t launch_linear(const LinearArgs &a, void *ws, cudaStream_t st) {
    return a.dtype == FK_F32 ? linear_t<float>(a, ws, st) : linear_t<uint16_t>(a, ws, st);
}

cudaError_t launch_linear_backward(const LinearArgs &a, void *ws, cudaStream_t st) {
    return a.dtype == FK_F32 ? linear_backward_t<float>(a, ws, st)
                             : linear_backward_t<uint16_t>(a, ws, st);
}

}  // namespace fk
