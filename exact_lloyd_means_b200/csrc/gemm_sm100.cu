// gemm_sm100.cu -- C = A B^T on the tensor cores, with its epilogue, for fk_linear and its
// gradients.
//
//   * persistent grid; a unit of work is one output tile (128 * CG rows by BN columns) over
//     one part of the depth.  CG = 2: a cluster of two CTAs, each with 128 rows of A, half
//     the columns of B and the 128 x 256 accumulator of its rows (cta_group::2, M = 256);
//   * warp 0: TMA producer, a ring of stages of 64 of the depth; warp 1: tcgen05.mma issuer,
//     two accumulators in tensor memory, so that a tile's epilogue overlaps the next tile's
//     products; warps 2..9: epilogue, two groups of four warps, half the columns each.  A
//     thread has one row of the tile and takes 32 columns at a time; it reads and writes
//     them in whole 32-byte sectors (fp32 threads exchange theirs first, so that a store covers
//     64 or 128 bytes of a row).  Only columns that do not start on 16 bytes pass through shared
//     memory, whose bandwidth the operands take (128 x 64 by 256 x 64 a chunk written and
//     read): staging the tile there as fp32 took 92 us where this takes 71 (10,000 x 768 x
//     4096, GELU, both outputs);
//   * either operand may be stored along the depth (K-major) or along its rows (MN-major):
//     both are 128-byte-swizzled TMA boxes, and the MMA descriptors say which.  So the three
//     products of a linear layer and its gradients read their operands as they lie;
//   * fp32 operands come as three bf16 planes (x = x0 + x1 + x2, 8 bits each, exact).  Six
//     of the nine products keep everything above 2^-24 of the result.  A stage holds all the
//     planes, each loaded once for its six products; x0 y0 goes into an accumulator of its
//     own and the five small products into another, so that these are not rounded to the
//     size of the sum, and the sum is rounded no more often than that of bf16 operands;
//   * every wait is bounded; on expiry the CTA records the timeout and winds down.
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gemm.cuh"
#include "ptx_sm100.cuh"

namespace fk {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encode_fn();  // assign_sm100.cu

namespace {

constexpr int kBandRows = 8;  // tiles of one column band that run side by side

// The tensor cores cut what they add to an accumulator (about 2^-24 of the sum a step of 16,
// always towards zero: 4.4e-6 of the result at a depth of 4096).  So fp32 products are
// accumulated in runs of 256 of the depth, 2e-7 each, and the runs added to fp32 registers; and
// the chain of those additions, whose roundings grow with its length (1e-6 of a sum of positive
// terms at a depth of 2^20), is ended every 65,536: deeper products are cut into parts, which
// are joined in order.  bf16 ones, whose result is rounded to 2^-9 anyway, take up to 131,072 of
// the depth in one accumulation.
constexpr int kRunChunks = 4;
constexpr int kMaxF32Chunks = 1024;
constexpr int kMaxBf16Chunks = 2048;
// Parts of a tile's depth that its join adds up one after the other: with up to 148 the gradients
// of 65536 x 64 x 64 bf16 took 53 us for 35.
constexpr int kMaxSplits = 32;

// OV = consecutive columns an epilogue thread writes at once: 32 or 16 bytes of them, or one
// column, where rows of the outputs do not start on such boundaries.
template <int CG, int BN, int NP, int OV>
struct GemmCfg {
    static constexpr int kABytes = kBM * kBK * 2;  // one plane
    static constexpr int kBRows = BN / CG;
    static constexpr int kBBytes = kBRows * kBK * 2;
    static constexpr int kStageBytes = NP * (kABytes + kBBytes);
    static constexpr int kEpiWarps = 8;
    static constexpr int kStageOut = OV == 1 ? 32 * 33 * 4 : 0;  // a warp's 32 x 32 fp32
    static constexpr int kBarBytes = 256;
    static constexpr int kSpace = 232448 - 1024 - kBarBytes - kEpiWarps * kStageOut;
    static constexpr int kStages = kSpace / kStageBytes < 8 ? kSpace / kStageBytes : 8;
    static constexpr int kSmemBytes =
        kStages * kStageBytes + kEpiWarps * kStageOut + kBarBytes + 1024;
    static constexpr int kThreads = 64 + kEpiWarps * 32;
    static constexpr int kAccCols = NP == 3 ? 2 * BN : BN;  // of one tile
    static constexpr int kTmemCols = 2 * kAccCols;
    static_assert(kTmemCols <= 512 && kStages >= 2, "two tiles, two stages");
    static constexpr int kGroupCols = BN / (kEpiWarps / 4);  // columns of one epilogue group
    static_assert(kSmemBytes <= 232448, "shared memory");
    static_assert(kStageBytes % 1024 == 0, "stage bases stay 1024-byte aligned");
    static_assert(8 * (2 * kStages + 5) + 8 <= kBarBytes, "barriers");
};

// Planes of an operand of type T.
template <typename T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;

struct GemmShape {
    int64_t rows, cols;
    int nkc;      // chunks of 64 in the depth
    int splits;
    int a_mn, b_mn;
    int64_t tiles_r, tiles_c;
    uint64_t inv_band;   // 2^64 / (tiles of a band), rounded down
    int64_t full, tail;  // tiles with the whole depth, tiles with their depth cut
};

// The products of a launch: the units of the first, then those of the second.
struct alignas(64) GemmJobs {
    CUtensorMap a[kMaxProducts], b[kMaxProducts];
    GemmShape shape[kMaxProducts];
    Epilogue ep[kMaxProducts];
    float *part[kMaxProducts];
    int bvec[kMaxProducts];  // the bias in 16-byte vectors
    int64_t second, units;   // first unit of the second product, all units
};

// Tile t in the order of work: bands of kBandRows row tiles, rows fastest within a band, so that
// the tiles running side by side share their operands in L2.  Each warp works this out before
// every tile, and where the depth is short nothing hides what it takes: without its two 64-bit
// divisions 65536 x 128 x 4096 takes 170 us, with them 173.
__device__ __forceinline__ void tile_of(const GemmShape &s, int64_t t, int64_t &tr, int64_t &tc) {
    const int64_t per_band = kBandRows * s.tiles_c;
    // (t < 2^34, so this is the quotient or one less)
    int64_t band = static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(t), s.inv_band));
    int64_t in = t - band * per_band;
    if (in >= per_band) {
        ++band;
        in -= per_band;
    }
    const int64_t left = s.tiles_r - band * kBandRows;
    if (left >= kBandRows) {
        tc = in / kBandRows;
        tr = band * kBandRows + in % kBandRows;
    } else {  // (a band has fewer than 2^29 tiles)
        const uint32_t i = static_cast<uint32_t>(in), h = static_cast<uint32_t>(left);
        tc = i / h;
        tr = band * kBandRows + i % h;
    }
}

// Unit u: its chunks of the depth, which part of it they are (0 of 1 for a whole one) ...
struct Chunks {
    int k0, k1, split;
};
__device__ __forceinline__ Chunks chunks_of(const GemmShape &s, int64_t u) {
    if (u < s.full || s.splits == 1) return Chunks{0, s.nkc, 0};
    const int split = static_cast<int>((u - s.full) / s.tail);
    return Chunks{static_cast<int>(static_cast<int64_t>(s.nkc) * split / s.splits),
                  static_cast<int>(static_cast<int64_t>(s.nkc) * (split + 1) / s.splits), split};
}
// ... its tile and, where its chunks are not all, its partial product.
struct Unit {
    int64_t tr, tc, part;
    int k0, k1;
};
__device__ __forceinline__ Unit unit_of(const GemmShape &s, int64_t u) {
    Unit r;
    const Chunks c = chunks_of(s, u);
    r.k0 = c.k0;
    r.k1 = c.k1;
    r.part = -1;
    if (u >= s.full && s.splits > 1) {
        u -= c.split * s.tail;
        r.part = (u - s.full) * s.splits + c.split;
    }
    tile_of(s, u, r.tr, r.tc);
    return r;
}

// f with the operands' majors as constants: the loops over the depth are the kernel's pulse,
// and deciding in them how to load cost a 65,536 x 768 x 4096 product 6%.  (An MN-major A
// comes with an MN-major B: dW.)
template <typename F>
__device__ __forceinline__ bool by_major(bool a_mn, bool b_mn, F &&f) {
    if (a_mn) return f(std::true_type{}, std::true_type{});
    if (b_mn) return f(std::false_type{}, std::true_type{});
    return f(std::false_type{}, std::false_type{});
}

__device__ __forceinline__ void gemm_timeout(volatile uint32_t *abort_flag, uint32_t *err) {
    *abort_flag = 1u;
    err[0] = kErrTimeout;
}

template <int CG, int BN, typename T, int OV>
__global__ void __launch_bounds__(GemmCfg<CG, BN, kPlanes<T>, OV>::kThreads, 1)
    gemm_kernel(const __grid_constant__ GemmJobs jobs, uint32_t *__restrict__ err,
                uint64_t wait_ns) {
    constexpr int NP = kPlanes<T>;
    using Cfg = GemmCfg<CG, BN, NP, OV>;
    constexpr int S = Cfg::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *stage_out = smem + S * Cfg::kStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(stage_out + Cfg::kEpiWarps * Cfg::kStageOut);
    uint64_t *empty = full + S;
    uint64_t *tfull = empty + S;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile uint32_t *abort_flag = tmem_slot + 1;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const int64_t first = blockIdx.x / CG;
    const int64_t step = gridDim.x / CG;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            ptx::mbar_init(&tfull[a], 1);
            ptx::mbar_init(&tempty[a], CG * Cfg::kEpiWarps);
        }
        ptx::mbar_init(drain, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&jobs.a[0]);
        ptx::prefetch_tmap(&jobs.b[0]);
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            ptx::tmem_alloc_pair(tmem_slot, Cfg::kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(tmem_slot, Cfg::kTmemCols);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) ptx::cluster_sync();
    ptx::tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            const uint32_t full_c =
                CG == 2 ? ptx::mapa_shared(ptx::smem_u32(full), 0) : 0u;
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (int64_t u = first; u < jobs.units && ok; u += step) {
                const bool j = u >= jobs.second;
                const Unit un = j ? unit_of(jobs.shape[1], u - jobs.second)
                                  : unit_of(jobs.shape[0], u);
                const CUtensorMap *ma = j ? &jobs.a[1] : &jobs.a[0];
                const CUtensorMap *mb = j ? &jobs.b[1] : &jobs.b[0];
                const int r0 = static_cast<int>(un.tr * (kBM * CG) + rank * kBM);
                const int c0 = static_cast<int>(un.tc * BN + rank * Cfg::kBRows);
                ok = by_major((j ? jobs.shape[1].a_mn : jobs.shape[0].a_mn) != 0,
                              (j ? jobs.shape[1].b_mn : jobs.shape[0].b_mn) != 0,
                              [&](auto a_mn, auto b_mn) {
                    for (int kc = un.k0; kc < un.k1; ++kc) {
                        if (!ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag, wait_ns)) {
                            gemm_timeout(abort_flag, err);
                            return false;
                        }
                        if (rank == 0)
                            ptx::mbar_arrive_expect_tx(&full[stage], CG * Cfg::kStageBytes);
                        const int k = kc * kBK;
                        auto load = [&](uint8_t *dst, const CUtensorMap *map, int x, int y,
                                        int p) {
                            if constexpr (CG == 2)
                                ptx::tma_load_3d_pair(dst, map, full_c + stage * 8, x, y, p);
                            else
                                ptx::tma_load_3d(dst, map, &full[stage], x, y, p);
                        };
#pragma unroll
                        for (int p = 0; p < NP; ++p) {
                            uint8_t *sa = smem + stage * Cfg::kStageBytes + p * Cfg::kABytes;
                            uint8_t *sb = smem + stage * Cfg::kStageBytes + NP * Cfg::kABytes +
                                          p * Cfg::kBBytes;
                            if constexpr (decltype(a_mn)::value) {
#pragma unroll
                                for (int b = 0; b < kBM / 64; ++b)
                                    load(sa + b * 8192, ma, r0 + b * 64, k, p);
                            } else {
                                load(sa, ma, k, r0, p);
                            }
                            if constexpr (decltype(b_mn)::value) {
#pragma unroll
                                for (int b = 0; b < Cfg::kBRows / 64; ++b)
                                    load(sb + b * 8192, mb, c0 + b * 64, k, p);
                            } else {
                                load(sb, mb, k, c0, p);
                            }
                        }
                        if (++stage == S) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    return true;
                });
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && rank == 0) {
            // chunks of one accumulation
            constexpr int kRun = NP == 3 ? kRunChunks : 0x40000000;
            uint32_t stage = 0, phase = 0, it = 0;
            bool ok = true;
            for (int64_t u = first; u < jobs.units && ok; u += step) {
                const bool j = u >= jobs.second;
                // (no more than it needs: what this thread does between tiles leaves the
                // tensor cores idle)
                const Chunks un = j ? chunks_of(jobs.shape[1], u - jobs.second)
                                    : chunks_of(jobs.shape[0], u);
                ok = by_major((j ? jobs.shape[1].a_mn : jobs.shape[0].a_mn) != 0,
                              (j ? jobs.shape[1].b_mn : jobs.shape[0].b_mn) != 0,
                              [&](auto a_mn, auto b_mn) {
                    constexpr bool AM = decltype(a_mn)::value, BM = decltype(b_mn)::value;
                    constexpr uint32_t idesc =
                        ptx::idesc_bf16_f32(kBM * CG, BN) | ptx::idesc_mn_major(AM, BM);
                    const uint32_t sa = ptx::smem_u32(smem);
                    const uint32_t sb = sa + NP * Cfg::kABytes;
                    const uint64_t da0 = AM ? ptx::sdesc_mn_sw128(sa) : ptx::sdesc_k_sw128(sa);
                    const uint64_t db0 = BM ? ptx::sdesc_mn_sw128(sb) : ptx::sdesc_k_sw128(sb);
                    for (int k0 = un.k0; k0 < un.k1; k0 += kRun, ++it) {
                        const uint32_t acc = it & 1u;
                        if (!ptx::mbar_wait(&tempty[acc], ((it >> 1) & 1u) ^ 1u, abort_flag,
                                            wait_ns)) {
                            gemm_timeout(abort_flag, err);
                            return false;
                        }
                        ptx::tc_fence_after();
                        const uint32_t dt = tmem + acc * Cfg::kAccCols;
                        const int n = un.k1 - k0 < kRun ? un.k1 - k0 : kRun;
                        for (int i = 0; i < n; ++i) {
                            if (!ptx::mbar_wait(&full[stage], phase, abort_flag, wait_ns)) {
                                gemm_timeout(abort_flag, err);
                                return false;
                            }
                            ptx::tc_fence_after();
                            // (an address field counts 16 bytes)
                            const uint64_t da = da0 + stage * (Cfg::kStageBytes / 16);
                            const uint64_t db = db0 + stage * (Cfg::kStageBytes / 16);
                            auto mma = [&](uint32_t d, int pa, int pb, int ks, uint32_t more) {
                                const uint64_t x =
                                    da + pa * (Cfg::kABytes / 16) + ks * (AM ? 128 : 2);
                                const uint64_t y =
                                    db + pb * (Cfg::kBBytes / 16) + ks * (BM ? 128 : 2);
                                if constexpr (CG == 2)
                                    ptx::mma_bf16_ss_pair(d, x, y, idesc, more);
                                else
                                    ptx::mma_bf16_ss(d, x, y, idesc, more);
                            };
#pragma unroll
                            for (int ks = 0; ks < kBK / 16; ++ks) {
                                const uint32_t more = i > 0 || ks > 0 ? 1u : 0u;
                                mma(dt, 0, 0, ks, more);
                                if constexpr (NP == 3) {
                                    mma(dt + BN, 0, 2, ks, more);
                                    mma(dt + BN, 1, 1, ks, 1u);
                                    mma(dt + BN, 2, 0, ks, 1u);
                                    mma(dt + BN, 0, 1, ks, 1u);
                                    mma(dt + BN, 1, 0, ks, 1u);
                                }
                            }
                            if constexpr (CG == 2)
                                ptx::mma_commit_pair(&empty[stage], 0x3);
                            else
                                ptx::mma_commit(&empty[stage]);
                            if (++stage == S) {
                                stage = 0;
                                phase ^= 1u;
                            }
                        }
                        if constexpr (CG == 2)
                            ptx::mma_commit_pair(&tfull[acc], 0x3);
                        else
                            ptx::mma_commit(&tfull[acc]);
                    }
                    return true;
                });
            }
            if (!ok) {
                if constexpr (CG == 2)
                    ptx::mma_commit_pair(drain, 0x1);
                else
                    ptx::mma_commit(drain);
                ptx::mbar_wait(drain, 0u, nullptr, wait_ns);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // thread = row of the tile (tensor-memory lane); 32 columns at a time
        const int g = (warp - 2) >> 2;
        const int q = warp & 3;
        [[maybe_unused]] float *st =
            reinterpret_cast<float *>(stage_out + (warp - 2) * Cfg::kStageOut);
        const uint32_t tempty_c =
            CG == 2 ? ptx::mapa_shared(ptx::smem_u32(tempty), 0) : 0u;
        constexpr int C = Cfg::kGroupCols / 32;
        uint32_t it = 0;
        bool ok = true;
        for (int64_t u = first; u < jobs.units && ok; u += step) {
            // (by value and by fixed index: a reference picked here is read from memory again
            // at every use)
            const bool j = u >= jobs.second;
            Epilogue ep = j ? jobs.ep[1] : jobs.ep[0];
            const float *bias = ep.bias;
            constexpr bool kBiasAhead = NP == 1 && OV > 1;
            if (kBiasAhead) ep.bias = nullptr;  // (added here)
            const int64_t rows = j ? jobs.shape[1].rows : jobs.shape[0].rows;
            const int bvec = j ? jobs.bvec[1] : jobs.bvec[0];
            float *part = j ? jobs.part[1] : jobs.part[0];
            const Unit un = j ? unit_of(jobs.shape[1], u - jobs.second)
                              : unit_of(jobs.shape[0], u);
            const int64_t r0 = un.tr * (kBM * CG) + rank * kBM + q * 32;
            const int64_t c0 = un.tc * BN + g * Cfg::kGroupCols;
            // columns c0 + 32 c .. + 31 of this thread's row, finished
            auto finish = [&](int c, float (&v)[32]) {
                const int64_t col = c0 + c * 32;
                if (un.part >= 0) {  // fp32 partial products, the whole tile
                    float *dst = part + (un.part * CG + rank) * (kBM * BN) +
                                 (q * 32 + lane) * BN + g * Cfg::kGroupCols + c * 32;
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        const float o[8] = {v[j],     v[j + 1], v[j + 2], v[j + 3],
                                            v[j + 4], v[j + 5], v[j + 6], v[j + 7]};
                        Raw<float, 8>::put(dst + j, o);
                    }
                } else if constexpr (OV > 1) {
                    if constexpr (NP == 3) {
                        if (r0 < rows && col < ep.cols)
                            epilogue_warp_f32<OV>(ep, r0, rows, col, bvec, lane, v);
                    } else {
                        float z[32 / OV][OV];
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j / OV][j % OV] = v[j];
                        Pieces o{(r0 + lane) * ep.cols + col, OV, col, OV, 0u};
                        const int64_t left = (ep.cols - col) / OV;  // pieces before the last column
                        if (r0 + lane >= rows || left <= 0) return;
                        if (left >= 32 / OV) {
                            epilogue_pieces<T, OV, true>(ep, o, bvec, z);
                        } else {
                            o.in = (1u << left) - 1u;
                            epilogue_pieces<T, OV, false>(ep, o, bvec, z);
                        }
                    }
                } else {  // turned in shared memory: thread = column, so that rows are coalesced
#pragma unroll
                    for (int j = 0; j < 32; ++j) st[lane * 33 + j] = v[j];
                    __syncwarp();
#pragma unroll 1
                    for (int rr = 0; rr < 32; rr += 8) {
                        float z[8][1];
#pragma unroll
                        for (int p = 0; p < 8; ++p) z[p][0] = st[(rr + p) * 33 + lane];
                        const int64_t left = rows - (r0 + rr);
                        const uint32_t n = left <= 0 ? 0u : (left < 8 ? (1u << left) - 1u : 0xffu);
                        const Pieces o{(r0 + rr) * ep.cols + col + lane, ep.cols, col + lane, 0,
                                       col + lane < ep.cols ? n : 0u};
                        epilogue_pieces<T, 1, false>(ep, o, 0, z);
                    }
                    __syncwarp();
                }
            };
            // bf16: the bias of columns c0 + 32 c .. + 31, read while the columns before are
            // still in TMEM; behind their stores it would wait for them in the load and store
            // unit.  10000 x 768 of depth 4096: 52 us, 54 with the read in the epilogue; 65536 x
            // 128 of depth 1024: 48 and 55.  In fp32 the registers for it spill: 182 and 162.
            // Where the outputs go column by column a thread needs one column's bias: 1001 columns
            // 123 us, and 152 with the registers for 32.
            [[maybe_unused]] float b[32];
            [[maybe_unused]] auto fetch_bias = [&](int c) {
                if (bias == nullptr) return;
                const int64_t col = c0 + c * 32;
                if (bvec && col + 32 <= ep.cols) {
                    load_params<32>(bias + col, 1, b);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) b[j] = col + j < ep.cols ? bias[col + j] : 0.f;
                }
            };
            [[maybe_unused]] auto add_bias = [&](float (&v)[32]) {
                if (bias == nullptr) return;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __fadd_rn(v[j], b[j]);
            };
            if (kBiasAhead && un.part < 0) fetch_bias(0);
            // Where tiles follow one another fast, the next one's residual is brought into L2.
            // 65536 x 1024 of depth 128, bf16: 76 us, 86 without; fp32 202 and 218; but 10000 x
            // 4096 of depth 1536 103 and 101, and 2500 x 4096 of depth 768 in fp32 98 and 97.
            constexpr int kAhead = 12 / NP;  // chunks of the depth
            if (ep.R != nullptr && u + step < jobs.units && un.k1 - un.k0 <= kAhead) {
                const bool jn = u + step >= jobs.second;
                const Unit nx = jn ? unit_of(jobs.shape[1], u + step - jobs.second)
                                   : unit_of(jobs.shape[0], u + step);
                const int64_t row = nx.tr * (kBM * CG) + rank * kBM + q * 32 + lane;
                const int64_t col = nx.tc * BN + g * Cfg::kGroupCols;
                if (jn == j && row < rows) {
                    const T *p = static_cast<const T *>(ep.R) + row * ep.cols + col;
                    constexpr int kLine = 128 / static_cast<int>(sizeof(T));
#pragma unroll
                    for (int x = 0; x < Cfg::kGroupCols; x += kLine)
                        if (col + x < ep.cols) ptx::prefetch_l2(p + x);
                }
            }
            auto wait_acc = [&]() -> bool {
                uint32_t good = 0;
                if (lane == 0)
                    good = ptx::mbar_wait(&tfull[it & 1u], (it >> 1) & 1u, abort_flag, wait_ns);
                if (__shfl_sync(0xffffffffu, good, 0)) {
                    ptx::tc_fence_after();
                    return true;
                }
                if (lane == 0) gemm_timeout(abort_flag, err);
                return false;
            };
            auto acc_cols = [&] {
                return tmem + (static_cast<uint32_t>(q * 32) << 16) + (it & 1u) * Cfg::kAccCols +
                       g * Cfg::kGroupCols;
            };
            auto release = [&] {  // the accumulator is free again
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        ptx::mbar_arrive_cluster(tempty_c + (it & 1u) * 8);
                    else
                        ptx::mbar_arrive(&tempty[it & 1u]);
                }
            };
            if constexpr (NP == 1) {
                if (!(ok = wait_acc())) break;
                const uint32_t tb = acc_cols();
#pragma unroll 1
                for (int c = 0; c < C; ++c) {
                    __syncwarp();
                    float v[32];
                    ptx::tmem_ld32_sync(tb + c * 32, v);
                    if (c == C - 1) release();
                    if (kBiasAhead && un.part < 0) {
                        add_bias(v);
                        if (c + 1 < C) fetch_bias(c + 1);
                    }
                    finish(c, v);
                }
                ++it;
            } else {
                // run by run of the depth into registers, both accumulators of each
                float sum[C][32];
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
                for (int k = un.k0; k < un.k1; k += kRunChunks, ++it) {
                    if (!(ok = wait_acc())) break;
                    const uint32_t tb = acc_cols();
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        __syncwarp();
                        float v[32];
                        ptx::tmem_ld32_sync(tb + BN + c * 32, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c][j] += v[j];
                        __syncwarp();
                        ptx::tmem_ld32_sync(tb + c * 32, v);
                        if (c == C - 1) release();
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c][j] += v[j];
                    }
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < C; ++c) finish(c, sum[c]);
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    ptx::tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) {
        __syncwarp();
        ptx::cluster_sync();
    }
    if (*abort_flag) {  // give copies already in flight a moment to land (bounded)
        const uint64_t t0 = ptx::globaltimer_ns();
        while (ptx::globaltimer_ns() - t0 < 200000ull) {
        }
    }
    if (warp == 1) {
        ptx::tc_fence_after();
        if constexpr (CG == 2)
            ptx::tmem_dealloc_pair(tmem, Cfg::kTmemCols);
        else
            ptx::tmem_dealloc(tmem, Cfg::kTmemCols);
    }
}

// Join the partial products of the tail tiles, in order, and apply the epilogue.  Block (x,
// y): rows of tail tile x, those of the first product (`split0` of them) before the second's.
// Behind all `tiles`, blocks of column sums.  MANY: some product has more parts than kMaxSplits,
// and they are added run by run, as one after the other they would round as a long chain does.
template <typename T, int V, bool MANY>
__global__ void __launch_bounds__(256)
    gemm_join_kernel(const __grid_constant__ GemmJobs jobs, int split0, int tiles, int tile_rows,
                     int bn, const ColSums sums) {
    __shared__ float red[32][33];
    pdl_wait();
    pdl_trigger();
    if (static_cast<int>(blockIdx.x) >= tiles) {
        if (blockIdx.y == 0) join_columns<256>(sums, blockIdx.x - tiles, red);
        return;
    }
    const int job = static_cast<int>(blockIdx.x) >= split0;
    const int64_t tile = static_cast<int64_t>(blockIdx.x) - (job ? split0 : 0);
    const GemmShape &s = jobs.shape[job];
    int64_t tr, tc;
    tile_of(s, s.full + tile, tr, tc);
    const int64_t size = static_cast<int64_t>(tile_rows) * bn;
    const float *base = jobs.part[job] + tile * s.splits * size;
    const int per_row = bn / V;
    for (int t = blockIdx.y * 256 + threadIdx.x; t < tile_rows * per_row; t += gridDim.y * 256) {
        const int lr = t / per_row, lc = (t - lr * per_row) * V;
        const int64_t row = tr * tile_rows + lr, col = tc * bn + lc;
        if (row >= s.rows || col >= s.cols) continue;
        const Pieces o{row * s.cols + col, 0, col, 0, 1u};
        float z[1][V];
#pragma unroll
        for (int j = 0; j < V; ++j) z[0][j] = 0.f;
        const float *p = base + lr * bn + lc;
        auto add = [&](int i, float (&sum)[V]) {
            float f[V];
            load_params<V>(p + i * size, 1, f);
#pragma unroll
            for (int j = 0; j < V; ++j) sum[j] += f[j];
        };
        const int head = MANY && s.splits > kMaxSplits ? kMaxSplits : s.splits;
#pragma unroll 4
        for (int i = 0; i < head; ++i) add(i, z[0]);
        for (int i0 = head; MANY && i0 < s.splits; i0 += kMaxSplits) {
            float run[V] = {};
            for (int i = i0; i < s.splits && i < i0 + kMaxSplits; ++i) add(i, run);
#pragma unroll
            for (int j = 0; j < V; ++j) z[0][j] += run[j];
        }
        epilogue_pieces<T, V, true>(jobs.ep[job], o, jobs.bvec[job], z);
    }
}

// Map of an operand's planes [planes][outer][inner] (rows of ld), boxes of 64 x box_outer.
bool operand_map(CUtensorMap *m, const GemmOperand &o, int64_t outer, int64_t inner, int planes,
                 int box_outer) {
    auto fn = tmap_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                          static_cast<cuuint64_t>(planes)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * 2,
                             static_cast<cuuint64_t>(o.ld) * 2 * static_cast<cuuint64_t>(outer)};
    cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_outer), 1u};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(o.base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, int BN, typename T, int OV>
cudaError_t launch_cfg(const GemmArgs *args, const GemmPlan *plans, int n, const ColSums &sums,
                       cudaStream_t st) {
    using Cfg = GemmCfg<CG, BN, kPlanes<T>, OV>;
    auto kernel = gemm_kernel<CG, BN, T, OV>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = smem_opt_in(kernel, Cfg::kSmemBytes, smem_set);
    if (e != cudaSuccess) return e;
    GemmJobs jobs{};
    int64_t joined[kMaxProducts] = {};  // tail tiles to join
    bool many = false;
    for (int i = 0; i < n; ++i) {
        const GemmArgs &a = args[i];
        const GemmPlan &p = plans[i];
        const bool ok =
            (a.A.mn_major ? operand_map(&jobs.a[i], a.A, a.depth, a.rows, kPlanes<T>, 64)
                          : operand_map(&jobs.a[i], a.A, a.rows, a.depth, kPlanes<T>, kBM)) &&
            (a.B.mn_major ? operand_map(&jobs.b[i], a.B, a.depth, a.cols, kPlanes<T>, 64)
                          : operand_map(&jobs.b[i], a.B, a.cols, a.depth, kPlanes<T>, Cfg::kBRows));
        if (!ok) return cudaErrorInvalidValue;
        GemmShape &s = jobs.shape[i];
        s.rows = a.rows;
        s.cols = a.cols;
        s.nkc = static_cast<int>(ceil_div(a.depth, kBK));
        s.splits = p.splits;
        s.a_mn = a.A.mn_major;
        s.b_mn = a.B.mn_major;
        s.tiles_r = ceil_div(a.rows, kBM * CG);
        s.tiles_c = ceil_div(a.cols, BN);
        s.inv_band = ~uint64_t(0) / static_cast<uint64_t>(kBandRows * s.tiles_c);
        s.full = p.full;
        s.tail = p.tail;
        jobs.bvec[i] = aligned(a.bias, 16);
        jobs.part[i] = a.part;
        Epilogue &ep = jobs.ep[i];
        ep.bias = a.bias;
        ep.R = a.R;
        ep.C = a.C;
        ep.Z = a.Z;
        ep.cols = a.cols;
        ep.act = a.act;
        jobs.units += p.full + p.tail * p.splits;
        if (i == 0) jobs.second = jobs.units;
        joined[i] = p.splits > 1 ? p.tail : 0;
        many = many || p.splits > kMaxSplits;
    }
    const int64_t slots = device_sm_count() / CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(CG * (jobs.units < slots ? jobs.units : slots)));
    cfg.blockDim = dim3(Cfg::kThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, jobs, args[0].err, kDefaultWaitNs);
    if (e != cudaSuccess) return e;
    note_launch();
    const int64_t tiles = joined[0] + joined[1];
    if (tiles > 0) {
        constexpr int JV = OV > kVec<T> ? kVec<T> : OV;  // 16 bytes of output a thread
        const int64_t want = ceil_div(static_cast<int64_t>(device_sm_count()) * 8, tiles);
        const int64_t most = int64_t(kBM) * CG * BN / JV / 256;
        const auto join = many ? gemm_join_kernel<T, JV, true> : gemm_join_kernel<T, JV, false>;
        e = launch_pdl(join,
                       dim3(static_cast<unsigned>(tiles + ceil_div(sums.db ? sums.cols : 0, 32)),
                            static_cast<unsigned>(want < most ? want : most)),
                       dim3(256), 0, st, jobs, static_cast<int>(joined[0]),
                       static_cast<int>(tiles), kBM * CG, BN, sums);
        if (e == cudaSuccess) note_launch();
    }
    return e;
}

template <typename T, int OV>
cudaError_t launch_v(const GemmArgs *a, const GemmPlan *p, int n, const ColSums &sums,
                     cudaStream_t st) {
    // (fp32: two accumulators a tile, so half the columns)
    constexpr int kPairCols = 256 / (kPlanes<T> == 3 ? 2 : 1);
    if (p->cg == 2) return launch_cfg<2, kPairCols, T, OV>(a, p, n, sums, st);
    if (p->bn == 128) return launch_cfg<1, 128, T, OV>(a, p, n, sums, st);
    return launch_cfg<1, 64, T, OV>(a, p, n, sums, st);
}

template <typename T>
cudaError_t launch_t(const GemmArgs *a, const GemmPlan *p, int n, const ColSums &sums,
                     cudaStream_t st) {
    constexpr int V = kVec<T>;
    auto rows_on = [&](int v) {
        const size_t b = v * sizeof(T);
        bool ok = true;
        for (int i = 0; i < n; ++i)
            ok = ok && a[i].cols % v == 0 && aligned(a[i].C, b) && aligned(a[i].Z, b) &&
                 aligned(a[i].R, b);
        return ok;
    };
    if (rows_on(2 * V)) return launch_v<T, 2 * V>(a, p, n, sums, st);
    if (rows_on(V)) return launch_v<T, V>(a, p, n, sums, st);
    return launch_v<T, 1>(a, p, n, sums, st);
}

}  // namespace

// The cheapest cut by a model in SM cycles: a chunk of 64 of the depth takes the time its
// operands take to arrive (64 bytes a cycle and SM) or that of its products, whichever is
// longer.  bf16: 512 for the pair's 256 x 256 tile, 512 for 128 x 128, 384 for 128 x 64; three
// planes: 1536 for 256 x 128 and for 128 x 128, 1152 for 128 x 64.  The ring fills and the last
// accumulator empties once (about 4000).  Tiles run in waves of as many as the GPU holds;
// those of the last, partial wave may have their depth cut so that it is spread over the
// GPU, in parts of at least four chunks: that costs a launch (about 4000) and the partial
// products' way through L2 (about 3000 bytes a cycle).
// Several products share a tile shape: the one with the least cost in all.
void gemm_plan(const GemmSize *sizes, int n, fk_dtype dtype, GemmPlan *plans) {
    struct Choice {
        int cg, bn, cycles;
    };
    static constexpr Choice kBf16[3] = {{2, 256, 512}, {1, 128, 512}, {1, 64, 384}};
    static constexpr Choice kF32[3] = {{2, 128, 1536}, {1, 128, 1536}, {1, 64, 1152}};
    double best_all = -1;
    for (const Choice &c : dtype == FK_F32 ? kF32 : kBf16) {
        double all = 0;
        GemmPlan mine[kMaxProducts] = {};
        for (int i = 0; i < n; ++i) {
            const int64_t nkc = ceil_div(sizes[i].depth, kBK);
            const int64_t tiles =
                ceil_div(sizes[i].rows, kBM * c.cg) * ceil_div(sizes[i].cols, c.bn);
            const int64_t slots = 148 / c.cg;
            const auto cost = [&](const GemmPlan &p) {
                const double waves = static_cast<double>(p.full / slots);
                const double last = static_cast<double>(ceil_div(p.tail * p.splits, slots));
                double t = 4000 + (waves + last) * 500 +
                           (waves * nkc + last * ceil_div(nkc, p.splits)) * c.cycles;
                if (p.splits > 1)
                    t += 4000 + 8.0 * static_cast<double>(p.tail * p.splits * p.tile()) / 3000;
                return t;
            };
            GemmPlan p{c.cg, c.bn, 1, tiles / slots * slots, tiles % slots};
            const int deepest = dtype == FK_F32 ? kMaxF32Chunks : kMaxBf16Chunks;
            if (nkc > deepest) {  // every tile's depth in parts
                p.full = 0;
                p.tail = tiles;
                p.splits = static_cast<int>(ceil_div(nkc, deepest));
            }
            const int least = p.splits, most = least > kMaxSplits ? least : kMaxSplits;
            double best = -1;
            for (; p.splits <= most; ++p.splits) {
                if (p.splits > least && (p.tail == 0 || nkc / p.splits < 4)) break;
                const double t = cost(p);
                if (best < 0 || t < best) {
                    best = t;
                    mine[i] = p;
                }
            }
            all += best;
        }
        if (best_all < 0 || all < best_all) {
            best_all = all;
            for (int i = 0; i < n; ++i) plans[i] = mine[i];
        }
    }
}

cudaError_t launch_gemm(const GemmArgs *args, const GemmPlan *plans, int n, const ColSums &sums,
                        cudaStream_t st) {
    return args[0].dtype == FK_F32 ? launch_t<float>(args, plans, n, sums, st)
                                   : launch_t<uint16_t>(args, plans, n, sums, st);
}

}  // namespace fk
