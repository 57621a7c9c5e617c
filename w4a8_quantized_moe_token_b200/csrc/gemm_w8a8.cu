// W8A8 GEMM for sm_100a: INT8 weights (one fp32 scale per output channel) x INT8 tokens
// (one fp32 scale per token), dense or grouped by expert, on the 5th-generation tensor
// cores.
//
// Mathematics: y[m][n] = sa[m] * sw[n] * sum_k qa[m][k] * qw[n][k].  The sum is an exact
// INT32 (K <= 2^17), so it may be cut anywhere along K and added in any order; both
// scales leave the sum, so one accumulator per tile lives in tensor memory for the whole
// K loop and the CUDA cores see each value once, in the epilogue.
//
// Weights take the MMA's M slot ("swap AB"): 128 output channels per CTA are always full,
// and N is the tile's number of tokens.  Weight blocks are packed as the tensor core reads
// them (128 rows x 128 bytes, 128-byte swizzle), one 16 KB copy per step; the tokens come
// through a tensor map, from row-major rows (dense; the copy swizzles) or from the layer's
// tiled rows (already swizzled).
//
// Two instances.  CG = 1: a CTA's tile is 128 channels x up to 128 tokens; what few tokens
// need, weights streamed from HBM.  CG = 2: a pair of CTAs (cta_group::2) works on 256
// channels x up to 256 tokens, each CTA holding its 128 channels and half of the tokens, so
// that a step of 2 x 128 x 256 x 128 products reads 32 KB per SM instead of the 48 KB that
// 128 x 256 alone would: at full rate (512 cycles a step) 64 bytes per cycle and SM.
//
// One persistent CTA per SM: a producer warp (TMA), an MMA warp (one elected thread issues,
// in the pair's first CTA) and 8 epilogue warps.  Steps are 128-wide K planes; two
// accumulators, so that a tile's epilogue overlaps the next tile's K loop.  Every wait is
// bounded.
#include <cuda.h>

#include <mutex>

#include "../../include/w8a8.h"
#include "w4a8_common.cuh"
#include "w8a8_internal.h"

namespace w4a8 {

namespace {

constexpr int kW8Stages = 7;
constexpr int kW8EpiWarps = 8;
constexpr int kW8ProdWarp = kW8EpiWarps;
constexpr int kW8MmaWarp = kW8EpiWarps + 1;
constexpr int kW8Threads = 32 * (kW8EpiWarps + 2);
constexpr int kW8RowsB = 128;                      // token rows per CTA and stage at most
constexpr int kW8OffA = 0;                         // 1024-aligned (swizzle atoms)
constexpr int kW8OffB = kW8OffA + kW8Stages * kW8BlockBytes;
constexpr int kW8OffBar = kW8OffB + kW8Stages * kW8RowsB * 128;
constexpr int kW8NumBars = 2 * kW8Stages + 4;      // full, empty, 2 x accumulator full / empty
constexpr int kW8OffMisc = kW8OffBar + kW8NumBars * 8;
constexpr int kW8Smem = kW8OffMisc + 16 + 1024;    // + alignment slack
static_assert(kW8Smem <= 227 * 1024, "shared memory over-subscribed");

// ---- PTX ----
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// the same for one CTA of a pair: `bar` may be the other CTA's
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T, s8 x s8 -> s32, K = 32
template <int CG>
__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// arrive on `bar` (in a pair: on both CTAs' barrier at that offset) when the MMAs issued so
// far by this thread are complete
template <int CG>
__device__ __forceinline__ void w8_commit(uint32_t bar) {
    if (CG == 1)
        tc_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// mbar_try_wait for a barrier that the other CTA of the pair arrives on
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
template <int CG>
__device__ __forceinline__ void w8_tmem_alloc(uint32_t dst, uint32_t cols) {
    if (CG == 1) {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void w8_tmem_dealloc(uint32_t addr, uint32_t cols) {
    if (CG == 1)
        tmem_dealloc(addr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// Bounded wait on an mbarrier phase: false (with the CTA and the error word flagged) when
// it runs out or another role already gave up.
template <bool kCluster = false>
__device__ __forceinline__ bool w8_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                        long long limit) {
    if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t n = 1;; ++n) {
        if (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((n & 15u) == 0) {
            if (*abort_flag) return false;
            if (clock64() - t0 > limit) {
                *abort_flag = 1;
                atomicOr(err, kErrTimeout);
                return false;
            }
        }
    }
}

// bounded wait without the abort bookkeeping, for draining at exit
__device__ __forceinline__ void w8_drain(uint32_t bar, uint32_t parity, long long limit) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > limit) return;
}

struct W8Tile {
    int e, nt, row0, nrows;  // nt: weight tile of this CTA
};

// Work item u of a CTA (or pair).  Grouped: row tile by row tile, weight tiles fastest, so
// that the CTAs at work share a row tile's tokens in L2.  Dense: blocks of 8 row tiles, row
// tiles fastest, so that the CTAs at work read about 8 row tiles and 9 (18) weight tiles,
// which stay in L2 together whatever M and N are.
template <int CG>
__device__ __forceinline__ W8Tile w8_tile(int u, const W8Args& a, uint32_t rank) {
    const int NP = (a.NT + CG - 1) / CG;
    W8Tile t;
    if (a.mt_tab != nullptr) {
        const int mt = u / NP;
        const int4 v = __ldg(a.mt_tab + mt);
        t.e = v.x;
        t.nt = (u - mt * NP) * CG + (int)rank;
        t.row0 = v.y;
        t.nrows = v.z;
    } else {
        constexpr int kBlk = 8;
        const int nmt = ceil_div(a.M, a.BN);
        const int g = u / (kBlk * NP), i = u - g * kBlk * NP;
        const int size = min(kBlk, nmt - g * kBlk);
        const int mt = g * kBlk + i % size;
        t.e = 0;
        t.nt = i / size * CG + (int)rank;
        t.row0 = mt * a.BN;
        t.nrows = min(a.BN, a.M - t.row0);
    }
    return t;
}

__device__ __forceinline__ float w8_silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ uint16_t to_bits16(float v, int type) {
    return type == W8A8_F16 ? __half_as_ushort(__float2half_rn(v)) : bf16_bits(v);
}

template <int CG>
__global__ void __launch_bounds__(kW8Threads, 1)
    gemm_w8a8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const W8Args a) {
    constexpr uint32_t kAccCols = 128 * CG;  // columns of one of the two accumulators
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();
    const uint32_t sA = base + kW8OffA, sB = base + kW8OffB;
    const uint32_t full = base + kW8OffBar, empty = full + 8 * kW8Stages;
    const uint32_t dfull = empty + 8 * kW8Stages, dempty = dfull + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kW8OffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kW8OffMisc + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kW8Stages; ++s) {
            mbar_init(full + 8 * s, 1);   // a pair's copies all report to its first CTA
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(dfull + 8 * b, 1);
            mbar_init(dempty + 8 * b, kW8EpiWarps * CG);  // in the first CTA, from both
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kW8MmaWarp) w8_tmem_alloc<CG>(smem_u32(tmem_slot), 2 * kAccCols);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    grid_dep_wait();  // the previous kernel on the stream has completed
    const int total = ceil_div(a.NT, CG) * (a.mt_tab != nullptr ? __ldg(a.n_mtiles) : ceil_div(a.M, a.BN));
    const int G = a.G;
    const int u0 = (int)blockIdx.x / CG, du = (int)gridDim.x / CG;

    if (warp == kW8ProdWarp) {
        // ---------------- producer ----------------
        if (lane == 0) {
            uint32_t j = 0;
            bool ok = true;
            for (int u = u0; u < total && ok; u += du) {
                const W8Tile t = w8_tile<CG>(u, a, rank);
                // this CTA's token rows: all of them, or half of the tile's N
                const int rows = CG == 1 ? t.nrows : round_up(t.nrows, 32) / 2;
                const int row0 = t.row0 + (int)rank * rows;
                const int boxes = ceil_div(rows, a.box_rows);
                const uint32_t bytes = (uint32_t)kW8BlockBytes + (uint32_t)(boxes * a.box_rows) * 128u;
                // (a pair's second tile may lie past the last one: read that one again)
                const int wrow = (t.e * a.NT + min(t.nt, a.NT - 1)) * G * kTileRows;
                for (int g = 0; g < G; ++g, ++j) {
                    const uint32_t s = j % kW8Stages;
                    if (!w8_wait(empty + 8 * s, ((j / kW8Stages) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit)) { ok = false; break; }
                    // test hook: leave the first step's stage empty, so that its consumers time out
                    if (j == 0 && blockIdx.x == 0 && (a.debug & kDebugSkipFirstCopy)) continue;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes * CG);
                    const uint32_t bar = CG == 1 ? full + 8 * s : mapa(full + 8 * s, 0);
                    const auto load = CG == 1 ? tma_load_2d : tma_load_2d_pair;
                    load(sA + s * kW8BlockBytes, &map_w, 0, wrow + g * kTileRows, bar);
                    for (int b = 0; b < boxes; ++b)
                        load(sB + s * (kW8RowsB * 128) + (uint32_t)(b * a.box_rows) * 128u, &map_x, g * a.plane_x,
                             row0 + b * a.box_rows + g * a.plane_y, bar);
                }
            }
            // Never leave with a copy or a barrier arrival still on its way into this CTA's
            // shared memory: the stages' copies have landed, and (in a run without a
            // timeout) the MMAs that read them have reported back.
            const uint32_t first = j > (uint32_t)kW8Stages ? j - kW8Stages : 0u;
            for (uint32_t q = first; q < j; ++q) {
                if (rank == 0) w8_drain(full + 8 * (q % kW8Stages), (q / kW8Stages) & 1u, a.wait_limit);
                if (ok && !*abort_flag) w8_drain(empty + 8 * (q % kW8Stages), (q / kW8Stages) & 1u, a.wait_limit);
            }
        }
        __syncwarp();
    } else if (warp == kW8MmaWarp) {
        // ---------------- MMA issue (the pair's first CTA) ----------------
        uint32_t j = 0, tile = 0;
        bool ok = rank == 0;
        for (int u = u0; u < total && ok; u += du, ++tile) {
            const W8Tile t = w8_tile<CG>(u, a, rank);
            const uint32_t idesc = idesc_i8(128 * CG, round_up(t.nrows, 16 * CG));
            const uint32_t b = tile & 1u;
            const uint32_t d = tmem + b * kAccCols;
            if (!w8_wait<CG == 2>(dempty + 8 * b, ((tile >> 1) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit)) break;
            tc_fence_after();
            for (int g = 0; g < G; ++g, ++j) {
                const uint32_t s = j % kW8Stages;
                if (!w8_wait<CG == 2>(full + 8 * s, (j / kW8Stages) & 1u, abort_flag, a.err, a.wait_limit)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_i8_ss<CG>(d, smem_desc_sw128(sA + s * kW8BlockBytes + kk * 32),
                                      smem_desc_sw128(sB + s * (kW8RowsB * 128) + kk * 32), idesc, (g | kk) != 0);
                    w8_commit<CG>(empty + 8 * s);
                    if (g == G - 1) w8_commit<CG>(dfull + 8 * b);
                }
                __syncwarp();
            }
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3, half = warp >> 2;  // tensor-memory lane quarter; chunks of 32 tokens: even / odd
        const int r = q * 32 + lane;               // tile row = tensor-memory lane
        const int odd = lane & 1;
        uint32_t tile = 0;
        for (int u = u0; u < total; u += du, ++tile) {
            const W8Tile t = w8_tile<CG>(u, a, rank);
            const uint32_t b = tile & 1u;
            const float sw = t.nt < a.NT ? __ldg(a.wscale + ((size_t)t.e * a.NT + t.nt) * kTileRows + r) : 0.f;
            // output column: channel n (past the last tile: none valid)
            const int n = a.mode == kW8Up ? t.nt * (kTileRows / 2) + (r >> 1) : t.nt * kTileRows + r;
            const float bias = (a.bias != nullptr && n < a.nvalid) ? __ldg(a.bias + n) : 0.f;
            if (!w8_wait(dfull + 8 * b, (tile >> 1) & 1u, abort_flag, a.err, a.wait_limit)) break;
            tc_fence_after();
            for (int c0 = half * 32; c0 < t.nrows; c0 += 64) {
                const int ncol = min(32, t.nrows - c0);  // tokens of this chunk
                const float sa = lane < ncol && a.act_scale != nullptr ? __ldg(a.act_scale + t.row0 + c0 + lane) : 0.f;
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + b * kAccCols + (uint32_t)c0, v);
                tmem_ld_wait();
                const size_t row = (size_t)(t.row0 + c0);
                if (a.mode == kW8Up) {
                    // even tile rows hold gate channel f, odd rows the matching up channel: per
                    // pair of tokens (i, i+1) the lanes of a pair swap one value, the even lane
                    // finishes token i, the odd lane token i+1
                    uint16_t* h = static_cast<uint16_t*>(a.out) + (row + odd) * a.ldo + n;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float p0 = __int2float_rn((int)v[i]) * sw, p1 = __int2float_rn((int)v[i + 1]) * sw;
                        const float recv = __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 1);
                        const float si = __shfl_sync(0xffffffffu, sa, i + odd);
                        const float gate = (odd ? recv : p0) * si, up = (odd ? p1 : recv) * si;
                        if (n < a.nvalid && i + odd < ncol) h[(size_t)i * a.ldo] = bf16_bits(w8_silu_mul(gate, up));
                    }
                } else if (a.out_type == W8A8_F32) {
                    float* y = static_cast<float*>(a.out) + row * a.ldo + n;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float si = __shfl_sync(0xffffffffu, sa, i);
                        if (n < a.nvalid && i < ncol) y[(size_t)i * a.ldo] = __int2float_rn((int)v[i]) * (sw * si) + bias;
                    }
                } else if (a.out_type == W8A8_I32) {
                    int32_t* y = static_cast<int32_t*>(a.out) + row * a.ldo + n;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (n < a.nvalid && i < ncol) y[(size_t)i * a.ldo] = (int32_t)v[i];
                } else if (a.pairs) {
                    // two channels per store: the lanes of a pair swap one value per pair of
                    // tokens, the even lane stores token i, the odd lane token i+1
                    uint16_t* y = static_cast<uint16_t*>(a.out) + (row + odd) * a.ldo + (n - odd);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float p0 = __int2float_rn((int)v[i]) * (sw * __shfl_sync(0xffffffffu, sa, i)) + bias;
                        const float p1 = __int2float_rn((int)v[i + 1]) * (sw * __shfl_sync(0xffffffffu, sa, i + 1)) + bias;
                        const float recv = __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 1);
                        const uint32_t lo = to_bits16(odd ? recv : p0, a.out_type), hi = to_bits16(odd ? p1 : recv, a.out_type);
                        if (n < a.nvalid && i + odd < ncol)
                            *reinterpret_cast<uint32_t*>(y + (size_t)i * a.ldo) = lo | (hi << 16);
                    }
                } else {
                    uint16_t* y = static_cast<uint16_t*>(a.out) + row * a.ldo + n;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float si = __shfl_sync(0xffffffffu, sa, i);
                        if (n < a.nvalid && i < ncol)
                            y[(size_t)i * a.ldo] = to_bits16(__int2float_rn((int)v[i]) * (sw * si) + bias, a.out_type);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 1)
                    mbar_arrive(dempty + 8 * b);
                else
                    mbar_arrive_cluster(mapa(dempty + 8 * b, 0));
            }
        }
    }

    __syncthreads();
    if (CG == 2) {
        // after a timeout the pair's copies and arrivals are not accounted for: give them
        // ample time (50 us) to land before either CTA's shared memory goes away
        if (*abort_flag) {
            const long long t0 = clock64();
            while (clock64() - t0 < 100000) {
            }
        }
        cluster_sync();
    }
    if (warp == kW8MmaWarp) {
        tc_fence_after();
        w8_tmem_dealloc<CG>(tmem, 2 * kAccCols);
    }
}

// ---------------------------------------------------------------------------
// Weight quantisation and packing: one warp per tile row.  A first pass over the row
// finds max|w|, a second one (from cache) writes the codes into the row's 128-byte line
// of every plane block.  Reads the weights once from memory and writes half as many bytes.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) pack_w8_kernel(const uint16_t* __restrict__ w, int E, int N, int K, int layout,
                                                      int NT, int G, float* __restrict__ scales,
                                                      uint8_t* __restrict__ blocks, int8_t* __restrict__ codes_out,
                                                      float* __restrict__ scale_out, PackHeader* __restrict__ header) {
    const long long id = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);  // (matrix, tile, row)
    const int lane = threadIdx.x & 31;
    if (id == 0 && lane == 0) {
        PackHeader h = {};
        h.magic = kW8PackMagic;
        h.version = 1;
        h.layout = (uint32_t)layout;
        h.E = (uint32_t)E;
        h.N = (uint32_t)N;
        h.K = (uint32_t)K;
        h.Kp = (uint32_t)(G * kGroup);
        h.G = (uint32_t)G;
        h.NT = (uint32_t)NT;
        h.rows_per_tile = kTileRows;
        h.block_bytes = kW8BlockBytes;
        h.group = 0;
        *header = h;
    }
    if (id >= (long long)E * NT * kTileRows) return;
    const int r = (int)(id % kTileRows);
    const long long tile = id / kTileRows;  // e * NT + t
    const int e = (int)(tile / NT), t = (int)(tile % NT);
    int src;
    bool valid;
    if (layout == W4A8_LAYOUT_GATEUP) {  // even tile rows gate channel f, odd rows up channel f
        const int F = N / 2, f = t * (kTileRows / 2) + (r >> 1);
        valid = f < F;
        src = (r & 1) ? F + f : f;
    } else {
        src = t * kTileRows + r;
        valid = src < N;
    }
    const uint16_t* row = valid ? w + ((size_t)e * N + src) * (size_t)K : nullptr;
    const bool vec = (K & 7) == 0;
    float v[16];
    auto load16 = [&](int k0) {
        if (vec && k0 + 16 <= K) {
            const uint4 p[2] = {*reinterpret_cast<const uint4*>(row + k0), *reinterpret_cast<const uint4*>(row + k0 + 8)};
            const uint32_t* pw = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[2 * i] = __uint_as_float(pw[i] << 16);
                v[2 * i + 1] = __uint_as_float(pw[i] & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = k0 + i < K ? __uint_as_float((uint32_t)row[k0 + i] << 16) : 0.f;
        }
    };
    float amax = 0.f;
    if (valid) {
        for (int ci = lane; ci < G * 8; ci += 32) {
            load16(ci * 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float sc = __fmul_rn(amax, kInv127);
    const float rinv = __fdiv_rn(1.0f, sc);
    for (int ci = lane; ci < G * 8; ci += 32) {
        uint32_t out[4] = {0u, 0u, 0u, 0u};
        if (valid && amax > 0.f) {
            load16(ci * 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) out[i >> 2] |= (uint32_t)(quant_i8_fast(v[i], sc, rinv) & 0xFF) << (8 * (i & 3));
        }
        const uint4 o = make_uint4(out[0], out[1], out[2], out[3]);
        *reinterpret_cast<uint4*>(blocks + (tile * G + ci / 8) * (size_t)kW8BlockBytes + act_tiled_offset(r, (ci & 7) * 16)) = o;
        if (valid && codes_out != nullptr)
            *reinterpret_cast<uint4*>(codes_out + ((size_t)e * N + src) * (size_t)(G * kGroup) + (size_t)ci * 16) = o;
    }
    if (lane == 0) {
        scales[id] = sc;
        if (valid && scale_out != nullptr) scale_out[(size_t)e * N + src] = sc;
    }
}

// cuTensorMapEncodeTiled, looked up in the driver once
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// rows of `width` bytes, `pitch` bytes apart, copied in boxes of 128 bytes x box_rows
cudaError_t make_map(CUtensorMap* m, const void* base, uint64_t width, uint64_t rows, uint64_t pitch, uint32_t box_rows,
                     bool swizzle) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {width, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {128, box_rows}, steps[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

}  // namespace

namespace {

template <int CG>
cudaError_t launch_instance(const CUtensorMap& mw, const CUtensorMap& mx, const W8Args& a, int num_ctas, cudaStream_t stream) {
    const auto kernel = gemm_w8a8_kernel<CG>;
    static std::mutex mu;
    static int clusters[64] = {0};  // per device: pairs that fit at once (CG = 2), 1 once prepared
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = num_ctas / CG * CG;
    cfg.blockDim = kW8Threads;
    cfg.dynamicSmemBytes = kW8Smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 1 ? 1 : 2;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (clusters[dev] == 0) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kW8Smem);
            if (e != cudaSuccess) return e;
            int n = 1;
            if (CG == 2) {
                cudaLaunchConfig_t q = cfg;
                q.attrs = attr + 1;
                q.numAttrs = 1;
                e = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
                if (e != cudaSuccess) return e;
                if (n < 1) return cudaErrorInvalidConfiguration;
            }
            clusters[dev] = n;
        }
        if (CG == 2 && (int)cfg.gridDim.x > clusters[dev] * CG) cfg.gridDim = clusters[dev] * CG;
    }
    return cudaLaunchKernelEx(&cfg, kernel, mw, mx, a);
}

}  // namespace

W8Plan w8_plan_grouped(int avg_tokens) {
    if (avg_tokens < 64) return {1, 128};
    const int want = avg_tokens + avg_tokens / 10;  // most experts' rows in equal tiles
    const int tiles = ceil_div(want, 256);
    return {2, round_up(ceil_div(want, tiles), 32)};
}

W8Plan w8_plan_dense(int M, int NT, int num_ctas) {
    if (M <= 128) return {1, round_up(M, 16)};
    W8Plan best = {2, 256};
    long long best_cost = 0;
    for (int bn = 256; bn >= 64; bn -= 32) {
        const long long tiles = (long long)ceil_div(M, bn) * ceil_div(NT, 2);
        const long long cost = (tiles + num_ctas / 2 - 1) / (num_ctas / 2) * (bn + 64);
        if (best_cost == 0 || cost < best_cost) {
            best_cost = cost;
            best = {2, bn};
        }
    }
    return best;
}

cudaError_t launch_gemm_w8a8(W8Args a, const W8Operands& op, int num_ctas, cudaStream_t stream) {
    CUtensorMap mw, mx;
    cudaError_t e = make_map(&mw, op.wblocks, 128, (uint64_t)op.matrices * a.NT * a.G * kTileRows, 128, kTileRows, false);
    if (e != cudaSuccess) return e;
    a.box_rows = op.cg == 1 ? 16 : 32;
    if (a.mt_tab != nullptr) {
        // tiled rows [G][rows][128]
        a.plane_x = 0;
        a.plane_y = op.x_rows;
        e = make_map(&mx, op.x, 128, (uint64_t)op.x_rows * a.G, 128, (uint32_t)a.box_rows, false);
    } else {
        // row-major rows of G * 128 bytes
        a.plane_x = 128;
        a.plane_y = 0;
        e = make_map(&mx, op.x, (uint64_t)a.G * 128, (uint64_t)op.x_rows, (uint64_t)a.G * 128, (uint32_t)a.box_rows, true);
    }
    if (e != cudaSuccess) return e;
    a.pairs = a.ldo % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
    return op.cg == 1 ? launch_instance<1>(mw, mx, a, num_ctas, stream) : launch_instance<2>(mw, mx, a, num_ctas, stream);
}

cudaError_t launch_pack_w8(const uint16_t* w, int E, int N, int K, int layout, uint8_t* packed, int8_t* codes, float* scale,
                           cudaStream_t stream) {
    const int NT = w8_tiles(N, layout), G = ceil_div(K, kGroup);
    float* scales = reinterpret_cast<float*>(packed + kHeaderBytes);
    uint8_t* blocks = packed + w8_blocks_offset(E, NT);
    const long long rows = (long long)E * NT * kTileRows;
    pack_w8_kernel<<<(unsigned)(rows / 8), 256, 0, stream>>>(w, E, N, K, layout, NT, G, scales, blocks, codes, scale,
                                                            reinterpret_cast<PackHeader*>(packed));
    return cudaGetLastError();
}

}  // namespace w4a8
