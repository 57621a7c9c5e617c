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
// and N is the tile's number of tokens, rounded up to 16.  Weight blocks are packed as the
// tensor core reads them (128 rows x 128 bytes, 128-byte swizzle), one 16 KB copy per
// step; the tokens come through a tensor map, from row-major rows (dense; the copy
// swizzles) or from the layer's tiled rows (already swizzled).
//
// One persistent CTA per SM: a producer warp (TMA), an MMA warp (one elected thread
// issues) and 8 epilogue warps.  Steps are 128-wide K planes; two accumulators, so that a
// tile's epilogue overlaps the next tile's K loop.  Every wait is bounded.
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
// D[tmem] (+)= A[smem] * B[smem]^T, s8 x s8 -> s32, K = 32
__device__ __forceinline__ void mma_i8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Bounded wait on an mbarrier phase: false (with the CTA and the error word flagged) when
// it runs out or another role already gave up.
__device__ __forceinline__ bool w8_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                        long long limit) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait(bar, parity)) return true;
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
    int e, nt, row0, nrows;
};

// Work item u.  Grouped: row tile by row tile, weight tiles fastest, so that the CTAs at
// work share a row tile's tokens in L2.  Dense: blocks of 8 row tiles, row tiles fastest,
// so that the CTAs at work read about 8 row tiles and 18 weight tiles, which stay in L2
// together whatever M and N are.
__device__ __forceinline__ W8Tile w8_tile(int u, const W8Args& a) {
    W8Tile t;
    if (a.mt_tab != nullptr) {
        const int mt = u / a.NT;
        const int4 v = __ldg(a.mt_tab + mt);
        t.e = v.x;
        t.nt = u - mt * a.NT;
        t.row0 = v.y;
        t.nrows = v.z;
    } else {
        constexpr int kBlk = 8;
        const int nmt = ceil_div(a.M, a.BN);
        const int g = u / (kBlk * a.NT), i = u - g * kBlk * a.NT;
        const int size = min(kBlk, nmt - g * kBlk);
        const int mt = g * kBlk + i % size;
        t.e = 0;
        t.nt = i / size;
        t.row0 = mt * a.BN;
        t.nrows = min(a.BN, a.M - t.row0);
    }
    return t;
}

__device__ __forceinline__ float w8_silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

__device__ __forceinline__ uint16_t to_bits16(float v, int type) {
    return type == W8A8_F16 ? __half_as_ushort(__float2half_rn(v)) : bf16_bits(v);
}

__global__ void __launch_bounds__(kW8Threads, 1)
    gemm_w8a8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const W8Args a) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sA = base + kW8OffA, sB = base + kW8OffB;
    const uint32_t full = base + kW8OffBar, empty = full + 8 * kW8Stages;
    const uint32_t dfull = empty + 8 * kW8Stages, dempty = dfull + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kW8OffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kW8OffMisc + 4);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kW8Stages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(dfull + 8 * b, 1);
            mbar_init(dempty + 8 * b, kW8EpiWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kW8MmaWarp) {
        tmem_alloc(smem_u32(tmem_slot), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    grid_dep_wait();  // the previous kernel on the stream has completed
    const int total = a.NT * (a.mt_tab != nullptr ? __ldg(a.n_mtiles) : ceil_div(a.M, a.BN));
    const int G = a.G;

    if (warp == kW8ProdWarp) {
        // ---------------- producer ----------------
        if (lane == 0) {
            uint32_t j = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < total && ok; u += gridDim.x) {
                const W8Tile t = w8_tile(u, a);
                const int boxes = ceil_div(t.nrows, a.box_rows);
                const uint32_t bytes = (uint32_t)kW8BlockBytes + (uint32_t)(boxes * a.box_rows) * 128u;
                const int wrow = (t.e * a.NT + t.nt) * G * kTileRows;
                for (int g = 0; g < G; ++g, ++j) {
                    const uint32_t s = j % kW8Stages;
                    if (!w8_wait(empty + 8 * s, ((j / kW8Stages) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit)) { ok = false; break; }
                    // test hook: leave the first step's stage empty, so that its consumers time out
                    if (j == 0 && blockIdx.x == 0 && (a.debug & kDebugSkipFirstCopy)) continue;
                    mbar_arrive_expect_tx(full + 8 * s, bytes);
                    tma_load_2d(sA + s * kW8BlockBytes, &map_w, 0, wrow + g * kTileRows, full + 8 * s);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(sB + s * (kW8RowsB * 128) + (uint32_t)(b * a.box_rows) * 128u, &map_x, g * a.plane_x,
                                    t.row0 + b * a.box_rows + g * a.plane_y, full + 8 * s);
                }
            }
            // Never leave with a copy or a barrier arrival still on its way into this CTA's
            // shared memory: the stages' copies have landed, and (in a run without a
            // timeout) the MMAs that read them have reported back.
            const uint32_t first = j > (uint32_t)kW8Stages ? j - kW8Stages : 0u;
            for (uint32_t q = first; q < j; ++q) {
                w8_drain(full + 8 * (q % kW8Stages), (q / kW8Stages) & 1u, a.wait_limit);
                if (ok && !*abort_flag) w8_drain(empty + 8 * (q % kW8Stages), (q / kW8Stages) & 1u, a.wait_limit);
            }
        }
        __syncwarp();
    } else if (warp == kW8MmaWarp) {
        // ---------------- MMA issue ----------------
        uint32_t j = 0, tile = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < total && ok; u += gridDim.x, ++tile) {
            const W8Tile t = w8_tile(u, a);
            const uint32_t idesc = idesc_i8(128, round_up(t.nrows, 16));
            const uint32_t b = tile & 1u;
            const uint32_t d = tmem + b * 128u;
            if (!w8_wait(dempty + 8 * b, ((tile >> 1) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit)) break;
            tc_fence_after();
            for (int g = 0; g < G; ++g, ++j) {
                const uint32_t s = j % kW8Stages;
                if (!w8_wait(full + 8 * s, (j / kW8Stages) & 1u, abort_flag, a.err, a.wait_limit)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_i8_ss(d, smem_desc_sw128(sA + s * kW8BlockBytes + kk * 32),
                                  smem_desc_sw128(sB + s * (kW8RowsB * 128) + kk * 32), idesc, (g | kk) != 0);
                    tc_commit(empty + 8 * s);
                    if (g == G - 1) tc_commit(dfull + 8 * b);
                }
                __syncwarp();
            }
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3, half = warp >> 2;  // tensor-memory lane quarter; chunks of 32 tokens: even / odd
        const int r = q * 32 + lane;               // tile row = tensor-memory lane
        uint32_t tile = 0;
        for (int u = blockIdx.x; u < total; u += gridDim.x, ++tile) {
            const W8Tile t = w8_tile(u, a);
            const uint32_t b = tile & 1u;
            const float sw = __ldg(a.wscale + ((size_t)t.e * a.NT + t.nt) * kTileRows + r);
            const int n = t.nt * kTileRows + r;
            const float bias = (a.bias != nullptr && n < a.nvalid) ? __ldg(a.bias + n) : 0.f;
            if (!w8_wait(dfull + 8 * b, (tile >> 1) & 1u, abort_flag, a.err, a.wait_limit)) break;
            tc_fence_after();
            for (int c0 = half * 32; c0 < t.nrows; c0 += 64) {
                const int ncol = min(32, t.nrows - c0);  // tokens of this chunk
                const float sa = lane < ncol && a.act_scale != nullptr ? __ldg(a.act_scale + t.row0 + c0 + lane) : 0.f;
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + b * 128u + (uint32_t)c0, v);
                tmem_ld_wait();
                const size_t row = (size_t)(t.row0 + c0);
                if (a.mode == kW8Up) {
                    // even tile rows hold gate channel f, odd rows the matching up channel: per
                    // pair of tokens (i, i+1) the lanes of a pair swap one value, the even lane
                    // finishes token i, the odd lane token i+1
                    const int f = t.nt * (kTileRows / 2) + (r >> 1), odd = r & 1;
                    uint16_t* h = static_cast<uint16_t*>(a.out) + row * a.ldo + f;
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float p0 = __int2float_rn((int)v[i]) * sw, p1 = __int2float_rn((int)v[i + 1]) * sw;
                        const float recv = __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 1);
                        const float si = __shfl_sync(0xffffffffu, sa, i + odd);
                        const float gate = (odd ? recv : p0) * si, up = (odd ? p1 : recv) * si;
                        if (f < a.nvalid && i + odd < ncol) h[(size_t)(i + odd) * a.ldo] = bf16_bits(w8_silu_mul(gate, up));
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
            if (lane == 0) mbar_arrive(dempty + 8 * b);
        }
    }

    __syncthreads();
    if (warp == kW8MmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
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

int w8_tile_tokens(int avg_tokens_per_group) {
    (void)avg_tokens_per_group;
    return 128;
}

cudaError_t launch_gemm_w8a8(W8Args a, const W8Operands& op, int num_ctas, cudaStream_t stream) {
    static std::mutex mu;
    static bool attr_done[64] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !attr_done[dev]) {
            e = cudaFuncSetAttribute(gemm_w8a8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kW8Smem);
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) attr_done[dev] = true;
        }
    }
    CUtensorMap mw, mx;
    e = make_map(&mw, op.wblocks, 128, (uint64_t)op.matrices * a.NT * a.G * kTileRows, 128, kTileRows, false);
    if (e != cudaSuccess) return e;
    a.box_rows = 16;
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
    return launch_pdl(gemm_w8a8_kernel, num_ctas, kW8Threads, kW8Smem, stream, mw, mx, a);
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
