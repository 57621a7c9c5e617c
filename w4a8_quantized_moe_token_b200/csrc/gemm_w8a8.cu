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
// One persistent CTA per SM: producer warps (TMA; a thread's time per step is a fixed few
// hundred cycles, longer than a step's arithmetic, so they take steps in turn), an MMA warp
// (one elected thread issues, in the pair's first CTA) and 8 epilogue warps.  Steps are
// 128-wide K planes; two accumulators, so that a tile's epilogue overlaps the next tile's K
// loop.  Every wait is bounded.
//
// Measured on B200.  16384 x 7168 -> 4096 (bf16 out): 285 us alone (3375 TOPS), 330-346 us
// repeated without a pause, when the power limit lowers the clock (tensor pipe 88 % active:
// bound by it, and by power).  64 tokens, 6 of 64 experts, H 4096, F 1408: up 117 us, 97 % of
// the measured copy rate, down 64 us, 88 % (bound by HBM).  One row, 2048 -> 7168: 6.0 us in a
// graph, of which the weights' 14.7 MB are 2.3 (bound by start-up and latency).
#include <cuda.h>

#include <mutex>

#include "../../include/w8a8.h"
#include "layer_internal.h"
#include "w4a8_common.cuh"
#include "w8a8_internal.h"

namespace w4a8 {

namespace {

constexpr int kW8EpiWarps = 8;
constexpr int kW8Producers = 2;
constexpr int kW8ProdWarp = kW8EpiWarps;
constexpr int kW8MmaWarp = kW8ProdWarp + kW8Producers;
constexpr int kW8Threads = 32 * (kW8MmaWarp + 1);
constexpr int kW8MaxStages = 12;
// shared memory: ns weight blocks, ns token blocks (both 1024-aligned: swizzle atoms), the
// receive buffer of a K split, barriers (full, empty, 2 x accumulator full / empty, receive),
// token scales
constexpr int kW8BarBytes = (2 * kW8MaxStages + 5) * 8 + 16 + kW8EpiWarps * 32 * 4;  // + token scales
constexpr int kW8SmemMax = 227 * 1024 - 1024;  // without the alignment slack
constexpr int kW8SplitSmem = 48 * 1024;        // five do not fit into an SM's 228 KB
inline int w8_smem(int ns, int b_stage, int recv) { return ns * (kW8BlockBytes + b_stage) + recv + kW8BarBytes + 1024; }

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
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// 16 bytes into another CTA's shared memory, reported to that CTA's barrier as such
__device__ __forceinline__ void st_async4(uint32_t cluster_addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w,
                                          uint32_t cluster_bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_addr),
                 "r"(x), "r"(y), "r"(z), "r"(w), "r"(cluster_bar)
                 : "memory");
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
template <bool kCluster>
__device__ __forceinline__ bool w8_test(uint32_t bar, uint32_t parity) {
    if (!kCluster) return mbar_test(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
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
                if (err != nullptr) atomicOr(err, kErrTimeout);
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

// tokens of a tile that each CTA of a K split finishes
__host__ __device__ inline int w8_tokens_per_part(int nrows, int parts) { return round_up(ceil_div(nrows, parts), 4); }

struct W8Tile {
    int e, nt, row0, nrows;  // nt: weight tile of this CTA
};

// Work item u of a CTA (or pair).  Grouped: row tile by row tile, weight tiles fastest, so
// that the CTAs at work share a row tile's tokens in L2.  Dense: blocks of 8 row tiles, row
// tiles fastest, so that the CTAs at work read about 8 row tiles and 9 (18) weight tiles,
// which stay in L2 together whatever M and N are.
template <int CG>
__device__ __forceinline__ W8Tile w8_tile(int u, const W8Args& a, uint32_t rank) {
    const int NP = a.NP;
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
        const int g = u / (kBlk * NP), i = u - g * kBlk * NP;
        const int size = min(kBlk, a.nmt - g * kBlk);
        const int mt = g * kBlk + i % size;
        t.e = 0;
        t.nt = i / size * CG + (int)rank;
        t.row0 = mt * a.BN;
        t.nrows = min(a.BN, a.M - t.row0);
    }
    return t;
}

// silu(g) * u = g / (1 + exp(-g)) * u, or g * exp(g) * u where exp(-g) alone counts (g < -64),
// within 7 roundings of fp32: expf (2 ulp), not __expf, whose error grows with |g|; a quotient
// corrected once by its residual (Markstein's method, for divisors between 1 and 2^93), not
// __fdividef, which returns 0 for divisors above 2^126.  Coarser, h rounds to another bf16 value
// now and then and its INT8 code follows.  (No __fdiv_rn: its branch keeps the values'
// arithmetic from overlapping.  Up projection, 600 tokens, 4 of 16 experts, H and F 2048: this
// 43.7 us, __fdiv_rn 51, the coarse form 40.9; H of 4096 and more: within 1 %.)
__device__ __forceinline__ float w8_silu_mul(float g, float u) {
    const bool far = g < -64.0f;
    const float e = expf(far ? g : -g);
    const float n = far ? g * e : g, d = far ? 1.0f : 1.0f + e;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    const float q = n * r;
    return __fmaf_rn(__fmaf_rn(-q, d, n), r, q) * u;
}

// A sum with the token's and the channel's scale, one after the other: |sum| >= 1, or 0, so that
// small scales cost no bits before the last product (the scales' own product may lie below
// fp32's range, or above it, where the result does not)
__device__ __forceinline__ float scaled(uint32_t sum, float sa, float sw) { return __int2float_rn((int)sum) * sa * sw; }

// Output kinds of the epilogue.  kOutPair: 16-bit rows that may be stored two columns at a time.
enum { kOutF32, kOutI32, kOutBf16, kOutF16, kOutPairBf16, kOutPairF16, kOutSwiglu };

template <int kOut>
__device__ __forceinline__ uint16_t to_bits16(float v) {
    return kOut == kOutF16 || kOut == kOutPairF16 ? __half_as_ushort(__float2half_rn(v)) : bf16_bits(v);
}

// predicated stores: a branch around each would keep the values' arithmetic from overlapping
// (SwiGLU tiles of 16 K planes 55.8 against 43.5 us)
__device__ __forceinline__ void st_if(bool p, void* at, uint32_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b32 [%0], %1;\n\t}" ::"l"(at), "r"(v), "r"((int)p)
                 : "memory");
}
__device__ __forceinline__ void st_if(bool p, void* at, uint16_t v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p st.global.b16 [%0], %1;\n\t}" ::"l"(at), "h"(v), "r"((int)p)
                 : "memory");
}

// One chunk of 16 tokens of this lane's channel: v[i] is token i's INT32 sum, sa[i] its scale
// (shared memory).  `out`: this lane's element of the chunk's first row (kOutPair: column
// n - odd of row `odd`; SwiGLU: column f of row `odd`), `pitch` bytes per row; the first ncol
// tokens exist.  Short on purpose, and called in a loop that is not unrolled: with 32 tokens
// and everything unrolled the epilogue waited for its instructions more than for anything
// else.
template <int kOut>
__device__ __forceinline__ void w8_store(const uint32_t (&v)[16], float sw, float bias, const float* sa, int ncol, bool valid,
                                         int odd, char* out, size_t pitch) {
    float s[16];
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        const float4 s4 = *reinterpret_cast<const float4*>(sa + i);
        s[i] = s4.x; s[i + 1] = s4.y; s[i + 2] = s4.z; s[i + 3] = s4.w;
    }
    if (kOut == kOutF32 || kOut == kOutI32 || kOut == kOutBf16 || kOut == kOutF16) {
#pragma unroll
        for (int i = 0; i < 16; ++i, out += pitch) {
            const float y = kOut == kOutI32 ? 0.f : scaled(v[i], s[i], sw) + bias;
            const bool p = valid && i < ncol;
            if (kOut == kOutF32) st_if(p, out, __float_as_uint(y));
            else if (kOut == kOutI32) st_if(p, out, v[i]);
            else st_if(p, out, to_bits16<kOut>(y));
        }
    } else if (kOut != kOutSwiglu) {
        // the lanes of a pair swap one value per pair of tokens: the even lane stores two
        // channels of token i, the odd lane of token i + 1
        float own[8], recv[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float p0 = scaled(v[i], s[i], sw) + bias;
            const float p1 = scaled(v[i + 1], s[i + 1], sw) + bias;
            own[i / 2] = odd ? p1 : p0;
            recv[i / 2] = __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 1);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2, out += 2 * pitch) {
            const uint32_t lo = to_bits16<kOut>(odd ? recv[i / 2] : own[i / 2]), hi = to_bits16<kOut>(odd ? own[i / 2] : recv[i / 2]);
            st_if(valid && i + odd < ncol, out, lo | (hi << 16));
        }
    } else {
        // even tile rows hold gate channel f, odd rows the matching up channel: per pair of
        // tokens the lanes of a pair swap one value, the even lane finishes token i, the odd
        // lane token i + 1 (shuffles first, then arithmetic, then stores: the first and the
        // last keep their order among themselves)
        float own[8], recv[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float p0 = scaled(v[i], s[i], sw), p1 = scaled(v[i + 1], s[i + 1], sw);
            own[i / 2] = odd ? p1 : p0;
            recv[i / 2] = __shfl_xor_sync(0xffffffffu, odd ? p0 : p1, 1);
        }
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = bf16_bits(w8_silu_mul(odd ? recv[i] : own[i], odd ? own[i] : recv[i]));
#pragma unroll
        for (int i = 0; i < 16; i += 2, out += 2 * pitch) st_if(valid && i + odd < ncol, out, h[i / 2]);
    }
}

// What a warp needs to write its part of a tile.
struct W8Out {
    float sw, bias;
    const float* sa;  // lane l's scale of each of its chunks of 32 tokens (registers)
    float* sa_w;      // 32 floats of shared memory of this warp (broadcast reads instead of a shuffle per token)
    uint32_t acc;     // tensor-memory address of the accumulator, this warp's lanes
    int c0;           // its first token; chunks of 32 are 64 apart
    int row0, nrows, n, odd;
};

template <int CG, int kOut>
__device__ __forceinline__ void w8_write_tile(const W8Args& a, const W8Out& o) {
    constexpr bool kPair = kOut == kOutPairBf16 || kOut == kOutPairF16;
    constexpr int kEl = kOut == kOutF32 || kOut == kOutI32 ? 4 : 2;
    const int lane = threadIdx.x & 31;
    const size_t pitch = (size_t)a.ldo * kEl;
    char* out = static_cast<char*>(a.out) + (size_t)(o.row0 + o.c0 + (kPair || kOut == kOutSwiglu ? o.odd : 0)) * pitch +
                (size_t)(o.n - (kPair ? o.odd : 0)) * kEl;
    const bool valid = o.n < a.nvalid;
    // 16 tokens at a time, the next 16 loading meanwhile
    uint32_t v[16];
    if (o.c0 < o.nrows) tmem_ld16(o.acc + (uint32_t)o.c0, v);
#pragma unroll 1
    for (int c = 0, c0 = o.c0; c0 < o.nrows; ++c, c0 += 64, out += 64 * pitch) {
        float sa = o.sa[0];
#pragma unroll
        for (int i = 1; i < CG * 2; ++i) sa = c == i ? o.sa[i] : sa;
        __syncwarp();
        o.sa_w[lane] = sa;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ncol = o.nrows - c0 - 16 * h;
            if (h == 1 && ncol <= 0) break;
            uint32_t x[16];
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = v[i];
            const int next = c0 + (h == 0 ? 16 : 64);
            if (next < o.nrows) tmem_ld16(o.acc + (uint32_t)next, v);
            w8_store<kOut>(x, o.sw, o.bias, o.sa_w + 16 * h, ncol, valid, o.odd, out + (size_t)(16 * h) * pitch, pitch);
        }
    }
}

// kSplit (CG = 1, dense): the CTAs of a cluster share one tile, each taking a part of its K
// planes.  Every CTA sends the INT32 partials of its peers' tokens into their shared memory
// (st.async, counted by the receiver's barrier) and finishes its own share of the tokens:
// exact sums, so the result does not depend on the split, no workspace and no second launch.
// Several such CTAs may share an SM, and each waits for its peers while it holds its 128
// columns of tensor memory; a peer that had to wait for columns could close a circle.  So the
// launcher asks for enough shared memory that no more than four fit on an SM (512 columns),
// and should another program's kernel hold columns there, the wait for the peer's data runs
// out and frees this CTA's.
template <int CG, bool kSplit>
__global__ void __launch_bounds__(kW8Threads, 1)
    gemm_w8a8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_small, const W8Args a) {
    constexpr uint32_t kAccCols = 128 * CG;  // columns of an accumulator
    constexpr uint32_t kTmemCols = kSplit ? kAccCols : 2 * kAccCols;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0u : cluster_rank();  // in the pair
    const uint32_t part = kSplit ? cluster_rank() : 0u, parts = kSplit ? cluster_size() : 1u;
    const uint32_t NS = (uint32_t)a.ns;
    const uint32_t sA = base, sB = sA + NS * kW8BlockBytes, recv = sB + NS * a.b_stage;
    const uint32_t full = recv + a.recv, empty = full + 8 * kW8MaxStages;
    const uint32_t dfull = empty + 8 * kW8MaxStages, dempty = dfull + 16, recv_full = dempty + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (recv_full + 8 - base));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < NS; ++s) {
            mbar_init(full + 8 * s, 1);   // a pair's copies all report to its first CTA
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(dfull + 8 * b, 1);
            mbar_init(dempty + 8 * b, kW8EpiWarps * CG);  // in the first CTA, from both
        }
        if (kSplit) mbar_init(recv_full, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kW8ProdWarp && lane < 2) {
        // the maps' first use would wait for them
        if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
        if (lane == 1) asm volatile("prefetch.tensormap [%0];" ::"l"(&map_x) : "memory");
    }
    // (before the allocation: a peer that has to wait for its columns holds up data, not barriers)
    if (kSplit) cluster_arrive();  // the epilogue warps wait, before they reach for their peers
    if (warp == kW8MmaWarp) w8_tmem_alloc<CG>(smem_u32(tmem_slot), kTmemCols);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    grid_dep_launch();
    grid_dep_wait();  // the previous kernel on the stream has completed
    const int total = a.NP * (a.mt_tab != nullptr ? __ldg(a.n_mtiles) : a.nmt);
    // this CTA's K planes [g0, g1) of a tile; kSplit: one tile per cluster
    const int g0 = kSplit ? (int)((long long)a.G * part / parts) : 0;
    const int g1 = kSplit ? (int)((long long)a.G * (part + 1) / parts) : a.G;
    const int u0 = (int)(blockIdx.x / (CG * parts)), du = (int)(gridDim.x / (CG * parts));

    if (warp >= kW8ProdWarp && warp < kW8MmaWarp) {
        // ---------------- producers: warp pi takes the steps j with j % kW8Producers == pi ----------------
        const uint32_t pi = (uint32_t)(warp - kW8ProdWarp);
        if (lane == 0) {
            uint32_t j = 0, s = 0, ph = 0;  // step, its stage and the stage's phase
            bool ok = true;
            for (int u = u0; u < total && ok; u += du) {
                const W8Tile t = w8_tile<CG>(u, a, rank);
                // this CTA's token rows: all of them, or half of the tile's N
                const int rows = CG == 1 ? t.nrows : round_up(t.nrows, 32) / 2;
                const int row0 = t.row0 + (int)rank * rows;
                // one box for a whole tile (every copy costs the producer and the TMA unit as
                // much as some KB of data: 256-token tiles in 32-row boxes ran at 2490 TOPS, in
                // one box at 3240), up to two small ones for the few rows of a ragged tile
                const bool small = rows <= 2 * a.small_rows;
                const CUtensorMap* map = small ? &map_small : &map_x;
                const int box_rows = small ? a.small_rows : a.box_rows;
                const int boxes = small ? ceil_div(rows, box_rows) : 1;
                const uint32_t bytes = (uint32_t)kW8BlockBytes + (uint32_t)(boxes * box_rows) * 128u;
                // (a pair's second tile may lie past the last one: read that one again)
                const int wunit = (t.e * a.NT + min(t.nt, a.NT - 1)) * a.G * (kTileRows / 16);
                const int unit0 = row0 / a.row_unit, box_units = box_rows / a.row_unit;
                for (int g = g0; g < g1; ++g, ++j) {
                    if (j > 0 && ++s == NS) { s = 0; ph ^= 1u; }
                    if (j % kW8Producers != pi) continue;
                    if (!w8_wait(empty + 8 * s, ph ^ 1u, abort_flag, a.err, a.wait_limit)) { ok = false; break; }
                    // test hook: leave the first step's stage empty, so that its consumers time out
                    if (j == 0 && blockIdx.x == 0 && (a.debug & kDebugSkipFirstCopy)) continue;
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes * CG);
                    const uint32_t bar = CG == 1 ? full + 8 * s : mapa(full + 8 * s, 0);
                    const auto load = CG == 1 ? tma_load_2d : tma_load_2d_pair;
                    load(sA + s * kW8BlockBytes, &map_w, 0, wunit + g * (kTileRows / 16), bar);
                    for (int b = 0; b < boxes; ++b)
                        load(sB + s * a.b_stage + (uint32_t)(b * box_rows) * 128u, map, g * a.plane_x,
                             unit0 + b * box_units + g * a.plane_y, bar);
                }
            }
            // Never leave with a copy or a barrier arrival still on its way into this CTA's
            // shared memory: the stages' copies have landed, and (in a run without a
            // timeout) the MMAs that read them have reported back.
            const uint32_t first = j > NS ? j - NS : 0u;
            for (uint32_t q = first; q < j; ++q) {
                if (q % kW8Producers != pi) continue;
                if (rank == 0) w8_drain(full + 8 * (q % NS), (q / NS) & 1u, a.wait_limit);
                if (ok && !*abort_flag) w8_drain(empty + 8 * (q % NS), (q / NS) & 1u, a.wait_limit);
            }
        }
        __syncwarp();
    } else if (warp == kW8MmaWarp) {
        // ---------------- MMA issue (the pair's first CTA) ----------------
        uint32_t s = 0, ph = 0, tile = 0;
        bool ok = rank == 0, ready = false;  // ready: an early test found this step's stage full
        for (int u = u0; u < total && ok; u += du, ++tile) {
            const W8Tile t = w8_tile<CG>(u, a, rank);
            const uint32_t idesc = idesc_i8(128 * CG, round_up(t.nrows, 16 * CG));
            const uint32_t b = tile & 1u;
            const uint32_t d = tmem + b * kAccCols;
            if (!w8_wait<CG == 2>(dempty + 8 * b, ((tile >> 1) & 1u) ^ 1u, abort_flag, a.err, a.wait_limit)) break;
            tc_fence_after();
            for (int g = g0; g < g1; ++g) {
                if (!ready && !w8_wait<CG == 2>(full + 8 * s, ph, abort_flag, a.err, a.wait_limit)) { ok = false; break; }
                const uint32_t s0 = s;
                if (++s == NS) { s = 0; ph ^= 1u; }
                ready = w8_test<CG == 2>(full + 8 * s, ph);
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_i8_ss<CG>(d, smem_desc_sw128(sA + s0 * kW8BlockBytes + kk * 32),
                                      smem_desc_sw128(sB + s0 * a.b_stage + kk * 32), idesc, g != g0 || kk != 0);
                    w8_commit<CG>(empty + 8 * s0);
                    if (g == g1 - 1) w8_commit<CG>(dfull + 8 * b);
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
        if (kSplit) cluster_wait();  // every CTA's barriers stand
        for (int u = u0; u < total; u += du, ++tile) {
            const W8Tile t = w8_tile<CG>(u, a, rank);
            const uint32_t b = tile & 1u;
            const float sw = t.nt < a.NT ? __ldg(a.wscale + ((size_t)t.e * a.NT + t.nt) * kTileRows + r) : 0.f;
            // output column: channel n (past the last tile: none valid)
            const int n = a.out_kind == kOutSwiglu ? t.nt * (kTileRows / 2) + (r >> 1) : t.nt * kTileRows + r;
            const float bias = (a.bias != nullptr && n < a.nvalid) ? __ldg(a.bias + n) : 0.f;
            // token scales, ahead of the accumulator: lane l's of each chunk of 32 tokens in a
            // register (kSplit: those of this CTA's tokens in shared memory)
            float* sa_s = reinterpret_cast<float*>(smem + (recv_full + 16 - base));
            float sa_r[CG * 2];
            if (kSplit) {
                const int tok = (int)part * w8_tokens_per_part(t.nrows, (int)parts) + (int)threadIdx.x;
                if (threadIdx.x < 64)
                    sa_s[threadIdx.x] = a.act_scale != nullptr && tok < t.nrows ? __ldg(a.act_scale + t.row0 + tok) : 0.f;
                named_bar_sync(1, kW8EpiWarps * 32);  // (one tile: every epilogue warp comes here once)
            } else {
#pragma unroll
                for (int c = 0; c < CG * 2; ++c) {
                    const int tok = half * 32 + c * 64 + lane;
                    sa_r[c] = a.act_scale != nullptr && tok < t.nrows ? __ldg(a.act_scale + t.row0 + tok) : 0.f;
                }
            }
            if (!w8_wait(dfull + 8 * b, (tile >> 1) & 1u, abort_flag, a.err, a.wait_limit)) break;
            tc_fence_after();
            if (kSplit) {
                // Tokens [p * per, (p + 1) * per) are finished by CTA p, which keeps the partials
                // of source s at recv[s][token / 4][channel][token % 4]: a lane sends four tokens
                // of its channel at a time, a warp 512 bytes in a row.
                const int per = w8_tokens_per_part(t.nrows, (int)parts);
                const int first = (int)part * per, count = max(0, min(per, t.nrows - first));
                if (threadIdx.x == 0) mbar_arrive_expect_tx(recv_full, parts * (uint32_t)round_up(count, 4) * (kTileRows * 4u));
                for (int c0 = half * 32; c0 < t.nrows; c0 += 64) {
                    uint32_t v[32];
                    tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)c0, v);
                    tmem_ld_wait();
                    int p = c0 / per, i0 = c0 - p * per;  // CTA and its token of the next four
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        if (c0 + i < t.nrows) {
                            if (i0 == per) { ++p; i0 = 0; }
                            st_async4(mapa(recv, (uint32_t)p) + (uint32_t)((((int)part * per + i0) / 4 * kTileRows + r) * 16), v[i],
                                      v[i + 1], v[i + 2], v[i + 3], mapa(recv_full, (uint32_t)p));
                            i0 += 4;
                        }
                    }
                }
                if (!w8_wait<true>(recv_full, 0, abort_flag, a.err, a.wait_limit)) break;
                const int4* rb = reinterpret_cast<const int4*>(smem + (recv - base)) + r;
                for (int i = half * 4; i < count; i += 8) {
                    int4 sum = make_int4(0, 0, 0, 0);
                    for (uint32_t src = 0; src < parts; ++src) {
                        const int4 x = rb[((int)src * per + i) / 4 * kTileRows];
                        sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
                    }
                    const int sums[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const size_t at = (size_t)(t.row0 + first + i + k) * a.ldo + n;
                        if (n < a.nvalid && i + k < count) {
                            const float y = scaled((uint32_t)sums[k], sa_s[i + k], sw) + bias;
                            if (a.out_kind == kOutI32) static_cast<int32_t*>(a.out)[at] = sums[k];
                            else if (a.out_kind == kOutF32) static_cast<float*>(a.out)[at] = y;
                            else if (a.out_kind == kOutF16 || a.out_kind == kOutPairF16)
                                static_cast<uint16_t*>(a.out)[at] = to_bits16<kOutF16>(y);
                            else static_cast<uint16_t*>(a.out)[at] = to_bits16<kOutBf16>(y);
                        }
                    }
                }
                break;
            }
            const W8Out o = {sw, bias, sa_r, sa_s + warp * 32, tmem + ((uint32_t)(q * 32) << 16) + b * kAccCols, half * 32,
                             t.row0, t.nrows, n, odd};
            switch (a.out_kind) {
                case kOutF32: w8_write_tile<CG, kOutF32>(a, o); break;
                case kOutI32: w8_write_tile<CG, kOutI32>(a, o); break;
                case kOutBf16: w8_write_tile<CG, kOutBf16>(a, o); break;
                case kOutF16: w8_write_tile<CG, kOutF16>(a, o); break;
                case kOutPairBf16: w8_write_tile<CG, kOutPairBf16>(a, o); break;
                case kOutPairF16: w8_write_tile<CG, kOutPairF16>(a, o); break;
                default: w8_write_tile<CG, kOutSwiglu>(a, o); break;
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
    if (kSplit && warp >= kW8ProdWarp) cluster_wait();  // (the epilogue warps have waited)
    if (CG == 2 || (kSplit && *abort_flag)) {
        // after a timeout the cluster's copies, stores and arrivals are not accounted for: give
        // them ample time (50 us) to land before this CTA's shared memory goes away, and stay
        // until every other CTA has come this far or left.  (kSplit without one: a CTA has
        // received all that is sent to it before it leaves.)
        if (*abort_flag) {
            const long long t0 = clock64();
            while (clock64() - t0 < 100000) {
            }
        }
        // (a split CTA frees its columns first: a peer may be waiting for some)
        if (kSplit && warp == kW8MmaWarp) {
            tc_fence_after();
            w8_tmem_dealloc<CG>(tmem, kTmemCols);
        }
        __syncwarp();
        cluster_sync();
    }
    if (a.status != nullptr) {
        // one word per CTA, every word written by every launch: nothing to clear beforehand
        if (threadIdx.x == 0) a.status[blockIdx.x] = *abort_flag ? kErrTimeout : 0u;
        if (blockIdx.x == 0)
            for (int i = (int)gridDim.x + (int)threadIdx.x; i < kW8StatusWords; i += kW8Threads) a.status[i] = 0u;
    }
    if (warp == kW8MmaWarp && !(kSplit && *abort_flag)) {
        tc_fence_after();
        w8_tmem_dealloc<CG>(tmem, kTmemCols);
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
    // the largest magnitude by its bits: a NaN is above infinity, and either becomes the scale,
    // with codes 0 (all outputs of the channel are 0 times it: NaN)
    uint32_t bits = 0u;
    if (valid) {
        for (int ci = lane; ci < G * 8; ci += 32) {
            load16(ci * 16);
#pragma unroll
            for (int i = 0; i < 16; ++i) bits = max(bits, __float_as_uint(fabsf(v[i])));
        }
    }
    const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
    const float sc = __fmul_rn(amax, kInv127);
    const float rinv = __fdiv_rn(1.0f, sc);
    for (int ci = lane; ci < G * 8; ci += 32) {
        uint32_t out[4] = {0u, 0u, 0u, 0u};
        if (valid && amax > 0.f && amax < INFINITY) {
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

// Row-major INT8 rows of `width` bytes (a multiple of 128), copied in boxes of 128 bytes x
// box_rows and swizzled on the way.
cudaError_t make_map_rows(CUtensorMap* m, const void* base, uint64_t width, uint64_t rows, uint32_t box_rows) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {width, rows}, strides[1] = {width};
    const cuuint32_t box[2] = {128, box_rows}, steps[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// Contiguous memory in units of 2 KB (16 tile rows of 128 bytes), copied `box` units at a
// time.  (The TMA unit's time goes by the box's rows: 2 KB rows, of 8-byte elements.)
cudaError_t make_map_linear(CUtensorMap* m, const void* base, uint64_t units, uint32_t box) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {256, units}, strides[1] = {2048};
    const cuuint32_t boxes[2] = {256, box}, steps[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, const_cast<void*>(base), dims, strides, boxes, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

}  // namespace

namespace {

// Per device, looked up once: the instances' shared-memory attribute is set, and how many
// clusters of 2, 4 and 8 CTAs run at once with one CTA per SM (clusters stay inside a GPC,
// whose SMs need not be a multiple of the cluster).
struct W8Device {
    int pairs = 0;         // CG = 2
    int clusters[4] = {};  // K split by 1 << i (index 0 unused)
};

template <int CG, bool kSplit>
cudaError_t max_clusters(int cluster, int* n) {
    const auto kernel = gemm_w8a8_kernel<CG, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess || cluster == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = (unsigned)cluster;
    cfg.blockDim = kW8Threads;
    cfg.dynamicSmemBytes = 227 * 1024;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
}

cudaError_t w8_device(W8Device* out) {
    static std::mutex mu;
    static W8Device devs[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (devs[dev].pairs == 0) {
        W8Device d;
        e = max_clusters<1, false>(1, nullptr);
        for (int i = 1; e == cudaSuccess && i <= 3; ++i) e = max_clusters<1, true>(1 << i, &d.clusters[i]);
        if (e == cudaSuccess) e = max_clusters<2, false>(2, &d.pairs);
        if (e != cudaSuccess) return e;
        if (d.pairs < 1) return cudaErrorInvalidConfiguration;
        devs[dev] = d;
    }
    *out = devs[dev];
    return cudaSuccess;
}

template <int CG, bool kSplit>
cudaError_t launch_instance(const CUtensorMap& mw, const CUtensorMap& mx, const CUtensorMap& ms, const W8Args& a, int smem, int grid,
                            int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = (unsigned)grid;
    cfg.blockDim = kW8Threads;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, gemm_w8a8_kernel<CG, kSplit>, mw, mx, ms, a);
}

// The cheapest of the dense tile shapes by a model of the kernel's time in cycles, fitted to
// measurements on B200: about 6200 (a pair: 7850) from launch to end for one step; per K
// plane the tensor core's 2 * bn or the arrival of its blocks (128 + bn / cg rows of 128
// bytes at 57 bytes per cycle and SM; a pair: 48), and not less than 480; the last tile's
// epilogue; the exchange of a K split.  At 4096 x 4096, 64 rows: 11.7 us unsplit, 7.9 us in
// four parts; 128 rows: 13.4 and 9.9 us.
W8Plan w8_plan_dense(int M, int NT, int G, int num_ctas, const W8Device& dev) {
    W8Plan best = {1, 128, 1};
    long long best_cost = -1;
    const auto consider = [&](int cg, int bn, int split, int slots) {
        const long long tiles = (long long)ceil_div(M, bn) * ceil_div(NT, cg);
        if (slots < 1 || split > G || (split > 1 && tiles > slots)) return;
        const long long arrival = cg == 1 ? (128 + bn) * 9 / 4 : (128 + bn / 2) * 53 / 20;
        const long long mma = 2 * bn > 480 ? 2 * bn : 480;
        const long long waves = (tiles + slots - 1) / slots;
        const long long cost = waves * (ceil_div(G, split) * (arrival > mma ? arrival : mma) + 300) + (cg == 1 ? 6200 : 7850) +
                               13 * bn + (split > 1 ? 600 + 56 * bn : 0);
        if (best_cost < 0 || cost < best_cost) {
            best_cost = cost;
            best = {cg, bn, split};
        }
    };
    const int top = M < 128 ? round_up(M, 16) : 128;
    for (int bn = top; bn >= 16; bn -= 16) {
        consider(1, bn, 1, num_ctas);
        for (int i = 1; i <= 3; ++i) consider(1, bn, 1 << i, dev.clusters[i]);
    }
    if (M > 64)
        for (int bn = 256; bn >= 64; bn -= 32) consider(2, bn, 1, dev.pairs);
    return best;
}

}  // namespace

// The grouped tile shape by the same model, for nslots rows spread evenly over the experts: a
// step's blocks come from L2 as above, but its weight block at least once per expert from
// memory (16 KB per CTA at 6.5 TB/s for all SMs: 700 cycles).  B200, up + down projections of
// 48 experts (H 4096, F 1408): 85 rows each, 170 us with 128 x 128 tiles, 176 us with pairs;
// 170 rows each (H 7168, F 2048): 558 against 405 us.
W8Plan w8_plan_grouped(int nslots, int E, int NT_up, int G_up, int NT_down, int G_down, int num_ctas) {
    const int experts = nslots < E ? nslots : E;
    const int rows = ceil_div(nslots, experts);
    const auto cost = [&](int cg, int bn) {
        const int mt = ceil_div(rows, bn), r = ceil_div(rows, mt);  // row tiles per expert, rows of one
        const long long slots = num_ctas / cg, memory = 700 / mt;
        long long plane = cg == 1 ? (128 + r) * 9 / 4 : (128 + r / 2) * 53 / 20;
        plane = plane > 480 ? plane : 480;
        plane = plane > memory ? plane : memory;
        plane = plane > 2 * r ? plane : 2 * r;
        long long sum = 0;
        for (int down = 0; down < 2; ++down) {
            const long long tiles = (long long)experts * mt * ceil_div(down ? NT_down : NT_up, cg);
            const long long loop = (down ? G_down : G_up) * plane;
            const long long epilogue = 16ll * r;  // overlaps the next tile's loop
            sum += (tiles + slots - 1) / slots * (loop > epilogue ? loop : epilogue) + epilogue + (cg == 1 ? 6200 : 7850);
        }
        return sum;
    };
    // (rows vary: tiles a tenth wider than the mean's equal shares)
    const int want = rows + rows / 10;
    W8Plan best = {1, 128, 1};
    long long best_cost = rows < 64 ? 0 : cost(1, 128);
    const auto consider = [&](int cg, int bn) {
        const long long c = cost(cg, bn);
        if (c < best_cost) {
            best_cost = c;
            best = {cg, bn, 1};
        }
    };
    consider(1, 64);
    for (int mt = ceil_div(want, 256); mt <= ceil_div(want, 128) + 1; ++mt) {
        const int bn = round_up(ceil_div(want, mt), 32);
        consider(2, bn < 64 ? 64 : bn);
    }
    return best;
}

cudaError_t launch_gemm_w8a8(W8Args a, const W8Operands& op, const W8Plan* grouped, int num_ctas, cudaStream_t stream) {
    W8Device dev;
    cudaError_t e = w8_device(&dev);
    if (e != cudaSuccess) return e;
    const W8Plan plan = grouped != nullptr ? *grouped : w8_plan_dense(a.M, a.NT, a.G, num_ctas, dev);
    CUtensorMap mw, mx, ms;
    e = make_map_linear(&mw, op.wblocks, (uint64_t)op.matrices * a.NT * a.G * (kTileRows / 16), kTileRows / 16);
    if (e != cudaSuccess) return e;
    a.BN = plan.bn;
    a.NP = ceil_div(a.NT, plan.cg);
    a.nmt = ceil_div(a.M, plan.bn);
    a.box_rows = plan.bn / plan.cg;  // 16 .. 128, a multiple of 16
    a.small_rows = 16;
    if (a.mt_tab != nullptr) {
        // tiled rows [G][rows][128]: a tile's rows of a plane lie together
        a.plane_x = 0;
        a.plane_y = op.x_rows / 16;
        a.row_unit = 16;
        e = make_map_linear(&mx, op.x, (uint64_t)op.x_rows / 16 * a.G, (uint32_t)a.box_rows / 16);
        if (e == cudaSuccess) e = make_map_linear(&ms, op.x, (uint64_t)op.x_rows / 16 * a.G, (uint32_t)a.small_rows / 16);
    } else {
        // row-major rows of G * 128 bytes
        a.plane_x = 128;
        a.plane_y = 0;
        a.row_unit = 1;
        e = make_map_rows(&mx, op.x, (uint64_t)a.G * 128, (uint64_t)op.x_rows, (uint32_t)a.box_rows);
        ms = mx;
        a.small_rows = 0;  // (rows past M are not read: the box costs what it holds)
    }
    if (e != cudaSuccess) return e;
    const bool pairs = a.ldo % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
    a.out_kind = a.mode == kW8Up            ? kOutSwiglu
                 : a.out_type == W8A8_F32   ? kOutF32
                 : a.out_type == W8A8_I32   ? kOutI32
                 : a.out_type == W8A8_BF16  ? (pairs ? kOutPairBf16 : kOutBf16)
                                            : (pairs ? kOutPairF16 : kOutF16);
    a.b_stage = (uint32_t)a.box_rows * 128u;
    a.recv = plan.split > 1 ? (uint32_t)(w8_tokens_per_part(plan.bn, plan.split) * plan.split * kTileRows * 4) : 0u;
    a.ns = (kW8SmemMax - kW8BarBytes - (int)a.recv) / (kW8BlockBytes + (int)a.b_stage);
    if (a.ns > kW8MaxStages) a.ns = kW8MaxStages;
    const int steps = ceil_div(a.G, plan.split);  // a short K needs no more stages
    if (plan.split > 1 && a.ns > steps) a.ns = steps;
    int smem = w8_smem(a.ns, (int)a.b_stage, (int)a.recv);
    if (plan.split > 1 && smem < kW8SplitSmem) smem = kW8SplitSmem;
    if (num_ctas > kW8StatusWords) num_ctas = kW8StatusWords;
    if (plan.split > 1) {
        const int grid = ceil_div(a.M, plan.bn) * a.NT * plan.split;
        return launch_instance<1, true>(mw, mx, ms, a, smem, grid, plan.split, stream);
    }
    if (plan.cg == 1) return launch_instance<1, false>(mw, mx, ms, a, smem, num_ctas, 1, stream);
    const int at_once = num_ctas / 2 < dev.pairs ? num_ctas / 2 : dev.pairs;
    return launch_instance<2, false>(mw, mx, ms, a, smem, at_once * 2, 2, stream);
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
