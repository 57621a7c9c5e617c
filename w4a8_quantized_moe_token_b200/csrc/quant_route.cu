// Quantisation, routing, permutation and combine kernels of the W4A8 MoE layer.
//
// Sources of the arithmetic:
//   weight INT4 (group 128, asymmetric, low nibble first):
//       «Kimi 2.7 Moe 从 4 bit 存储到 INT8 拆解» (pptc.cn) sections 2.1 and 2.2;
//   activation INT8 (per token, symmetric, scale = max|x| / (2^(b-1) - 1)):
//       LLM quantisation primer (hotelren.com 5982361) section 2.1 and the Kimi 2.7T
//       MoE W4A8 article (hotelren.com 5173946) section 4.3, step 3;
//   routing kept in 16-bit float: the Kimi 2.7T MoE W4A8 article, section 5.2.
// Every "round" is round-half-to-even, every division a correctly rounded fp32
// division, so codes agree bit for bit with any other IEEE implementation.
#include <climits>

#include "layer_internal.h"
#include "w4a8_common.cuh"
#include "w4a8_internal.h"

namespace w4a8 {

namespace {

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------------------
// a1: weight quantisation + packing.  One block per (group gq, tile t, matrix e);
// thread r quantises tiled row r's GRP weights of group gq, 64 at a time: a first
// pass over the group finds its range, a second one (re-reading the row from cache)
// computes the codes and writes them into the group's 128-wide plane blocks.
// ---------------------------------------------------------------------------
// 64 weights of a row from K index k0 on (zero past K and for rows past N)
__device__ __forceinline__ void load_w64(const uint16_t* row, int K, int k0, float (&v)[64]) {
    if (row != nullptr && (K & 7) == 0 && k0 + 64 <= K) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint4 p = *reinterpret_cast<const uint4*>(row + k0 + 8 * i);
            const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                v[8 * i + 2 * h] = bf16_to_f32((uint16_t)(pw[h] & 0xFFFFu));
                v[8 * i + 2 * h + 1] = bf16_to_f32((uint16_t)(pw[h] >> 16));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 64; ++i) v[i] = (row != nullptr && k0 + i < K) ? bf16_to_f32(row[k0 + i]) : 0.f;
    }
}

// sym: 0 asymmetric min/max, 1 symmetric, 2 asymmetric on the 0.1th..99.9th percentile
// range (128-value groups only); G = 128-wide planes per row
template <int GRP>
__global__ void __launch_bounds__(128) pack_kernel(const uint16_t* __restrict__ w, int N, int K, int layout, int sym,
                                                   int NT, int G, uint8_t* __restrict__ blocks,
                                                   uint8_t* __restrict__ codes_out, uint16_t* __restrict__ scale_out,
                                                   uint16_t* __restrict__ zp_out) {
    constexpr int kChunks = GRP / 64;
    constexpr int kBB = block_bytes_for(GRP);
    const int gq = blockIdx.x, t = blockIdx.y, e = blockIdx.z;
    const int Gq = G * kGroup / GRP;
    const int r = threadIdx.x;
    int src;
    bool valid;
    if (layout == 1) {  // gate|up interleave: even tiled rows gate channel f, odd rows up channel f
        const int F = N / 2;
        const int f = t * (kTileRows / 2) + (r >> 1);
        valid = f < F;
        src = (r & 1) ? F + f : f;
    } else {
        src = t * kTileRows + r;
        valid = src < N;
    }
    const uint16_t* row = valid ? w + ((size_t)e * N + src) * (size_t)K : nullptr;
    float v[64];
    __half sh;
    int zp;
    if (sym != 1) {
        float lo, hi;
        // min / max, and the two smallest and two largest values (a0 <= a1, b0 >= b1)
        float mn0 = INFINITY, mx0 = -INFINITY;
        float a0 = INFINITY, a1 = INFINITY, b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
            load_w64(row, K, gq * GRP + c * 64, v);
#pragma unroll
            for (int i = 0; i < 64; ++i) {
                mn0 = fminf(mn0, v[i]);
                mx0 = fmaxf(mx0, v[i]);
                if (sym == 2) {
                    a1 = fminf(a1, fmaxf(v[i], a0));
                    a0 = fminf(a0, v[i]);
                    b1 = fmaxf(b1, fminf(v[i], b0));
                    b0 = fmaxf(b0, v[i]);
                }
            }
        }
        if (sym == 2) {
            // the 0.1th and 99.9th percentiles of a 128-value group: linear interpolation
            // between the order statistics around positions 0.127 and 126.873
            lo = __fadd_rn(a0, __fmul_rn(0.127f, __fsub_rn(a1, a0)));
            hi = __fadd_rn(b1, __fmul_rn(0.873f, __fsub_rn(b0, b1)));
        } else {
            lo = mn0;
            hi = mx0;
        }
        // range widened to contain 0
        const float mn = fminf(lo, 0.f), mx = fmaxf(hi, 0.f);
        // scale = (max - min) / (2^4 - 1), stored as fp16; the fp16 value is the one used
        sh = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
        if (__half2float(sh) == 0.f) sh = __float2half_rn(1.0f);
        // zero_point = round(-min / scale)
        zp = (int)fminf(fmaxf(rintf(__fdiv_rn(-mn, __half2float(sh))), 0.f), 15.f);
    } else {
        // symmetric (b = 4): scale = max|w| / (2^3 - 1), stored as code q + 8 with zero point 8
        float amax = 0.f;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
            load_w64(row, K, gq * GRP + c * 64, v);
#pragma unroll
            for (int i = 0; i < 64; ++i) amax = fmaxf(amax, fabsf(v[i]));
        }
        sh = __float2half_rn(__fdiv_rn(amax, 7.0f));
        if (__half2float(sh) == 0.f) sh = __float2half_rn(1.0f);
        zp = 8;
    }
    const float shf = __half2float(sh);
    const size_t tile_blk = (size_t)(e * NT + t) * G;
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c) {
        const int k0 = gq * GRP + c * 64;  // K index of this chunk's first weight
        load_w64(row, K, k0, v);
        uint32_t code[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            if (sym != 1) {
                // index = clamp(round(w / scale) + zero_point, 0, 15)
                const int cc = (int)rintf(__fdiv_rn(v[i], shf)) + zp;
                code[i] = (uint32_t)min(max(cc, 0), 15);
            } else {
                // q = clamp(round(w / scale), -7, 7)
                const int q = (int)rintf(__fdiv_rn(v[i], shf));
                code[i] = (uint32_t)(min(max(q, -7), 7) + 8);
            }
        }
        // tiled block of plane k0 / 128: word i of the plane (K = 8i .. 8i+7):
        // byte b = code[8i+b] | code[8i+4+b] << 4; this chunk is the plane's half k0 / 64 % 2
        uint8_t* blk = blocks + (tile_blk + (size_t)(k0 / kGroup)) * kBB;
        const int hh = (k0 / 64) & 1;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
            uint32_t wd[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int l = 32 * cc + 8 * q;  // chunk-local index of the word's first code
                uint32_t x = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) x |= (code[l + b] | (code[l + 4 + b] << 4)) << (8 * b);
                wd[q] = x;
            }
            *reinterpret_cast<uint4*>(blk + code_chunk_offset(r, 2 * hh + cc)) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
        }
        if (valid && codes_out != nullptr) {
            // canonical order: byte j = code[2j] | code[2j+1] << 4
            uint8_t* dst = codes_out + ((size_t)e * N + src) * (size_t)(G * kGroup / 2) + (size_t)k0 / 2;
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                uint32_t wd[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t x = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int j = 16 * cc + 4 * q + b;
                        x |= (code[2 * j] | (code[2 * j + 1] << 4)) << (8 * b);
                    }
                    wd[q] = x;
                }
                *reinterpret_cast<uint4*>(dst + 16 * cc) = make_uint4(wd[0], wd[1], wd[2], wd[3]);
            }
        }
    }
    // scale and zero point: in the plane block (group 64: the plane's sub-group slot;
    // group 256: both of the group's planes)
    const __half zh = __float2half_rn((float)zp);
#pragma unroll
    for (int pp = 0; pp < (GRP > kGroup ? GRP / kGroup : 1); ++pp) {
        const int plane = GRP > kGroup ? gq * (GRP / kGroup) + pp : gq * GRP / kGroup;
        const int sub = GRP < kGroup ? (gq & 1) : 0;
        uint8_t* blk = blocks + (tile_blk + (size_t)plane) * kBB + sub * 512;
        reinterpret_cast<__half*>(blk + kScaleOff)[r] = sh;
        reinterpret_cast<__half*>(blk + kZpOff)[r] = zh;
    }
    if (valid) {
        if (scale_out != nullptr) scale_out[((size_t)e * N + src) * Gq + gq] = __half_as_ushort(sh);
        if (zp_out != nullptr) zp_out[((size_t)e * N + src) * Gq + gq] = __half_as_ushort(zh);
    }
    if (e == 0 && t == 0 && gq == 0 && r == 0) {
        PackHeader* h = reinterpret_cast<PackHeader*>(blocks - kHeaderBytes);
        h->magic = kPackMagic;
        h->version = 2;
        h->layout = (uint32_t)layout | (sym == 1 ? 0x100u : sym == 2 ? 0x200u : 0u);
        h->E = gridDim.z;
        h->N = (uint32_t)N;
        h->K = (uint32_t)K;
        h->Kp = (uint32_t)(G * kGroup);
        h->G = (uint32_t)G;
        h->NT = (uint32_t)NT;
        h->rows_per_tile = kTileRows;
        h->block_bytes = kBB;
        h->group = GRP;
    }
}

// ---------------------------------------------------------------------------
// a2: per-token INT8, natural layout [T][Kp].  One warp per row.  With K a multiple
// of 8 the row is read in 16-byte vectors (8 bf16 per lane and step) and the codes are
// written 8 bytes at a time; other K take the scalar path.  The codes are the same.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) quant_act_kernel(const uint16_t* __restrict__ x, int T, int K, int Kp,
                                                        int8_t* __restrict__ q, float* __restrict__ s) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= T) return;
    const uint16_t* xr = x + (size_t)row * K;
    int8_t* qr = q + (size_t)row * Kp;
    float amax = 0.f;
    if ((K & 7) == 0) {
        const uint4* xv = reinterpret_cast<const uint4*>(xr);
        for (int c = lane; c < K / 8; c += 32) {
            const uint4 p = __ldg(xv + c);
            const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int h = 0; h < 4; ++h)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(pw[h] << 16)), fabsf(__uint_as_float(pw[h] & 0xFFFF0000u))));
        }
        amax = warp_max(amax);
        const float sc = __fdiv_rn(amax, 127.0f);
        const float rinv = __fdiv_rn(1.0f, sc);
        for (int c = lane; c < Kp / 8; c += 32) {
            uint32_t out[2] = {0u, 0u};
            if (c < K / 8 && amax > 0.f) {
                const uint4 p = __ldg(xv + c);
                const uint32_t pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const uint32_t lo = (uint32_t)(quant_i8_fast(__uint_as_float(pw[h] << 16), sc, rinv) & 0xFF);
                    const uint32_t hi = (uint32_t)(quant_i8_fast(__uint_as_float(pw[h] & 0xFFFF0000u), sc, rinv) & 0xFF);
                    out[h >> 1] |= (lo | (hi << 8)) << (16 * (h & 1));
                }
            }
            *reinterpret_cast<uint2*>(qr + 8 * c) = make_uint2(out[0], out[1]);
        }
        if (lane == 0) s[row] = sc;
        return;
    }
    for (int k = lane; k < K; k += 32) amax = fmaxf(amax, fabsf(bf16_to_f32(xr[k])));
    amax = warp_max(amax);
    const float sc = __fdiv_rn(amax, 127.0f);
    const float rinv = __fdiv_rn(1.0f, sc);
    for (int k = lane; k < Kp; k += 32) {
        int c = 0;
        if (k < K && amax > 0.f) c = quant_i8_fast(bf16_to_f32(xr[k]), sc, rinv);
        qr[k] = (int8_t)c;
    }
    if (lane == 0) s[row] = sc;
}

// ---------------------------------------------------------------------------
// a3: top-k softmax routing.  One warp per token; lane l owns experts l, l+32, ...
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) route_topk_kernel(const uint16_t* __restrict__ logits, int T, int E, int k,
                                                         int32_t* __restrict__ ids, float* __restrict__ wout) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= T) return;
    const uint16_t* lr = logits + (size_t)t * E;
    const int per_lane = (E + 31) >> 5;
    uint32_t taken = 0;
    float top = -INFINITY;
    for (int j = 0; j < k; ++j) {
        float bv = -INFINITY;
        int be = INT_MAX;
        for (int i = 0; i < per_lane; ++i) {
            const int e = lane + 32 * i;
            if (e < E && !((taken >> i) & 1u)) {
                float v = bf16_to_f32(lr[e]);
                if (isnan(v)) v = -INFINITY;
                if (v > bv || (v == bv && e < be)) { bv = v; be = e; }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; }
        }
        if (lane == (be & 31)) taken |= 1u << (be >> 5);
        if (j == 0) top = bv;
        if (lane == 0) {
            ids[(size_t)t * k + j] = be;
            wout[(size_t)t * k + j] = bv;  // logit for now, turned into a probability below
        }
    }
    float sum = 0.f;
    for (int i = 0; i < per_lane; ++i) {
        const int e = lane + 32 * i;
        if (e < E) {
            const float v = bf16_to_f32(lr[e]);
            if (!isnan(v)) sum += expf(v - top);
        }
    }
    sum = warp_sum(sum);
    __syncwarp();
    if (lane < k) {
        const float lv = wout[(size_t)t * k + lane];
        wout[(size_t)t * k + lane] = expf(lv - top) / sum;
    }
}

// ---------------------------------------------------------------------------
// a4: stable grouping of slots by expert (counting sort in three passes)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPermChunk) perm_hist_kernel(const int32_t* __restrict__ ids, int nslots, int E,
                                                              int* __restrict__ chist, uint32_t* err) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    __shared__ int h[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += blockDim.x) h[e] = 0;
    __syncthreads();
    const int i = blockIdx.x * kPermChunk + threadIdx.x;
    if (i < nslots) {
        const int e = ids[i];
        if (e >= 0 && e < E) atomicAdd(&h[e], 1);
        else atomicOr(err, kErrBadExpert);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) chist[(size_t)blockIdx.x * E + e] = h[e];
}

// block-wide exclusive scan (blockDim.x == 1024) of one int per thread
__device__ int block_exclusive_scan(int v, int* sh, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += n;
        }
        sh[lane] = w;  // inclusive over warps
    }
    __syncthreads();
    const int before = (warp > 0 ? sh[warp - 1] : 0) + incl - v;
    *total = sh[31];
    __syncthreads();
    return before;
}

__global__ void __launch_bounds__(1024) perm_scan_kernel(int* __restrict__ chist, int nchunk, int E, int tile_tokens,
                                                        int* __restrict__ counts, int* __restrict__ offs,
                                                        int* __restrict__ poffs, int* __restrict__ mtstart,
                                                        int4* __restrict__ mt_tab, int* __restrict__ row_src) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    __shared__ int sh[32];
    const int e = threadIdx.x;
    int c_e = 0;
    if (e < E) {
        // per-chunk histogram -> slots of e in all earlier chunks (in place)
        for (int c = 0; c < nchunk; ++c) {
            const int v = chist[(size_t)c * E + e];
            chist[(size_t)c * E + e] = c_e;
            c_e += v;
        }
    }
    int t0, t1, t2;
    const int o0 = block_exclusive_scan(c_e, sh, &t0);
    const int o1 = block_exclusive_scan(round_up(c_e, kRowPad), sh, &t1);
    const int o2 = block_exclusive_scan(ceil_div(c_e, tile_tokens), sh, &t2);
    if (e < E) {
        counts[e] = c_e;
        offs[e] = o0;
        poffs[e] = o1;
        mtstart[e] = o2;
        for (int rr = o1 + c_e; rr < o1 + round_up(c_e, kRowPad); ++rr) row_src[rr] = -1;
        // one entry per row tile of this expert: (expert, first row, rows)
        for (int t = 0; t < ceil_div(c_e, tile_tokens); ++t)
            mt_tab[o2 + t] = make_int4(e, o1 + t * tile_tokens, min(tile_tokens, c_e - t * tile_tokens), 0);
    }
    if (e == 0) {
        offs[E] = t0;
        poffs[E] = t1;
        mtstart[E] = t2;
    }
}

__global__ void __launch_bounds__(kPermChunk) perm_scatter_kernel(const int32_t* __restrict__ ids, int nslots, int E,
                                                                 const int* __restrict__ chist,
                                                                 const int* __restrict__ offs,
                                                                 const int* __restrict__ poffs, int* __restrict__ perm,
                                                                 int* __restrict__ inv, int* __restrict__ row_src) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    constexpr int kWarps = kPermChunk / 32;
    __shared__ int wcnt[kWarps][kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int idx = threadIdx.x; idx < kWarps * E; idx += blockDim.x) wcnt[idx / E][idx % E] = 0;
    __syncthreads();
    const int i = blockIdx.x * kPermChunk + threadIdx.x;
    const bool valid = i < nslots;
    const int e = valid ? ids[i] : -1;
    const bool good = valid && e >= 0 && e < E;
    const int key = good ? e : E + lane;  // unmatched keys for slots that take no part
    const uint32_t mask = __match_any_sync(0xffffffffu, key);
    const int rank_w = __popc(mask & ((1u << lane) - 1u));
    if (good && lane == __ffs(mask) - 1) wcnt[warp][e] = __popc(mask);
    __syncthreads();
    if (good) {
        int p = chist[(size_t)blockIdx.x * E + e] + rank_w;
        for (int w2 = 0; w2 < warp; ++w2) p += wcnt[w2][e];
        perm[offs[e] + p] = i;
        const int rr = poffs[e] + p;
        inv[i] = rr;
        row_src[rr] = i;
    } else if (valid) {
        inv[i] = -1;
    }
}

// a4 for small batches (up to kPermSmallSlots slots): histogram, scans and the
// stable scatter in one CTA, in slot order, 1024 slots at a time.
__global__ void __launch_bounds__(1024) perm_small_kernel(const int32_t* __restrict__ ids, int nslots, int E,
                                                         int tile_tokens, int* __restrict__ counts,
                                                         int* __restrict__ offs, int* __restrict__ poffs,
                                                         int* __restrict__ mtstart, int4* __restrict__ mt_tab,
                                                         int* __restrict__ perm, int* __restrict__ inv,
                                                         int* __restrict__ row_src, uint32_t* err) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    extern __shared__ int psm[];
    int* s_off = psm;          // [E] counts, then the exclusive offsets
    int* s_poff = psm + E;     // [E] padded offsets
    int* s_run = psm + 2 * E;  // [E] slots of e placed so far
    int* s_wcnt = psm + 3 * E; // [32][E] slots of e in each warp of the current chunk
    __shared__ int sh[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int e = tid; e < E; e += blockDim.x) {
        s_off[e] = 0;
        s_run[e] = 0;
    }
    __syncthreads();
    for (int i = tid; i < nslots; i += blockDim.x) {
        const int e = ids[i];
        if (e >= 0 && e < E) atomicAdd(&s_off[e], 1);
        else atomicOr(err, kErrBadExpert);
    }
    __syncthreads();
    const int c_e = tid < E ? s_off[tid] : 0;
    int t0, t1, t2;
    const int o0 = block_exclusive_scan(c_e, sh, &t0);
    const int o1 = block_exclusive_scan(round_up(c_e, kRowPad), sh, &t1);
    const int o2 = block_exclusive_scan(ceil_div(c_e, tile_tokens), sh, &t2);
    if (tid < E) {
        counts[tid] = c_e;
        offs[tid] = o0;
        poffs[tid] = o1;
        mtstart[tid] = o2;
        s_off[tid] = o0;
        s_poff[tid] = o1;
        for (int rr = o1 + c_e; rr < o1 + round_up(c_e, kRowPad); ++rr) row_src[rr] = -1;
        for (int t = 0; t < ceil_div(c_e, tile_tokens); ++t)
            mt_tab[o2 + t] = make_int4(tid, o1 + t * tile_tokens, min(tile_tokens, c_e - t * tile_tokens), 0);
    }
    if (tid == 0) {
        offs[E] = t0;
        poffs[E] = t1;
        mtstart[E] = t2;
    }
    for (int c0 = 0; c0 < nslots; c0 += blockDim.x) {
        for (int idx = tid; idx < 32 * E; idx += blockDim.x) s_wcnt[idx] = 0;
        __syncthreads();
        const int i = c0 + tid;
        const bool valid = i < nslots;
        const int e = valid ? ids[i] : -1;
        const bool good = valid && e >= 0 && e < E;
        const uint32_t mask = __match_any_sync(0xffffffffu, good ? e : E + lane);
        const int rank_w = __popc(mask & ((1u << lane) - 1u));
        if (good && lane == __ffs(mask) - 1) s_wcnt[warp * E + e] = __popc(mask);
        __syncthreads();
        if (good) {
            int p = s_run[e] + rank_w;
            for (int w2 = 0; w2 < warp; ++w2) p += s_wcnt[w2 * E + e];
            perm[s_off[e] + p] = i;
            inv[i] = s_poff[e] + p;
            row_src[s_poff[e] + p] = i;
        } else if (valid) {
            inv[i] = -1;
        }
        __syncthreads();
        for (int ee = tid; ee < E; ee += blockDim.x) {
            int add = 0;
            for (int w2 = 0; w2 < 32; ++w2) add += s_wcnt[w2 * E + ee];
            s_run[ee] += add;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// a2 / a6 in the layer: per-row symmetric INT8 into the tiled token rows.  One CTA
// of 128 threads per grouped row; thread t owns the 16-value chunks t, t+128, ...
// of the row and keeps up to kRowCache of them in registers between the max pass
// and the quantisation pass.  Pad rows (row_src < 0) get zero codes and scale 0.
// ---------------------------------------------------------------------------
constexpr int kRowCache = 4;

struct Chunk16 {
    float v[16];
};

// (aligned: the row starts on 16 bytes, whatever its length)
__device__ __forceinline__ void load_chunk(const uint16_t* row, int len, int k0, Chunk16& c, bool aligned = false) {
    if ((aligned || (len & 15) == 0) && k0 + 16 <= len) {
        const uint4 p0 = *reinterpret_cast<const uint4*>(row + k0);
        const uint4 p1 = *reinterpret_cast<const uint4*>(row + k0 + 8);
        const uint32_t pw[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            c.v[2 * h] = bf16_to_f32((uint16_t)(pw[h] & 0xFFFFu));
            c.v[2 * h + 1] = bf16_to_f32((uint16_t)(pw[h] >> 16));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) c.v[i] = (k0 + i < len) ? bf16_to_f32(row[k0 + i]) : 0.f;
    }
}
__device__ __forceinline__ void load_chunk(const float* row, int len, int k0, Chunk16& c) {
    if ((len & 15) == 0 && k0 + 16 <= len) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 p = *reinterpret_cast<const float4*>(row + k0 + 4 * i);
            c.v[4 * i] = p.x; c.v[4 * i + 1] = p.y; c.v[4 * i + 2] = p.z; c.v[4 * i + 3] = p.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) c.v[i] = (k0 + i < len) ? row[k0 + i] : 0.f;
    }
}

// scale of a row with largest magnitude amax: the correctly rounded quotient amax / 127,
// or (W8A8) the fp32 product amax * (1 / 127)
template <bool kW8>
__device__ __forceinline__ float row_scale(float amax) {
    return kW8 ? __fmul_rn(amax, kInv127) : __fdiv_rn(amax, 127.0f);
}

// the larger of amax and |v|: NaN are passed over, or (W8A8) larger than everything, as the
// magnitudes' bits order them
template <bool kW8>
__device__ __forceinline__ float larger(float amax, float v) {
    if (kW8) return __uint_as_float(max(__float_as_uint(amax), __float_as_uint(fabsf(v))));
    return fmaxf(amax, fabsf(v));
}

template <int kCache, bool kW8, typename TIn>
__device__ __forceinline__ void quant_row_cta(const TIn* row, int len, int Kp, int r, int RB,
                                              int8_t* __restrict__ act, float* __restrict__ s) {
    __shared__ float red[4];
    const int nch = Kp / 16;
    const int G = Kp / kGroup;
    const int t = threadIdx.x;
    Chunk16 cache[kCache];
    float amax = 0.f;
    if (row != nullptr) {
#pragma unroll
        for (int c = 0; c < kCache; ++c) {
            const int ci = t + c * 128;
            if (ci < nch) {
                load_chunk(row, len, ci * 16, cache[c], kW8);
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = larger<kW8>(amax, cache[c].v[i]);
            }
        }
        for (int ci = t + kCache * 128; ci < nch; ci += 128) {
            Chunk16 tmp;
            load_chunk(row, len, ci * 16, tmp, kW8);
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = larger<kW8>(amax, tmp.v[i]);
        }
    }
    amax = kW8 ? __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))) : warp_max(amax);
    if ((t & 31) == 0) red[t >> 5] = amax;
    __syncthreads();
    amax = larger<kW8>(larger<kW8>(red[0], red[1]), larger<kW8>(red[2], red[3]));
    const float sc = row_scale<kW8>(amax);
    const float rinv = __fdiv_rn(1.0f, sc);
    auto emit = [&](int ci, const Chunk16& c) {
        uint32_t out[4] = {0u, 0u, 0u, 0u};
        if (amax > 0.f && (!kW8 || amax < INFINITY)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t q = (uint32_t)(quant_i8_fast(c.v[i], sc, rinv) & 0xFF);
                out[i >> 2] |= q << (8 * (i & 3));
            }
        }
        *reinterpret_cast<uint4*>(act + act_offset(r, ci * 16, G, RB)) = make_uint4(out[0], out[1], out[2], out[3]);
    };
#pragma unroll
    for (int c = 0; c < kCache; ++c) {
        const int ci = t + c * 128;
        if (ci < nch) {
            if (row == nullptr) {
#pragma unroll
                for (int i = 0; i < 16; ++i) cache[c].v[i] = 0.f;
            }
            emit(ci, cache[c]);
        }
    }
    for (int ci = t + kCache * 128; ci < nch; ci += 128) {
        Chunk16 tmp;
        if (row != nullptr) load_chunk(row, len, ci * 16, tmp, kW8);
        else {
#pragma unroll
            for (int i = 0; i < 16; ++i) tmp.v[i] = 0.f;
        }
        emit(ci, tmp);
    }
    if (t == 0) s[r] = sc;
}

// x rows (bf16) -> INT8 rows in expert-grouped order.  CTA t < T quantises token t
// once (one read of x) and writes the codes to each of its k grouped rows; CTA T + e
// writes zero codes and scale 0 into the pad rows of expert e.
__global__ void __launch_bounds__(128) act_scatter_kernel(const uint16_t* __restrict__ x, int T, int H, int Kp, int k,
                                                          const int* __restrict__ inv,
                                                          const int* __restrict__ offs,
                                                          const int* __restrict__ poffs, int RB,
                                                          int8_t* __restrict__ act, float* __restrict__ s) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int nch = Kp / 16;
    const int G = Kp / kGroup;
    const int t = threadIdx.x;
    if ((int)blockIdx.x >= T) {
        const int e = (int)blockIdx.x - T;
        const int r0 = __ldg(poffs + e) + (__ldg(offs + e + 1) - __ldg(offs + e));
        const int r1 = __ldg(poffs + e + 1);
        for (int r = r0; r < r1; ++r) {
            for (int ci = t; ci < nch; ci += 128)
                *reinterpret_cast<uint4*>(act + act_offset(r, ci * 16, G, RB)) = make_uint4(0u, 0u, 0u, 0u);
            if (t == 0) s[r] = 0.f;
        }
        return;
    }
    const int tok = blockIdx.x;
    const uint16_t* row = x + (size_t)tok * H;
    __shared__ int dst[32];
    __shared__ float red[4];
    if (t < k) dst[t] = __ldg(inv + (size_t)tok * k + t);
    Chunk16 cache[kRowCache];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < kRowCache; ++c) {
        const int ci = t + c * 128;
        if (ci < nch) {
            load_chunk(row, H, ci * 16, cache[c]);
#pragma unroll
            for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(cache[c].v[i]));
        }
    }
    for (int ci = t + kRowCache * 128; ci < nch; ci += 128) {
        Chunk16 tmp;
        load_chunk(row, H, ci * 16, tmp);
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(tmp.v[i]));
    }
    amax = warp_max(amax);
    if ((t & 31) == 0) red[t >> 5] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float sc = __fdiv_rn(amax, 127.0f);
    const float rinv = __fdiv_rn(1.0f, sc);
    auto emit = [&](int ci, const Chunk16& c) {
        uint32_t out[4] = {0u, 0u, 0u, 0u};
        if (amax > 0.f) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t q = (uint32_t)(quant_i8_fast(c.v[i], sc, rinv) & 0xFF);
                out[i >> 2] |= q << (8 * (i & 3));
            }
        }
        const uint4 o = make_uint4(out[0], out[1], out[2], out[3]);
        for (int j = 0; j < k; ++j) {
            const int r = dst[j];
            if (r >= 0) *reinterpret_cast<uint4*>(act + act_offset(r, ci * 16, G, RB)) = o;
        }
    };
#pragma unroll
    for (int c = 0; c < kRowCache; ++c) {
        const int ci = t + c * 128;
        if (ci < nch) emit(ci, cache[c]);
    }
    for (int ci = t + kRowCache * 128; ci < nch; ci += 128) {
        Chunk16 tmp;
        load_chunk(row, H, ci * 16, tmp);
        emit(ci, tmp);
    }
    if (t < k && dst[t] >= 0) s[dst[t]] = sc;
}

// h rows (fp32, SwiGLU output of the up GEMM) -> INT8 rows for the down GEMM
// (kCache chunks of 16 per thread stay in registers: 1 covers F <= 2048)
template <int kCache, bool kW8>
__global__ void __launch_bounds__(128) requant_kernel(const uint16_t* __restrict__ h, int ldh, int F, int Kp,
                                                      const int* __restrict__ row_src, const int* __restrict__ poffs,
                                                      int E, int RB, int8_t* __restrict__ act, float* __restrict__ s) {
    if (kW8) grid_dep_launch();
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int r = blockIdx.x;
    if (r >= __ldg(poffs + E)) return;
    if (kW8 && row_src[r] < 0) return;  // (a pad row's codes and scale reach no output that is stored)
    quant_row_cta<kCache, kW8, uint16_t>(row_src[r] < 0 ? nullptr : h + (size_t)r * ldh, F, Kp, r, RB, act, s);
}

// ---------------------------------------------------------------------------
// W8A8 layer: rows kept as the bf16 pairs that were loaded, 16 values (two 16-byte words) at a
// time, and quantised with a rounding constant.
// ---------------------------------------------------------------------------
struct Raw16 {
    uint32_t w[8];
};

// 16 values of a row from k0 on, zero past len (aligned: the row starts on 16 bytes)
__device__ __forceinline__ void load_raw(const uint16_t* row, int len, int k0, bool aligned, Raw16& c) {
    if (aligned && k0 + 16 <= len) {
        const uint4 p0 = *reinterpret_cast<const uint4*>(row + k0);
        const uint4 p1 = *reinterpret_cast<const uint4*>(row + k0 + 8);
        c.w[0] = p0.x; c.w[1] = p0.y; c.w[2] = p0.z; c.w[3] = p0.w;
        c.w[4] = p1.x; c.w[5] = p1.y; c.w[6] = p1.z; c.w[7] = p1.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = k0 + 2 * i < len ? row[k0 + 2 * i] : 0u, hi = k0 + 2 * i + 1 < len ? row[k0 + 2 * i + 1] : 0u;
            c.w[i] = lo | (hi << 16);
        }
    }
}

// The largest magnitude of a row as bf16 bits, which order magnitudes, infinity above them and
// NaN above that: the row's scale tells of either (`m`: two maxima side by side).
__device__ __forceinline__ uint32_t raw_max(const Raw16& c, uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, c.w[i] & 0x7FFF7FFFu);
    return m;
}
__device__ __forceinline__ uint32_t warp_max_raw(uint32_t m) { return __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xFFFFu)); }
// Rows with a NaN or an infinity, and rows of zeros, have codes 0; with the first two's scale
// every output that they enter is 0 * NaN or 0 * infinity.
__device__ __forceinline__ bool raw_has_codes(uint32_t bits) { return bits > 0u && bits < 0x7F80u; }

// INT8 codes of 16 values, the codes of quant_i8 bit for bit, where no |value| exceeds the
// amax behind sc (so that nothing saturates).  t = x * inv + 1.5 * 2^23 holds rint(x * inv) in
// its low bits; a value within 6.1e-5 of a rounding boundary (see quant_i8_fast), or not
// finite, sends the chunk to the exact divisions: five instructions per value instead of
// twelve.
__device__ __forceinline__ uint4 quant16(const Raw16& c, float sc, float inv) {
    constexpr float kMagic = 12582912.0f;
    uint32_t out[4];
    bool exact = false;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t w = c.w[2 * g + i / 2];
            const float y = __fmul_rn(__uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16)), inv);
            const float t = __fadd_rn(y, kMagic);
            exact = exact || !(fabsf(__fsub_rn(y, __fsub_rn(t, kMagic))) < 0.5f - 6.103515625e-05f);
            b[i] = __float_as_uint(t);
        }
        out[g] = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    }
    if (exact) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            out[g] = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t w = c.w[2 * g + i / 2];
                out[g] |= (uint32_t)(quant_i8(__uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16)), sc) & 0xFF) << (8 * i);
            }
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Requantisation of short rows (F <= 512 * kChunks): a warp per row, which stays in registers.
// (With F = 256 a CTA per row spends its time on being launched: 12000 rows 20 us, so 12 us;
// launch_w8_requant() has the rule and both sides at longer rows.)
template <int kChunks>
__global__ void __launch_bounds__(256) requant_short_kernel(const uint16_t* __restrict__ h, int ldh, int F, int Kp,
                                                            const int* __restrict__ row_src, const int* __restrict__ poffs,
                                                            int E, int RB, int8_t* __restrict__ act, float* __restrict__ s) {
    grid_dep_launch();
    grid_dep_wait();
    const int r = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint16_t* row = h + (size_t)r * ldh;
    const int nch = Kp / 16;
    const bool exists = r < __ldg(poffs + E);  // (false: inside the workspace all the same, or past it)
    if (!exists) return;
    const int src = row_src[r];  // (a pad row is read, not written)
    Raw16 c[kChunks];
    uint32_t m = 0u;
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
        if (lane + 32 * q < nch) load_raw(row, F, (lane + 32 * q) * 16, true, c[q]);
    if (src < 0) return;
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
        if (lane + 32 * q < nch) m = raw_max(c[q], m);
    m = warp_max_raw(m);
    const float sc = row_scale<true>(__uint_as_float(m << 16));
    const float rinv = __fdiv_rn(1.0f, sc);
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
        const int ci = lane + 32 * q;
        if (ci < nch)
            *reinterpret_cast<uint4*>(act + act_offset(r, ci * 16, Kp / kGroup, RB)) =
                raw_has_codes(m) ? quant16(c[q], sc, rinv) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (lane == 0) s[r] = sc;
}

// Activation quantisation of short rows (H <= 512 * kChunks): a warp per token, its row in
// registers, written to the token's k places.
template <int kChunks>
__global__ void __launch_bounds__(256) act_scatter_short_kernel(const uint16_t* __restrict__ x, int T, int H, int Kp, int k,
                                                                const int* __restrict__ inv, int RB, int8_t* __restrict__ act,
                                                                float* __restrict__ s) {
    grid_dep_launch();
    grid_dep_wait();
    const int tok = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (tok >= T) return;
    const uint16_t* row = x + (size_t)tok * H;
    const int nch = Kp / 16, G = Kp / kGroup;
    const int my_dst = lane < k ? __ldg(inv + (size_t)tok * k + lane) : -1;
    Raw16 c[kChunks];
    uint32_t m = 0u;
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
        if (lane + 32 * q < nch) load_raw(row, H, (lane + 32 * q) * 16, (H & 7) == 0, c[q]);
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
        if (lane + 32 * q < nch) m = raw_max(c[q], m);
    m = warp_max_raw(m);
    const float sc = row_scale<true>(__uint_as_float(m << 16));
    const float rinv = __fdiv_rn(1.0f, sc);
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
        const int ci = lane + 32 * q;
        const uint4 o = ci < nch && raw_has_codes(m) ? quant16(c[q], sc, rinv) : make_uint4(0u, 0u, 0u, 0u);
        for (int j = 0; j < k; ++j) {
            const int r = __shfl_sync(0xffffffffu, my_dst, j);
            if (r >= 0 && ci < nch) *reinterpret_cast<uint4*>(act + act_offset(r, ci * 16, G, RB)) = o;
        }
    }
    if (my_dst >= 0) s[my_dst] = sc;
}

// The quantisation of one row by a CTA of 256 threads, written to the places dst[0 .. k): two
// chunks per thread in registers (loaded by the caller), longer rows read again.
__device__ __forceinline__ void quant_row_places(const uint16_t* row, int H, int Kp, int k, const Raw16 (&cache)[2],
                                                 const int* dst, uint32_t* red, int RB, int8_t* __restrict__ act,
                                                 float* __restrict__ s) {
    const int tid = threadIdx.x, nch = Kp / 16, G = Kp / kGroup;
    const bool aligned = (H & 7) == 0;
    uint32_t m = 0u;
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (tid + c * 256 < nch) m = raw_max(cache[c], m);
    for (int ci = tid + 512; ci < nch; ci += 256) {
        Raw16 tmp;
        load_raw(row, H, ci * 16, aligned, tmp);
        m = raw_max(tmp, m);
    }
    m = warp_max_raw(m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();  // (dst, too, is complete)
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, red[w]);
    const float sc = row_scale<true>(__uint_as_float(m << 16));
    const float rinv = __fdiv_rn(1.0f, sc);
    auto emit = [&](int ci, const Raw16& c) {
        const uint4 q = raw_has_codes(m) ? quant16(c, sc, rinv) : make_uint4(0u, 0u, 0u, 0u);
        for (int j = 0; j < k; ++j)
            if (dst[j] >= 0) *reinterpret_cast<uint4*>(act + act_offset(dst[j], ci * 16, G, RB)) = q;
    };
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (tid + c * 256 < nch) emit(tid + c * 256, cache[c]);
    for (int ci = tid + 512; ci < nch; ci += 256) {
        Raw16 tmp;
        load_raw(row, H, ci * 16, aligned, tmp);
        emit(ci, tmp);
    }
    if (tid < k && dst[tid] >= 0) s[dst[tid]] = sc;
}

// Activation quantisation, a CTA per token.  Pad rows are left alone: they reach no output
// that is stored.
__global__ void __launch_bounds__(256) act_scatter_w8_kernel(const uint16_t* __restrict__ x, int H, int Kp, int k,
                                                             const int* __restrict__ inv, int RB, int8_t* __restrict__ act,
                                                             float* __restrict__ s) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ int dst[32];
    __shared__ uint32_t red[8];
    const int tid = threadIdx.x, nch = Kp / 16;
    const uint16_t* row = x + (size_t)blockIdx.x * H;
    Raw16 cache[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (tid + c * 256 < nch) load_raw(row, H, (tid + c * 256) * 16, (H & 7) == 0, cache[c]);
    if (tid < k) dst[tid] = __ldg(inv + (size_t)blockIdx.x * k + tid);
    quant_row_places(row, H, Kp, k, cache, dst, red, RB, act, s);
}

// ---------------------------------------------------------------------------
// W8A8 layer, up to kPrepareSlots slots: the permutation and the activation quantisation in
// one kernel.  CTA t quantises token t; every CTA counts all ids for itself (a few thousand
// integers from L2, cheaper than a kernel of its own in front: 8 us of the one-token layer's
// chain), and a slot's place among its expert's rows is the number of earlier slots with the
// same id, so the grouping is that of the permutation kernels.  CTA 0 writes the tables and
// the error word.  Pad rows are not written: nothing that depends on them is ever read.
// ---------------------------------------------------------------------------
// exclusive scan over 256 threads
__device__ __forceinline__ int scan256(int v, int* sh, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < warp) before += sh[w];
        all += sh[w];
    }
    *total = all;
    return before + incl - v;
}

__global__ void __launch_bounds__(256) w8_prepare_kernel(const int32_t* __restrict__ ids, const uint16_t* __restrict__ x,
                                                         int T, int H, int Kp, int k, int E, int tile_tokens,
                                                         int* __restrict__ counts, int* __restrict__ offs,
                                                         int* __restrict__ poffs, int* __restrict__ mtstart,
                                                         int4* __restrict__ mt_tab, int* __restrict__ perm,
                                                         int* __restrict__ inv, int* __restrict__ row_src, int RB,
                                                         int8_t* __restrict__ act, float* __restrict__ s,
                                                         uint32_t* __restrict__ err) {
    grid_dep_launch();
    grid_dep_wait();
    __shared__ int s_ids[kPrepareSlots];
    __shared__ int s_off[kMaxExperts], s_poff[kMaxExperts];  // counts first, then offsets
    __shared__ int sh[8], dst[32], s_bad;
    __shared__ uint32_t red[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tok = blockIdx.x, nslots = T * k;
    const int nch = Kp / 16;
    const uint16_t* row = x + (size_t)tok * H;
    // the token's row, loading while the ids are counted
    Raw16 cache[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (tid + c * 256 < nch) load_raw(row, H, (tid + c * 256) * 16, (H & 7) == 0, cache[c]);
    if (tid == 0) s_bad = 0;
    for (int e = tid; e < E; e += 256) s_off[e] = 0;
    __syncthreads();
    for (int i = tid; i < nslots; i += 256) {
        const int e = __ldg(ids + i);
        const bool good = e >= 0 && e < E;
        s_ids[i] = good ? e : -1;
        if (good) atomicAdd(&s_off[e], 1);
        else s_bad = 1;
    }
    __syncthreads();
    // thread t scans experts 4t .. 4t + 3
    int c4[4], o = 0, p = 0, m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c4[i] = 4 * tid + i < E ? s_off[4 * tid + i] : 0;
        o += c4[i];
        p += round_up(c4[i], kRowPad);
        m += ceil_div(c4[i], tile_tokens);
    }
    int ot, pt, mt;
    o = scan256(o, sh, &ot);
    p = scan256(p, sh, &pt);
    if (tok == 0) m = scan256(m, sh, &mt);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * tid + i;
        if (e < E) {
            if (tok == 0) {
                counts[e] = c4[i];
                offs[e] = o;
                poffs[e] = p;
                mtstart[e] = m;
                for (int r = p + c4[i]; r < p + round_up(c4[i], kRowPad); ++r) row_src[r] = -1;
                for (int q = 0; q < ceil_div(c4[i], tile_tokens); ++q)
                    mt_tab[m + q] = make_int4(e, p + q * tile_tokens, min(tile_tokens, c4[i] - q * tile_tokens), 0);
            }
            s_off[e] = o;
            s_poff[e] = p;
            o += c4[i];
            p += round_up(c4[i], kRowPad);
            m += ceil_div(c4[i], tile_tokens);
        }
    }
    if (tok == 0 && tid == 0) {
        offs[E] = ot;
        poffs[E] = pt;
        mtstart[E] = mt;
        *err = s_bad ? kErrBadExpert : 0u;
    }
    __syncthreads();
    // a warp per slot of the token: how many earlier slots chose the same expert
    for (int j = warp; j < k; j += 8) {
        const int slot = tok * k + j, e = s_ids[slot];
        int n = 0;
        for (int i = lane; i < slot; i += 32) n += s_ids[i] == e;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) n += __shfl_xor_sync(0xffffffffu, n, w);
        if (lane == 0) {
            const int r = e >= 0 ? s_poff[e] + n : -1;
            dst[j] = r;
            inv[slot] = r;
            if (e >= 0) {
                perm[s_off[e] + n] = slot;
                row_src[r] = slot;
            }
        }
    }
    quant_row_places(row, H, Kp, k, cache, dst, red, RB, act, s);
}

// ---------------------------------------------------------------------------
// a8: out[t] = sum_j w[t][j] * y2[inv[t*k+j]]  (fp32, j ascending) -> bf16
// ---------------------------------------------------------------------------
template <bool kW8>
__global__ void __launch_bounds__(256) combine_kernel(const float* __restrict__ y2, int H, const int* __restrict__ inv,
                                                      const float* __restrict__ w, int T, int k,
                                                      uint16_t* __restrict__ out) {
    if (kW8) grid_dep_launch();
    grid_dep_wait();  // the previous kernel of the forward has completed
    __shared__ int rows[32];
    __shared__ float wts[32];
    const int t = blockIdx.x;
    if (threadIdx.x < k) {
        rows[threadIdx.x] = inv[(size_t)t * k + threadIdx.x];
        wts[threadIdx.x] = w[(size_t)t * k + threadIdx.x];
    }
    __syncthreads();
    const bool vec = (H & 7) == 0;
    for (int c0 = (blockIdx.y * blockDim.x + threadIdx.x) * 8; c0 < H; c0 += gridDim.y * blockDim.x * 8) {
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const int rr = rows[j];
            if (rr < 0) continue;
            const float wt = wts[j];
            const float* row = y2 + (size_t)rr * H + c0;
            if (vec) {
                const float4 a = *reinterpret_cast<const float4*>(row);
                const float4 b = *reinterpret_cast<const float4*>(row + 4);
                acc[0] = fmaf(wt, a.x, acc[0]); acc[1] = fmaf(wt, a.y, acc[1]);
                acc[2] = fmaf(wt, a.z, acc[2]); acc[3] = fmaf(wt, a.w, acc[3]);
                acc[4] = fmaf(wt, b.x, acc[4]); acc[5] = fmaf(wt, b.y, acc[5]);
                acc[6] = fmaf(wt, b.z, acc[6]); acc[7] = fmaf(wt, b.w, acc[7]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + i < H) acc[i] = fmaf(wt, row[i], acc[i]);
            }
        }
        uint16_t* o = out + (size_t)t * H + c0;
        if (vec) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                pk[i] = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * i])) |
                        ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(acc[2 * i + 1])) << 16);
            *reinterpret_cast<uint4*>(o) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c0 + i < H) o[i] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i]));
        }
    }
}

// dense GEMM: copy INT8 rows into the tiled planes (pad rows zero) and describe
// them as one "expert" with M rows.
__global__ void __launch_bounds__(256) dense_prep_kernel(const int8_t* __restrict__ qa, int M, int Kq, int Kp, int tile_tokens,
                                                         int RB, int8_t* __restrict__ act, int4* mt_tab, int* n_mtiles) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int Mp = round_up(M, kRowPad);
    const int nch = Kp / 16;
    const size_t idx = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int nmt = ceil_div(M, tile_tokens);
    if (idx == 0) *n_mtiles = nmt;
    if (idx < (size_t)nmt) mt_tab[idx] = make_int4(0, (int)idx * tile_tokens, min(tile_tokens, M - (int)idx * tile_tokens), 0);
    if (idx >= (size_t)Mp * nch) return;
    const int r = (int)(idx / nch);
    const int ci = (int)(idx % nch);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < M && ci * 16 < Kq) v = *reinterpret_cast<const uint4*>(qa + (size_t)r * Kq + ci * 16);
    *reinterpret_cast<uint4*>(act + act_offset(r, ci * 16, Kp / kGroup, RB)) = v;
}

// ---------------------------------------------------------------------------
// W4A16 token rows: bf16 values copied (not quantised) into the tiled bf16 layout
// of act16_offset, 16-row blocks, 8 values (16 bytes) per thread and step.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint4 load8_bf16(const uint16_t* row, int len, int k0) {
    if ((len & 7) == 0 && k0 + 8 <= len) return *reinterpret_cast<const uint4*>(row + k0);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = k0 + 2 * i < len ? row[k0 + 2 * i] : 0u;
        const uint32_t hi = k0 + 2 * i + 1 < len ? row[k0 + 2 * i + 1] : 0u;
        w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// CTA t copies token t's row to each of its k grouped rows (pad K columns zero) and
// zeroes the pad columns [F, Fp) of the same rows of the h buffer, which the up
// projection's epilogue leaves unwritten (chunks that straddle F are zeroed whole;
// the epilogue writes their valid part afterwards, in stream order)
__global__ void __launch_bounds__(128) act_gather_bf16_kernel(const uint16_t* __restrict__ x, int H, int k,
                                                              const int* __restrict__ inv, uint8_t* __restrict__ x16,
                                                              uint8_t* __restrict__ h16, int F) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int Hp = round_up(H, kGroup), G1 = Hp / kGroup;
    const int Fp = round_up(F, kGroup), G2 = Fp / kGroup;
    const int tok = blockIdx.x;
    __shared__ int dst[32];
    if ((int)threadIdx.x < k) dst[threadIdx.x] = __ldg(inv + (size_t)tok * k + threadIdx.x);
    __syncthreads();
    const uint16_t* row = x + (size_t)tok * H;
    for (int ci = threadIdx.x; ci < Hp / 8; ci += blockDim.x) {
        const uint4 v = load8_bf16(row, H, ci * 8);
        for (int j = 0; j < k; ++j) {
            const int r = dst[j];
            if (r >= 0) *reinterpret_cast<uint4*>(x16 + act16_offset(r, ci * 8, G1, 16)) = v;
        }
    }
    for (int ci = F / 8 + threadIdx.x; ci < Fp / 8; ci += blockDim.x) {
        for (int j = 0; j < k; ++j) {
            const int r = dst[j];
            if (r >= 0) *reinterpret_cast<uint4*>(h16 + act16_offset(r, ci * 8, G2, 16)) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

// dense W4A16 GEMM: x rows into the tiled bf16 layout (pad rows and columns zero),
// described as one "expert" of 16-row tiles
__global__ void __launch_bounds__(256) dense_prep_bf16_kernel(const uint16_t* __restrict__ x, int M, int K,
                                                              uint8_t* __restrict__ act16, int4* mt_tab,
                                                              int* n_mtiles) {
    grid_dep_wait();  // the previous kernel of the forward has completed
    const int Kp = round_up(K, kGroup), G = Kp / kGroup;
    const int Mp = round_up(M, kRowPad);
    const int nch = Kp / 8;
    const size_t idx = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int nmt = ceil_div(M, 16);
    if (idx == 0) *n_mtiles = nmt;
    if (idx < (size_t)nmt) mt_tab[idx] = make_int4(0, (int)idx * 16, min(16, M - (int)idx * 16), 0);
    if (idx >= (size_t)Mp * nch) return;
    const int r = (int)(idx / nch);
    const int ci = (int)(idx % nch);
    const uint4 v = r < M ? load8_bf16(x + (size_t)r * K, K, ci * 8) : make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(act16 + act16_offset(r, ci * 8, G, 16)) = v;
}

}  // namespace

// ------------------------------- launchers ---------------------------------
cudaError_t launch_pack(const uint16_t* w, int E, int N, int K, int layout, int scheme, int group, uint8_t* packed,
                        uint8_t* codes, uint16_t* scale, uint16_t* zp, cudaStream_t stream) {
    const int G = k_padded_for(K, group) / kGroup;
    const int NT = layout == 1 ? ceil_div(N / 2, kTileRows / 2) : ceil_div(N, kTileRows);
    dim3 grid(G * kGroup / group, NT, E);
    uint8_t* blocks = packed + kHeaderBytes;
    if (group == 64)
        pack_kernel<64><<<grid, 128, 0, stream>>>(w, N, K, layout, scheme, NT, G, blocks, codes, scale, zp);
    else if (group == 256)
        pack_kernel<256><<<grid, 128, 0, stream>>>(w, N, K, layout, scheme, NT, G, blocks, codes, scale, zp);
    else
        pack_kernel<128><<<grid, 128, 0, stream>>>(w, N, K, layout, scheme, NT, G, blocks, codes, scale, zp);
    return cudaGetLastError();
}

cudaError_t launch_quant_act(const uint16_t* x, int T, int K, int8_t* q, float* s, cudaStream_t stream) {
    return launch_pdl(quant_act_kernel, ceil_div(T, 8), 256, 0, stream, x, T, K, round_up(K, kGroup), q, s);
}

cudaError_t launch_route_topk(const uint16_t* logits, int T, int E, int k, int32_t* ids, float* w,
                              cudaStream_t stream) {
    return launch_pdl(route_topk_kernel, ceil_div(T, 8), 256, 0, stream, logits, T, E, k, ids, w);
}

int perm_launch_count(int nslots, int small_slots) { return nslots <= small_slots ? 1 : 3; }
int perm_launch_count(int nslots) { return perm_launch_count(nslots, kPermSmallSlots); }

cudaError_t launch_perm(const int32_t* ids, int nslots, int E, int tile_tokens, int* chist, int nchunk, int* counts,
                        int* offs, int* poffs, int* mtstart, int4* mt_tab, int* perm, int* inv, int* row_src,
                        uint32_t* err, cudaStream_t stream, int small_slots) {
    if (nslots <= small_slots) {
        const size_t smem = (size_t)35 * E * sizeof(int);
        static int attr_done[64] = {0};
        int dev = 0;
        cudaGetDevice(&dev);
        if (dev < 0 || dev >= 64 || !attr_done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(perm_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       35 * kMaxExperts * (int)sizeof(int));
            if (e != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) attr_done[dev] = 1;
        }
        return launch_pdl(perm_small_kernel, 1, 1024, smem, stream, ids, nslots, E, tile_tokens, counts, offs, poffs,
                          mtstart, mt_tab, perm, inv, row_src, err);
    }
    cudaError_t e = launch_pdl(perm_hist_kernel, nchunk, kPermChunk, 0, stream, ids, nslots, E, chist, err);
    if (e != cudaSuccess) return e;
    e = launch_pdl(perm_scan_kernel, 1, 1024, 0, stream, chist, nchunk, E, tile_tokens, counts, offs, poffs, mtstart,
                   mt_tab, row_src);
    if (e != cudaSuccess) return e;
    return launch_pdl(perm_scatter_kernel, nchunk, kPermChunk, 0, stream, ids, nslots, E, chist, offs, poffs, perm, inv,
                      row_src);
}

cudaError_t launch_perm(const int32_t* ids, int nslots, int E, int tile_tokens, int* chist, int nchunk, int* counts,
                        int* offs, int* poffs, int* mtstart, int4* mt_tab, int* perm, int* inv, int* row_src,
                        uint32_t* err, cudaStream_t stream) {
    return launch_perm(ids, nslots, E, tile_tokens, chist, nchunk, counts, offs, poffs, mtstart, mt_tab, perm, inv, row_src,
                       err, stream, kPermSmallSlots);
}

cudaError_t launch_act_scatter(const uint16_t* x, int T, int H, int Kp, int k, const int* inv, const int* offs,
                               const int* poffs, int E, int rb, int8_t* act, float* s, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    return launch_pdl(act_scatter_kernel, T + E, 128, 0, stream, x, T, H, Kp, k, inv, offs, poffs, rb, act, s);
}

cudaError_t launch_w8_act_scatter(const uint16_t* x, int T, int H, int Kp, int k, const int* inv, int rb, int8_t* act, float* s,
                                  cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    // 3000 tokens of 1024 values to 4 places each: 12.7 us with a warp per token, 16 us with a CTA
    if (H <= 1024)
        return launch_pdl(H <= 512 ? act_scatter_short_kernel<1> : act_scatter_short_kernel<2>, ceil_div(T, 8), 256, 0, stream, x,
                          T, H, Kp, k, inv, rb, act, s);
    return launch_pdl(act_scatter_w8_kernel, T, 256, 0, stream, x, H, Kp, k, inv, rb, act, s);
}

cudaError_t launch_w8_prepare(const int32_t* ids, const uint16_t* x, int T, int H, int Kp, int k, int E, int tile_tokens,
                              int* counts, int* offs, int* poffs, int* mtstart, int4* mt_tab, int* perm, int* inv, int* row_src,
                              int rb, int8_t* act, float* s, uint32_t* err, cudaStream_t stream) {
    return launch_pdl(w8_prepare_kernel, T, 256, 0, stream, ids, x, T, H, Kp, k, E, tile_tokens, counts, offs, poffs, mtstart,
                      mt_tab, perm, inv, row_src, rb, act, s, err);
}

cudaError_t launch_requant(const uint16_t* h, int ldh, int F, int Kp, const int* row_src, const int* poffs, int E,
                           int rows_cap, int rb, int8_t* act, float* s, cudaStream_t stream) {
    if (rows_cap == 0) return cudaSuccess;
    return launch_pdl(F <= 128 * 16 ? requant_kernel<1, false> : requant_kernel<kRowCache, false>, rows_cap, 128, 0, stream, h,
                      ldh, F, Kp, row_src, poffs, E, rb, act, s);
}

cudaError_t launch_w8_requant(const uint16_t* h, int ldh, int F, int Kp, const int* row_src, const int* poffs, int E,
                              int rows_cap, int rb, int8_t* act, float* s, cudaStream_t stream) {
    if (rows_cap == 0) return cudaSuccess;
    // A warp per row up to F = 2048, unless a CTA per row fits the GPU at once and a row keeps
    // most of a CTA busy (F > 1024). CTA against warp at F = 1408: 384 rows 8.7 against 10.5 us,
    // 1536 rows 10.7 and 10.8, 3840 rows 14.7 and 12.7, 49152 rows (F = 1536) 104.7 and 60.9; at
    // F = 2048: 1920 rows 11.5 and 12.3, 3840 rows 16.4 and 14.8; at F = 1024, 160 rows of 512
    // experts 8.7 both.
    if (F <= 2048 && (F <= 1024 || rows_cap > 16 * sm_count()))
        return launch_pdl(F <= 512    ? requant_short_kernel<1>
                          : F <= 1024 ? requant_short_kernel<2>
                                      : requant_short_kernel<4>,
                          ceil_div(rows_cap, 8), 256, 0, stream, h, ldh, F, Kp, row_src, poffs, E, rb, act, s);
    return launch_pdl(F <= 128 * 16 ? requant_kernel<1, true> : requant_kernel<kRowCache, true>, rows_cap, 128, 0, stream, h, ldh,
                      F, Kp, row_src, poffs, E, rb, act, s);
}

cudaError_t launch_combine(const float* y2, int H, const int* inv, const float* w, int T, int k, uint16_t* out,
                           cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    return launch_pdl(combine_kernel<false>, T, 256, 0, stream, y2, H, inv, w, T, k, out);
}

cudaError_t launch_w8_combine(const float* y2, int H, const int* inv, const float* w, int T, int k, uint16_t* out,
                              cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    // Few tokens are spread over several CTAs each.  The layer (F 256, 4 of 32 experts) with and
    // without: 1 token, H 7168, 33.1 and 36.7 us; 64 tokens 60.2 and 68.6, H 4096 47.9 and 51.9,
    // H 2048 (one CTA either way) 29.4; 290 tokens, H 7168, 69.4 and 79.4.  (Beyond the rule's two
    // CTAs per SM it would still gain: 600 tokens, H 7168, 92.6 and 102.5.)
    const dim3 grid(T, T < 2 * sm_count() ? ceil_div(H, 256 * 8) : 1);
    return launch_pdl(combine_kernel<true>, grid, 256, 0, stream, y2, H, inv, w, T, k, out);
}

cudaError_t launch_dense_prep(const int8_t* qa, int M, int Kq, int Kp, int tile_tokens, int rb, int8_t* act, int4* mt_tab,
                              int* n_mtiles, cudaStream_t stream) {
    const size_t n = (size_t)round_up(M, kRowPad) * (Kp / 16);
    return launch_pdl(dense_prep_kernel, (unsigned)((n + 255) / 256 + 1), 256, 0, stream, qa, M, Kq, Kp, tile_tokens, rb,
                      act, mt_tab, n_mtiles);
}

cudaError_t launch_dense_prep_bf16(const uint16_t* x, int M, int K, uint8_t* act16, int4* mt_tab, int* n_mtiles,
                                   cudaStream_t stream) {
    const size_t n = (size_t)round_up(M, kRowPad) * (round_up(K, kGroup) / 8);
    return launch_pdl(dense_prep_bf16_kernel, (unsigned)((n + 255) / 256 + 1), 256, 0, stream, x, M, K, act16, mt_tab,
                      n_mtiles);
}

cudaError_t launch_act_gather_bf16(const uint16_t* x, int T, int H, int k, const int* inv, uint8_t* x16, uint8_t* h16,
                                   int F, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    return launch_pdl(act_gather_bf16_kernel, T, 128, 0, stream, x, H, k, inv, x16, h16, F);
}

}  // namespace w4a8
