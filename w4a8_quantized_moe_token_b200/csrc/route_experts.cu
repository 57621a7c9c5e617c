// Routing to experts with softmax or sigmoid scores, a per-expert bias that enters the
// choice only, a restriction to the best groups of experts, and renormalised weights
// (w4a8_route_experts; the contract is in include/w4a8.h).
//
// One warp per token, its choice values in registers as order-preserving 32-bit keys, four
// consecutive experts per lane and step where E allows.  The k-th largest of the lanes' own
// maxima bounds the k-th largest value from below, so that only about k experts remain; each
// goes to a lane of its own, which counts how many of the others come before it.  (Rows in
// which more than 32 remain, for example of equal logits, take a round per expert.)
//
// The contract orders experts by their 64-bit choice values.  The values here are fp32 with
// an error of at most `delta` (from the documented bounds of __expf, expf and rcp.approx,
// doubled), so a gap of more than that between neighbours in the result decides their order
// for good, and equal inputs are true ties.  A row with a closer pair among the k chosen and
// the next one, or at the border of the kept groups, is done again in 64 bits (about one row
// in a few hundred for random inputs): exact order at the price of fp32 arithmetic.  Without
// a bias the keys are the logits themselves and nothing is ever in doubt.
//
// Bound by instruction issue, not by memory: 16384 x 384 fp32 logits (sigmoid, bias, 4 of 8
// groups) take 32-34 us on B200, 1482 warp instructions per token, for 4 us of bytes; one
// token 4.9 us, 64 x 64 (softmax) 3.2 us, both in a graph.  (At 40 registers the rare 64-bit
// functions, called out of line, cost every instance a stack frame of 104 to 128 bytes and some
// spills: 44 bytes stored and 100 loaded with 384 experts.)
#include <math_constants.h>

#include <type_traits>

#include "../../include/w4a8.h"
#include "layer_internal.h"
#include "w4a8_common.cuh"
#include "w4a8_internal.h"

namespace w4a8 {

namespace {

constexpr int kRouteWarps = 4;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

__device__ __forceinline__ bool masked(float v) { return !(v > -CUDART_INF_F); }  // -inf or NaN

// order-preserving keys of fp32 values (both zeros alike); kept below every real value:
constexpr uint32_t kKeyNone = 0, kKeyMasked = 1;
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

// doubles of shared memory per warp: E, and room for E floats and 32 ints; even (16-byte rows)
__host__ __device__ inline int route_smem_doubles(int E) {
    const int fl = (E + 1) / 2 + 16;
    return ((E > fl ? E : fl) + 1) / 2 * 2;
}

struct RouteArgs {
    const void* logits;
    const float* bias;
    int T, E, k, flags, n_group, topk_group;
    int gsize;        // experts per group
    uint32_t ginv;    // group of expert e: e * ginv >> 20
    float scale;
    int32_t* ids;
    float* w;
};

// 64-bit score of an unmasked expert; top = the largest logit of the row
__device__ __forceinline__ double score64(float x, float top, double sum, bool sigmoid) {
    if (sigmoid) return 1.0 / (1.0 + exp(-(double)x));
    return exp(x == top ? 0.0 : (double)x - (double)top) / sum;
}

// 64-bit sum of a row's exponentials relative to its largest logit
template <typename T>
__device__ __noinline__ double sum64(const T* x, int E, float top) {
    double sum = 0.0;
    for (int e = threadIdx.x & 31; e < E; e += 32) {
        const float v = to_f32(x[e]);
        if (!masked(v)) sum += score64(v, top, 1.0, false);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    return sum;
}

// The 64-bit choice values of a row into `choice` (E doubles of shared memory of this warp).
template <typename T>
__device__ __forceinline__ void choice64(const RouteArgs& a, const T* x, double* choice, float top, double sum) {
    __syncwarp();
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float v = to_f32(x[e]), b = a.bias != nullptr ? __ldg(a.bias + e) : 0.f;
        choice[e] = masked(v) || masked(b) ? -CUDART_INF
                                           : score64(v, top, sum, a.flags & W4A8_ROUTE_SIGMOID) + (double)b;
    }
    __syncwarp();
}

// The 64-bit score of group lane / lpg (lpg lanes scan a group).
template <typename T>
__device__ __noinline__ double group_score64(const RouteArgs& a, const T* x, double* choice, float top, int lpg) {
    choice64(a, x, choice, top, a.flags & W4A8_ROUTE_SIGMOID ? 1.0 : sum64(x, a.E, top));
    const int lane = threadIdx.x & 31, g = lane / lpg;
    double b0 = -CUDART_INF, b1 = -CUDART_INF;
    if (g < a.n_group) {
        for (int i = lane & (lpg - 1); i < a.gsize; i += lpg) {
            const double c = choice[g * a.gsize + i];
            b1 = fmax(b1, fmin(b0, c));
            b0 = fmax(b0, c);
        }
    }
    for (int o = 1; o < lpg; o <<= 1) {
        const double o0 = __shfl_xor_sync(kAll, b0, o), o1 = __shfl_xor_sync(kAll, b1, o);
        b1 = fmax(fmin(b0, o0), fmax(b1, o1));
        b0 = fmax(b0, o0);
    }
    __syncwarp();
    return (a.flags & W4A8_ROUTE_GROUP_TOP2) && b1 > -CUDART_INF ? b0 + b1 : b0;
}

// The choice of one row among the experts of the kept groups in 64 bits, a round per expert
// (rows with more than 32 experts in doubt): lane j < k returns the j-th, masked in
// *is_masked.  group_bit: the bit of group g in `kept` is g * group_bit.
template <typename T>
__device__ __noinline__ int route_row64(const RouteArgs& a, const T* x, double* choice, float top, double sum, uint32_t kept,
                                        int group_bit, bool* is_masked) {
    const int lane = threadIdx.x & 31, E = a.E;
    choice64(a, x, choice, top, sum);
    uint32_t taken = 0;
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        double bv = -CUDART_INF;
        int be = E;
        for (int e = lane, i = 0; e < E; e += 32, ++i) {
            if ((taken >> i) & 1u || !((kept >> ((((uint32_t)e * a.ginv) >> 20) * group_bit & 31)) & 1u)) continue;
            const double c = choice[e];
            if (be == E || c > bv) { bv = c; be = e; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(kAll, bv, o);
            const int oe = __shfl_xor_sync(kAll, be, o);
            if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; }
        }
        if ((be & 31) == lane) taken |= 1u << (be >> 5);
        if (lane == j) {
            mine = be;
            *is_masked = bv == -CUDART_INF;
        }
    }
    return mine;
}

__device__ __forceinline__ float rcp_approx(float v) {  // 1 ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// The logits of one row as loaded.  kVec: lane l owns experts 4 (32 i + l) .. + 3
// (E % 4 == 0), otherwise l, l + 32, ...
template <typename T, int kPL, bool kVec>
struct Row {
    using Vec = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
    Vec raw[kVec ? kPL / 4 : 1];
    T one[kVec ? 1 : kPL];

    static __device__ __forceinline__ int expert(int i, int lane) {
        return kVec ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane;
    }
    __device__ __forceinline__ void load(const T* x, int E, int lane) {
        if (kVec) {
#pragma unroll
            for (int i = 0; i < kPL / 4; ++i)
                if (expert(4 * i, lane) < E) raw[i] = __ldg(reinterpret_cast<const Vec*>(x + expert(4 * i, lane)));
        } else {
#pragma unroll
            for (int i = 0; i < kPL; ++i)
                if (expert(i, lane) < E) one[i] = x[expert(i, lane)];
        }
    }
    __device__ __forceinline__ void values(float (&v)[kPL], int E, int lane) const {
#pragma unroll
        for (int i = 0; i < kPL; ++i) {
            T t;
            if (kVec)
                t = reinterpret_cast<const T*>(&raw[i / 4])[i & 3];
            else
                t = one[i];
            v[i] = expert(i, lane) < E ? to_f32(t) : -CUDART_INF_F;
        }
    }
};

// (a row's own chain of loads and reductions takes about 3 us: warps in flight matter more
// than the registers of one)
template <typename T, int kPL, bool kVec>
__global__ void __launch_bounds__(kRouteWarps * 32, kPL <= 12 ? 12 : kPL <= 16 ? 8 : 4) route_experts_kernel(const RouteArgs a) {
    grid_dep_launch();
    grid_dep_wait();
    extern __shared__ double sm_choice[];
    const int lane = threadIdx.x & 31;
    const int E = a.E, k = a.k;
    const T* logits = static_cast<const T*>(a.logits);
    const bool sigmoid = a.flags & W4A8_ROUTE_SIGMOID, top2 = a.flags & W4A8_ROUTE_GROUP_TOP2;
    const bool by_logit = a.bias == nullptr && !top2;
    double* const sm64 = sm_choice + (size_t)(threadIdx.x >> 5) * route_smem_doubles(E);
    auto expert = [&](int i) { return Row<T, kPL, kVec>::expert(i, lane); };

    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const T* x = logits + (size_t)t * E;
    float v[kPL];
    {
        Row<T, kPL, kVec> row;
        row.load(x, E, lane);
        row.values(v, E, lane);
    }

    // scores, choice values and their keys
    float top = 0.f, inv_sum = 0.f, delta = 0.f;
    uint32_t key[kPL];
    if (!sigmoid) {
        top = -CUDART_INF_F;
#pragma unroll
        for (int i = 0; i < kPL; ++i) top = fmaxf(top, v[i]);  // (fmaxf passes over NaN)
        const uint32_t m = __reduce_max_sync(kAll, key_of(top));
        top = value_of(m);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPL; ++i) {
            const float p = masked(v[i]) ? 0.f : expf(v[i] == top ? 0.f : v[i] - top);
            sum += p;
            key[i] = __float_as_uint(p);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        inv_sum = sum > 0.f ? __fdiv_rn(1.0f, sum) : 0.f;
        // scores s = e^-d / sum: expf 2 ulp, the difference d half an ulp of it (s d <= 0.37 of
        // the largest score), at most 37 additions, the quotient and product: below
        // 32 * 2^-23 of the largest score, 1 / sum
        delta = inv_sum * 7.62939453e-06f;  // 2^-17
    } else {
        // 1 / (1 + e^-x): __expf (2 + 1.17 |x|) ulp, weighted by s e^-x / (1 + e^-x); sum and
        // reciprocal 1.5 ulp: below 4 * 2^-23
        delta = 9.5367432e-07f;  // 2^-20
    }
    float* sm = reinterpret_cast<float*>(sm64);
#pragma unroll
    for (int i = 0; i < kPL; i += 4) {
        float bv[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.bias != nullptr) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (expert(i + q) < E) bv[q] = __ldg(a.bias + expert(i + q));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int e = expert(i + q);
            uint32_t kk = kKeyNone;
            if (e < E) {
                float c = v[i + q];
                const bool out = masked(c) || masked(bv[q]);
                if (!by_logit) c = (sigmoid ? rcp_approx(1.0f + __expf(-c)) : __uint_as_float(key[i + q]) * inv_sum) + bv[q];
                kk = out ? kKeyMasked : key_of(c);
            }
            key[i + q] = kk;
        }
    }
    auto store_values = [&] {  // this lane's choice values into the row's array, masked as -inf
#pragma unroll
        for (int i = 0; i < kPL; i += 4) {
            float c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) c[q] = key[i + q] == kKeyMasked ? -CUDART_INF_F : value_of(key[i + q]);
            if (kVec) {
                if (expert(i) < E) *reinterpret_cast<float4*>(sm + expert(i)) = make_float4(c[0], c[1], c[2], c[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (expert(i + q) < E) sm[expert(i + q)] = c[q];
            }
        }
    };
    store_values();
    __syncwarp();
    // lpg lanes per group (a power of two) scan its values; bit g * lpg of `kept`: group g stays
    const int lpg = a.n_group > 16 ? 1 : a.n_group > 8 ? 2 : a.n_group > 4 ? 4 : a.n_group > 2 ? 8 : 16;
    uint32_t kept = kAll;
    if (a.n_group > 1) {
        const int g = lane / lpg;
        float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F;
        if (g < a.n_group) {
            for (int i = lane & (lpg - 1); i < a.gsize; i += lpg) {
                const float c = sm[g * a.gsize + i];
                b1 = fmaxf(b1, fminf(b0, c));
                b0 = fmaxf(b0, c);
            }
        }
        for (int o = 1; o < lpg; o <<= 1) {
            const float o0 = __shfl_xor_sync(kAll, b0, o), o1 = __shfl_xor_sync(kAll, b1, o);
            b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
            b0 = fmaxf(b0, o0);
        }
        const float gs = top2 && b1 > -CUDART_INF_F ? b0 + b1 : b0;
        int beaten = 0;
        for (int q = 0; q < a.n_group; ++q) {
            const float o = __shfl_sync(kAll, gs, q * lpg);
            beaten += o > gs || (o == gs && q < g);
        }
        bool keep = g < a.n_group && beaten < a.topk_group;
        if (!by_logit && a.topk_group < a.n_group) {
            // Error of a group's score: of its one or two values delta and 2^-24 of the value each,
            // of their sum 2^-24 of it; together below 2 delta + 2^-23 of the values' magnitudes,
            // which may be far above a sum that cancels.  Twice the second part covers the bounds'
            // own roundings.  The worst group kept, at its lowest, against the best one left out,
            // at its highest (a masked group is exact; an infinite one is always in doubt).
            const float size = fabsf(b0) + (top2 && b1 > -CUDART_INF_F ? fabsf(b1) : 0.f);
            const float err = b0 > -CUDART_INF_F ? 2.0f * delta + 2.38418579e-07f * size : 0.f;
            const float lo = value_of(__reduce_min_sync(kAll, keep ? key_of(fmaxf(gs - err, -CUDART_INF_F)) : kAll));
            const float hi = value_of(__reduce_max_sync(kAll, g < a.n_group && !keep ? key_of(gs + err) : 0x007FFFFFu));
            if (hi > -CUDART_INF_F && !(lo > hi)) {
                const double gs64 = group_score64<T>(a, x, sm64, top, lpg);
                beaten = 0;
                for (int q = 0; q < a.n_group; ++q) {
                    const double o = __shfl_sync(kAll, gs64, q * lpg);
                    beaten += o > gs64 || (o == gs64 && q < g);
                }
                keep = g < a.n_group && beaten < a.topk_group;
                store_values();  // (the 64-bit values lay over them)
                __syncwarp();
            }
        }
        kept = __ballot_sync(kAll, keep);
        if (kVec && a.gsize % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kPL; i += 4)
                if (!((kept >> ((((uint32_t)expert(i) * a.ginv) >> 20) * lpg & 31)) & 1u))
                    key[i] = key[i + 1] = key[i + 2] = key[i + 3] = kKeyNone;
        } else {
#pragma unroll
            for (int i = 0; i < kPL; ++i)
                if (!((kept >> ((((uint32_t)expert(i) * a.ginv) >> 20) * lpg & 31)) & 1u)) key[i] = kKeyNone;
        }
    }

    // a bound from below of the k-th largest: the k-th largest of the lanes' maxima
    uint32_t mine = kKeyNone, bound = kKeyNone;
#pragma unroll
    for (int i = 0; i < kPL; ++i) mine = max(mine, key[i]);
    for (int j = 0; j < k; ++j) {
        bound = __reduce_max_sync(kAll, mine);
        if (mine == bound) mine = kKeyNone;
    }
    // within `slack` fp32 does not decide the order: what lies that close below stays too
    const float kth = value_of(bound);
    const float slack = by_logit ? 0.f : 2.0f * delta + 4.76837158e-07f * fabsf(kth);
    uint32_t low = bound <= kKeyMasked ? kKeyMasked : by_logit ? bound : key_of(kth - slack);
    if (low <= kKeyMasked || !(kth - slack > -CUDART_INF_F)) low = kKeyMasked;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < kPL; ++i) bits |= key[i] >= low ? 1u << i : 0u;
    int* list = reinterpret_cast<int*>(sm64 + (E + 1) / 2);  // behind the E floats: 32 experts
    int n = 0;
    for (uint32_t m = bits;;) {
        const uint32_t who = __ballot_sync(kAll, m != 0);
        if (who == 0 || n > 32) break;
        const int at = n + __popc(who & ((1u << lane) - 1u));
        if (m != 0 && at < 32) list[at] = expert(__ffs(m) - 1);
        m &= m - 1;
        n += __popc(who);
    }
    __syncwarp();

    int my_id = 0;
    uint32_t my_key = kKeyNone;
    float xv = 0.f;
    if (n <= 32) {
        int id = lane < n ? list[lane] : E;
        uint32_t c = kKeyNone;
        if (lane < n) {
            const float f = sm[id];
            c = f > -CUDART_INF_F ? key_of(f) : kKeyMasked;
        }
        int rank = 0;
        for (int q = 0; q < n; ++q) {
            const uint32_t o = __shfl_sync(kAll, c, q);
            const int oid = __shfl_sync(kAll, id, q);
            rank += o > c || (o == c && oid < id);
        }
        // rank r moves to lane r
        __syncwarp();
        if (lane < n) list[rank] = id | (lane << 16);
        __syncwarp();
        const int from = lane < n ? list[lane] : 0;
        c = __shfl_sync(kAll, c, from >> 16);
        id = from & 0xffff;
        if (lane >= n) c = kKeyNone;
        if (lane < n) xv = to_f32(x[id]);
        if (!by_logit) {
            // neighbours in the order (of the k chosen and the next one) that fp32 leaves open
            const float b = a.bias != nullptr && lane < n ? __ldg(a.bias + id) : 0.f;
            const uint32_t nc = __shfl_down_sync(kAll, c, 1);
            const float nx = __shfl_down_sync(kAll, xv, 1), nb = __shfl_down_sync(kAll, b, 1);
            bool doubt = false;
            if (lane < k && lane + 1 < n && nc > kKeyMasked) {
                const float f = value_of(c), g = value_of(nc);
                // (the same inputs beyond the border may hide a close value behind them)
                doubt = !(f - g > 2.0f * delta + 2.38418579e-07f * (fabsf(f) + fabsf(g))) &&
                        !(xv == nx && b == nb && lane + 1 < k);
            }
            if (__any_sync(kAll, doubt)) {
                const double sum = sigmoid ? 1.0 : sum64(x, E, top);
                const double cv = c > kKeyMasked ? score64(xv, top, sum, sigmoid) + (double)b : -CUDART_INF;
                rank = 0;
                for (int q = 0; q < n; ++q) {
                    const double o = __shfl_sync(kAll, cv, q);
                    const int oid = __shfl_sync(kAll, id, q);
                    rank += o > cv || (o == cv && oid < id);
                }
                __syncwarp();
                if (lane < n) list[rank] = id | (lane << 16);
                __syncwarp();
                const int now = lane < n ? list[lane] : 0;
                c = __shfl_sync(kAll, c, now >> 16);
                xv = __shfl_sync(kAll, xv, now >> 16);
                id = now & 0xffff;
            }
        }
        my_id = id;
        my_key = c;
    } else if (by_logit) {
        // a round per expert: the largest key after (key m, expert e), ties to the lower id
        uint32_t m = kAll;
        int e = -1;
        for (int j = 0; j < k; ++j) {
            uint32_t best = kKeyNone;
            int be = E;
#pragma unroll
            for (int i = 0; i < kPL; ++i) {
                const bool left = key[i] < m || (key[i] == m && expert(i) > e);
                if (left && key[i] > best) { best = key[i]; be = expert(i); }
            }
            m = __reduce_max_sync(kAll, best);
            e = (int)__reduce_min_sync(kAll, best == m ? (uint32_t)be : kAll);
            if (lane == j) { my_key = m; my_id = e; }
        }
        xv = lane < k ? to_f32(x[my_id]) : 0.f;
    } else {
        bool out = false;
        my_id = route_row64(a, x, sm64, top, sigmoid ? 1.0 : sum64(x, E, top), kept, lpg, &out);
        my_key = out ? kKeyMasked : kAll;
        xv = lane < k ? to_f32(x[my_id]) : 0.f;
    }
    const bool is_masked = my_key == kKeyMasked;

    // weights: sigmoid as e^min(x,0) / (1 + e^-|x|).  With renormalisation the exponents are
    // taken relative to the largest chosen one, so that the sum never underflows.
    const bool renorm = a.flags & W4A8_ROUTE_RENORM;
    const bool live = lane < k && !is_masked;
    const float ex = sigmoid ? fminf(xv, 0.f) : xv;
    float ref = sigmoid ? 0.f : top;
    if (renorm) ref = value_of(__reduce_max_sync(kAll, live ? key_of(ex) : 0x007FFFFFu));
    // A difference of tens is rounded by some 2^-19, and its exponential by as much of itself:
    // what the subtraction lost (exact, the two-sum's second half) corrects it.
    const float d = ex == ref ? 0.f : ex - ref, v0 = d - ex;
    const float lost = ex == ref ? 0.f : (ex - (d - v0)) - (ref + v0);
    float s = live ? expf(d) : 0.f;
    if (s > 0.f) s = __fmaf_rn(s, lost, s);  // (0: too far below, or beside an infinite one)
    if (live && sigmoid) s = __fdiv_rn(s, 1.0f + expf(-fabsf(xv)));
    if (renorm) {
        float total = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
        s = total > 0.f ? __fdiv_rn(s, total) : 0.f;
    } else if (!sigmoid) {
        s *= inv_sum;
    }
    if (lane < k) {
        a.ids[(size_t)t * k + lane] = my_id;
        a.w[(size_t)t * k + lane] = s * a.scale;
    }
}

template <typename T>
cudaError_t launch_typed(const RouteArgs& a, cudaStream_t stream) {
    const int grid = ceil_div(a.T, kRouteWarps);
    // per warp: E choice values in fp32 and 32 experts, or E choice values in 64 bits
    const size_t smem = (size_t)kRouteWarps * route_smem_doubles(a.E) * sizeof(double);
    const bool vec = a.E % 4 == 0;
    // values per lane: the smallest that holds E / 32 (registers, and scans of empty values)
#define W4A8_ROUTE_LAUNCH(PL)                                                                                       \
    return vec ? launch_pdl(route_experts_kernel<T, PL, true>, grid, kRouteWarps * 32, smem, stream, a)             \
               : launch_pdl(route_experts_kernel<T, PL, false>, grid, kRouteWarps * 32, smem, stream, a)
    if (a.E <= 128) W4A8_ROUTE_LAUNCH(4);
    if (a.E <= 256) W4A8_ROUTE_LAUNCH(8);
    if (a.E <= 384) W4A8_ROUTE_LAUNCH(12);
    if (a.E <= 512) W4A8_ROUTE_LAUNCH(16);
    W4A8_ROUTE_LAUNCH(32);
#undef W4A8_ROUTE_LAUNCH
}

}  // namespace

cudaError_t launch_route_experts(const void* logits, int type, int T, int E, int k, int flags, const float* bias, int n_group,
                                 int topk_group, float scale, int32_t* ids, float* w, cudaStream_t stream) {
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.flags = flags;
    a.n_group = n_group;
    a.topk_group = topk_group;
    a.gsize = E / n_group;
    // exact for e < 1024: e * (rounding of 2^20 / gsize) < 2^10 <= 2^20 / gsize
    a.ginv = (uint32_t)(((1u << 20) + a.gsize - 1) / a.gsize);
    a.scale = scale;
    a.ids = ids;
    a.w = w;
    if (type == W4A8_LOGITS_F32) return launch_typed<float>(a, stream);
    if (type == W4A8_LOGITS_F16) return launch_typed<__half>(a, stream);
    return launch_typed<__nv_bfloat16>(a, stream);
}

}  // namespace w4a8
