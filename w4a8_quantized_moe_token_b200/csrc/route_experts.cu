// Routing to experts with softmax or sigmoid scores, a per-expert bias that enters the
// choice only, a restriction to the best groups of experts, and renormalised weights
// (w4a8_route_experts; the contract is in include/w4a8.h).
//
// One warp per token, its choice values in registers as order-preserving 32-bit keys, four
// consecutive experts per lane and step where E allows.  Each lane keeps its two best; every
// round of the top-k is then two warp reductions and a pop, and a lane scans its values
// again only when both are gone.
//
// The contract orders experts by their 64-bit choice values.  The values here are fp32 with
// an error of at most `delta` (from the documented bounds of __expf, expf and __fdividef,
// doubled), so a gap of more than that between neighbours in the result decides their order
// for good, and equal inputs are true ties.  A row with a closer pair among the k chosen and
// the next one, or at the border of the kept groups, is done again in 64 bits (about one row
// in a few hundred for random inputs): exact order at the price of fp32 arithmetic.  Without
// a bias the keys are the logits themselves and nothing is ever in doubt.
#include <math_constants.h>

#include "../../include/w4a8.h"
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

// The choice of one row in 64 bits: lane j < k returns the j-th expert, kKeyMasked's case in
// *is_masked.  `choice`: E doubles of shared memory of this warp.
template <typename T>
__device__ __noinline__ int route_row64(const RouteArgs& a, const T* x, double* choice, bool* is_masked) {
    const int lane = threadIdx.x & 31, E = a.E;
    const bool sigmoid = a.flags & W4A8_ROUTE_SIGMOID;
    float top = -CUDART_INF_F;
    double sum = 0.0;
    if (!sigmoid) {
        for (int e = lane; e < E; e += 32) top = fmaxf(top, to_f32(x[e]));
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        for (int e = lane; e < E; e += 32) {
            const float v = to_f32(x[e]);
            if (!masked(v)) sum += score64(v, top, 1.0, false);
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    }
    __syncwarp();
    for (int e = lane; e < E; e += 32) {
        const float v = to_f32(x[e]), b = a.bias != nullptr ? __ldg(a.bias + e) : 0.f;
        choice[e] = masked(v) || masked(b) ? -CUDART_INF : score64(v, top, sum, sigmoid) + (double)b;
    }
    __syncwarp();
    uint32_t kept = kAll;
    if (a.n_group > 1) {
        double b0 = -CUDART_INF, b1 = -CUDART_INF;
        if (lane < a.n_group) {
            for (int i = 0; i < a.gsize; ++i) {
                const double c = choice[lane * a.gsize + i];
                b1 = fmax(b1, fmin(b0, c));
                b0 = fmax(b0, c);
            }
        }
        const double gs = (a.flags & W4A8_ROUTE_GROUP_TOP2) && b1 > -CUDART_INF ? b0 + b1 : b0;
        int beaten = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double o = __shfl_sync(kAll, gs, g);
            beaten += o > gs || (o == gs && g < lane);
        }
        kept = __ballot_sync(kAll, lane < a.n_group && beaten < a.topk_group);
    }
    uint32_t taken = 0;
    int mine = 0;
    for (int j = 0; j < a.k; ++j) {
        double bv = -CUDART_INF;
        int be = E;
        for (int e = lane, i = 0; e < E; e += 32, ++i) {
            if ((taken >> i) & 1u || !((kept >> (((uint32_t)e * a.ginv) >> 20)) & 1u)) continue;
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

// kPL: values per lane at most; kVec: lane l owns experts 4 (32 i + l) .. + 3 (E % 4 == 0),
// otherwise l, l + 32, ...
template <typename T, int kPL, bool kVec>
__global__ void __launch_bounds__(kRouteWarps * 32) route_experts_kernel(const RouteArgs a) {
    grid_dep_wait();
    extern __shared__ double sm_choice[];
    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    const T* x = static_cast<const T*>(a.logits) + (size_t)t * E;
    const bool sigmoid = a.flags & W4A8_ROUTE_SIGMOID, top2 = a.flags & W4A8_ROUTE_GROUP_TOP2;
    const bool by_logit = a.bias == nullptr && !top2;
    auto expert = [&](int i) { return kVec ? ((i >> 2) * 32 + lane) * 4 + (i & 3) : i * 32 + lane; };

    float v[kPL];
    if (kVec) {
#pragma unroll
        for (int i = 0; i < kPL; i += 4) {
            const int e = expert(i);
            if (e < E) {
                if (sizeof(T) == 4) {
                    const float4 p = *reinterpret_cast<const float4*>(x + e);
                    v[i] = p.x; v[i + 1] = p.y; v[i + 2] = p.z; v[i + 3] = p.w;
                } else {
                    const uint2 p = *reinterpret_cast<const uint2*>(x + e);
                    const T* h = reinterpret_cast<const T*>(&p);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[i + q] = to_f32(h[q]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[i + q] = -CUDART_INF_F;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPL; ++i) v[i] = expert(i) < E ? to_f32(x[expert(i)]) : -CUDART_INF_F;
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
        // __fdividef 2.5 ulp: below 4 * 2^-23
        delta = 9.5367432e-07f;  // 2^-20
    }
    float* sm = reinterpret_cast<float*>(sm_choice + (size_t)(threadIdx.x >> 5) * E);
#pragma unroll
    for (int i = 0; i < kPL; ++i) {
        const int e = expert(i);
        uint32_t kk = kKeyNone;
        if (e < E) {
            float c = v[i];
            bool out = masked(c);
            if (!by_logit) {
                const float b = a.bias != nullptr ? __ldg(a.bias + e) : 0.f;
                out = out || masked(b);
                c = (sigmoid ? __fdividef(1.0f, 1.0f + __expf(-v[i])) : __uint_as_float(key[i]) * inv_sum) + b;
            }
            kk = out ? kKeyMasked : key_of(c);
            if (a.n_group > 1) sm[e] = out ? -CUDART_INF_F : c;
        }
        key[i] = kk;
    }

    bool doubt = false;
    if (a.n_group > 1) {
        // lpg lanes per group (a power of two) scan its values
        const int lpg = a.n_group > 16 ? 1 : a.n_group > 8 ? 2 : a.n_group > 4 ? 4 : a.n_group > 2 ? 8 : 16;
        const int g = lane / lpg;
        float b0 = -CUDART_INF_F, b1 = -CUDART_INF_F;
        __syncwarp();
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
        const bool keep = g < a.n_group && beaten < a.topk_group;
        const uint32_t kept = __ballot_sync(kAll, keep);
        if (!by_logit && a.topk_group < a.n_group) {
            // the worst group kept against the best one left out
            const float lo = value_of(__reduce_min_sync(kAll, keep ? key_of(gs) : kAll));
            const float hi = value_of(__reduce_max_sync(kAll, g < a.n_group && !keep ? key_of(gs) : 0x007FFFFFu));
            if (hi > -CUDART_INF_F)
                doubt = !(lo - hi > 4.0f * delta + 4.76837158e-07f * (fabsf(lo) + fabsf(hi)));
        }
#pragma unroll
        for (int i = 0; i < kPL; ++i)
            if (!((kept >> ((((uint32_t)expert(i) * a.ginv) >> 20) * lpg & 31)) & 1u)) key[i] = kKeyNone;
    }

    // this lane's two best after (bm, be) in the order (key descending, expert ascending)
    uint32_t k0, k1;
    int e0, e1;
    auto scan = [&](uint32_t bm, int be) {
        k0 = k1 = kKeyNone;
        e0 = e1 = 0;
#pragma unroll
        for (int i = 0; i < kPL; ++i) {
            const int e = expert(i);
            const bool left = key[i] < bm || (key[i] == bm && e > be);
            if (left && key[i] > k0) {
                k1 = k0; e1 = e0;
                k0 = key[i]; e0 = e;
            } else if (left && key[i] > k1) {
                k1 = key[i]; e1 = e;
            }
        }
    };
    scan(kAll, -1);
    uint32_t my_key = kKeyNone, next_key = kKeyNone;
    int my_id = 0, next_id = 0;
    bool second = true;  // k1 is still this lane's next best after k0
    const int rounds = by_logit ? k : k + 1;  // one more, to see what was just left out
    for (int j = 0; j < rounds; ++j) {
        const uint32_t m = __reduce_max_sync(kAll, k0);
        const int e = (int)__reduce_min_sync(kAll, k0 == m ? (uint32_t)e0 : kAll);
        if (j < k) {
            if (lane == j) { my_key = m; my_id = e; }
        } else {
            next_key = m;
            next_id = e;
        }
        if (k0 == m && e0 == e && m != kKeyNone) {
            if (second) {
                k0 = k1; e0 = e1;
                second = false;
            } else {
                scan(m, e);
                second = true;
            }
        }
    }

    float xv = lane < k ? to_f32(x[my_id]) : 0.f;
    bool is_masked = my_key == kKeyMasked;
    if (!by_logit) {
        // neighbours (j, j + 1) of the chosen ones, the last against the next one left out
        const float b = a.bias != nullptr && lane < k ? __ldg(a.bias + my_id) : 0.f;
        uint32_t nk = __shfl_down_sync(kAll, my_key, 1);
        float nx = __shfl_down_sync(kAll, xv, 1), nb = __shfl_down_sync(kAll, b, 1);
        bool border = false;
        if (lane == k - 1) {
            nk = next_key;
            if (nk > kKeyMasked) {
                nx = to_f32(x[next_id]);
                nb = a.bias != nullptr ? __ldg(a.bias + next_id) : 0.f;
            }
        }
        if (lane < k && nk > kKeyMasked) {
            const float c = value_of(my_key), n = value_of(nk);
            const bool close = !(c - n > 2.0f * delta + 2.38418579e-07f * (fabsf(c) + fabsf(n)));
            const bool tie = xv == nx && b == nb;
            doubt = doubt || (close && !tie);
            border = close && tie && lane == k - 1;
        }
        if (__any_sync(kAll, border)) {
            // a true tie across the border: another value close to it may lie behind it
            const float c = value_of(__shfl_sync(kAll, my_key, k - 1));
            const float bx = __shfl_sync(kAll, xv, k - 1), bb = __shfl_sync(kAll, b, k - 1);
            const float slack = 2.0f * delta + 4.76837158e-07f * fabsf(c);
#pragma unroll
            for (int i = 0; i < kPL; ++i)
                if (key[i] > kKeyMasked && !(c - value_of(key[i]) > slack) && !(value_of(key[i]) - c > slack)) {
                    const float ob = a.bias != nullptr ? __ldg(a.bias + expert(i)) : 0.f;
                    doubt = doubt || v[i] != bx || ob != bb;
                }
        }
        if (__any_sync(kAll, doubt)) {
            my_id = route_row64(a, x, sm_choice + (size_t)(threadIdx.x >> 5) * E, &is_masked);
            xv = lane < k ? to_f32(x[my_id]) : 0.f;
        }
    }

    // weights: sigmoid as e^min(x,0) / (1 + e^-|x|).  With renormalisation the exponents are
    // taken relative to the largest chosen one, so that the sum never underflows.
    const bool renorm = a.flags & W4A8_ROUTE_RENORM;
    const bool live = lane < k && !is_masked;
    const float ex = sigmoid ? fminf(xv, 0.f) : xv;
    float ref = sigmoid ? 0.f : top;
    if (renorm) ref = value_of(__reduce_max_sync(kAll, live ? key_of(ex) : 0x007FFFFFu));
    float s = live ? expf(ex == ref ? 0.f : ex - ref) : 0.f;
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
    const bool by_logit = a.bias == nullptr && !(a.flags & W4A8_ROUTE_GROUP_TOP2);
    const size_t smem = a.n_group > 1 || !by_logit ? (size_t)kRouteWarps * a.E * sizeof(double) : 0;
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
