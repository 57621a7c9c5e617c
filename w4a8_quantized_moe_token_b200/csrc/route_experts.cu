// Routing to experts with softmax or sigmoid scores, a per-expert bias that enters the
// choice only, a restriction to the best groups of experts, and renormalised weights
// (w4a8_route_experts; the contract is in include/w4a8.h).
//
// One warp per token; lane l owns experts l, l + 32, ...  The choice values of a token lie
// in shared memory as doubles: the order of two experts whose scores differ by less than
// fp32 holds is then the order of their 64-bit scores.
#include <math_constants.h>

#include "../../include/w4a8.h"
#include "w4a8_common.cuh"
#include "w4a8_internal.h"

namespace w4a8 {

namespace {

constexpr int kRouteWarps = 4;

template <typename T>
__device__ __forceinline__ float logit(const T* p);
template <>
__device__ __forceinline__ float logit(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float logit(const __half* p) { return __half2float(*p); }

__device__ __forceinline__ bool masked(float v) { return !(v > -CUDART_INF_F); }  // -inf or NaN

// 64-bit score of an unmasked expert; top = the largest logit of the row
__device__ __forceinline__ double score64(float x, float top, double sum, bool sigmoid) {
    if (sigmoid) return 1.0 / (1.0 + exp(-(double)x));
    return exp(x == top ? 0.0 : (double)x - (double)top) / sum;
}

template <typename T>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_experts_kernel(const T* __restrict__ logits, int ntok, int E, int k, int flags, const float* __restrict__ bias,
                         int n_group, int topk_group, float scale, int32_t* __restrict__ ids, float* __restrict__ w) {
    grid_dep_wait();
    extern __shared__ double sm_choice[];
    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t >= ntok) return;
    double* choice = sm_choice + (size_t)(threadIdx.x >> 5) * E;
    const T* x = logits + (size_t)t * E;
    const bool sigmoid = flags & W4A8_ROUTE_SIGMOID;
    const bool by_logit = bias == nullptr && !(flags & W4A8_ROUTE_GROUP_TOP2);
    float top = -CUDART_INF_F;
    double sum = 0.0;
    if (!sigmoid) {
        for (int e = lane; e < E; e += 32) top = fmaxf(top, logit(x + e));
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (int e = lane; e < E; e += 32) {
            const float v = logit(x + e);
            if (!masked(v)) sum += score64(v, top, 1.0, false);
        }
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    for (int e = lane; e < E; e += 32) {
        const float v = logit(x + e), b = bias != nullptr ? __ldg(bias + e) : 0.f;
        choice[e] = masked(v) || masked(b) ? -CUDART_INF : by_logit ? (double)v : score64(v, top, sum, sigmoid) + (double)b;
    }
    __syncwarp();
    // the groups kept: those that fewer than topk_group groups beat
    uint32_t kept = 0xffffffffu;
    const int gsize = E / n_group;
    if (n_group > 1) {
        double b0 = -CUDART_INF, b1 = -CUDART_INF;
        if (lane < n_group) {
            for (int i = 0; i < gsize; ++i) {
                const double c = choice[lane * gsize + i];
                b1 = fmax(b1, fmin(b0, c));
                b0 = fmax(b0, c);
            }
        }
        const double gs = (flags & W4A8_ROUTE_GROUP_TOP2) && b1 > -CUDART_INF ? b0 + b1 : b0;
        int beaten = 0;
        for (int g = 0; g < n_group; ++g) {
            const double o = __shfl_sync(0xffffffffu, gs, g);
            beaten += o > gs || (o == gs && g < lane);
        }
        kept = __ballot_sync(0xffffffffu, lane < n_group && beaten < topk_group);
    }
    // k times the largest choice value left, ties to the lower id
    uint32_t taken = 0;
    float mine = 0.f;  // lane j: the j-th expert's logit
    int mine_id = 0;
    bool mine_masked = false;
    for (int j = 0; j < k; ++j) {
        double bv = -CUDART_INF;
        int be = E;
        for (int e = lane, i = 0; e < E; e += 32, ++i) {
            if ((taken >> i) & 1u || !((kept >> (n_group > 1 ? e / gsize : 0)) & 1u)) continue;
            const double c = choice[e];
            if (be == E || c > bv) { bv = c; be = e; }
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oe = __shfl_xor_sync(0xffffffffu, be, o);
            if (ov > bv || (ov == bv && oe < be)) { bv = ov; be = oe; }
        }
        if ((be & 31) == lane) taken |= 1u << (be >> 5);
        if (lane == j) {
            mine_id = be;
            mine = logit(x + be);
            mine_masked = bv == -CUDART_INF;
        }
    }
    double s = lane < k && !mine_masked ? score64(mine, top, sigmoid ? 1.0 : sum, sigmoid) : 0.0;
    if (flags & W4A8_ROUTE_RENORM) {
        double total = s;
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        s = total > 0.0 ? s / total : 0.0;
    }
    if (lane < k) {
        ids[(size_t)t * k + lane] = mine_id;
        w[(size_t)t * k + lane] = (float)(s * (double)scale);
    }
}

}  // namespace

cudaError_t launch_route_experts(const void* logits, int type, int T, int E, int k, int flags, const float* bias, int n_group,
                                 int topk_group, float scale, int32_t* ids, float* w, cudaStream_t stream) {
    const int grid = ceil_div(T, kRouteWarps);
    const size_t smem = (size_t)kRouteWarps * E * sizeof(double);
    if (type == W4A8_LOGITS_F32)
        return launch_pdl(route_experts_kernel<float>, grid, kRouteWarps * 32, smem, stream, static_cast<const float*>(logits),
                          T, E, k, flags, bias, n_group, topk_group, scale, ids, w);
    if (type == W4A8_LOGITS_F16)
        return launch_pdl(route_experts_kernel<__half>, grid, kRouteWarps * 32, smem, stream, static_cast<const __half*>(logits),
                          T, E, k, flags, bias, n_group, topk_group, scale, ids, w);
    return launch_pdl(route_experts_kernel<__nv_bfloat16>, grid, kRouteWarps * 32, smem, stream,
                      static_cast<const __nv_bfloat16*>(logits), T, E, k, flags, bias, n_group, topk_group, scale, ids, w);
}

}  // namespace w4a8
