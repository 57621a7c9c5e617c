// C ABI of the W8A8 scheme (declarations and contract: include/w8a8.h): argument
// validation, workspace carve-up and launch sequences.
#include "../../include/w8a8.h"
#include "layer_internal.h"
#include "w4a8_common.cuh"
#include "w8a8_internal.h"

#define W4A8_EXPORT extern "C" __attribute__((visibility("default")))

namespace w4a8 {
namespace {

constexpr size_t kAlign = 256;
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int to_status(cudaError_t e) { return e == cudaSuccess ? W4A8_OK : W4A8_ECUDA; }

#define W8_TRY(expr)                              \
    do {                                          \
        cudaError_t _e = (expr);                  \
        if (_e != cudaSuccess) return W4A8_ECUDA; \
    } while (0)

// 0 for an invalid shape, else the packed bytes; *fits is false when the tensor map's
// 32-bit row coordinate or the INT32 sum cannot hold the shape
size_t packed_bytes_of(int E, int N, int K, int layout, bool* fits) {
    *fits = false;
    if (E < 1 || N < 1 || K < 1) return 0;
    if (layout != W4A8_LAYOUT_PLAIN && layout != W4A8_LAYOUT_GATEUP) return 0;
    if (layout == W4A8_LAYOUT_GATEUP && (N & 1)) return 0;
    if (N > INT32_MAX - kTileRows || K > INT32_MAX - kGroup) return 0;
    const size_t tiles = (size_t)E * w8_tiles(N, layout), G = ceil_div(K, kGroup);
    *fits = K <= kW8MaxK && tiles * G * kTileRows < (1ull << 31);
    return kHeaderBytes + tiles * kTileRows * 4 + tiles * G * kW8BlockBytes;
}

using Layout = MoeLayout;

// the regions of w4a8_moe_forward's workspace, whose limits and the tensor maps' hold
bool layout_of(int T, int E, int k, int H, int F, Layout* L) {
    if (H > kW8MaxK || F > kW8MaxK || !moe_layout(T, E, k, H, F, false, L)) return false;
    return (long long)L->R * (L->G1 > L->G2 ? L->G1 : L->G2) < (1ll << 31);
}

template <typename T>
T* at(void* base, const Layout& L, Region r) {
    return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + L.off[r]);
}

}  // namespace
}  // namespace w4a8

using namespace w4a8;

W4A8_EXPORT size_t w8a8_packed_bytes(int E, int N, int K, int layout) {
    bool fits;
    return packed_bytes_of(E, N, K, layout, &fits);
}

W4A8_EXPORT int w8a8_pack_weights(const void* w_bf16, int E, int N, int K, int layout, void* packed, size_t packed_bytes,
                                  int8_t* codes_opt, float* scale_opt, void* stream) {
    bool fits;
    const size_t need = packed_bytes_of(E, N, K, layout, &fits);
    if (need == 0 || w_bf16 == nullptr || packed == nullptr) return W4A8_EINVAL;
    if (!fits) return W4A8_EUNSUPPORTED;
    if (!aligned(w_bf16, 16) || !aligned(packed, kAlign) || !aligned(codes_opt, 16) || !aligned(scale_opt, 4))
        return W4A8_EALIGN;
    if (packed_bytes < need) return W4A8_ENOSPACE;
    return to_status(launch_pack_w8(static_cast<const uint16_t*>(w_bf16), E, N, K, layout, static_cast<uint8_t*>(packed),
                                    codes_opt, scale_opt, static_cast<cudaStream_t>(stream)));
}

W4A8_EXPORT size_t w8a8_gemm_workspace_bytes(int M, int N, int K) {
    if (M < 0 || N < 1 || K < 1 || K > kW8MaxK) return 0;
    return kW8StatusWords * 4;  // one error word per CTA
}

W4A8_EXPORT int w8a8_gemm(const int8_t* qa, const float* sa, int M, const void* packed, int N, int K, const float* bias_opt,
                          void* y, int out_type, void* ws, size_t ws_bytes, void* stream) {
    if (M < 0 || N < 1 || K < 1 || out_type < W8A8_F32 || out_type > W8A8_I32) return W4A8_EINVAL;
    bool fits;
    packed_bytes_of(1, N, K, W4A8_LAYOUT_PLAIN, &fits);
    if (!fits || ((long long)M / 16 + 1) * w8_tiles(N, W4A8_LAYOUT_PLAIN) > INT32_MAX / 2) return W4A8_EUNSUPPORTED;
    if (packed == nullptr || ws == nullptr) return W4A8_EINVAL;
    if (!aligned(packed, kAlign) || !aligned(ws, kAlign)) return W4A8_EALIGN;
    if (ws_bytes < w8a8_gemm_workspace_bytes(M, N, K)) return W4A8_ENOSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M > 0) {
        if (qa == nullptr || y == nullptr || (sa == nullptr && out_type != W8A8_I32)) return W4A8_EINVAL;
        const size_t el = out_type == W8A8_F32 || out_type == W8A8_I32 ? 4 : 2;
        if (!aligned(qa, 16) || !aligned(sa, 4) || !aligned(bias_opt, 4) || !aligned(y, el)) return W4A8_EALIGN;
    }
    if (M == 0) return to_status(cudaMemsetAsync(ws, 0, kW8StatusWords * 4, s));
    W8Args a{};
    W8Operands op{};
    a.NT = w8_tiles(N, W4A8_LAYOUT_PLAIN);
    a.G = ceil_div(K, kGroup);
    a.wscale = reinterpret_cast<const float*>(static_cast<const uint8_t*>(packed) + kHeaderBytes);
    a.act_scale = out_type == W8A8_I32 ? nullptr : sa;
    a.M = M;
    a.mode = kW8Dense;
    a.out_type = out_type;
    a.out = y;
    a.ldo = N;
    a.nvalid = N;
    a.bias = out_type == W8A8_I32 ? nullptr : bias_opt;
    a.status = static_cast<uint32_t*>(ws);
    a.wait_limit = debug_wait_limit();
    a.debug = debug_flags();
    op.wblocks = static_cast<const uint8_t*>(packed) + w8_blocks_offset(1, a.NT);
    op.matrices = 1;
    op.x = qa;
    op.x_rows = M;
    ProfScope prof(W4A8_KERNEL_GEMM_DENSE, 1, s);
    W8_TRY(launch_gemm_w8a8(a, op, nullptr, sm_count(), s));
    return W4A8_OK;
}

W4A8_EXPORT int w8a8_gemm_last_error(const void* ws, void* stream) {
    if (ws == nullptr) return W4A8_EINVAL;
    uint32_t v[kW8StatusWords];
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(v, ws, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess) return W4A8_ECUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return W4A8_ECUDA;
    uint32_t all = 0;
    for (uint32_t w : v) all |= w;
    return (int)all;
}

W4A8_EXPORT size_t w8a8_moe_workspace_bytes(int T, int E, int k, int H, int F) {
    Layout L;
    if (!layout_of(T, E, k, H, F, &L)) return 0;
    return L.off[R_COUNT];
}

W4A8_EXPORT int w8a8_moe_forward(const void* packed_up, const void* packed_down, int E, int H, int F, const void* x_bf16,
                                 int T, const int32_t* ids, const float* w, int k, void* out_bf16, void* ws,
                                 size_t ws_bytes, void* stream) {
    Layout L;
    if (T < 0 || E < 1 || k < 1 || k > E || H < 1 || F < 1) return W4A8_EINVAL;
    bool fits_up, fits_down;
    if (F > INT32_MAX / 2 - kTileRows) return W4A8_EUNSUPPORTED;
    packed_bytes_of(E, 2 * F, H, W4A8_LAYOUT_GATEUP, &fits_up);
    packed_bytes_of(E, H, F, W4A8_LAYOUT_PLAIN, &fits_down);
    if (!fits_up || !fits_down || !layout_of(T, E, k, H, F, &L)) return W4A8_EUNSUPPORTED;
    if (packed_up == nullptr || packed_down == nullptr || ws == nullptr) return W4A8_EINVAL;
    if (!aligned(packed_up, kAlign) || !aligned(packed_down, kAlign) || !aligned(ws, kAlign)) return W4A8_EALIGN;
    if (ws_bytes < L.off[R_COUNT]) return W4A8_ENOSPACE;
    if (T > 0) {
        if (x_bf16 == nullptr || ids == nullptr || w == nullptr || out_bf16 == nullptr) return W4A8_EINVAL;
        if (!aligned(x_bf16, 16) || !aligned(ids, 16) || !aligned(w, 16) || !aligned(out_bf16, 16)) return W4A8_EALIGN;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t* err = at<uint32_t>(ws, L, R_ERR);
    if (T == 0 || L.nslots > kPrepareSlots) W8_TRY(cudaMemsetAsync(err, 0, 16, st));
    if (T == 0) return W4A8_OK;
    int* offs = at<int>(ws, L, R_OFFS);
    int* poffs = at<int>(ws, L, R_POFFS);
    int* mtstart = at<int>(ws, L, R_MTSTART);
    int* row_src = at<int>(ws, L, R_ROWSRC);
    int* inv = at<int>(ws, L, R_INV);
    int8_t* act1 = at<int8_t>(ws, L, R_ACT1);
    int8_t* act2 = at<int8_t>(ws, L, R_ACT2);
    float* s1 = at<float>(ws, L, R_S1);
    float* s2 = at<float>(ws, L, R_S2);
    uint16_t* h = at<uint16_t>(ws, L, R_H);
    float* y2 = at<float>(ws, L, R_Y2);
    const W8Plan plan = w8_plan_grouped(L.nslots, E, w8_tiles(2 * F, W4A8_LAYOUT_GATEUP), L.G1, w8_tiles(H, W4A8_LAYOUT_PLAIN), L.G2,
                                        sm_count());
    const uint16_t* x = static_cast<const uint16_t*>(x_bf16);
    if (L.nslots <= kPrepareSlots) {
        ProfScope p(W4A8_KERNEL_ACT_QUANT, 1, st);
        W8_TRY(launch_w8_prepare(ids, x, T, H, L.Hp, k, E, plan.bn, at<int>(ws, L, R_COUNTS), offs, poffs, mtstart,
                                 at<int4>(ws, L, R_MTTAB), at<int>(ws, L, R_PERM), inv, row_src, L.R, act1, s1, err, st));
    } else {
        {
            // (always in three kernels: of 2560 slots over 16 experts the layer takes 46.3 us against
            // 47.6 with one CTA, of 4096 57.9 and 61.2, of 16000 125 and 152; over 384 experts 156.5
            // and 162, 158.5 and 168, 215 and 269)
            ProfScope p(W4A8_KERNEL_PERM, perm_launch_count(L.nslots, 0), st);
            W8_TRY(launch_perm(ids, L.nslots, E, plan.bn, at<int>(ws, L, R_CHIST), L.nchunk, at<int>(ws, L, R_COUNTS), offs,
                               poffs, mtstart, at<int4>(ws, L, R_MTTAB), at<int>(ws, L, R_PERM), inv, row_src, err, st, 0));
        }
        ProfScope p(W4A8_KERNEL_ACT_QUANT, 1, st);
        W8_TRY(launch_w8_act_scatter(x, T, H, L.Hp, k, inv, L.R, act1, s1, st));
    }
    W8Args a{};
    W8Operands op{};
    a.NT = w8_tiles(2 * F, W4A8_LAYOUT_GATEUP);
    a.G = L.Hp / kGroup;
    a.wscale = reinterpret_cast<const float*>(static_cast<const uint8_t*>(packed_up) + kHeaderBytes);
    a.act_scale = s1;
    a.mt_tab = at<int4>(ws, L, R_MTTAB);
    a.n_mtiles = mtstart + E;
    a.mode = kW8Up;
    a.out_type = W8A8_BF16;
    a.out = h;
    a.ldo = L.Fp;
    a.nvalid = F;
    a.err = err;
    a.wait_limit = debug_wait_limit();
    a.debug = debug_flags();
    op.wblocks = static_cast<const uint8_t*>(packed_up) + w8_blocks_offset(E, a.NT);
    op.matrices = E;
    op.x = act1;
    op.x_rows = L.R;
    {
        ProfScope p(W4A8_KERNEL_GEMM_UP, 1, st);
        W8_TRY(launch_gemm_w8a8(a, op, &plan, sm_count(), st));
    }
    {
        ProfScope p(W4A8_KERNEL_REQUANT, 1, st);
        W8_TRY(launch_w8_requant(h, L.Fp, F, L.Fp, row_src, poffs, E, L.R, L.R, act2, s2, st));
    }
    a.NT = w8_tiles(H, W4A8_LAYOUT_PLAIN);
    a.G = L.Fp / kGroup;
    a.wscale = reinterpret_cast<const float*>(static_cast<const uint8_t*>(packed_down) + kHeaderBytes);
    a.act_scale = s2;
    a.mode = kW8Down;
    a.out_type = W8A8_F32;
    a.out = y2;
    a.ldo = H;
    a.nvalid = H;
    op.wblocks = static_cast<const uint8_t*>(packed_down) + w8_blocks_offset(E, a.NT);
    op.x = act2;
    {
        ProfScope p(W4A8_KERNEL_GEMM_DOWN, 1, st);
        W8_TRY(launch_gemm_w8a8(a, op, &plan, sm_count(), st));
    }
    {
        ProfScope p(W4A8_KERNEL_COMBINE, 1, st);
        W8_TRY(launch_w8_combine(y2, H, inv, w, T, k, static_cast<uint16_t*>(out_bf16), st));
    }
    return W4A8_OK;
}
