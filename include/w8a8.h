/*
 * w8a8.h -- C ABI of libw4a8.so, second part: the W8A8 scheme (INT8 weights with one
 * scale per output channel, INT8 activations with one scale per token).
 *
 * Where it stands: the W4A16 / W4A8 / W8A8 table of «Kimi 2.7 Moe 从 4 bit 存储到 INT8
 * 拆解» (pptc.cn), section 3.3, names W8A8 as the scheme that costs twice the weight
 * memory of W4A8 and the least accuracy.  Weights (per output channel) and, inside the
 * layer, activations (per token) follow the symmetric formula of the LLM quantisation
 * primer (hotelren.com 5982361, section 2.1):
 *       s = max|v| * (1 / 127) (constant and product in fp32),
 *       q = clamp(round(v / s), -127, 127) (correctly rounded fp32 quotient),
 * round half to even; an all-zero row has s = 0 and q = 0.  A row with a NaN has s = NaN, one
 * with an infinity and no NaN s = infinity, both q = 0: a channel of weights, a token or a row
 * of h that holds one makes every output that it enters NaN (W8A8_I32 sums: 0).
 * (w4a8_quant_act divides by 127 instead, so that its scales may be one fp32 step away, and
 * passes over NaN; w8a8_gemm takes any codes and scales.)
 *
 * The conventions of w4a8.h hold for every entry point here: caller-owned device memory,
 * caller's workspace and stream, argument errors as a w4a8_status, device errors in the
 * workspace (w8a8_gemm_last_error, and w4a8_last_device_error for the layer), nothing
 * allocated.  Serving only: no backward pass.
 */
#ifndef W8A8_H
#define W8A8_H

#include "w4a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Output types of w8a8_gemm. */
enum {
    W8A8_F32 = 0,
    W8A8_BF16 = 1,
    W8A8_F16 = 2,
    W8A8_I32 = 3 /* the exact INT32 sums, without scales or bias */
};

/* Bytes of a packed weight buffer for E matrices [N][K] in `layout` (W4A8_LAYOUT_PLAIN or
 * W4A8_LAYOUT_GATEUP, no scheme flags): a 256-byte header; the fp32 scale of every tile row
 * [E][tiles][128]; then, per (matrix, 128-row tile, 128-wide K plane), 128 rows of 128
 * codes (16384 bytes), the 16-byte chunk c of row r at chunk position c ^ (r & 7).  Rows
 * past N and columns past K are zero.  Returns 0 for invalid shapes or flags. */
size_t w8a8_packed_bytes(int E, int N, int K, int layout);

/* Quantise and pack E weight matrices (offline, once).
 *   w_bf16    : device, bf16 [E][N][K].      packed: device, 256-byte aligned.
 *   codes_opt : device or NULL; int8 [E][N][Kp], Kp = K rounded up to 128.
 *   scale_opt : device or NULL; float [E][N].
 * W4A8_ENOSPACE if packed_bytes is too small; W4A8_EUNSUPPORTED for K > 131072 (the INT32
 * sum could overflow) or more than 2^31 - 1 packed rows (tiles x planes x 128). */
int w8a8_pack_weights(const void* w_bf16, int E, int N, int K, int layout, void* packed, size_t packed_bytes,
                      int8_t* codes_opt, float* scale_opt, void* stream);

/* One dense W8A8 linear layer:
 *   y[m][n] = sa[m] * sw[n] * sum_k qa[m][k] * qw[n][k] (+ bias[n]),
 * the sum exact in INT32, the rest fp32 (the sum times sa, times sw, plus the bias, in this
 * order), rounded once to the output type.
 *   qa       : device int8 [M][Kp], Kp = K rounded up to 128, padding 0 (as w4a8_quant_act
 *              writes it), 16-byte aligned.
 *   sa       : device float [M] (may be NULL for W8A8_I32).
 *   packed   : from w8a8_pack_weights(1, N, K, W4A8_LAYOUT_PLAIN).
 *   bias_opt : device float [N] or NULL (ignored for W8A8_I32).
 *   y        : device [M][N] of out_type, aligned to its element.
 *   ws       : w8a8_gemm_workspace_bytes(M, N, K) bytes, 256-byte aligned.
 * W4A8_EUNSUPPORTED: K > 131072, packed rows as in w8a8_pack_weights, or (M / 16 + 1) *
 * ceil(N / 128) >= 2^30. */
size_t w8a8_gemm_workspace_bytes(int M, int N, int K);
int w8a8_gemm(const int8_t* qa, const float* sa, int M, const void* packed, int N, int K, const float* bias_opt, void* y,
              int out_type, void* ws, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then return the device error bits of the last w8a8_gemm call on
 * workspace `ws` (0 = none; bit 0 = a bounded wait timed out). */
int w8a8_gemm_last_error(const void* ws, void* stream);

/* The MoE expert FFN with W8A8 experts: the arguments, routing, permutation, activation
 * quantisation and combine of w4a8_moe_forward,
 *   out[t] = sum_j w[t][j] * Down_e(SwiGLU(Up_e(x[t]))),  e = ids[t][j],
 * h = silu(gate) * up (fp32, within 7 roundings) rounded to bf16 and requantised per token
 * before Down, the experts' outputs summed in fp32, j ascending, and rounded once to bf16.
 * An id out of range drops its slot and sets bit 1 of the error word.
 *   packed_up   : from w8a8_pack_weights(E, 2F, H, W4A8_LAYOUT_GATEUP).
 *   packed_down : from w8a8_pack_weights(E, H, F, W4A8_LAYOUT_PLAIN).
 * The workspace is laid out as w4a8_moe_forward's, its stages readable with w4a8_debug_dump
 * (tiled rows in one block, RB = R).
 * Limits: E <= 1024, k <= 32, H, F <= 131072, (T * k + 15 E) * ceil(max(H, F) / 128) < 2^31. */
size_t w8a8_moe_workspace_bytes(int T, int E, int k, int H, int F);
int w8a8_moe_forward(const void* packed_up, const void* packed_down, int E, int H, int F, const void* x_bf16, int T,
                     const int32_t* ids, const float* w, int k, void* out_bf16, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
