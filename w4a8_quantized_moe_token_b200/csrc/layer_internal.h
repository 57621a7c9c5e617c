// Host-side declarations shared by the entry points of both schemes' layers (api.cu,
// w8a8_api.cu), and the launchers that only some of them use.
#pragma once

#include "w4a8_common.cuh"
#include "w4a8_internal.h"

namespace w4a8 {

// Lets the next kernel of the stream start its set-up once every CTA of this grid has come
// here.  A kernel that allocates tensor memory calls it only after its allocation: a later
// kernel, which waits for this one, must not be able to take the columns first.
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// the W8A8 scheme's scales are max|v| * (1 / 127), the constant and the product in fp32
constexpr float kInv127 = 1.0f / 127.0f;

// the debug hook's current values on the calling host thread (wait_limit: the default if unset)
long long debug_wait_limit();
uint32_t debug_flags();

// multiprocessors of the current device
int sm_count();

// records an event pair around the kernels launched in its scope while the per-kernel
// timing (w4a8_profile_start) is on
struct ProfScope {
    int kind, nlaunch;
    cudaStream_t st;
    cudaEvent_t a = nullptr;
    ProfScope(int kind, int nlaunch, cudaStream_t st);
    ~ProfScope();
};

// Workspace of w4a8_moe_forward: regions in the order of the enum below.
enum Region {
    R_ERR, R_CHIST, R_COUNTS, R_OFFS, R_POFFS, R_MTSTART, R_MTTAB, R_PERM, R_INV, R_ROWSRC,
    R_ACT1, R_S1, R_H, R_ACT2, R_S2, R_Y2,
    R_XIN, R_IDSIN, R_WIN, R_OUT, R_LOGITS,  // host-buffer variants only
    R_COUNT
};

struct MoeLayout {
    size_t off[R_COUNT + 1];
    size_t bytes[R_COUNT];
    int nslots, nchunk, R, Hp, Fp, G1, G2;
};
// false for a shape outside the layer's limits
bool moe_layout(int T, int E, int k, int H, int F, bool host_io, MoeLayout* L, bool w4a16 = false, int group = 128);

cudaError_t launch_route_experts(const void* logits, int type, int T, int E, int k, int flags, const float* bias, int n_group,
                                 int topk_group, float scale, int32_t* ids, float* w, cudaStream_t stream);

// the permutation as launch_perm's, in one CTA for up to small_slots slots, else in three kernels
int perm_launch_count(int nslots, int small_slots);
cudaError_t launch_perm(const int32_t* ids, int nslots, int E, int tile_tokens, int* chist, int nchunk, int* counts,
                        int* offs, int* poffs, int* mtstart, int4* mt_tab, int* perm, int* inv, int* row_src,
                        uint32_t* err, cudaStream_t stream, int small_slots);

// The W8A8 layer's own: scales as the scheme defines them, pad rows left alone.
cudaError_t launch_w8_act_scatter(const uint16_t* x, int T, int H, int Kp, int k, const int* inv, int rb, int8_t* act, float* s,
                                  cudaStream_t stream);
cudaError_t launch_w8_requant(const uint16_t* h, int ldh, int F, int Kp, const int* row_src, const int* poffs, int E,
                              int rows_cap, int rb, int8_t* act, float* s, cudaStream_t stream);
cudaError_t launch_w8_combine(const float* y2, int H, const int* inv, const float* w, int T, int k, uint16_t* out,
                              cudaStream_t stream);
// T * k <= kPrepareSlots: permutation and activation quantisation in one kernel, which also
// sets the error word.  The layer (H 2048, F 256, 8 of 16 experts) with it against the
// permutation's three kernels and the quantisation: 256 slots 30.9 and 37.0 us, 1024 34.6 and
// 39.3, 2048 39.1 and 43.1, 2560 41.7 and 46.3, 4096 52.8 and 57.9, 8192 78.5 and 72.1: every CTA
// counts all ids.  (2048 is below the crossing: 8 KB of shared memory for the ids.)
constexpr int kPrepareSlots = 2048;
cudaError_t launch_w8_prepare(const int32_t* ids, const uint16_t* x, int T, int H, int Kp, int k, int E, int tile_tokens,
                              int* counts, int* offs, int* poffs, int* mtstart, int4* mt_tab, int* perm, int* inv, int* row_src,
                              int rb, int8_t* act, float* s, uint32_t* err, cudaStream_t stream);

}  // namespace w4a8
