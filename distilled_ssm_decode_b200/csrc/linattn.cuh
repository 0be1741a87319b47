// linattn.cuh -- arguments and plan shared by the two routes of the linear-attention prefill.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace hyena {

// decay^n in fp64 by binary powering (decay^0 = 1 also for decay = 0).
__device__ __forceinline__ double decay_pow(double g, long long n) {
    double r = 1.0;
    while (n > 0) {
        if (n & 1) r *= g;
        g *= g;
        n >>= 1;
    }
    return r;
}

struct LinArgs {
    const void *q, *k, *v;
    void *o;
    int B, L, H, Hk, dk, dv;
    long long ldq, ldk, ldv;
    const float *decay;
    float scale;
    const int *lens;
    const float *init;       // state entering segment s: init + s * init_stride (null: zero)
    long long init_stride;
    float *states;           // states_only: contribution of segment s -> states + (s + 1) * init_stride
    float *state_out;        // else: the state after the last segment
    int seg_tokens, nseg;    // segments of this launch (states_only leaves out the last one)
    int vtiles, nv;          // column tiles of a state, their width
    int *err;                // an error word for each block of the tensor-core route (the other route clears them)
    int nerr;
    int hold;                // tests: block 0 never signals its state products, so that a wait runs out
};

// tokens of row b
__device__ __forceinline__ int row_tokens(const LinArgs &a, int b) {
    if (!a.lens) return a.L;
    return min(max(a.lens[HB_IDX(b, a.B)], 0), a.L);
}

// A prompt is split into segments of whole tiles of tokens when there are too few (sequence, head,
// column tile) units to fill the GPU: the segments' own contributions to the state are computed
// first, then combined into the state entering each segment, then every segment runs by itself.
struct LinPlan {
    int vtiles, nv, nseg, seg_tokens;
};

// linattn_tc.cu
constexpr int kLinMaxBlocks = 148;       // one block per SM
bool linattn_tc_dims(int dtype, int dk, int dv);
LinPlan linattn_tc_plan(int B, int L, int H, int Hk, int dk, int dv, bool lens);
cudaError_t launch_linattn_tc(LinArgs a, bool states_only, cudaStream_t s);

}  // namespace hyena
