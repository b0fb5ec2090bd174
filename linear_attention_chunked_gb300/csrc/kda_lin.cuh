// Shared parts of the linear attention with a decay for each head (walk, single tokens).
//
// Per document and head, lambda = exp(slope):  S_t = lambda S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.
// Its gradient is three more walks of the same recurrence with the roles changed (G_t is the gradient of S_t):
//   dq_t = scale S_t dO_t                              query dO, key v, value k, forwards, the state is S^T
//   dv_t = G_t^T k_t,  G_t = lambda G_{t+1} + scale q_t dO_t^T   query k, key q, value dO, backwards
//   dk_t = G_t v_t                                     query v, key dO, value q, backwards, the state is G^T
// so one walk serves the forward and the backward, and the backward needs no states of single chunks.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// One walk over the documents.  Its state X [key channel][value channel] is
//   forwards:   X_t = lambda X_{t-1} + key_t value_t^T (X before the first token: s0, after the last: s_end)
//   backwards:  X_t = Y_t + in key_t value_t^T,  Y_{t-1} = lambda X_t (Y at the last token: s0, past the first: s_end)
// and out_t = by X_t^T query_t.
struct LinPass {
    const __nv_bfloat16 *query, *key, *value;
    int64_t ldq, ldk, ldv;  // token strides (elements)
    int rq, rk, rv;         // heads that share a row of each
    void* out;              // dense [T, H, 128]
    int out_fp32;
    const float* s0;        // [N, H, 128, 128] or null
    float* s_end;           // likewise
    int trans;              // the states in memory are X^T
    int back;
    float in, by;
};

struct LinArgs {
    int64_t T;
    int N, H;
    const int* cu;
    const float* slope;
    int* status;
    int4 sizes;            // of this call
    int4* made_for;        // forward with a saved set: where it notes them
    const int4* expected;  // backward from a saved set: what its forward noted
    int passes;
    LinPass pass[3];
};

// single tokens (kda_lin_step.cu)
struct LinStepArgs {
    int N, H, share;
    int64_t ldq, ldk, ldv, nslots;
    float scale;
    const __nv_bfloat16 *q, *k, *v;
    const float *slope, *hin;
    const int* slots;
    float* hout;
    __nv_bfloat16* o;
    int* status;
};
void launch_lin_step(const LinStepArgs& a, cudaStream_t st);

void launch_lin_walk(const LinArgs& a, cudaStream_t st);

}  // namespace kda
