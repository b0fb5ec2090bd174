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
    int query, key, value;  // tensors of LinMaps
    int store;              // the output's (bf16 outputs)
    int rq, rk, rv;         // heads that share a row of each
    void* out;              // dense [T, H, 128]
    int out_fp32;
    const float* s0;        // [N, H, 128, 128] or null
    float* s_end;           // likewise
    int trans;              // the states in memory are X^T
    int back;
    float in, by;
};

constexpr int LC = 128;  // tokens of a chunk


// With few heads, documents longer than LIN_WHOLE tokens are cut into segments of `seg` tokens (the last one shorter),
// which are walked side by side; the others are one segment.  The state between two segments of a document lies in a
// slot.
constexpr int LIN_WHOLE = 2048;

struct LinPlan {
    int4* tab;     // per segment: {document, first token, length | first << 16 | last << 17, w}: w is the slot behind
                   // the segment, w - 1 the one in front of it
    int4* multi;   // per document of more than one segment: {document, slot behind its first segment, segments, tokens}
    int* counts;   // segments, documents in multi
};

struct LinArgs {
    int64_t T;
    int N, H;
    int seg;               // tokens of a segment
    int direct;            // no document is cut: no plan
    const int* cu;
    const float* slope;
    int* status;
    int4 sizes;            // of this call
    int4* made_for;        // forward with a saved set: where it notes them
    const int4* expected;  // backward from a saved set: what its forward noted
    LinPlan plan;
    float *front, *back;   // slots [][H][128][128] of the forward and of the backward walks
    int passes;
    LinPass pass[3];
};

// The rows of a call as TMA tensors: {64 channels, tokens, half of the head, head}, boxes of 128 tokens x one head,
// which land as two 128-byte-swizzled tiles [64 channels of 128 tokens]; the outputs likewise.  LinPass names them.
struct LinMaps {
    CUtensorMap m[7];
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

cudaError_t lin_setup();  // shared memory limits
void launch_lin_plan(const LinArgs& a, cudaStream_t st);
// the slots' states: what each segment adds (pass of a.pass whose walk they stand for), then their sums
void launch_lin_states(const LinArgs& a, const LinMaps& tm, int pass, cudaStream_t st);
void launch_lin_walk(const LinArgs& a, const LinMaps& tm, cudaStream_t st);

}  // namespace kda
