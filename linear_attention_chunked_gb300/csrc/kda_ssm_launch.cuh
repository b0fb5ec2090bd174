// Launchers of the selective state-space scan's kernels, per translation unit.
#pragma once

#include "kda_ssm.cuh"

namespace kda {

// states into a.hs and, where given, y and the final states (kda_ssm_fwd.cu)
void launch_ssm_scan(const SsmArgs& a, int dtype, cudaStream_t st);
// the chunks' start gradients from zero ends into a.gs
void launch_ssm_rstate(const SsmArgs& a, int dtype, cudaStream_t st);

// backward from a.hs (kda_ssm_bwd.cu)
struct SsmBwdPlan {
    int lanes;   // lanes per channel (four states each)
    int tiles;   // channel tiles per group
    int nl;      // tiles per block: 1, or SSM_QUAD where there are blocks enough
    int splits;  // blocks per group and chunk = ceil(tiles / nl)
};
constexpr int SSM_QUAD = 4;
SsmBwdPlan ssm_bwd_plan(int64_t maxC, int C, int S, int G);
cudaError_t ssm_bwd_setup();
void launch_ssm_bwd(const SsmArgs& a, int dtype, cudaStream_t st);

// single tokens (kda_ssm_step.cu)
struct SsmStepArgs {
    int N, C, S, G, softplus;
    int64_t ldu, lddt, ldb, ldc, ldz, nslots;
    const void *u, *dt, *B, *Cm, *z;
    const float *A, *D, *bias, *hin;
    const int* slots;
    float* hout;
    void* y;
    int* status;
};
void launch_ssm_step(const SsmStepArgs& a, int dtype, cudaStream_t st);

}  // namespace kda
