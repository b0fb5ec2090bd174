// Selective state-space scan for single tokens: one step of every sequence's state.
//
// Bound by HBM: the state is read and written once (8 S bytes per channel against ~10 bytes of
// inputs and output), so four consecutive states (one 16-byte access) belong to a lane, the lanes
// of a channel are neighbours, and a warp reads and writes 512 consecutive bytes.  The channel's
// scalars (delta, the gate) are recomputed by each of its lanes: their cost is hidden behind the
// state's traffic.
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

constexpr int STEP_THREADS = 256;

// four consecutive elements, one access when VEC
template <class E, bool VEC>
__device__ __forceinline__ float4 ld_e4(const void* p, int64_t i, int s, int S) {
    if constexpr (VEC) {
        if constexpr (sizeof(E) == 4) {
            return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const E*>(p) + i);
            const E* e = reinterpret_cast<const E*>(&u);
            return make_float4(ssm_ld<E>(e, 0), ssm_ld<E>(e, 1), ssm_ld<E>(e, 2), ssm_ld<E>(e, 3));
        }
    } else {
        return make_float4(s < S ? ssm_ld<E>(p, i) : 0.f, s + 1 < S ? ssm_ld<E>(p, i + 1) : 0.f,
                           s + 2 < S ? ssm_ld<E>(p, i + 2) : 0.f, s + 3 < S ? ssm_ld<E>(p, i + 3) : 0.f);
    }
}

// P lanes per channel; VEC: S = 4 P and every row of B, C, A and the state allows the wide access.  A block
// takes R rows (sequences) of its channels: A and the other weights are read once for them, and R states
// are in flight per thread.
template <class E, int P, bool VEC, int R>
__global__ void __launch_bounds__(STEP_THREADS) k_ssm_step(SsmStepArgs a, int blocks_per_row) {
    const int n0 = blockIdx.x / blocks_per_row * R;
    const int c = (blockIdx.x % blocks_per_row) * (STEP_THREADS / P) + threadIdx.x / P;
    const int p = threadIdx.x % P, s0 = 4 * p, S = a.S;
    const bool on = c < a.C;  // whole channels: the lanes of a channel agree
    const int cc = on ? c : a.C - 1, Cg = a.C / a.G, g = cc / Cg;
    int64_t hi[R];
    bool use[R];
    float4 h4[R], B4[R], C4[R];
    float u[R], raw[R], z[R];
    const float4 A4 = ld_e4<float, VEC>(a.A, int64_t(cc) * S + s0, s0, S);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t n = n0 + r;
        int64_t slot = n;
        use[r] = n < a.N;
        if (use[r] && a.slots) {
            slot = a.slots[n];
            if (slot >= a.nslots && a.status && threadIdx.x == 0) *a.status = KDA_ERR_DEVICE_CHECK;
            use[r] = slot >= 0 && slot < a.nslots;
        }
        hi[r] = (slot * a.C + cc) * S + s0;
        if (use[r]) {
            h4[r] = ld_e4<float, VEC>(a.hin, hi[r], s0, S);
            B4[r] = ld_e4<E, VEC>(a.B, n * a.ldb + int64_t(g) * S + s0, s0, S);
            C4[r] = ld_e4<E, VEC>(a.Cm, n * a.ldc + int64_t(g) * S + s0, s0, S);
            u[r] = ssm_ld<E>(a.u, n * a.ldu + cc);
            raw[r] = ssm_ld<E>(a.dt, n * a.lddt + cc);
            z[r] = a.z ? ssm_ld<E>(a.z, n * a.ldz + cc) : 0.f;
        }
    }
    const float bias = a.bias ? a.bias[cc] : 0.f, skip = a.D ? a.D[cc] : 0.f;
    const float* Av = &A4.x;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (n0 + r >= a.N) break;
        if (!use[r]) {  // an unused row: y is zero and no state is touched
            if (on && p == 0) ssm_st<E>(a.y, int64_t(n0 + r) * a.C + c, 0.f);
            continue;
        }
        const float dl = ssm_delta(__fadd_rn(raw[r], bias), a.softplus), du = dl * u[r];
        const float *hv = &h4[r].x, *Bv = &B4[r].x, *Cv = &C4[r].x;
        float4 o4;
        float* ov = &o4.x;
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ov[j] = fmaf(ex2(Av[j] * LOG2E * dl), hv[j], Bv[j] * du);
            if (VEC || s0 + j < S) y = fmaf(ov[j], Cv[j], y);
        }
#pragma unroll
        for (int o = 1; o < P; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (!on) continue;
        if constexpr (VEC) {
            *reinterpret_cast<float4*>(a.hout + hi[r]) = o4;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (s0 + j < S) a.hout[hi[r] + j] = ov[j];
        }
        if (p == 0) {
            y = fmaf(skip, u[r], y);
            if (a.z) y *= ssm_silu(z[r]);
            ssm_st<E>(a.y, int64_t(n0 + r) * a.C + c, y);
        }
    }
}

template <class E, int P, int R>
void launch(const SsmStepArgs& a, int bpr, cudaStream_t st) {
    const unsigned grid = unsigned(int64_t(bpr) * ((a.N + R - 1) / R));
    auto wide = [&](const void* p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * int64_t(sizeof(E)))) % (4 * sizeof(E)) == 0;
    };
    ProfScope ps(KK_SSM_STEP, st);
    if (a.S == 4 * P && wide(a.B, a.ldb) && wide(a.Cm, a.ldc))
        k_ssm_step<E, P, true, R><<<grid, STEP_THREADS, 0, st>>>(a, bpr);
    else
        k_ssm_step<E, P, false, R><<<grid, STEP_THREADS, 0, st>>>(a, bpr);
}

template <class E, int P>
void launch(const SsmStepArgs& a, cudaStream_t st) {
    const int bpr = (a.C * P + STEP_THREADS - 1) / STEP_THREADS;
    // four rows a block once that leaves the 152 multiprocessors four blocks each
    if (int64_t(bpr) * a.N >= 4 * 608) launch<E, P, 4>(a, bpr, st);
    else launch<E, P, 1>(a, bpr, st);
}

template <class E>
void launch_e(const SsmStepArgs& a, cudaStream_t st) {
    if (a.S <= 4) launch<E, 1>(a, st);
    else if (a.S <= 8) launch<E, 2>(a, st);
    else if (a.S <= 16) launch<E, 4>(a, st);
    else if (a.S <= 32) launch<E, 8>(a, st);
    else launch<E, 16>(a, st);
}

}  // namespace

void launch_ssm_step(const SsmStepArgs& a, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) launch_e<__nv_bfloat16>(a, st);
    else if (dtype == KDA_DT_FP16) launch_e<__half>(a, st);
    else launch_e<float>(a, st);
}

}  // namespace kda
