// Selective state-space scan for single tokens: one step of every sequence's state.
//
// Bound by HBM: the state is read and written once (8 S bytes per channel against ~10 bytes of
// inputs and output), so four consecutive states (one 16-byte access) belong to a lane, the lanes
// of a channel are neighbours, and a warp reads and writes 512 consecutive bytes.  What then costs
// is instructions, so a thread takes four sequences: the weights are read once for them, each of a
// channel's lanes computes the scalars (delta, the gate) of one sequence and hands them to the others, and
// the sums over states go back by halving, so that a lane finishes the sequence it began.  256 sequences x
// 8192 channels x 16 states: 63 us, 4.6 TB/s (three blocks per multiprocessor; 68 us with four, 97 with
// five, whose registers no longer hold the loads in flight).
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

constexpr int STEP_THREADS = 256;

// four consecutive elements as they lie in memory, one access when VEC
template <class E> struct alignas(4 * sizeof(E)) Four { E e[4]; };
template <class E, bool VEC>
__device__ __forceinline__ Four<E> ld4e(const void* p, int64_t i, int s, int S) {
    const E* q = static_cast<const E*>(p) + i;
    if constexpr (VEC) {
        return *reinterpret_cast<const Four<E>*>(q);
    } else {
        Four<E> r;
        const E zero = E(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.e[j] = s + j < S ? q[j] : zero;
        return r;
    }
}
template <class E>
__device__ __forceinline__ f2 low(const Four<E>& v) { return pk2(ssm_f<E>(v.e[0]), ssm_f<E>(v.e[1])); }
template <class E>
__device__ __forceinline__ f2 high(const Four<E>& v) { return pk2(ssm_f<E>(v.e[2]), ssm_f<E>(v.e[3])); }

constexpr int R = 4;  // sequences that a block takes together

// P lanes per channel; VEC: S = 4 P and every row of B, C, A and the state allows the wide access.
template <class E, int P, bool VEC>
__global__ void __launch_bounds__(STEP_THREADS, 3) k_ssm_step(SsmStepArgs a) {
    constexpr int RL = P < R ? R / P : 1;  // sequences whose scalars a lane computes: p, p + P, ..
    const int c = blockIdx.x * (STEP_THREADS / P) + threadIdx.x / P;
    const int p = threadIdx.x % P, s0 = 4 * p, S = a.S;
    const bool on = c < a.C;  // whole channels: the lanes of a channel agree
    const int cc = on ? c : a.C - 1, g = a.G == 1 ? 0 : cc / (a.C / a.G);
    const Four<float> A4 = ld4e<float, VEC>(a.A, int64_t(cc) * S + s0, s0, S);
    const f2 A0 = mul2(low(A4), pk2(LOG2E, LOG2E)), A1 = mul2(high(A4), pk2(LOG2E, LOG2E));
    const float bias = a.bias ? a.bias[cc] : 0.f, skip = a.D ? a.D[cc] : 0.f;
    const int64_t CS = int64_t(a.C) * S, own = int64_t(cc) * S + s0;
    for (int n0 = blockIdx.y * R; n0 < a.N; n0 += gridDim.y * R) {
        int64_t hi[R];
        bool use[R];
        Four<float> h4[R];
        Four<E> B4[R], C4[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int n = n0 + r;
            int slot = n;
            use[r] = n < a.N;
            if (use[r] && a.slots) {
                slot = a.slots[n];
                if (slot >= a.nslots && a.status && threadIdx.x == 0) *a.status = KDA_ERR_DEVICE_CHECK;
                use[r] = slot >= 0 && slot < a.nslots;
            }
            hi[r] = slot * CS + own;
            if (use[r]) {
                h4[r] = ld4e<float, VEC>(a.hin, hi[r], s0, S);
                B4[r] = ld4e<E, VEC>(a.B, n * a.ldb + g * S + s0, s0, S);
                C4[r] = ld4e<E, VEC>(a.Cm, n * a.ldc + g * S + s0, s0, S);
            }
        }
        float u[RL], z[RL], dl[RL], du[RL];
#pragma unroll
        for (int i = 0; i < RL; ++i) {
            const int n = min(n0 + ((p + i * P) & (R - 1)), a.N - 1);
            u[i] = ssm_ld<E>(a.u, n * a.ldu + cc);
            z[i] = a.z ? ssm_ld<E>(a.z, n * a.ldz + cc) : 0.f;
            dl[i] = ssm_delta(__fadd_rn(ssm_ld<E>(a.dt, n * a.lddt + cc), bias), a.softplus);
            du[i] = __fmul_rn(dl[i], u[i]);
        }
        float y[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float d = dl[P < R ? r / P : 0], v = du[P < R ? r / P : 0];
            if (P > 1) {
                d = __shfl_sync(0xffffffffu, d, r % P, P);
                v = __shfl_sync(0xffffffffu, v, r % P, P);
            }
            y[r] = 0.f;
            if (use[r]) {
                const f2 d2 = pk2(d, d), v2 = pk2(v, v);
                f2 o0 = fma2(ex2_2(mul2(A0, d2)), low(h4[r]), mul2(low(B4[r]), v2));
                f2 o1 = fma2(ex2_2(mul2(A1, d2)), high(h4[r]), mul2(high(B4[r]), v2));
                if (!VEC) {
                    o0 = keep2(o0, s0, S);
                    o1 = keep2(o1, s0 + 2, S);
                }
                y[r] = hsum2(fma2(o1, high(C4[r]), mul2(o0, low(C4[r]))));
                if (on) {
                    if constexpr (VEC) {
                        *reinterpret_cast<ulonglong2*>(a.hout + hi[r]) = make_ulonglong2(o0, o1);
                    } else {
                        float o[4];
                        up2(o0, o[0], o[1]);
                        up2(o1, o[2], o[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (s0 + j < S) a.hout[hi[r] + j] = o[j];
                    }
                }
            }
        }
        // lane p ends with the sums of sequences p, p + P, .. (P of 4 and more: sequence p mod 4)
        if (P > 1) {
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
                const float give = p & 1 ? y[2 * i] : y[2 * i + 1], keep = p & 1 ? y[2 * i + 1] : y[2 * i];
                y[i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            }
        }
        if (P > 2) {
            const float give = p & 2 ? y[0] : y[1], keep = p & 2 ? y[1] : y[0];
            y[0] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        }
#pragma unroll
        for (int o = 4; o < P; o <<= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
        if (on && (P <= R || p < R))
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                const int r = (p + i * P) & (R - 1);
                if (n0 + r >= a.N) continue;
                bool used = false;
#pragma unroll
                for (int j = 0; j < R; ++j) used |= j == r && use[j];
                float v = fmaf(skip, u[i], y[i]);
                if (a.z) v *= ssm_silu(z[i]);
                // an unused row: y is zero and no state was touched
                ssm_st<E>(a.y, int64_t(n0 + r) * a.C + c, used ? v : 0.f);
            }
    }
}

template <class E, int P>
void launch(const SsmStepArgs& a, cudaStream_t st) {
    // a block takes one group of R sequences, or several once the launch would pass eight waves of three blocks on
    // each of the 152 multiprocessors (256 sequences x 8192 channels: 65.5 us so, 68 with a block for every group)
    const int groups = (a.N + R - 1) / R, gx = (a.C + STEP_THREADS / P - 1) / (STEP_THREADS / P);
    constexpr int most = 8 * 3 * 152;
    const int per = int((int64_t(gx) * groups + most - 1) / most);
    const dim3 grid(unsigned(gx), unsigned((groups + per - 1) / per));
    auto wide = [&](const void* p, int64_t ld) {
        return (reinterpret_cast<uintptr_t>(p) | uintptr_t(ld * int64_t(sizeof(E)))) % (4 * sizeof(E)) == 0;
    };
    ProfScope ps(KK_SSM_STEP, st);
    if (a.S == 4 * P && wide(a.B, a.ldb) && wide(a.Cm, a.ldc)) k_ssm_step<E, P, true><<<grid, STEP_THREADS, 0, st>>>(a);
    else k_ssm_step<E, P, false><<<grid, STEP_THREADS, 0, st>>>(a);
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
