// Shared parts of the selective state-space scan (prompt, backward and single-token kernels); the layer norm
// uses its element types and packed arithmetic.
//
// Per document, channel c, state s and the channel's group g of B and C:
//   delta = softplus(dt + bias)   (or dt + bias),   a = exp(delta A[c, s])
//   h_t = a h_{t-1} + (delta u) B[t, g, s],   y = (sum_s C[t, g, s] h_t + D u) silu(z)
//
// A thread holds SPT states of one channel in registers as pairs (packed fp32 arithmetic: one
// instruction per two states); P neighbouring groups of lanes share a channel when it has more
// than SPT states.  A is scaled by log2(e) once, so a decay is one multiply and one ex2.
#pragma once

#include <cuda_fp16.h>

#include "kda_internal.cuh"

namespace kda {

constexpr int SSM_THREADS = 128;
constexpr int SSM_MAXS = 64;  // states per channel
constexpr int SSM_UT = 16;           // tokens between the states kept for the backward
constexpr int SSM_SUB = CH / SSM_UT;
constexpr float LOG2E = 1.4426950408889634f;

struct SsmArgs {
    int64_t T, maxC;
    int N, C, S, G;
    int softplus;
    int64_t ldu, lddt, ldb, ldc, ldz;  // row strides (elements) of u, dt, B, C, z
    const int* cu;
    const void *u, *dt, *B, *Cm, *z, *dy;
    const float *A, *D, *bias, *h0, *dht;
    void *y, *du, *ddt, *dB, *dC, *dz;  // dense rows
    float *ht, *dA, *dD, *dbias, *dh0;
    // workspace
    int *status, *nchunks, *doc_off;  // the chunk plan's (a saved set holds its forward's plan)
    int* call_status;                 // the first word of this call's workspace
    int4* chunk_tab;                  // {doc, first token, length, chunk index within the doc}
    int4* made_for;                   // beside a saved set's plan: the sizes of the forward that wrote it
    int4 sizes;                       // this call's
    int from_saved;                   // the plan is a saved set's (backward)
    int direct;                       // every document fits one chunk: no plan, no carry
    int sub;          // states kept per chunk: 1 (its start) or SSM_SUB (every SSM_UT-th token: the backward's set)
    float* sumdt;     // [maxC][C] sum of delta over the chunk
    float* hs;        // [maxC][sub][C][S] those states (a document's first: h0)
    float* gs;        // [maxC][C][S] gradient of the state at each chunk's end (last chunk: dht)
    float* pBC;       // [channel blocks][T][2 S] partial sums of dB and dC
    float* pA;        // [maxC][C][S + 2] partial sums of dA, dD, dbias
};

// Whether the call's plan may be followed: well-formed offsets, and a saved set that was written for these
// sizes (the plan of another problem, or what a buffer held that no forward wrote, would lead outside the
// tensors).
__device__ __forceinline__ bool ssm_plan_ok(const SsmArgs& a) {
    if (*a.status != KDA_OK) return false;
    if (!a.from_saved) return true;
    const int4 m = *a.made_for;
    return m.x == a.sizes.x && m.y == a.sizes.y && m.z == a.sizes.z && m.w == a.sizes.w;
}

// ---- element types ----
template <class E> __device__ __forceinline__ float ssm_ld(const void* p, int64_t i);
template <> __device__ __forceinline__ float ssm_ld<float>(const void* p, int64_t i) {
    return static_cast<const float*>(p)[i];
}
template <> __device__ __forceinline__ float ssm_ld<__nv_bfloat16>(const void* p, int64_t i) {
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <> __device__ __forceinline__ float ssm_ld<__half>(const void* p, int64_t i) {
    return __half2float(static_cast<const __half*>(p)[i]);
}
template <class E> __device__ __forceinline__ void ssm_st(void* p, int64_t i, float v);
template <> __device__ __forceinline__ void ssm_st<float>(void* p, int64_t i, float v) {
    static_cast<float*>(p)[i] = v;
}
template <> __device__ __forceinline__ void ssm_st<__nv_bfloat16>(void* p, int64_t i, float v) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
template <> __device__ __forceinline__ void ssm_st<__half>(void* p, int64_t i, float v) {
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// ---- packed fp32 pairs ----
typedef unsigned long long f2;
__device__ __forceinline__ f2 pk2(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void up2(f2 v, float& x, float& y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
    float x, y;
    up2(v, x, y);
    return pk2(ex2(x), ex2(y));
}
__device__ __forceinline__ float hsum2(f2 v) {
    float x, y;
    up2(v, x, y);
    return x + y;
}
// the pair with the states at or past S cleared (channels whose S does not fill the lanes' slots:
// an infinite input times a padded zero must not reach y)
__device__ __forceinline__ f2 keep2(f2 v, int s, int S) {
    float x, y;
    up2(v, x, y);
    return pk2(s < S ? x : 0.f, s + 1 < S ? y : 0.f);
}

__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// z sigmoid(z).  Past z = -87 the divisor leaves the range of its reciprocal: the limit there is 0
__device__ __forceinline__ float ssm_silu(float z) {
    return __fmul_rn(z, z < -87.f ? 0.f : rcp(__fadd_rn(1.f, ex2(-LOG2E * z))));
}

// two logistic functions; gate: exactly 0 below -87, so that z times it has silu's limit
template <bool GATE = false>
__device__ __forceinline__ f2 ssm_sigmoid2(f2 z) {
    float x, y, p, q;
    up2(z, x, y);
    up2(mul2(z, pk2(-LOG2E, -LOG2E)), p, q);
    up2(add2(pk2(ex2(p), ex2(q)), pk2(1.f, 1.f)), p, q);
    return GATE ? pk2(x < -87.f ? 0.f : rcp(p), y < -87.f ? 0.f : rcp(q)) : pk2(rcp(p), rcp(q));
}
__device__ __forceinline__ f2 ssm_gate2(f2 z) { return ssm_sigmoid2<true>(z); }

// softplus(x) = max(x, 0) + log1p(u), u = e^-|x| in (0, 1], with log1p(u) = 2 atanh(z), z = u / (2 + u) in
// (0, 1/3].  2 atanh(z) / z is a polynomial in z^2 (its minimax fit on [0, 1/9] by Remez exchange:
// relative error 7.8e-9 with the coefficients as rounded, below fp32's rounding).  Two values at a time.
__device__ __forceinline__ f2 ssm_delta2(f2 raw, int softplus) {
    if (!softplus) return raw;
    float x, y;
    up2(raw, x, y);
    const f2 u = pk2(ex2(-LOG2E * fabsf(x)), ex2(-LOG2E * fabsf(y)));
    float d, e;
    up2(add2(u, pk2(2.f, 2.f)), d, e);
    const f2 z = mul2(u, pk2(rcp(d), rcp(e))), z2 = mul2(z, z);
    f2 p = fma2(z2, pk2(0.28178334f, 0.28178334f), pk2(0.279606f, 0.279606f));
    p = fma2(z2, p, pk2(0.4002491f, 0.4002491f));
    p = fma2(z2, p, pk2(0.66666317f, 0.66666317f));
    p = fma2(z2, p, pk2(2.f, 2.f));
    return fma2(z, p, pk2(fmaxf(x, 0.f), fmaxf(y, 0.f)));
}
// one value (the same operations)
__device__ __forceinline__ float ssm_delta(float raw, int softplus) {
    if (!softplus) return raw;
    const float u = ex2(-LOG2E * fabsf(raw));
    const float z = __fmul_rn(u, rcp(__fadd_rn(u, 2.f))), z2 = __fmul_rn(z, z);
    float p = fmaf(z2, 0.28178334f, 0.279606f);
    p = fmaf(z2, p, 0.4002491f);
    p = fmaf(z2, p, 0.66666317f);
    p = fmaf(z2, p, 2.f);
    return fmaf(z, p, fmaxf(raw, 0.f));
}

// An element as it lies in memory: rows loaded ahead are kept so, and widened where they are used (a
// widening right behind the load would wait for it)
template <class E> __device__ __forceinline__ float ssm_f(E v) { return ssm_ld<E>(&v, 0); }

// SP = P SPT states per channel slot; the block's B (and C) rows of a chunk as fp32 [CH][SP]
template <class E, int SP, int NTH = SSM_THREADS>
__device__ __forceinline__ void ssm_load_rows(float* s, const void* g, int64_t ld, int64_t t0,
                                              int len, int col0, int S) {
    constexpr int N = CH * SP / NTH, U = N < 8 ? N : 8;  // loads of a thread, in flight together
    const E* p = static_cast<const E*>(g) + t0 * ld + col0;
#pragma unroll
    for (int j = 0; j < N; j += U) {
        E raw[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = threadIdx.x + (j + i) * NTH, r = e / SP, k = e % SP;
            if (r < len && k < S) raw[i] = p[r * ld + k];
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int e = threadIdx.x + (j + i) * NTH, r = e / SP, k = e % SP;
            s[e] = r < len && k < S ? ssm_f<E>(raw[i]) : 0.f;
        }
    }
}

}  // namespace kda
