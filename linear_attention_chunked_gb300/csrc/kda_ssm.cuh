// Shared parts of the selective state-space scan (prompt, backward and single-token kernels).
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
    int *status, *nchunks, *doc_off;
    int4* chunk_tab;  // {doc, first token, length, chunk index within the doc}
    float* sumdt;     // [maxC][C] sum of delta over the chunk
    float* hs;        // [maxC][C][S] state at each chunk's start (a document's first chunk: h0)
    float* gs;        // [maxC][C][S] gradient of the state at each chunk's end (last chunk: dht)
    float* pBC;       // [channel blocks][T][2 S] partial sums of dB and dC
    float* pA;        // [maxC][C][S + 2] partial sums of dA, dD, dbias
    int nsplit;       // channel blocks per group of the backward
};

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

// z silu'(..) helpers: the fast reciprocal is 0 once 1 + e^-z exceeds 2^126, the limit there
__device__ __forceinline__ float ssm_sigmoid(float z) { return __fdividef(1.f, 1.f + ex2(-LOG2E * z)); }
__device__ __forceinline__ float ssm_silu(float z) {
    // below -87 the quotient's divisor overflows the fast division's range: the limit there is 0
    return z < -87.f ? 0.f * z : __fdividef(z, 1.f + ex2(-LOG2E * z));
}

__device__ __forceinline__ float ssm_delta(float raw, int softplus) {
    return softplus ? softplus_f(raw) : raw;
}

// SP = P SPT states per channel slot; the block's B (and C) rows of a chunk as fp32 [CH][SP]
template <class E, int SP, int NTH = SSM_THREADS>
__device__ __forceinline__ void ssm_load_rows(float* s, const void* g, int64_t ld, int64_t t0,
                                              int len, int col0, int S) {
    for (int i = threadIdx.x; i < CH * SP; i += NTH) {
        const int r = i / SP, k = i % SP;
        s[i] = r < len && k < S ? ssm_ld<E>(g, (t0 + r) * ld + col0 + k) : 0.f;
    }
}

// Slots of a lane for S states per channel: SPT states per lane, P lanes per channel.
struct SsmShape { int spt, p; };

// ---- launches ----
enum { SSM_BF16 = KDA_DT_BF16, SSM_FP16 = KDA_DT_FP16, SSM_FP32 = KDA_DT_FP32 };

}  // namespace kda
