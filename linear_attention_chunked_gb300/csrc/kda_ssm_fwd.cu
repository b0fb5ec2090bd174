// Selective state-space scan over packed documents, forward (kda_ssm.cuh has the formulas).
//
// A document is cut into chunks of 64 tokens.  Three launches after the chunk plan:
//   k_ssm_state  per chunk that has a successor: its end state from a zero start, and sum(delta)
//   k_ssm_carry  per (document, channel, state): start_{k+1} = exp(A sum(delta)_k) start_k + end_k
//   k_ssm_out    per chunk: the recurrence from its start state, y, and the final state
// so a long document fills the machine whatever its batch, at the price of a second evaluation of
// the decays in the chunks that have a successor.  Lanes are channels: u, dt, z and y rows are read and
// written as they lie, a lane's B and C values are shared-memory broadcasts, and the sum over
// states stays in the lane.
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

constexpr int GR = 8;  // tokens loaded ahead of their use

// Places a block's threads on (group, channel, first state): CB channels of one group per block.
template <int SPT, int P>
struct Place {
    static constexpr int CB = SSM_THREADS / P;  // channels per block
    static constexpr int CW = 32 / P;           // channels per warp
    int g, c, s0;                               // group, channel, first state of the lane
    bool on;
    __device__ __forceinline__ Place(const SsmArgs& a, int tile) {
        const int Cg = a.C / a.G, tg = (Cg + CB - 1) / CB;
        g = tile / tg;
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        const int ci = (tile - g * tg) * CB + w * CW + lane % CW;
        on = ci < Cg;
        c = g * Cg + (on ? ci : Cg - 1);  // lanes past the group repeat its last channel, unwritten
        s0 = lane / CW * SPT;
    }
};

template <int SPT>
__device__ __forceinline__ void load_A(const SsmArgs& a, int c, int s0, f2 (&A2)[SPT / 2]) {
#pragma unroll
    for (int j = 0; j < SPT / 2; ++j) {
        const int s = s0 + 2 * j;
        const float* row = a.A + int64_t(c) * a.S;
        A2[j] = pk2(s < a.S ? LOG2E * row[s] : 0.f, s + 1 < a.S ? LOG2E * row[s + 1] : 0.f);
    }
}

template <class E, int SPT, int P, bool FULL>
__global__ void __launch_bounds__(SSM_THREADS) k_ssm_state(SsmArgs a, int tiles) {
    constexpr int SP = SPT * P, H2 = SPT / 2;
    __shared__ __align__(16) float sB[CH * SP];
    const int k = blockIdx.x / tiles;
    if (k >= *a.nchunks) return;
    const int4 t = a.chunk_tab[k];
    if (t.y + t.z == a.cu[t.x + 1]) return;  // no successor
    const Place<SPT, P> pl(a, blockIdx.x % tiles);
    ssm_load_rows<E, SP>(sB, a.B, a.ldb, t.y, CH, pl.g * a.S, a.S);
    f2 A2[H2], h[H2];
    load_A<SPT>(a, pl.c, pl.s0, A2);
#pragma unroll
    for (int j = 0; j < H2; ++j) h[j] = 0;
    const float bias = a.bias ? a.bias[pl.c] : 0.f;
    float sum = 0.f;
    Ahead<E, GR> u(a.u, t.y, a.ldu, pl.c), d(a.dt, t.y, a.lddt, pl.c);
    u.load(GR);
    d.load(GR);
    __syncthreads();
#pragma unroll 1
    for (int q = 0; q < CH; q += GR) {  // a chunk with a successor is full
        E cu[GR], cd[GR];
#pragma unroll
        for (int i = 0; i < GR; ++i) cu[i] = u.raw[i], cd[i] = d.raw[i];
        if (q + GR < CH) {
            u.load(GR);
            d.load(GR);
        }
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            const float dl = ssm_delta(ssm_f<E>(cd[i]) + bias, a.softplus), du = dl * ssm_f<E>(cu[i]);
            sum += dl;
            const f2 dl2 = pk2(dl, dl), du2 = pk2(du, du);
            const ulonglong2* Bp = reinterpret_cast<const ulonglong2*>(sB + (q + i) * SP + pl.s0);
#pragma unroll
            for (int j = 0; j < H2; j += 2) {
                const ulonglong2 b2 = Bp[j / 2];
                h[j] = fma2(ex2_2(mul2(A2[j], dl2)), h[j], mul2(b2.x, du2));
                h[j + 1] = fma2(ex2_2(mul2(A2[j + 1], dl2)), h[j + 1], mul2(b2.y, du2));
            }
        }
    }
    if (!pl.on) return;
    if (pl.s0 == 0) a.sumdt[int64_t(k) * a.C + pl.c] = sum;
    float* out = a.hs + (int64_t(k + 1) * a.sub * a.C + pl.c) * a.S + pl.s0;  // the next chunk's slot
#pragma unroll
    for (int j = 0; j < H2; ++j) {
        float x, y;
        up2(h[j], x, y);
        if (FULL || pl.s0 + 2 * j < a.S) out[2 * j] = x;
        if (FULL || pl.s0 + 2 * j + 1 < a.S) out[2 * j + 1] = y;
    }
}

// One thread per (document, channel, state).  Chunk k + 1's slot of hs holds chunk k's end from a zero
// start and receives chunk k + 1's start state.
constexpr int CARRY_THREADS = 128;
__global__ void __launch_bounds__(CARRY_THREADS) k_ssm_carry(SsmArgs a, int blocks_per_doc) {
    if (*a.status != KDA_OK) return;
    const int n = blockIdx.x / blocks_per_doc;
    const int64_t CS = int64_t(a.C) * a.S;
    const int64_t i = int64_t(blockIdx.x % blocks_per_doc) * CARRY_THREADS + threadIdx.x;
    if (i >= CS) return;
    const int c = int(i / a.S);
    const int k0 = a.doc_off[n], k1 = a.doc_off[n + 1];
    float h = a.h0 ? a.h0[n * CS + i] : 0.f;
    if (k0 == k1) {  // an empty document's final state
        if (a.ht) a.ht[n * CS + i] = h;
        return;
    }
    const float A2 = LOG2E * a.A[i];
    const int64_t hstep = CS * a.sub;
    float* hs = a.hs + k0 * hstep + i;
    const float* sd = a.sumdt + int64_t(k0) * a.C + c;
    hs[0] = h;
    constexpr int U = 8;  // chunks loaded together
    for (int k = 0; k < k1 - k0 - 1; k += U) {
        float e[U], d[U];
        const int m = min(U, k1 - k0 - 1 - k);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j < m) {
                e[j] = hs[(k + j + 1) * hstep];
                d[j] = sd[int64_t(k + j) * a.C];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j < m) {
                h = fmaf(ex2(A2 * d[j]), h, e[j]);
                hs[(k + j + 1) * hstep] = h;
            }
    }
}

template <class E, int SPT, int P, bool FULL>
__global__ void __launch_bounds__(SSM_THREADS) k_ssm_out(SsmArgs a, int tiles) {
    constexpr int SP = SPT * P, H2 = SPT / 2;
    __shared__ __align__(16) float sB[CH * SP], sC[CH * SP];
    const int k = blockIdx.x / tiles;
    if (k >= *a.nchunks) return;
    const int4 t = a.chunk_tab[k];
    const int len = t.z;
    const Place<SPT, P> pl(a, blockIdx.x % tiles);
    ssm_load_rows<E, SP>(sB, a.B, a.ldb, t.y, len, pl.g * a.S, a.S);
    ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t.y, len, pl.g * a.S, a.S);
    f2 A2[H2], h[H2];
    load_A<SPT>(a, pl.c, pl.s0, A2);
    {
        const float* in = a.hs + (int64_t(k) * a.sub * a.C + pl.c) * a.S + pl.s0;
#pragma unroll
        for (int j = 0; j < H2; ++j)
            h[j] = pk2(FULL || pl.s0 + 2 * j < a.S ? in[2 * j] : 0.f,
                       FULL || pl.s0 + 2 * j + 1 < a.S ? in[2 * j + 1] : 0.f);
    }
    const float bias = a.bias ? a.bias[pl.c] : 0.f, skip = a.D ? a.D[pl.c] : 0.f;
    // (the backward's replay takes the states alone: no y, no ht)
    const bool writer = a.y && pl.on && pl.s0 == 0, gated = a.z, keep = a.sub > 1;
    Ahead<E, GR> u(a.u, t.y, a.ldu, pl.c), d(a.dt, t.y, a.lddt, pl.c), z(a.z, t.y, a.ldz, pl.c);
    E* yp = static_cast<E*>(a.y) + int64_t(t.y) * a.C + pl.c;
    u.load(len);
    d.load(len);
    if (gated) z.load(len);
    __syncthreads();
    E cu[GR], cd[GR], cz[GR];
    auto token = [&](int q, int i) {
        const float x = ssm_f<E>(cu[i]);
        const float dl = ssm_delta(ssm_f<E>(cd[i]) + bias, a.softplus), du = dl * x;
        const f2 dl2 = pk2(dl, dl), du2 = pk2(du, du);
        const ulonglong2* Bp = reinterpret_cast<const ulonglong2*>(sB + (q + i) * SP + pl.s0);
        const ulonglong2* Cp = reinterpret_cast<const ulonglong2*>(sC + (q + i) * SP + pl.s0);
        f2 acc = 0;
#pragma unroll
        for (int j = 0; j < H2; j += 2) {
            const ulonglong2 b2 = Bp[j / 2], c2 = Cp[j / 2];
            h[j] = fma2(ex2_2(mul2(A2[j], dl2)), h[j], mul2(b2.x, du2));
            h[j + 1] = fma2(ex2_2(mul2(A2[j + 1], dl2)), h[j + 1], mul2(b2.y, du2));
            if (!FULL) {
                h[j] = keep2(h[j], pl.s0 + 2 * j, a.S);
                h[j + 1] = keep2(h[j + 1], pl.s0 + 2 * j + 2, a.S);
            }
            acc = fma2(h[j], c2.x, acc);
            acc = fma2(h[j + 1], c2.y, acc);
        }
        float y = hsum2(acc);
#pragma unroll
        for (int o = 32 / P; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        y = fmaf(skip, x, y);
        if (gated) y *= ssm_silu(ssm_f<E>(cz[i]));
        if (writer) ssm_st<E>(yp, int64_t(i) * a.C, y);
    };
#pragma unroll 1
    for (int q = 0; q < len; q += GR) {
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            cu[i] = u.raw[i], cd[i] = d.raw[i];
            if (gated) cz[i] = z.raw[i];
        }
        if (q + GR < len) {
            u.load(len - q - GR);
            d.load(len - q - GR);
            if (gated) z.load(len - q - GR);
        }
        if (keep && q % SSM_UT == 0 && q > 0 && pl.on) {
            float* out = a.hs + ((int64_t(k) * a.sub + q / SSM_UT) * a.C + pl.c) * a.S + pl.s0;
#pragma unroll
            for (int j = 0; j < H2; ++j) {
                float x, y;
                up2(h[j], x, y);
                if (FULL) {
                    *reinterpret_cast<float2*>(out + 2 * j) = make_float2(x, y);
                } else {
                    if (pl.s0 + 2 * j < a.S) out[2 * j] = x;
                    if (pl.s0 + 2 * j + 1 < a.S) out[2 * j + 1] = y;
                }
            }
        }
        if (q + GR <= len) {
#pragma unroll
            for (int i = 0; i < GR; ++i) token(q, i);
        } else {
#pragma unroll
            for (int i = 0; i < GR - 1; ++i)
                if (q + i < len) token(q, i);
        }
        yp += GR * int64_t(a.C);
    }
    if (a.ht && pl.on && t.y + len == a.cu[t.x + 1]) {  // the document's last chunk
        float* out = a.ht + (int64_t(t.x) * a.C + pl.c) * a.S + pl.s0;
#pragma unroll
        for (int j = 0; j < H2; ++j) {
            float x, y;
            up2(h[j], x, y);
            if (FULL || pl.s0 + 2 * j < a.S) out[2 * j] = x;
            if (FULL || pl.s0 + 2 * j + 1 < a.S) out[2 * j + 1] = y;
        }
    }
}

template <class E, int SPT, int P, bool FULL>
void launch(const SsmArgs& a, cudaStream_t st) {
    const int Cg = a.C / a.G, CB = SSM_THREADS / P;
    const int tiles = a.G * ((Cg + CB - 1) / CB);
    const unsigned grid = unsigned(a.maxC * tiles);
    if (a.T > CH) {  // a pack of at most one chunk of tokens has no chunk with a successor
        ProfScope ps(KK_SSM_STATE, st);
        k_ssm_state<E, SPT, P, FULL><<<grid, SSM_THREADS, 0, st>>>(a, tiles);
    }
    {
        ProfScope ps(KK_SSM_CARRY, st);
        const int64_t CS = int64_t(a.C) * a.S;
        const int bpd = int((CS + CARRY_THREADS - 1) / CARRY_THREADS);
        k_ssm_carry<<<unsigned(int64_t(bpd) * a.N), CARRY_THREADS, 0, st>>>(a, bpd);
    }
    if (grid) {
        ProfScope ps(KK_SSM_OUT, st);
        k_ssm_out<E, SPT, P, FULL><<<grid, SSM_THREADS, 0, st>>>(a, tiles);
    }
}

template <class E>
void launch_e(const SsmArgs& a, cudaStream_t st) {
    switch (a.S) {  // the usual state counts fill their lanes; others are padded to the next one
        case 4: return launch<E, 4, 1, true>(a, st);
        case 8: return launch<E, 8, 1, true>(a, st);
        case 16: return launch<E, 16, 1, true>(a, st);
        case 32: return launch<E, 16, 2, true>(a, st);
        case 64: return launch<E, 16, 4, true>(a, st);
        default: break;
    }
    if (a.S < 8) return launch<E, 8, 1, false>(a, st);
    if (a.S < 16) return launch<E, 16, 1, false>(a, st);
    if (a.S < 32) return launch<E, 16, 2, false>(a, st);
    return launch<E, 16, 4, false>(a, st);
}

}  // namespace

void launch_ssm_scan(const SsmArgs& a, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) launch_e<__nv_bfloat16>(a, st);
    else if (dtype == KDA_DT_FP16) launch_e<__half>(a, st);
    else launch_e<float>(a, st);
}

}  // namespace kda
