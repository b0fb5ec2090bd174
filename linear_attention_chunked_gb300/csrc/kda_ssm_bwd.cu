// Selective state-space scan, backward.  With dY = dy silu(z) and G_t the gradient of h_t
// (G_t = C_t dY_t + a_{t+1} G_{t+1}, from dht at a document's last token):
//   dC_t[s] = sum_c dY h_t        dB_t[s] = sum_c G delta u       (sums over the group's channels)
//   sB = sum_s G B, w = a G h_{t-1}:  du = delta sB + D dY,  ddelta = u sB + sum_s A w
//   dA = sum_t delta w,  dD = sum_t dY u,  ddt = ddelta softplus'(dt + bias),  dbias = sum_t ddt
//   dz = dy y0 silu'(z),  y0 = sum_s C h + D u,  dh0 = a_1 G_1
//
//   k_ssm_rstate   per chunk with a predecessor: its start gradient from a zero end,
//                  sum_t exp(A (delta_1 + .. + delta_t)) C_t dY_t, and sum(delta)
//   k_ssm_rcarry   per (document, channel, state): the chunks' end gradients, last to first
//   k_ssm_bwd      per (chunk, channel tile): the gradients
//   k_ssm_reduce_* the sums over channel tiles (dB, dC) and over chunks (dA, dD, dbias), in order
//
// k_ssm_bwd needs h_{t-1} in reverse.  A chunk is swept forward once from its start state, the
// states every SB = 8 tokens kept in shared memory; each run of 8 tokens is then recomputed from
// its start with states and decays in registers and walked backwards.  Four lanes hold a channel's 16
// states (four each).  A lane's eight dB / dC terms per token are summed over two channels in
// registers before they cross lanes, and cross them by halving (each step a lane gives away half
// of its values), 7 shuffles for 8 values over 8 lanes.
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

constexpr int SB = 8;        // tokens per run
constexpr int NSB = CH / SB; // runs per chunk
constexpr int NP = 2;        // channel passes per warp
constexpr int NW = SSM_THREADS / 32;
constexpr int SPT = 4;       // states per lane

__device__ __forceinline__ float4 ld4(const float* p, int s, int S) {
    return make_float4(s < S ? p[s] : 0.f, s + 1 < S ? p[s + 1] : 0.f, s + 2 < S ? p[s + 2] : 0.f,
                       s + 3 < S ? p[s + 3] : 0.f);
}
__device__ __forceinline__ void st4(float* p, int s, int S, float4 v) {
    if (s < S) p[s] = v.x;
    if (s + 1 < S) p[s + 1] = v.y;
    if (s + 2 < S) p[s + 2] = v.z;
    if (s + 3 < S) p[s + 3] = v.w;
}

// ---- gradient at a chunk's start from a zero end ----

template <class E, int SPTR, int P>
__global__ void __launch_bounds__(SSM_THREADS) k_ssm_rstate(SsmArgs a, int tiles) {
    constexpr int SP = SPTR * P, H2 = SPTR / 2, CB = SSM_THREADS / P, CW = 32 / P, GR = 8;
    __shared__ __align__(16) float sC[CH * SP];
    const int k = blockIdx.x / tiles;
    if (k >= *a.nchunks) return;
    const int4 t = a.chunk_tab[k];
    if (t.w == 0) return;  // no predecessor
    const int len = t.z;
    const int Cg = a.C / a.G, tg = (Cg + CB - 1) / CB, tile = blockIdx.x % tiles, g = tile / tg;
    const int lane = threadIdx.x & 31;
    const int ci = (tile - g * tg) * CB + (threadIdx.x >> 5) * CW + lane % CW;
    const bool on = ci < Cg;
    const int c = g * Cg + (on ? ci : Cg - 1), s0 = lane / CW * SPTR;
    ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t.y, len, g * a.S, a.S);
    f2 A2[H2], acc[H2];
#pragma unroll
    for (int j = 0; j < H2; ++j) {
        const int s = s0 + 2 * j;
        const float* row = a.A + int64_t(c) * a.S;
        A2[j] = pk2(s < a.S ? LOG2E * row[s] : 0.f, s + 1 < a.S ? LOG2E * row[s + 1] : 0.f);
        acc[j] = 0;
    }
    const float bias = a.bias ? a.bias[c] : 0.f;
    const int64_t id = int64_t(t.y) * a.lddt + c, iz = int64_t(t.y) * a.ldz + c;
    const int64_t iy = int64_t(t.y) * a.C + c;
    float rd[GR], rz[GR], ry[GR], sum = 0.f;
    auto load = [&](int q) {
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            const int r = min(q + i, len - 1);
            rd[i] = ssm_ld<E>(a.dt, id + r * a.lddt);
            ry[i] = ssm_ld<E>(a.dy, iy + int64_t(r) * a.C);
            rz[i] = a.z ? ssm_ld<E>(a.z, iz + r * a.ldz) : 0.f;
        }
    };
    load(0);
    __syncthreads();
    for (int q = 0; q < len; q += GR) {
        float cd[GR], cy[GR], cz[GR];
#pragma unroll
        for (int i = 0; i < GR; ++i) cd[i] = rd[i], cy[i] = ry[i], cz[i] = rz[i];
        if (q + GR < len) load(q + GR);
#pragma unroll
        for (int i = 0; i < GR; ++i) {
            if (q + i >= len) break;
            sum += ssm_delta(cd[i] + bias, a.softplus);
            const float dY = a.z ? cy[i] * ssm_silu(cz[i]) : cy[i];
            const f2 s2 = pk2(sum, sum), d2 = pk2(dY, dY);
            const f2* Cp = reinterpret_cast<const f2*>(sC + (q + i) * SP + s0);
#pragma unroll
            for (int j = 0; j < H2; ++j)
                acc[j] = fma2(ex2_2(mul2(A2[j], s2)), mul2(Cp[j], d2), acc[j]);
        }
    }
    if (!on) return;
    if (s0 == 0) a.sumdt[int64_t(k) * a.C + c] = sum;
    float* out = a.gs + (int64_t(k - 1) * a.C + c) * a.S;  // the chunk before: its end
#pragma unroll
    for (int j = 0; j < H2; ++j) {
        float x, y;
        up2(acc[j], x, y);
        if (s0 + 2 * j < a.S) out[s0 + 2 * j] = x;
        if (s0 + 2 * j + 1 < a.S) out[s0 + 2 * j + 1] = y;
    }
}

constexpr int CARRY_THREADS = 128;
__global__ void __launch_bounds__(CARRY_THREADS) k_ssm_rcarry(SsmArgs a, int blocks_per_doc) {
    if (*a.status != KDA_OK) return;
    const int n = blockIdx.x / blocks_per_doc;
    const int64_t CS = int64_t(a.C) * a.S;
    const int64_t i = int64_t(blockIdx.x % blocks_per_doc) * CARRY_THREADS + threadIdx.x;
    if (i >= CS) return;
    const int c = int(i / a.S);
    const int k0 = a.doc_off[n], nc = a.doc_off[n + 1] - k0;
    float g = a.dht ? a.dht[n * CS + i] : 0.f;
    if (nc == 0) {  // an empty document hands its end gradient on
        if (a.dh0) a.dh0[n * CS + i] = g;
        return;
    }
    const float A2 = LOG2E * a.A[i];
    float* gs = a.gs + int64_t(k0) * CS + i;
    const float* sd = a.sumdt + int64_t(k0) * a.C + c;
    gs[int64_t(nc - 1) * CS] = g;
    constexpr int U = 8;
    for (int k = nc - 1; k > 0; k -= U) {
        float e[U], d[U];
        const int m = min(U, k);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j < m) {
                e[j] = gs[(k - j - 1) * CS];
                d[j] = sd[int64_t(k - j) * a.C];
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j < m) {
                g = fmaf(ex2(A2 * d[j]), g, e[j]);
                gs[(k - j - 1) * CS] = g;
            }
    }
}

// ---- the gradients ----

// Sums v[0 .. NV-1] over the CL channel lanes of a warp (lane bits from P up), halving: on return a
// lane holds the sums of values idx .. idx + n - 1 in v[0 .. n-1], n = max(1, NV / CL).
template <int NV, int P>
__device__ __forceinline__ void reduce_lanes(float (&v)[NV], int lane) {
    int n = NV;
#pragma unroll
    for (int o = P; o < 32; o <<= 1) {
        if (n > 1) {
            const bool up = lane & o;
#pragma unroll
            for (int i = 0; i < NV / 2; ++i)
                if (i < n / 2) {
                    const float give = up ? v[i] : v[i + n / 2];
                    const float keep = up ? v[i + n / 2] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            n /= 2;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
}
template <int NV, int P>
__device__ __forceinline__ int reduce_index(int lane) {
    int n = NV, idx = 0;
#pragma unroll
    for (int o = P; o < 32; o <<= 1)
        if (n > 1) {
            n /= 2;
            if (lane & o) idx += n;
        }
    return idx;
}

template <int P>
struct BwdShape {
    static constexpr int CL = 32 / P;       // channels of a pass
    static constexpr int CW = NP * CL;      // channels of a warp
    static constexpr int CB = NW * CW;      // channels of a tile
    static constexpr int SP = SPT * P;      // state slots
    // shared memory, in floats
    static constexpr int oB = 0, oC = oB + CH * SP, oPre = oC + CH * SP;
    static constexpr int oCk = oPre + NW * SB * CW * 4;
    static constexpr int oG = oCk + NSB * NP * SSM_THREADS * 4;
    static constexpr int oRed = oG + 2 * NP * SSM_THREADS * 4;
    static constexpr int oBC = oRed + NW * SB * 2 * SP;
    static constexpr int floats = oBC + CH * 2 * SP;
};

template <class E, int P>
__global__ void __launch_bounds__(SSM_THREADS) k_ssm_bwd(SsmArgs a, SsmBwdPlan pl) {
    using L = BwdShape<P>;
    constexpr int CL = L::CL, CW = L::CW, SP = L::SP;
    extern __shared__ __align__(16) float sm[];
    const int per_chunk = a.G * pl.splits;
    const int k = blockIdx.x / per_chunk;
    if (k >= *a.nchunks) return;
    const int4 tab = a.chunk_tab[k];
    const int t0 = tab.y, len = tab.z, nsub = (len + SB - 1) / SB;
    const int gsp = blockIdx.x % per_chunk, g_ = gsp / pl.splits, split = gsp % pl.splits;
    const int Cg = a.C / a.G, S = a.S;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int p = lane % P, cl = lane / P, s0 = SPT * p;
    float *sB = sm + L::oB, *sC = sm + L::oC, *sBC = sm + L::oBC;
    float4* pre = reinterpret_cast<float4*>(sm + L::oPre) + w * SB * CW;  // [token][channel]
    float4* ck = reinterpret_cast<float4*>(sm + L::oCk) + tid;            // [run][pass], stride 128
    float4* gA = reinterpret_cast<float4*>(sm + L::oG) + tid;             // g, dA: [2][pass]
    float* red = sm + L::oRed;                                            // [warp][token][2 SP]
    ssm_load_rows<E, SP>(sB, a.B, a.ldb, t0, len, g_ * S, S);
    ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t0, len, g_ * S, S);
    if (pl.nl > 1)
        for (int i = tid; i < CH * 2 * SP; i += SSM_THREADS) sBC[i] = 0.f;
    __syncthreads();

    for (int it = 0; it < pl.nl; ++it) {
        const int cb = (split * pl.nl + it) * L::CB;  // the tile's first channel in the group
        if (cb >= Cg) break;
        const int cw = cb + w * CW;  // the warp's
        auto chan = [&](int j) { return g_ * Cg + min(cw + j, Cg - 1); };  // its j-th channel
        float4 A4[NP];
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            A4[q] = ld4(a.A + int64_t(chan(q * CL + cl)) * S, s0, S);
            // lanes past the group's channels stay zero: they add nothing to dB and dC
            ck[q * SSM_THREADS] = ld4(a.hs + (int64_t(k) * a.C + chan(q * CL + cl)) * S, s0,
                                      cw + q * CL + cl < Cg ? S : 0);
        }
        // the warp's delta, delta u and dY of run b; tokens past the chunk are the identity step
        auto stage = [&](int b, bool grad) {
#pragma unroll
            for (int i = lane; i < SB * CW; i += 32) {
                const int r = b * SB + i / CW, c = chan(i % CW);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < len && cw + i % CW < Cg) {
                    const int64_t t = t0 + r;
                    v.x = ssm_delta(ssm_ld<E>(a.dt, t * a.lddt + c) + (a.bias ? a.bias[c] : 0.f), a.softplus);
                    v.y = v.x * ssm_ld<E>(a.u, t * a.ldu + c);
                    if (grad) {
                        v.z = ssm_ld<E>(a.dy, t * a.C + c);
                        if (a.z) v.z *= ssm_silu(ssm_ld<E>(a.z, t * a.ldz + c));
                    }
                }
                pre[i] = v;
            }
            __syncwarp();
        };
        // forward sweep: the states at every run's start
        for (int b = 0; b + 1 < nsub; ++b) {
            stage(b, false);
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const float4 h4 = ck[(b * NP + q) * SSM_THREADS];
                const f2 Aa = pk2(LOG2E * A4[q].x, LOG2E * A4[q].y), Ab = pk2(LOG2E * A4[q].z, LOG2E * A4[q].w);
                f2 ha = pk2(h4.x, h4.y), hb = pk2(h4.z, h4.w);
#pragma unroll
                for (int i = 0; i < SB; ++i) {
                    const float2 v = *reinterpret_cast<const float2*>(pre + i * CW + q * CL + cl);
                    const f2 d2 = pk2(v.x, v.x), u2 = pk2(v.y, v.y);
                    const f2* Bp = reinterpret_cast<const f2*>(sB + (b * SB + i) * SP + s0);
                    ha = fma2(ex2_2(mul2(Aa, d2)), ha, mul2(Bp[0], u2));
                    hb = fma2(ex2_2(mul2(Ab, d2)), hb, mul2(Bp[1], u2));
                }
                float4 o;
                up2(ha, o.x, o.y);
                up2(hb, o.z, o.w);
                ck[((b + 1) * NP + q) * SSM_THREADS] = o;
            }
            __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            gA[q * SSM_THREADS] = ld4(a.gs + (int64_t(k) * a.C + chan(q * CL + cl)) * S, s0,
                                      cw + q * CL + cl < Cg ? S : 0);
            gA[(NP + q) * SSM_THREADS] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float accD[CW > 32 ? 2 : 1] = {}, accb[CW > 32 ? 2 : 1] = {};
        for (int b = nsub - 1; b >= 0; --b) {
            stage(b, true);
            float bc[SB][2 * SPT];  // dB, dC of the run's tokens, summed over the passes
#pragma unroll
            for (int i = 0; i < SB; ++i)
#pragma unroll
                for (int j = 0; j < 2 * SPT; ++j) bc[i][j] = 0.f;
#pragma unroll 1
            for (int q = 0; q < NP; ++q) {
                const float4 A_ = A4[0], A__ = A4[NP - 1];
                const float4 Aq = q ? A__ : A_;
                const float* av = &Aq.x;
                float h[SB + 1][SPT], dec[SB][SPT];
                {
                    const float4 h4 = ck[(b * NP + q) * SSM_THREADS];
                    h[0][0] = h4.x, h[0][1] = h4.y, h[0][2] = h4.z, h[0][3] = h4.w;
                }
                const float4* pq = pre + q * CL + cl;
#pragma unroll
                for (int i = 0; i < SB; ++i) {
                    const float2 v = *reinterpret_cast<const float2*>(pq + i * CW);
                    const float4 B4 = *reinterpret_cast<const float4*>(sB + (b * SB + i) * SP + s0);
                    const float* bv = &B4.x;
#pragma unroll
                    for (int j = 0; j < SPT; ++j) {
                        dec[i][j] = ex2(av[j] * LOG2E * v.x);
                        h[i + 1][j] = fmaf(dec[i][j], h[i][j], bv[j] * v.y);
                    }
                }
                float4 g4 = gA[q * SSM_THREADS], dA4 = gA[(NP + q) * SSM_THREADS];
                float *g = &g4.x, *dA = &dA4.x;
                float sums[3][SB];
#pragma unroll
                for (int i = SB - 1; i >= 0; --i) {
                    const float4 v = pq[i * CW];
                    const float4 B4 = *reinterpret_cast<const float4*>(sB + (b * SB + i) * SP + s0);
                    const float4 C4 = *reinterpret_cast<const float4*>(sC + (b * SB + i) * SP + s0);
                    const float *bv = &B4.x, *cv = &C4.x;
                    float xB = 0.f, xw = 0.f, xy = 0.f;
#pragma unroll
                    for (int j = 0; j < SPT; ++j) {
                        const float G = fmaf(cv[j], v.z, g[j]);
                        bc[i][j] = fmaf(G, v.y, bc[i][j]);
                        bc[i][SPT + j] = fmaf(h[i + 1][j], v.z, bc[i][SPT + j]);
                        xB = fmaf(G, bv[j], xB);
                        xy = fmaf(cv[j], h[i + 1][j], xy);
                        g[j] = dec[i][j] * G;
                        const float wj = g[j] * h[i][j];
                        xw = fmaf(wj, av[j], xw);
                        dA[j] = fmaf(wj, v.x, dA[j]);
                    }
                    sums[0][i] = xB, sums[1][i] = xw, sums[2][i] = xy;
                }
                gA[q * SSM_THREADS] = g4;
                gA[(NP + q) * SSM_THREADS] = dA4;
                // sums over the channel's lanes
#pragma unroll
                for (int i = 0; i < SB; ++i)
#pragma unroll
                    for (int x = 0; x < 3; ++x)
#pragma unroll
                        for (int o = 1; o < P; o <<= 1)
                            sums[x][i] += __shfl_xor_sync(0xffffffffu, sums[x][i], o);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < SB; ++i)
                    if (p == i % P) {
                        float* o = reinterpret_cast<float*>(pre + i * CW + q * CL + cl);
                        o[1] = sums[0][i];
                        o[2] = sums[1][i];
                        o[3] = sums[2][i];
                    }
            }
            // dB, dC of the run over the warp's channels
#pragma unroll
            for (int i = 0; i < SB; ++i) {
                constexpr int NV = 2 * SPT, n = NV / CL > 1 ? NV / CL : 1;
                reduce_lanes<NV, P>(bc[i], lane);
                // (with more channel lanes than values, several lanes write the same sum)
                const int idx = reduce_index<NV, P>(lane);
#pragma unroll
                for (int j = 0; j < n; ++j) {
                    const int vi = idx + j;  // 0 .. 3: dB, 4 .. 7: dC
                    red[(w * SB + i) * 2 * SP + (vi / SPT) * SP + s0 + vi % SPT] = bc[i][j];
                }
            }
            __syncwarp();
            // the run's du, ddt, dz: lanes are channels again
#pragma unroll
            for (int i = lane, x = 0; i < SB * CW; i += 32, ++x) {
                const int r = b * SB + i / CW, ci = cw + i % CW;
                if (r < len && ci < Cg) {
                    const int c = g_ * Cg + ci;
                    const int64_t t = t0 + r;
                    const float4 v = pre[i];  // delta, sum G B, sum A w, sum C h
                    const float u = ssm_ld<E>(a.u, t * a.ldu + c), raw = ssm_ld<E>(a.dt, t * a.lddt + c) + (a.bias ? a.bias[c] : 0.f);
                    const float skip = a.D ? a.D[c] : 0.f;
                    float dY = ssm_ld<E>(a.dy, t * a.C + c);
                    if (a.z) {
                        const float z = ssm_ld<E>(a.z, t * a.ldz + c), sg = ssm_sigmoid(z);
                        ssm_st<E>(a.dz, t * a.C + c, dY * fmaf(skip, u, v.w) * sg * fmaf(z, 1.f - sg, 1.f));
                        dY *= ssm_silu(z);
                    }
                    ssm_st<E>(a.du, t * a.C + c, fmaf(v.x, v.y, skip * dY));
                    float dd = fmaf(u, v.y, v.z);
                    if (a.softplus) dd *= ssm_sigmoid(raw);
                    ssm_st<E>(a.ddt, t * a.C + c, dd);
                    accD[CW > 32 ? x & 1 : 0] += dY * u;
                    accb[CW > 32 ? x & 1 : 0] += dd;
                }
            }
            __syncthreads();  // every warp's sums are written
            for (int i = tid; i < SB * 2 * SP; i += SSM_THREADS) {
                float s = red[i];
#pragma unroll
                for (int j = 1; j < NW; ++j) s += red[j * SB * 2 * SP + i];
                const int r = b * SB + i / (2 * SP), v = i % (2 * SP), x = v / SP, st = v % SP;
                if (pl.nl > 1) sBC[r * 2 * SP + v] += s;
                else if (r < len && st < S) a.pBC[(int64_t(gsp) * a.T + t0 + r) * 2 * S + x * S + st] = s;
            }
            __syncthreads();  // read before the next run's are written
        }
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const int ci = cw + q * CL + cl;
            if (ci < Cg) {
                const int c = g_ * Cg + ci;
                st4(a.pA + (int64_t(k) * a.C + c) * (S + 2), s0, S, gA[(NP + q) * SSM_THREADS]);
                if (a.dh0 && tab.w == 0) st4(a.dh0 + (int64_t(tab.x) * a.C + c) * S, s0, S, gA[q * SSM_THREADS]);
            }
        }
        // lanes that share a channel hold its tokens' terms of dD and dbias
#pragma unroll
        for (int x = 0; x < (CW > 32 ? 2 : 1); ++x) {
#pragma unroll
            for (int o = CW; o < 32; o <<= 1) {
                accD[x] += __shfl_xor_sync(0xffffffffu, accD[x], o);
                accb[x] += __shfl_xor_sync(0xffffffffu, accb[x], o);
            }
            const int j = lane % CW + 32 * x, ci = cw + j;
            if (ci < Cg && lane < CW) {
                float* o = a.pA + (int64_t(k) * a.C + g_ * Cg + ci) * (S + 2) + S;
                o[0] = accD[x];
                o[1] = accb[x];
            }
        }
    }
    if (pl.nl > 1)
        for (int i = tid; i < len * 2 * S; i += SSM_THREADS) {
            const int r = i / (2 * S), v = i % (2 * S);
            a.pBC[(int64_t(gsp) * a.T + t0) * 2 * S + i] = sBC[r * 2 * SP + v / S * SP + v % S];
        }
}

// dB, dC: the channel blocks' sums in order, in runs of SSM_QUAD tiles whatever a block covered
// (so that a document's gradients do not depend on the rest of its pack)
template <class E>
__global__ void k_ssm_reduce_bc(SsmArgs a, SsmBwdPlan pl) {
    if (*a.status != KDA_OK) return;
    const int64_t n = a.T * a.G * 2 * a.S;
    const int per = pl.nl > 1 ? 1 : SSM_QUAD;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int v = int(i % (2 * a.S));
        const int64_t tg = i / (2 * a.S);
        const int g = int(tg % a.G);
        const int64_t t = tg / a.G;
        float sum = 0.f;
        for (int q = 0; q < pl.splits; q += per) {
            float part = 0.f;
            for (int j = q; j < min(q + per, pl.splits); ++j)
                part += a.pBC[((int64_t(g) * pl.splits + j) * a.T + t) * 2 * a.S + v];
            sum += part;
        }
        const int64_t o = (t * a.G + g) * a.S + v % a.S;
        ssm_st<E>(v < a.S ? a.dB : a.dC, o, sum);
    }
}

// dA, dD, dbias: the chunks' sums in order
__global__ void k_ssm_reduce_par(SsmArgs a) {
    if (*a.status != KDA_OK) return;
    const int W = a.S + 2;
    const int64_t n = int64_t(a.C) * W, i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int nc = *a.nchunks;
    float sum = 0.f;
#pragma unroll 8
    for (int k = 0; k < nc; ++k) sum += a.pA[k * n + i];
    const int c = int(i / W), s = int(i % W);
    if (s < a.S) a.dA[int64_t(c) * a.S + s] = sum;
    else if (s == a.S) { if (a.dD) a.dD[c] = sum; }
    else if (a.dbias) a.dbias[c] = sum;
}

template <class E, int SPTR, int P>
void launch_rstate(const SsmArgs& a, cudaStream_t st) {
    const int Cg = a.C / a.G, CB = SSM_THREADS / P, tiles = a.G * ((Cg + CB - 1) / CB);
    if (a.T > CH) {
        ProfScope ps(KK_SSM_RSTATE, st);
        k_ssm_rstate<E, SPTR, P><<<unsigned(a.maxC * tiles), SSM_THREADS, 0, st>>>(a, tiles);
    }
    ProfScope ps(KK_SSM_RCARRY, st);
    const int64_t CS = int64_t(a.C) * a.S;
    const int bpd = int((CS + CARRY_THREADS - 1) / CARRY_THREADS);
    k_ssm_rcarry<<<unsigned(int64_t(bpd) * a.N), CARRY_THREADS, 0, st>>>(a, bpd);
}

template <class E, int P>
void launch_main(const SsmArgs& a, const SsmBwdPlan& pl, cudaStream_t st) {
    const unsigned grid = unsigned(a.maxC * a.G * pl.splits);
    if (grid) {
        ProfScope ps(KK_SSM_BWD, st);
        k_ssm_bwd<E, P><<<grid, SSM_THREADS, BwdShape<P>::floats * 4, st>>>(a, pl);
    }
    {
        ProfScope ps(KK_SSM_REDUCE, st);
        const int64_t n = a.T * a.G * 2 * a.S, blocks = (n + 255) / 256;
        if (blocks) k_ssm_reduce_bc<E><<<unsigned(blocks < 8192 ? blocks : 8192), 256, 0, st>>>(a, pl);
    }
    {
        ProfScope ps(KK_SSM_REDUCE, st);
        const int64_t n = int64_t(a.C) * (a.S + 2);
        k_ssm_reduce_par<<<unsigned((n + 127) / 128), 128, 0, st>>>(a);
    }
}

template <class E>
void launch_e(const SsmArgs& a, cudaStream_t st) {
    if (a.S <= 8) launch_rstate<E, 8, 1>(a, st);
    else if (a.S <= 16) launch_rstate<E, 16, 1>(a, st);
    else if (a.S <= 32) launch_rstate<E, 16, 2>(a, st);
    else launch_rstate<E, 16, 4>(a, st);
    const SsmBwdPlan pl = ssm_bwd_plan(a.maxC, a.C, a.S, a.G);
    switch (pl.lanes) {
        case 1: return launch_main<E, 1>(a, pl, st);
        case 2: return launch_main<E, 2>(a, pl, st);
        case 4: return launch_main<E, 4>(a, pl, st);
        case 8: return launch_main<E, 8>(a, pl, st);
        default: return launch_main<E, 16>(a, pl, st);
    }
}

template <class E>
cudaError_t setup_e() {
    const void* f[] = {(const void*)k_ssm_bwd<E, 1>, (const void*)k_ssm_bwd<E, 2>, (const void*)k_ssm_bwd<E, 4>,
                       (const void*)k_ssm_bwd<E, 8>, (const void*)k_ssm_bwd<E, 16>};
    const int n[] = {BwdShape<1>::floats, BwdShape<2>::floats, BwdShape<4>::floats, BwdShape<8>::floats,
                     BwdShape<16>::floats};
    for (int i = 0; i < 5; ++i)
        if (cudaError_t e = cudaFuncSetAttribute(f[i], cudaFuncAttributeMaxDynamicSharedMemorySize, n[i] * 4)) return e;
    return cudaSuccess;
}

}  // namespace

SsmBwdPlan ssm_bwd_plan(int64_t maxC, int C, int S, int G) {
    SsmBwdPlan pl{};
    pl.lanes = S <= 4 ? 1 : S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16;
    const int CB = NW * NP * (32 / pl.lanes), Cg = C / G;
    pl.tiles = (Cg + CB - 1) / CB;
    // four tiles per block keep the partial sums of dB and dC small; with fewer blocks than the
    // machine holds at once, one tile per block spreads the work
    const int64_t quads = (pl.tiles + SSM_QUAD - 1) / SSM_QUAD;
    pl.nl = maxC * G * quads >= 456 ? SSM_QUAD : 1;
    pl.splits = (pl.tiles + pl.nl - 1) / pl.nl;
    return pl;
}

cudaError_t ssm_bwd_setup() {
    if (cudaError_t e = setup_e<__nv_bfloat16>()) return e;
    if (cudaError_t e = setup_e<__half>()) return e;
    return setup_e<float>();
}

void launch_ssm_bwd(const SsmArgs& a, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) launch_e<__nv_bfloat16>(a, st);
    else if (dtype == KDA_DT_FP16) launch_e<__half>(a, st);
    else launch_e<float>(a, st);
}

}  // namespace kda
