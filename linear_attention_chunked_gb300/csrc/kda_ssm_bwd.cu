// Selective state-space scan, backward.  With dY = dy silu(z) and G_t the gradient of h_t
// (G_t = C_t dY_t + a_{t+1} G_{t+1}, from dht at a document's last token):
//   dC_t[s] = sum_c dY h_t        dB_t[s] = sum_c G delta u       (sums over the group's channels)
//   sB = sum_s G B, w = a G h_{t-1}:  du = delta sB + D dY,  ddelta = u sB + sum_s A w
//   dA = sum_t delta w,  dD = sum_t dY u,  ddt = ddelta softplus'(dt + bias),  dbias = sum_t ddt
//   dz = dy y0 silu'(z),  y0 = sum_s C h + D u,  dh0 = a_1 G_1
//
//   k_ssm_rstate   per chunk with a predecessor: its start gradient from a zero end (kda_ssm_fwd.cu)
//   k_ssm_rcarry   per (document, channel, state): the chunks' end gradients, last to first
//   k_ssm_bwd      per (chunk, channel tile): the gradients
//   k_ssm_reduce_* the sums over channel tiles (dB, dC) and over chunks (dA, dD, dbias), in order
//
// k_ssm_bwd needs h_{t-1} in reverse.  The forward leaves the state at every 16th token; a unit of 16
// tokens is swept forward once from there, the states every 4 tokens kept in shared memory, and
// each run of 4 tokens is recomputed from its start with states and decays in registers and walked
// backwards.  Four lanes hold a channel's 16 states (four each), a warp 16 channels in two passes.
// The channels' scalars (delta, delta u, dY, u and what the gradients are multiplied with at the end) are
// computed once per token by lanes laid out as (token, channel) items and handed over through shared
// memory, one unit ahead of their use.  Sums cross lanes by halving (each step a lane gives away half
// of its values): a channel's three sums over states for 4 tokens leave each of its four lanes with one
// token, whose du, ddt and dz that lane finishes; the eight dB / dC terms per token, summed over the two
// passes in registers first, take 7 shuffles over 8 lanes.
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

#ifndef BB
#define BB (P <= 4 ? 3 : 2)
#endif
constexpr int RT = 4;           // tokens per run
constexpr int UT = SSM_UT;      // tokens per unit
constexpr int NR = UT / RT;     // runs per unit
constexpr int NP = 2;           // channel passes per warp
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

// Sums of a run's three values per token over the P lanes of a channel, halving over the tokens: on return
// a lane holds its tokens' sums in v[.][0 .. NT-1], the first of them token first_token(p).
template <int P> __device__ constexpr int lane_tokens() { return P == 1 ? 4 : P == 2 ? 2 : 1; }
template <int P> __device__ __forceinline__ int first_token(int p) {
    return (P > 1 && (p & 1) ? 2 : 0) + (P > 2 && (p & 2) ? 1 : 0);
}
template <int P>
__device__ __forceinline__ void reduce_tokens(float (&v)[3][RT], int p) {
    static_assert(RT == 4, "two halvings");
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (P > 1)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float give = p & 1 ? v[x][i] : v[x][i + 2], keep = p & 1 ? v[x][i + 2] : v[x][i];
                v[x][i] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
            }
        if (P > 2) {
            const float give = p & 2 ? v[x][0] : v[x][1], keep = p & 2 ? v[x][1] : v[x][0];
            v[x][0] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
        }
#pragma unroll
        for (int o = 4; o < P; o <<= 1) v[x][0] += __shfl_xor_sync(0xffffffffu, v[x][0], o);
    }
}

template <int P>
struct BwdShape {
    static constexpr int CL = 32 / P;       // channels of a pass
    static constexpr int CW = NP * CL;      // channels of a warp
    static constexpr int CB = NW * CW;      // channels of a tile
    static constexpr int SP = SPT * P;      // state slots
    static constexpr int NI = RT * CW > 32 ? RT * CW / 32 : 1;  // (token, channel) items of a run per lane
    // shared memory, in floats
    static constexpr int oB = 0, oC = oB + CH * SP, oPre = oC + CH * SP;
    static constexpr int oFin = oPre + NW * UT * CW * 4;
    static constexpr int oCk = oFin + NW * UT * CW * 2;
    static constexpr int oRed = oCk + (NR - 1) * NP * SSM_THREADS * 4;
    static constexpr int oBC = oRed + 2 * NW * RT * 2 * SP;
    static constexpr int floats = oBC + CH * 2 * SP;
};

template <class E, int P>
__global__ void __launch_bounds__(SSM_THREADS, BB) k_ssm_bwd(SsmArgs a, SsmBwdPlan pl) {
    using L = BwdShape<P>;
    constexpr int CL = L::CL, CW = L::CW, SP = L::SP, NI = L::NI, NB = CW > 32 ? 2 : 1, LT = lane_tokens<P>();
    extern __shared__ __align__(16) float sm[];
    const int per_chunk = a.G * pl.splits;
    const int k = blockIdx.x / per_chunk;
    if (k >= *a.nchunks) return;
    const int4 tab = a.chunk_tab[k];
    const int t0 = tab.y, len = tab.z;
    const int gsp = blockIdx.x % per_chunk, g_ = gsp / pl.splits, split = gsp % pl.splits;
    const int Cg = a.C / a.G, S = a.S;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int p = lane % P, cl = lane / P, s0 = SPT * p;
    float *sB = sm + L::oB, *sC = sm + L::oC;
    // a unit's scalars; a run's give way to the next unit's as soon as it is done
    float4* pre = reinterpret_cast<float4*>(sm + L::oPre) + w * UT * CW;  // [token][channel]: delta, delta u, dY, u
    float2* fin = reinterpret_cast<float2*>(sm + L::oFin) + w * UT * CW;  // d delta / d dt, dz / y0
    ulonglong2* ck = reinterpret_cast<ulonglong2*>(sm + L::oCk) + tid;    // [run][pass], stride 128
    float *red = sm + L::oRed, *sBC = sm + L::oBC;                        // [parity][warp][token][2 SP]; [token][2 SP]
    ssm_load_rows<E, SP>(sB, a.B, a.ldb, t0, len, g_ * S, S);
    ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t0, len, g_ * S, S);
    __syncthreads();
    const int nu = (len + UT - 1) / UT;  // units
    const bool gated = a.z;
    int par = 0;

    for (int it = 0; it < pl.nl; ++it) {
        const int cb = (split * pl.nl + it) * L::CB;  // the tile's first channel in the group
        if (cb >= Cg) break;
        const int cw = cb + w * CW;                                         // the warp's
        auto chan = [&](int j) { return g_ * Cg + min(cw + j, Cg - 1); };  // its j-th channel
        // lanes as states: pass q's channel.  Lanes past the group's channels stay zero: they add
        // nothing to dB and dC
        f2 A2[NP][2], g[NP][2], dA[NP][2], hs[NP][2];
        float skip[NP], accD[NP] = {}, accb[NP] = {};
        auto lim = [&](int q) { return cw + q * CL + cl < Cg ? S : 0; };
        auto pair2 = [](float4 v, f2(&o)[2]) { o[0] = pk2(v.x, v.y), o[1] = pk2(v.z, v.w); };
        auto start = [&](int u, int q) {  // the state at unit u's start
            return ld4(a.hs + ((int64_t(k) * SSM_SUB + u) * a.C + chan(q * CL + cl)) * S, s0, lim(q));
        };
        float4 nh[NP];
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const int64_t row = int64_t(chan(q * CL + cl)) * S;
            float4 v = ld4(a.A + row, s0, S);
            v.x *= LOG2E, v.y *= LOG2E, v.z *= LOG2E, v.w *= LOG2E;
            pair2(v, A2[q]);
            pair2(ld4(a.gs + int64_t(k) * a.C * S + row, s0, lim(q)), g[q]);
            dA[q][0] = dA[q][1] = 0;
            nh[q] = start(nu - 1, q);
            skip[q] = a.D ? a.D[chan(q * CL + cl)] : 0.f;
        }
        // lanes as (token, channel) items of a run: item x is token (lane + 32 x) / CW of the run and
        // channel (lane + 32 x) % CW of the warp
        float bias[NB];
#pragma unroll
        for (int x = 0; x < NB; ++x) bias[x] = a.bias ? a.bias[chan(lane % CW + 32 * x)] : 0.f;
        struct Raw { E dt, u, dy, z; };
        auto at = [&](const void* base, int64_t ld, int row, int c) {
            return static_cast<const E*>(base)[(int64_t(t0) + row) * ld + c];
        };
        auto fetch = [&](Raw(&r)[NI], int row0) {
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                const int i = lane + 32 * x, c = chan(i % CW), row = min(row0 + i / CW, len - 1);
                r[x].dt = at(a.dt, a.lddt, row, c);
                r[x].u = at(a.u, a.ldu, row, c);
                r[x].dy = at(a.dy, a.C, row, c);
                if (gated) r[x].z = at(a.z, a.ldz, row, c);
            }
        };
        // the scalars of a run into a unit's buffer; tokens past the chunk are the identity step
        auto stage = [&](const Raw(&r)[NI], int u, int run) {
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                const int i = lane + 32 * x;
                if (RT * CW < 32 && i >= RT * CW) break;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                float2 f = make_float2(0.f, 0.f);
                if (u * UT + run * RT + i / CW < len && cw + i % CW < Cg) {
                    const float raw = __fadd_rn(ssm_f<E>(r[x].dt), bias[x % NB]);
                    v.x = ssm_delta(raw, a.softplus);
                    v.w = ssm_f<E>(r[x].u);
                    v.y = __fmul_rn(v.x, v.w);
                    v.z = ssm_f<E>(r[x].dy);
                    f.x = a.softplus ? ssm_sigmoid(raw) : 1.f;
                    if (gated) {
                        const float z = ssm_f<E>(r[x].z), sg = z < -87.f ? 0.f : ssm_sigmoid(z), zs = z * sg;
                        f.y = v.z * fmaf(zs, 1.f - sg, sg);  // silu'(z) = sg + z sg (1 - sg)
                        v.z = __fmul_rn(v.z, zs);
                    }
                }
                pre[run * RT * CW + i] = v;
                fin[run * RT * CW + i] = f;
            }
        };
        Raw nxt[NI];
#pragma unroll 1
        for (int r = 0; r < NR; ++r) {
            fetch(nxt, (nu - 1) * UT + r * RT);
            stage(nxt, nu - 1, r);
        }
#pragma unroll 1
        for (int u = nu - 1; u >= 0; --u) {
            const float4* pu = pre + cl;
            const float2* fu = fin + cl;
            const int nr = (min(UT, len - u * UT) + RT - 1) / RT;  // runs of the unit
            __syncwarp();
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                pair2(nh[q], hs[q]);
                if (u > 0) nh[q] = start(u - 1, q);
            }
            // forward sweep: the states at every run's start
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                f2 ha = hs[q][0], hb = hs[q][1];
#pragma unroll 1
                for (int r = 0; r + 1 < nr; ++r) {
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float2 v = *reinterpret_cast<const float2*>(pu + (r * RT + i) * CW + q * CL);
                        const f2 d2 = pk2(v.x, v.x), u2 = pk2(v.y, v.y);
                        const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(sB + (u * UT + r * RT + i) * SP + s0);
                        ha = fma2(ex2_2(mul2(A2[q][0], d2)), ha, mul2(b2.x, u2));
                        hb = fma2(ex2_2(mul2(A2[q][1], d2)), hb, mul2(b2.y, u2));
                    }
                    ck[(r * NP + q) * SSM_THREADS] = make_ulonglong2(ha, hb);
                }
            }
            // runs the unit lacks (its chunk ends inside it) still stage the next unit's tokens
#pragma unroll 1
            for (int r = nr; u > 0 && r < NR; ++r) {
                fetch(nxt, (u - 1) * UT + r * RT);
                stage(nxt, u - 1, r);
            }
#pragma unroll 1
            for (int r = nr - 1; r >= 0; --r) {
                const int row0 = u * UT + r * RT;
                if (u > 0) fetch(nxt, row0 - UT);
                f2 bc[RT][4];  // dB, dC of the run's tokens, summed over the passes
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) bc[i][j] = 0;
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    f2 h[RT + 1][2], dec[RT][2];
                    h[0][0] = hs[q][0], h[0][1] = hs[q][1];
                    if (r > 0) {
                        const ulonglong2 v = ck[((r - 1) * NP + q) * SSM_THREADS];
                        h[0][0] = v.x, h[0][1] = v.y;
                    }
                    const float4* pq = pu + r * RT * CW + q * CL;
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
                        const float2 v = *reinterpret_cast<const float2*>(pq + i * CW);
                        const f2 d2 = pk2(v.x, v.x), u2 = pk2(v.y, v.y);
                        const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(sB + (row0 + i) * SP + s0);
                        dec[i][0] = ex2_2(mul2(A2[q][0], d2));
                        dec[i][1] = ex2_2(mul2(A2[q][1], d2));
                        h[i + 1][0] = fma2(dec[i][0], h[i][0], mul2(b2.x, u2));
                        h[i + 1][1] = fma2(dec[i][1], h[i][1], mul2(b2.y, u2));
                    }
                    float sums[3][RT];  // over the states: G B, log2(e) A w, C h
#pragma unroll
                    for (int i = RT - 1; i >= 0; --i) {
                        const float4 v = pq[i * CW];
                        const f2 d2 = pk2(v.x, v.x), u2 = pk2(v.y, v.y), y2 = pk2(v.z, v.z);
                        const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(sB + (row0 + i) * SP + s0);
                        const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(sC + (row0 + i) * SP + s0);
                        const f2 G0 = fma2(c2.x, y2, g[q][0]), G1 = fma2(c2.y, y2, g[q][1]);
                        bc[i][0] = fma2(G0, u2, bc[i][0]);
                        bc[i][1] = fma2(G1, u2, bc[i][1]);
                        bc[i][2] = fma2(h[i + 1][0], y2, bc[i][2]);
                        bc[i][3] = fma2(h[i + 1][1], y2, bc[i][3]);
                        sums[0][i] = hsum2(fma2(G1, b2.y, mul2(G0, b2.x)));
                        sums[2][i] = hsum2(fma2(h[i + 1][1], c2.y, mul2(h[i + 1][0], c2.x)));
                        g[q][0] = mul2(dec[i][0], G0);
                        g[q][1] = mul2(dec[i][1], G1);
                        const f2 w0 = mul2(g[q][0], h[i][0]), w1 = mul2(g[q][1], h[i][1]);
                        sums[1][i] = hsum2(fma2(w1, A2[q][1], mul2(w0, A2[q][0])));
                        dA[q][0] = fma2(w0, d2, dA[q][0]);
                        dA[q][1] = fma2(w1, d2, dA[q][1]);
                    }
                    reduce_tokens<P>(sums, p);
                    if (P <= 4 || p < 4)
#pragma unroll
                        for (int i = 0; i < LT; ++i) {
                            const int tk = first_token<P>(p) + i, row = row0 + tk, ci = cw + q * CL + cl;
                            if (row < len && ci < Cg) {
                                const int64_t o = (int64_t(t0) + row) * a.C + g_ * Cg + ci;
                                const float4 v = pq[tk * CW];
                                const float2 f = fu[(r * RT + tk) * CW + q * CL];
                                const float dd = fmaf(v.w, sums[0][i], sums[1][i] * 0.6931471805599453f) * f.x;
                                ssm_st<E>(a.du, o, fmaf(v.x, sums[0][i], skip[q] * v.z));
                                ssm_st<E>(a.ddt, o, dd);
                                if (gated) ssm_st<E>(a.dz, o, f.y * fmaf(skip[q], v.w, sums[2][i]));
                                accD[q] = fmaf(v.z, v.w, accD[q]);
                                accb[q] += dd;
                            }
                        }
                }
                // dB, dC of the run over the warp's channels
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    constexpr int NV = 2 * SPT, n = NV / CL > 1 ? NV / CL : 1;
                    float v[NV];
#pragma unroll
                    for (int j = 0; j < 4; ++j) up2(bc[i][j], v[2 * j], v[2 * j + 1]);
                    reduce_lanes<NV, P>(v, lane);
                    // (with more channel lanes than values, several lanes write the same sum)
                    const int idx = reduce_index<NV, P>(lane);
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        const int vi = idx + j;  // 0 .. 3: dB, 4 .. 7: dC
                        red[((par * NW + w) * RT + i) * 2 * SP + (vi / SPT) * SP + s0 + vi % SPT] = v[j];
                    }
                }
                __syncwarp();
                if (u > 0) stage(nxt, u - 1, r);
                // the warps' sums are written; two buffers, so that one barrier a run is enough
                __syncthreads();
                for (int i = tid; i < RT * 2 * SP; i += SSM_THREADS) {
                    const float* rp = red + par * NW * RT * 2 * SP + i;
                    float s = rp[0];
#pragma unroll
                    for (int j = 1; j < NW; ++j) s += rp[j * RT * 2 * SP];
                    float* o = sBC + row0 * 2 * SP + i;  // the same thread adds every tile of the block
                    *o = it ? *o + s : s;
                }
                par ^= 1;
            }
        }
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            // the channel's lanes hold its tokens' terms of dD and dbias
#pragma unroll
            for (int o = 1; o < P; o <<= 1) {
                accD[q] += __shfl_xor_sync(0xffffffffu, accD[q], o);
                accb[q] += __shfl_xor_sync(0xffffffffu, accb[q], o);
            }
            const int ci = cw + q * CL + cl;
            if (ci < Cg) {
                const int c = g_ * Cg + ci;
                float* row = a.pA + (int64_t(k) * a.C + c) * (S + 2);
                float4 v;
                up2(dA[q][0], v.x, v.y);
                up2(dA[q][1], v.z, v.w);
                st4(row, s0, S, v);
                if (p == 0) row[S] = accD[q], row[S + 1] = accb[q];
                up2(g[q][0], v.x, v.y);
                up2(g[q][1], v.z, v.w);
                if (a.dh0 && tab.w == 0) st4(a.dh0 + (int64_t(tab.x) * a.C + c) * S, s0, S, v);
            }
        }
        __syncwarp();
    }
    __syncthreads();
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
    launch_ssm_rstate(a, dtype, st);
    {
        ProfScope ps(KK_SSM_RCARRY, st);
        const int64_t CS = int64_t(a.C) * a.S;
        const int bpd = int((CS + CARRY_THREADS - 1) / CARRY_THREADS);
        k_ssm_rcarry<<<unsigned(int64_t(bpd) * a.N), CARRY_THREADS, 0, st>>>(a, bpd);
    }
    if (dtype == KDA_DT_BF16) launch_e<__nv_bfloat16>(a, st);
    else if (dtype == KDA_DT_FP16) launch_e<__half>(a, st);
    else launch_e<float>(a, st);
}

}  // namespace kda
