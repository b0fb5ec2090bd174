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
//   k_ssm_reduce   the sums over channel tiles (dB, dC) and over chunks (dA, dD, dbias), in a fixed order
//
// k_ssm_bwd needs h_{t-1} in reverse.  The forward leaves the state at every 16th token; a unit of 16
// tokens is swept forward once from there, the states every 4 tokens kept in shared memory, and
// each run of 4 tokens is recomputed from its start with states and decays in registers and walked
// backwards.  Four lanes hold a channel's 16 states (four each), and a lane holds two channels, as the two
// halves of packed arithmetic: the channels' scalars are pairs as they lie, and B and C are read once for
// both.  The scalars (delta, delta u, dY, u and what the gradients are multiplied with at the end) are
// computed once per token by lanes laid out as (token, channel pair) items and handed over through
// shared memory, one unit ahead of their use.  Sums cross lanes by halving (each step a lane gives away
// half of its values): a channel's three sums over states for 4 tokens leave each of its four lanes with
// one token, whose du, ddt and dz that lane finishes; the eight dB / dC terms per token, summed over the
// two channels first, take 7 shuffles over 8 lanes.
//
// Bound by instruction issue and shared-memory operands together (16384 x 2048 x 16: 768 us, about 29
// instructions per channel, state and token, half of the issue slots, 12 warps per multiprocessor by
// registers).  Measured and worse: B and C doubled in shared memory, which saves the copies into
// pairs (+51 us: the operand reads double); their products as two scalar instructions (+24 us); four
// blocks per multiprocessor (spills, +380 us); two channel tiles a block (+20 us with the larger reduction).
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

constexpr int RT = 4;           // tokens per run
constexpr int UT = SSM_UT;      // tokens per unit
constexpr int NR = UT / RT;     // runs per unit
constexpr int NW = SSM_THREADS / 32;
constexpr int SPT = 4;          // states per lane

// four states from s of a row of S (those past S: zero, unwritten); vec: rows are whole vectors
__device__ __forceinline__ float4 ld4(const float* p, int s, int S, bool vec) {
    if (vec) return s < S ? *reinterpret_cast<const float4*>(p + s) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(s < S ? p[s] : 0.f, s + 1 < S ? p[s + 1] : 0.f, s + 2 < S ? p[s + 2] : 0.f,
                       s + 3 < S ? p[s + 3] : 0.f);
}
__device__ __forceinline__ void st4(float* p, int s, int S, float4 v) {
    if (s < S) p[s] = v.x;
    if (s + 1 < S) p[s + 1] = v.y;
    if (s + 2 < S) p[s + 2] = v.z;
    if (s + 3 < S) p[s + 3] = v.w;
}

// A decay rate of -inf as the lowest finite one: the decay is 0 either way (from steps of 4e-37 on), and the
// steps of 0 that stand for tokens past the chunk and for lanes past the group's channels keep their decay
// of 1, where 0 times infinity would reach dB and dC of every channel.  (NaN stays.)
__device__ __forceinline__ f2 above_inf2(f2 v) {
    constexpr float low = -3.402823466e38f;
    float x, y;
    up2(v, x, y);
    return pk2(x < low ? low : x, y < low ? low : y);
}

constexpr int CARRY_THREADS = 128;
__global__ void __launch_bounds__(CARRY_THREADS) k_ssm_rcarry(SsmArgs a, int blocks_per_doc) {
    const bool ok = ssm_plan_ok(a);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.call_status = ok ? KDA_OK : KDA_ERR_DEVICE_CHECK;  // (the plan may be a saved one)
    if (!ok) return;
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
    constexpr int U = 16;
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
// a lane holds its tokens' sums in v[.][0 .. lane_tokens - 1], the first of them token first_token(p).
template <int P> __device__ constexpr int lane_tokens() { return P == 1 ? 4 : P == 2 ? 2 : 1; }
template <int P> __device__ __forceinline__ int first_token(int p) {
    return (P > 1 && (p & 1) ? 2 : 0) + (P > 2 && (p & 2) ? 1 : 0);
}
template <int P>
__device__ __forceinline__ void reduce_tokens(f2 (&v)[3][RT], int p) {
    static_assert(RT == 4, "two halvings");
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        if (P > 1)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f2 give = p & 1 ? v[x][i] : v[x][i + 2], keep = p & 1 ? v[x][i + 2] : v[x][i];
                v[x][i] = add2(keep, __shfl_xor_sync(0xffffffffu, give, 1));
            }
        if (P > 2) {
            const f2 give = p & 2 ? v[x][0] : v[x][1], keep = p & 2 ? v[x][1] : v[x][0];
            v[x][0] = add2(keep, __shfl_xor_sync(0xffffffffu, give, 2));
        }
#pragma unroll
        for (int o = 4; o < P; o <<= 1) v[x][0] = add2(v[x][0], __shfl_xor_sync(0xffffffffu, v[x][0], o));
    }
}

template <int P>
struct BwdShape {
    static constexpr int CL = 32 / P;       // channel pairs of a warp: channels i and i + CL
    static constexpr int CB = NW * 2 * CL;  // channels of a tile
    static constexpr int SP = SPT * P;      // state slots
    static constexpr int NI = RT * CL > 32 ? RT * CL / 32 : 1;  // (token, channel pair) items of a run per lane
    // shared memory, in floats: B and C rows; three vectors of scalars per item; states at the
    // runs' starts; the warps' dB, dC; the chunk's
    static constexpr int oB = 0, oC = oB + CH * SP, oPre = oC + CH * SP;
    static constexpr int oCk = oPre + 3 * NW * UT * CL * 4;
    static constexpr int oRed = oCk + (NR - 1) * 2 * SSM_THREADS * 4;
    static constexpr int oBC = oRed + 2 * NW * RT * 2 * SP;
    static constexpr int floats = oBC + CH * 2 * SP;
};

template <class E, int P>
__global__ void __launch_bounds__(SSM_THREADS, P == 1 ? 2 : P <= 4 ? 3 : 1) k_ssm_bwd(SsmArgs a, SsmBwdPlan pl) {
    using L = BwdShape<P>;
    constexpr int CL = L::CL, SP = L::SP, NI = L::NI, LT = lane_tokens<P>();
    extern __shared__ __align__(16) float sm[];
    const int per_chunk = a.G * pl.splits;
    const int k = blockIdx.x / per_chunk;
    if (!ssm_plan_ok(a) || k >= *a.nchunks) return;
    const int4 tab = a.chunk_tab[k];
    const int t0 = tab.y, len = tab.z;
    const int gsp = blockIdx.x % per_chunk, g_ = gsp / pl.splits, split = gsp % pl.splits;
    const int Cg = a.C / a.G, S = a.S;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int p = lane % P, cl = lane / P, s0 = SPT * p;
    float *sB = sm + L::oB, *sC = sm + L::oC;
    auto four = [&](const float* rows, int row, f2(&o)[SPT]) {  // the lane's states of a row, doubled
        const float4 v = *reinterpret_cast<const float4*>(rows + row * SP + s0);
        o[0] = pk2(v.x, v.x), o[1] = pk2(v.y, v.y), o[2] = pk2(v.z, v.z), o[3] = pk2(v.w, v.w);
    };
    // a unit's scalars [token][pair]; a run's give way to the next unit's as soon as it is done
    ulonglong2* pX = reinterpret_cast<ulonglong2*>(sm + L::oPre) + w * UT * CL;  // delta, delta u
    ulonglong2* pY = pX + NW * UT * CL;                                          // dY, u
    ulonglong2* pF = pY + NW * UT * CL;                                          // d delta / d dt, dz / y0
    ulonglong2* ck = reinterpret_cast<ulonglong2*>(sm + L::oCk) + tid;           // [run][2], stride 128
    float *red = sm + L::oRed, *sBC = sm + L::oBC;                               // [parity][warp][token][2 SP]; [token][2 SP]
    ssm_load_rows<E, SP>(sB, a.B, a.ldb, t0, len, g_ * S, S);
    ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t0, len, g_ * S, S);
    __syncthreads();
    const int nu = (len + UT - 1) / UT;  // units
    const bool gated = a.z;
    int par = 0;

    for (int it = 0; it < pl.nl; ++it) {
        const int cb = (split * pl.nl + it) * L::CB;  // the tile's first channel in the group
        if (cb >= Cg) break;
        const int cw = cb + w * 2 * CL;                                    // the warp's
        auto chan = [&](int j) { return g_ * Cg + min(cw + j, Cg - 1); };  // its j-th channel
        // lanes as states: channels cl and cl + CL.  Lanes past the group's channels stay zero: they add
        // nothing to dB and dC
        const int c0 = chan(cl), c1 = chan(cl + CL);
        const bool on0 = cw + cl < Cg, on1 = cw + cl + CL < Cg;
        f2 A2[SPT], g[SPT], dA[SPT], hs[SPT];
        auto both4 = [&](const float* base, bool mask, float4(&o)[2]) {
            o[0] = ld4(base + int64_t(c0) * S, s0, !mask || on0 ? S : 0, S % 4 == 0);
            o[1] = ld4(base + int64_t(c1) * S, s0, !mask || on1 ? S : 0, S % 4 == 0);
        };
        auto paired = [](const float4(&v)[2], f2(&o)[SPT]) {
            o[0] = pk2(v[0].x, v[1].x), o[1] = pk2(v[0].y, v[1].y), o[2] = pk2(v[0].z, v[1].z), o[3] = pk2(v[0].w, v[1].w);
        };
        float4 nh[2];                  // the next unit's states, paired where they are used (pairing waits for them)
        auto start = [&](int u) {  // the states at unit u's start
            both4(a.hs + (int64_t(k) * SSM_SUB + u) * a.C * S, true, nh);
        };
        {
            float4 va[2], vg[2];
            both4(a.A, false, va);
            both4(a.gs + int64_t(k) * a.C * S, true, vg);
            start(nu - 1);
            paired(va, A2);
            paired(vg, g);
        }
#pragma unroll
        for (int j = 0; j < SPT; ++j) A2[j] = above_inf2(mul2(A2[j], pk2(LOG2E, LOG2E))), dA[j] = 0;
        const f2 skip = a.D ? pk2(a.D[c0], a.D[c1]) : 0;
        f2 accD = 0, accb = 0;
        // lanes as items: item x of a run is token (lane + 32 x) / CL, channels lane % CL and lane % CL + CL
        const int ic = lane % CL, i0 = chan(ic), i1 = chan(ic + CL);
        const f2 bias = a.bias ? pk2(a.bias[i0], a.bias[i1]) : 0;
        const bool ion0 = cw + ic < Cg, ion1 = cw + ic + CL < Cg;
        struct Raw { E dt[2], u[2], dy[2], z[2]; };
        auto fetch = [&](Raw(&r)[NI], int row0) {
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                const int64_t t = t0 + min(row0 + (lane + 32 * x) / CL, len - 1);
                auto two = [&](E(&o)[2], const void* base, int64_t ld) {
                    const E* q = static_cast<const E*>(base) + t * ld;
                    o[0] = q[i0], o[1] = q[i1];
                };
                two(r[x].dt, a.dt, a.lddt);
                two(r[x].u, a.u, a.ldu);
                two(r[x].dy, a.dy, a.C);
                if (gated) two(r[x].z, a.z, a.ldz);
            }
        };
        auto wide = [](const E(&v)[2]) { return pk2(ssm_f<E>(v[0]), ssm_f<E>(v[1])); };
        // the scalars of a run; tokens past the chunk are the identity step
        auto stage = [&](const Raw(&r)[NI], int u, int run) {
#pragma unroll
            for (int x = 0; x < NI; ++x) {
                const int i = lane + 32 * x;
                if (RT * CL < 32 && i >= RT * CL) break;
                const bool in = u * UT + run * RT + i / CL < len;
                const f2 raw = add2(wide(r[x].dt), bias), dl = ssm_delta2(raw, a.softplus);
                f2 uu = wide(r[x].u), dY = wide(r[x].dy), sg = pk2(1.f, 1.f), F = 0;
                if (a.softplus) sg = ssm_sigmoid2(raw);
                if (gated) {
                    const f2 z = wide(r[x].z), q = ssm_gate2(z), zs = mul2(z, q);
                    // silu'(z) = q + z q (1 - q)
                    F = mul2(dY, fma2(zs, fma2(q, pk2(-1.f, -1.f), pk2(1.f, 1.f)), q));
                    dY = mul2(dY, zs);
                }
                auto only = [&](f2 v) {
                    float y0, y1;
                    up2(v, y0, y1);
                    return pk2(in && ion0 ? y0 : 0.f, in && ion1 ? y1 : 0.f);
                };
                const int o = run * RT * CL + i;
                if (in && ion0 && ion1) {
                    pX[o] = make_ulonglong2(dl, mul2(dl, uu));
                    pY[o] = make_ulonglong2(dY, uu);
                    pF[o] = make_ulonglong2(sg, F);
                } else {
                    pX[o] = make_ulonglong2(only(dl), only(mul2(dl, uu)));
                    pY[o] = make_ulonglong2(only(dY), only(uu));
                    pF[o] = make_ulonglong2(only(sg), only(F));
                }
            }
        };
        {
            constexpr int NF = NI <= 2 ? NR : 1;  // runs in flight
            Raw first[NF][NI];
#pragma unroll
            for (int r0 = 0; r0 < NR; r0 += NF) {
#pragma unroll
                for (int r = 0; r < NF; ++r) fetch(first[r], (nu - 1) * UT + (r0 + r) * RT);
#pragma unroll
                for (int r = 0; r < NF; ++r) stage(first[r], nu - 1, r0 + r);
            }
        }
        Raw nxt[NI];
#pragma unroll 1
        for (int u = nu - 1; u >= 0; --u) {
            const int nr = (min(UT, len - u * UT) + RT - 1) / RT;  // runs of the unit
            __syncwarp();
            paired(nh, hs);
            if (u > 0) start(u - 1);
            // one token forward: decays and states
            auto ahead = [&](int i, int row, const f2(&h)[SPT], f2(&dec)[SPT], f2(&o)[SPT]) {
                const ulonglong2 v = pX[i * CL + cl];
                f2 b[SPT];
                four(sB, row, b);
#pragma unroll
                for (int j = 0; j < SPT; ++j) {
                    dec[j] = ex2_2(mul2(A2[j], v.x));
                    o[j] = fma2(dec[j], h[j], mul2(b[j], v.y));
                }
            };
            // forward sweep: the states at every run's start
            {
                f2 h[SPT], d[SPT];
#pragma unroll
                for (int j = 0; j < SPT; ++j) h[j] = hs[j];
#pragma unroll 1
                for (int r = 0; r + 1 < nr; ++r) {
#pragma unroll
                    for (int i = 0; i < RT; ++i) ahead(r * RT + i, u * UT + r * RT + i, h, d, h);
                    ck[(2 * r) * SSM_THREADS] = make_ulonglong2(h[0], h[1]);
                    ck[(2 * r + 1) * SSM_THREADS] = make_ulonglong2(h[2], h[3]);
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
                f2 h[RT + 1][SPT], dec[RT][SPT];
                if (r > 0) {
                    const ulonglong2 x = ck[(2 * r - 2) * SSM_THREADS], y = ck[(2 * r - 1) * SSM_THREADS];
                    h[0][0] = x.x, h[0][1] = x.y, h[0][2] = y.x, h[0][3] = y.y;
                } else {
#pragma unroll
                    for (int j = 0; j < SPT; ++j) h[0][j] = hs[j];
                }
#pragma unroll
                for (int i = 0; i < RT; ++i) ahead(r * RT + i, row0 + i, h[i], dec[i], h[i + 1]);
                f2 sums[3][RT];  // over the states: G B, log2(e) A w, C h
#pragma unroll
                for (int i = RT - 1; i >= 0; --i) {
                    const ulonglong2 x = pX[(r * RT + i) * CL + cl];
                    const f2 dY = pY[(r * RT + i) * CL + cl].x;
                    f2 b[SPT], c[SPT];
                    four(sB, row0 + i, b);
                    four(sC, row0 + i, c);
                    constexpr int NV = 2 * SPT, n = NV / CL > 1 ? NV / CL : 1;
                    float v[NV];  // dB, dC terms of the two channels
#pragma unroll
                    for (int j = 0; j < SPT; ++j) {
                        const f2 G = fma2(c[j], dY, g[j]);
                        v[j] = hsum2(mul2(G, x.y));
                        v[SPT + j] = hsum2(mul2(h[i + 1][j], dY));
                        sums[0][i] = j ? fma2(G, b[j], sums[0][i]) : mul2(G, b[j]);
                        sums[2][i] = j ? fma2(h[i + 1][j], c[j], sums[2][i]) : mul2(h[i + 1][j], c[j]);
                        g[j] = mul2(dec[i][j], G);
                        const f2 wj = mul2(g[j], h[i][j]);
                        sums[1][i] = j ? fma2(wj, A2[j], sums[1][i]) : mul2(wj, A2[j]);
                        dA[j] = fma2(wj, x.x, dA[j]);
                    }
                    reduce_lanes<NV, P>(v, lane);
                    // (with more channel lanes than values, several lanes write the same sum)
                    const int idx = reduce_index<NV, P>(lane);
#pragma unroll
                    for (int j = 0; j < n; ++j) {
                        const int vi = idx + j;  // 0 .. 3: dB, 4 .. 7: dC
                        red[((par * NW + w) * RT + i) * 2 * SP + (vi / SPT) * SP + s0 + vi % SPT] = v[j];
                    }
                }
                reduce_tokens<P>(sums, p);
                if (P <= 4 || p < 4)
#pragma unroll
                    for (int i = 0; i < LT; ++i) {
                        const int tk = first_token<P>(p) + i, row = row0 + tk;
                        if (row < len && on0) {
                            const ulonglong2 x = pX[(r * RT + tk) * CL + cl], y = pY[(r * RT + tk) * CL + cl];
                            const ulonglong2 f = pF[(r * RT + tk) * CL + cl];
                            const f2 du = fma2(x.x, sums[0][i], mul2(skip, y.x));
                            const f2 dd = mul2(fma2(y.y, sums[0][i], mul2(sums[1][i], pk2(0.6931471805599453f, 0.6931471805599453f))), f.x);
                            const f2 dz = mul2(f.y, fma2(skip, y.y, sums[2][i]));
                            accD = fma2(y.x, y.y, accD);
                            accb = add2(accb, dd);
                            const int64_t o = (int64_t(t0) + row) * a.C + g_ * Cg + cw + cl;
                            auto put = [&](void* base, f2 val) {
                                float q0, q1;
                                up2(val, q0, q1);
                                ssm_st<E>(base, o, q0);
                                if (on1) ssm_st<E>(base, o + CL, q1);
                            };
                            put(a.du, du);
                            put(a.ddt, dd);
                            if (gated) put(a.dz, dz);
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
        // the channel's lanes hold its tokens' terms of dD and dbias
#pragma unroll
        for (int o = 1; o < P; o <<= 1) {
            accD = add2(accD, __shfl_xor_sync(0xffffffffu, accD, o));
            accb = add2(accb, __shfl_xor_sync(0xffffffffu, accb, o));
        }
        float v[2][4], e[2][4], d[2], b[2];
#pragma unroll
        for (int j = 0; j < SPT; ++j) {
            up2(dA[j], v[0][j], v[1][j]);
            up2(g[j], e[0][j], e[1][j]);
        }
        up2(accD, d[0], d[1]);
        up2(accb, b[0], b[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (q ? on1 : on0) {
                const int c = q ? c1 : c0;
                float* row = a.pA + (int64_t(k) * a.C + c) * (S + 2);
                st4(row, s0, S, make_float4(v[q][0], v[q][1], v[q][2], v[q][3]));
                if (p == 0) row[S] = d[q], row[S + 1] = b[q];
                if (a.dh0 && tab.w == 0)
                    st4(a.dh0 + (int64_t(tab.x) * a.C + c) * S, s0, S, make_float4(e[q][0], e[q][1], e[q][2], e[q][3]));
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
__device__ __forceinline__ void reduce_bc(const SsmArgs& a, const SsmBwdPlan& pl, int block, int blocks) {
    const int64_t n = a.T * a.G * 2 * a.S;
    const int per = pl.nl > 1 ? 1 : SSM_QUAD;
    for (int64_t i = int64_t(block) * blockDim.x + threadIdx.x; i < n; i += int64_t(blocks) * blockDim.x) {
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

// dA, dD, dbias: the chunks' sums.  32 values x 16 strands of chunks per block; a strand's chunks are added
// in order, then the strands.
constexpr int PAR_STRANDS = 16;
__device__ __forceinline__ void reduce_par(const SsmArgs& a, int block) {
    __shared__ float part[PAR_STRANDS][33];
    const int W = a.S + 2, x = threadIdx.x & 31, st = threadIdx.x >> 5, nc = *a.nchunks;
    const int64_t n = int64_t(a.C) * W, i = int64_t(block) * 32 + x;
    float sum = 0.f;
    if (i < n)
#pragma unroll 8
        for (int k = st; k < nc; k += PAR_STRANDS) sum += a.pA[k * n + i];
    part[st][x] = sum;
    __syncthreads();
    if (st || i >= n) return;
#pragma unroll
    for (int j = 1; j < PAR_STRANDS; ++j) sum += part[j][x];
    const int c = int(i / W), s = int(i % W);
    if (s < a.S) a.dA[int64_t(c) * a.S + s] = sum;
    else if (s == a.S) { if (a.dD) a.dD[c] = sum; }
    else if (a.dbias) a.dbias[c] = sum;
}

// the first par_blocks blocks take the parameters, the others dB and dC
template <class E>
__global__ void __launch_bounds__(32 * PAR_STRANDS) k_ssm_reduce(SsmArgs a, SsmBwdPlan pl, int par_blocks) {
    if (!ssm_plan_ok(a)) return;
    if (int(blockIdx.x) < par_blocks) reduce_par(a, blockIdx.x);
    else reduce_bc<E>(a, pl, blockIdx.x - par_blocks, gridDim.x - par_blocks);
}

template <class E, int P>
void launch_main(const SsmArgs& a, const SsmBwdPlan& pl, cudaStream_t st) {
    const unsigned grid = unsigned(a.maxC * a.G * pl.splits);
    {
        ProfScope ps(KK_SSM_BWD, st);
        k_ssm_bwd<E, P><<<grid, SSM_THREADS, BwdShape<P>::floats * 4, st>>>(a, pl);
    }
    constexpr int NT = 32 * PAR_STRANDS;
    const int64_t n = a.T * a.G * 2 * a.S, bc = (n + NT - 1) / NT;
    const int par_blocks = int((int64_t(a.C) * (a.S + 2) + 31) / 32);
    ProfScope ps(KK_SSM_REDUCE, st);
    k_ssm_reduce<E><<<unsigned(par_blocks + (bc < 4096 ? bc : 4096)), NT, 0, st>>>(a, pl, par_blocks);
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
    const int CB = NW * 2 * (32 / pl.lanes), Cg = C / G;
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
