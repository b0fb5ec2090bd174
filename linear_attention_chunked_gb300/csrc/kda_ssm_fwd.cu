// Selective state-space scan over packed documents: the chunked recurrence (kda_ssm.cuh has the formulas).
//
// A document is cut into chunks of 64 tokens.  Three launches after the chunk plan:
//   k_ssm_state  per chunk that has a successor: its end state from a zero start, and sum(delta)
//   k_ssm_carry  per (document, channel, state): start_{k+1} = exp(A sum(delta)_k) start_k + end_k
//   k_ssm_out    per chunk: the recurrence from its start state, y, and the final state
// so a long document fills the machine whatever its batch, at the price of a second evaluation of
// the decays in the chunks that have a successor.  The backward adds
//   k_ssm_rstate per chunk with a predecessor: its start gradient from a zero end,
//                sum_t exp(A (delta_1 + .. + delta_t)) C_t dY_t, and sum(delta)
//
// One walk serves the three (k_ssm_walk).  Lanes are channels: rows are read and written as they lie, the
// sum over up to 16 states stays in the lane, and a lane's B and C values are shared-memory broadcasts.
// The walk loads several pipes at once (per token and 16 states: 16 of 32 ex2 a clock, 16 packed fp32
// instructions, and 4 clocks of register write-back for each shared 16-byte operand) and runs at 0.7
// instructions a clock per scheduler.  Measured and worse on 16384 x 8192 x 16 (the call's kernels 1067 us:
// states 390, output 614, carry 57, plan 6): two channels a lane, which halves the operand reads but leaves
// 12 warps (1270); two lanes a channel with the scalars handed over through shared memory, 32 warps (1295);
// scalars computed a group ahead (1121).
//
// Small problems (k_ssm_small) are bound by the latency of the serial walk instead: there a channel's
// states are spread four to a lane, and the scalars of the whole chunk are computed before the walk by
// all threads at once.  Both forms do the same arithmetic in the same order -- the sum over states goes
// by fours, then by a tree -- so which one runs leaves no trace in the results.
#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

namespace kda {

namespace {

enum Mode { STATE, OUT, RSTATE };

// SPT states at `p` (the states from s0 of a channel's S); FULL: whole 16-byte vectors
template <int SPT, bool FULL>
__device__ __forceinline__ void load_state(const float* p, int s0, int S, f2 (&h)[SPT / 2]) {
#pragma unroll
    for (int j = 0; j < SPT / 2; j += 2) {
        if (FULL) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p + s0 + 2 * j);
            h[j] = v.x, h[j + 1] = v.y;
        } else {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = s0 + 2 * j + i < S ? p[s0 + 2 * j + i] : 0.f;
            h[j] = pk2(v[0], v[1]), h[j + 1] = pk2(v[2], v[3]);
        }
    }
}
template <int SPT, bool FULL>
__device__ __forceinline__ void store_state(float* p, int s0, int S, const f2 (&h)[SPT / 2]) {
#pragma unroll
    for (int j = 0; j < SPT / 2; j += 2) {
        if (FULL) {
            *reinterpret_cast<ulonglong2*>(p + s0 + 2 * j) = make_ulonglong2(h[j], h[j + 1]);
        } else {
            float v[4];
            up2(h[j], v[0], v[1]);
            up2(h[j + 1], v[2], v[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s0 + 2 * j + i < S) p[s0 + 2 * j + i] = v[i];
        }
    }
}
template <int SPT, bool FULL>
__device__ __forceinline__ void load_A(const SsmArgs& a, int c, int s0, f2 (&A2)[SPT / 2]) {
    load_state<SPT, FULL>(a.A + int64_t(c) * a.S, s0, a.S, A2);
#pragma unroll
    for (int j = 0; j < SPT / 2; ++j) A2[j] = mul2(A2[j], pk2(LOG2E, LOG2E));
}

// One thread per (document, channel, state).  Chunk k + 1's slot of hs holds chunk k's end from a zero
// start and receives chunk k + 1's start state.
constexpr int CARRY_THREADS = 128;
__global__ void __launch_bounds__(CARRY_THREADS) k_ssm_carry(SsmArgs a, int blocks_per_doc) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *a.call_status = *a.status;  // (the plan may lie in the saved set)
        if (a.made_for) *a.made_for = a.sizes;
    }
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
    constexpr int U = 16;  // chunks loaded together (few threads, each a serial walk: latency)
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

// The sum over 16 (or fewer) states from its sums over four: by a tree
template <int N>
__device__ __forceinline__ f2 tree4(const f2 (&v)[N]) {
    if constexpr (N == 1) return v[0];
    else if constexpr (N == 2) return add2(v[0], v[1]);
    else return add2(add2(v[0], v[1]), add2(v[2], v[3]));
}


// Rows of a channel, read GR tokens ahead of their use.  The rows past the chunk's end repeat its last one.
template <class E, int GR>
struct Ahead {
    const E* p;  // the next group's first row
    int64_t ld;
    E raw[GR];
    __device__ __forceinline__ Ahead(const void* base, int64_t row, int64_t ld_, int c)
        : p(static_cast<const E*>(base) + row * ld_ + c), ld(ld_) {}
    // left: rows from the group's first to the chunk's end
    __device__ __forceinline__ void load(int left) {
        if (left >= GR) {
#pragma unroll
            for (int i = 0; i < GR; ++i) raw[i] = p[i * ld];
        } else {
#pragma unroll
            for (int i = 0; i < GR; ++i) raw[i] = p[min(i, left - 1) * ld];
        }
        p += GR * ld;
    }
    __device__ __forceinline__ void take(E (&o)[GR]) const {
#pragma unroll
        for (int i = 0; i < GR; ++i) o[i] = raw[i];
    }
};

template <int SPT, int P>
struct Walk {
    static constexpr int CW = 32 / P;           // channels of a warp
    static constexpr int CB = SSM_THREADS / P;  // channels of a block
    static constexpr int SP = SPT * P;          // state slots
};

template <class E, int SPT, int P, bool FULL, int MODE>
__global__ void __launch_bounds__(SSM_THREADS, MODE == STATE ? 6 : MODE == OUT ? 5 : 4) k_ssm_walk(SsmArgs a, int tiles) {
    using L = Walk<SPT, P>;
    constexpr int CW = L::CW, SP = L::SP, H2 = SPT / 2, GR = MODE == RSTATE ? 8 : 4;
    __shared__ __align__(16) float sB[MODE == RSTATE ? 4 : CH * SP], sC[MODE == STATE ? 4 : CH * SP];
    const int k = blockIdx.x / tiles, tile = blockIdx.x % tiles, S = a.S;
    if (MODE == RSTATE && !ssm_plan_ok(a)) return;
    if (k >= *a.nchunks) return;
    const int4 t = a.chunk_tab[k];
    const int t0 = t.y, len = t.z;
    const bool last = t0 + len == a.cu[t.x + 1];
    if (MODE == STATE && last) return;      // no successor
    if (MODE == RSTATE && t.w == 0) return; // no predecessor
    const int Cg = a.C / a.G, tg = (Cg + L::CB - 1) / L::CB, g = tile / tg;
    const int lane = threadIdx.x & 31;
    const int ci = (tile - g * tg) * L::CB + (threadIdx.x >> 5) * CW + lane % CW;
    const bool on = ci < Cg;
    const int c = g * Cg + min(ci, Cg - 1), s0 = lane / CW * SPT;  // lanes past the group repeat its last channel, unwritten
    if (MODE != RSTATE) ssm_load_rows<E, SP>(sB, a.B, a.ldb, t0, len, g * S, S);
    if (MODE != STATE) ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t0, len, g * S, S);
    f2 A2[H2], h[H2];
    load_A<SPT, FULL>(a, c, s0, A2);
    if (MODE == OUT) {
        load_state<SPT, FULL>(a.hs + (int64_t(k) * a.sub * a.C + c) * S, s0, S, h);
    } else {
#pragma unroll
        for (int j = 0; j < H2; ++j) h[j] = 0;
    }
    const float bias = a.bias ? a.bias[c] : 0.f, skip = MODE == OUT && a.D ? a.D[c] : 0.f;
    // (the backward's replay takes the states alone: no y, no ht)
    const bool gated = MODE != STATE && a.z, keep = MODE == OUT && a.sub > 1, writer = MODE == OUT && a.y && on && s0 == 0;
    // (RSTATE: dy in u's place)
    Ahead<E, GR> u(MODE == RSTATE ? a.dy : a.u, t0, MODE == RSTATE ? a.C : a.ldu, c), d(a.dt, t0, a.lddt, c), z(a.z, t0, a.ldz, c);
    E* yp = static_cast<E*>(a.y) + int64_t(t0) * a.C + c;
    u.load(len);
    d.load(len);
    if (gated) z.load(len);
    __syncthreads();
    E cu[GR] = {}, cd[GR] = {}, cz[GR] = {};
    float sum = 0.f;
    auto token = [&](int q, int i) {
        const float dl = ssm_delta(__fadd_rn(ssm_f<E>(cd[i]), bias), a.softplus);
        float v = ssm_f<E>(cu[i]);
        if (MODE != RSTATE) v = __fmul_rn(dl, v);
        else if (gated) v = __fmul_rn(v, ssm_silu(ssm_f<E>(cz[i])));
        if (MODE != OUT) sum += dl;
        const float x = MODE == RSTATE ? sum : dl;
        const f2 d2 = pk2(x, x), u2 = pk2(v, v);
        const ulonglong2* Bp = reinterpret_cast<const ulonglong2*>(sB + (q + i) * SP + s0);
        const ulonglong2* Cp = reinterpret_cast<const ulonglong2*>(sC + (q + i) * SP + s0);
        f2 acc[SPT / 4];
#pragma unroll
        for (int j = 0; j < H2; j += 2) {
            if (MODE == RSTATE) {
                const ulonglong2 c2 = Cp[j / 2];
                h[j] = fma2(ex2_2(mul2(A2[j], d2)), mul2(c2.x, u2), h[j]);
                h[j + 1] = fma2(ex2_2(mul2(A2[j + 1], d2)), mul2(c2.y, u2), h[j + 1]);
            } else {
                const ulonglong2 b2 = Bp[j / 2];
                h[j] = fma2(ex2_2(mul2(A2[j], d2)), h[j], mul2(b2.x, u2));
                h[j + 1] = fma2(ex2_2(mul2(A2[j + 1], d2)), h[j + 1], mul2(b2.y, u2));
            }
            if (MODE == OUT) {
                if (!FULL) {
                    h[j] = keep2(h[j], s0 + 2 * j, S);
                    h[j + 1] = keep2(h[j + 1], s0 + 2 * j + 2, S);
                }
                const ulonglong2 c2 = Cp[j / 2];
                acc[j / 2] = fma2(h[j + 1], c2.y, mul2(h[j], c2.x));
            }
        }
        if (MODE == OUT) {
            float y = hsum2(tree4(acc));
#pragma unroll
            for (int o = CW; o < 32; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            y = fmaf(skip, ssm_f<E>(cu[i]), y);
            if (gated) y = __fmul_rn(y, ssm_silu(ssm_f<E>(cz[i])));
            if (writer) ssm_st<E>(yp, int64_t(i) * a.C, y);
        }
    };
#pragma unroll 1
    for (int q = 0; q < len; q += GR) {
        u.take(cu);
        d.take(cd);
        if (gated) z.take(cz);
        if (q + GR < len) {
            u.load(len - q - GR);
            d.load(len - q - GR);
            if (gated) z.load(len - q - GR);
        }
        if (keep && q % SSM_UT == 0 && q > 0 && on)
            store_state<SPT, FULL>(a.hs + ((int64_t(k) * a.sub + q / SSM_UT) * a.C + c) * S, s0, S, h);
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
    if (!on) return;
    if (MODE == OUT) {
        if (a.ht && last) store_state<SPT, FULL>(a.ht + (int64_t(t.x) * a.C + c) * S, s0, S, h);
        return;
    }
    if (s0 == 0) a.sumdt[int64_t(k) * a.C + c] = sum;
    // into the next chunk's slot; RSTATE: the end gradient of the chunk before
    float* out = MODE == STATE ? a.hs + (int64_t(k + 1) * a.sub * a.C + c) * S : a.gs + (int64_t(k - 1) * a.C + c) * S;
    store_state<SPT, FULL>(out, s0, S, h);
}

// ---- small problems ----

// P lanes per channel, four states each; channels are neighbours in the warp's lanes' upper bits.
template <int P>
struct Small {
    static constexpr int SP = 4 * P, CB = SSM_THREADS / P;  // channels per block
    static constexpr int NI = CH * CB / SSM_THREADS;        // (token, channel) items per thread
    // shared memory, in floats: B and C rows; delta and delta u (y in its place); y before the gate
    static constexpr int oB = 0, oC = CH * SP, oPre = 2 * CH * SP, floats = oPre + 2 * CH * CB;
};

// direct: one block row per document of at most one chunk, without plan and carry; the block checks
// the offsets itself.
template <class E, int P, bool FULL, int MODE>
__global__ void __launch_bounds__(SSM_THREADS) k_ssm_small(SsmArgs a, int tiles, int direct) {
    using L = Small<P>;
    constexpr int SP = L::SP, CB = L::CB;
    extern __shared__ __align__(16) float sm[];
    float *sB = sm + L::oB, *sC = sm + L::oC;
    float2* pre = reinterpret_cast<float2*>(sm + L::oPre);  // [token][channel]
    const int tid = threadIdx.x, k = blockIdx.x / tiles, tile = blockIdx.x % tiles, S = a.S;
    int doc, t0, len;
    bool last, first;
    if (direct) {
        bool ok = true;
        for (int i = tid; i <= a.N; i += SSM_THREADS)
            ok &= i == 0 ? a.cu[0] == 0 : a.cu[i] >= a.cu[i - 1] && (i < a.N || a.cu[i] == a.T);
        ok = __syncthreads_and(ok);
        if (blockIdx.x == 0 && tid == 0) *a.status = ok ? KDA_OK : KDA_ERR_DEVICE_CHECK;
        if (!ok) return;
        doc = k, t0 = a.cu[k], len = a.cu[k + 1] - t0;
        last = first = true;
    } else {
        if (MODE == RSTATE && !ssm_plan_ok(a)) return;
        if (k >= *a.nchunks) return;
        const int4 t = a.chunk_tab[k];
        doc = t.x, t0 = t.y, len = t.z;
        last = t0 + len == a.cu[doc + 1];
        first = false;  // (the carry has written every chunk's start state)
        if (MODE == STATE && last) return;
        if (MODE == RSTATE && t.w == 0) return;
    }
    const int Cg = a.C / a.G, tg = (Cg + CB - 1) / CB, g = tile / tg, cb = (tile - g * tg) * CB;
    const int p = tid % P, cl = tid / P, s0 = 4 * p, c = g * Cg + min(cb + cl, Cg - 1);
    const bool on = cb + cl < Cg;
    // items: channel tid % CB, tokens tid / CB + i SSM_THREADS / CB
    constexpr int TS = SSM_THREADS / CB;
    const int ic = g * Cg + min(cb + tid % CB, Cg - 1), it = tid / CB;
    const bool gated = MODE != STATE && a.z, ion = cb + tid % CB < Cg;
    const float bias = a.bias ? a.bias[ic] : 0.f, skip = MODE == OUT && a.D ? a.D[ic] : 0.f;
    constexpr int NB = L::NI < 16 ? L::NI : 16;  // items in flight
    E ru[NB], rd[NB], rz[NB];  // (RSTATE: dy in u's place)
    auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int r = it + (i0 + i) * TS;
            if (r < len) {
                const int64_t row = t0 + r;
                ru[i] = static_cast<const E*>(MODE == RSTATE ? a.dy : a.u)[row * (MODE == RSTATE ? a.C : a.ldu) + ic];
                rd[i] = static_cast<const E*>(a.dt)[row * a.lddt + ic];
                if (gated) rz[i] = static_cast<const E*>(a.z)[row * a.ldz + ic];
            }
        }
    };
    fetch(0);
    if (MODE != RSTATE) ssm_load_rows<E, SP>(sB, a.B, a.ldb, t0, len, g * S, S);
    if (MODE != STATE) ssm_load_rows<E, SP>(sC, a.Cm, a.ldc, t0, len, g * S, S);
    f2 A2[2], h[2] = {0, 0};
    load_A<4, FULL>(a, c, s0, A2);
    if (MODE == OUT) {
        if (!first) load_state<4, FULL>(a.hs + (int64_t(k) * a.sub * a.C + c) * S, s0, S, h);
        else if (a.h0) load_state<4, FULL>(a.h0 + (int64_t(doc) * a.C + c) * S, s0, S, h);
    }
#pragma unroll
    for (int i0 = 0; i0 < L::NI; i0 += NB) {
        if (i0) fetch(i0);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int r = it + (i0 + i) * TS;
            if (r < len) {
                const float dl = ssm_delta(__fadd_rn(ssm_f<E>(rd[i]), bias), a.softplus);
                float v = ssm_f<E>(ru[i]);
                if (MODE != RSTATE) v = __fmul_rn(dl, v);
                else if (gated) v = __fmul_rn(v, ssm_silu(ssm_f<E>(rz[i])));
                pre[r * CB + tid % CB] = make_float2(dl, v);
            }
        }
    }
    __syncthreads();
    float sum = 0.f;
    auto token = [&](int r) {
        const float2 v = pre[r * CB + cl];
        if (MODE != OUT) sum += v.x;
        const float x = MODE == RSTATE ? sum : v.x;
        const f2 d2 = pk2(x, x), u2 = pk2(v.y, v.y);
        const ulonglong2* Bp = reinterpret_cast<const ulonglong2*>(sB + r * SP + s0);
        const ulonglong2* Cp = reinterpret_cast<const ulonglong2*>(sC + r * SP + s0);
        if (MODE == RSTATE) {
            h[0] = fma2(ex2_2(mul2(A2[0], d2)), mul2(Cp->x, u2), h[0]);
            h[1] = fma2(ex2_2(mul2(A2[1], d2)), mul2(Cp->y, u2), h[1]);
        } else {
            h[0] = fma2(ex2_2(mul2(A2[0], d2)), h[0], mul2(Bp->x, u2));
            h[1] = fma2(ex2_2(mul2(A2[1], d2)), h[1], mul2(Bp->y, u2));
        }
        if (MODE == OUT) {
            if (!FULL) {
                h[0] = keep2(h[0], s0, S);
                h[1] = keep2(h[1], s0 + 2, S);
            }
            const ulonglong2 c2 = *Cp;
            f2 acc = fma2(h[1], c2.y, mul2(h[0], c2.x));
#pragma unroll
            for (int o = 1; o < P && o < 4; o <<= 1) acc = add2(acc, __shfl_xor_sync(0xffffffffu, acc, o));
            float y = hsum2(acc);
#pragma unroll
            for (int o = 4; o < P; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
            if (p == 0) pre[r * CB + cl].x = y;  // delta has been read by all of the channel's lanes
        }
    };
    constexpr int UR = 4;
    for (int r0 = 0; r0 < len; r0 += UR) {
        if (MODE == OUT && a.sub > 1 && r0 % SSM_UT == 0 && r0 > 0 && on)
            store_state<4, FULL>(a.hs + ((int64_t(k) * a.sub + r0 / SSM_UT) * a.C + c) * S, s0, S, h);
        if (r0 + UR <= len) {
#pragma unroll
            for (int i = 0; i < UR; ++i) token(r0 + i);
        } else {
            for (int r = r0; r < len; ++r) token(r);
        }
    }
    if (MODE != OUT) {
        if (on) {
            if (p == 0) a.sumdt[int64_t(k) * a.C + c] = sum;
            float* out = MODE == STATE ? a.hs + (int64_t(k + 1) * a.sub * a.C + c) * S : a.gs + (int64_t(k - 1) * a.C + c) * S;
            store_state<4, FULL>(out, s0, S, h);
        }
        return;
    }
    if (a.ht && last && on) store_state<4, FULL>(a.ht + (int64_t(doc) * a.C + c) * S, s0, S, h);
    if (!a.y) return;
    __syncthreads();
#pragma unroll
    for (int i0 = 0; i0 < L::NI; i0 += NB) {
        if (L::NI > NB) fetch(i0);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int r = it + (i0 + i) * TS;
            if (r < len && ion) {
                float y = fmaf(skip, ssm_f<E>(ru[i]), pre[r * CB + tid % CB].x);
                if (gated) y = __fmul_rn(y, ssm_silu(ssm_f<E>(rz[i])));
                ssm_st<E>(a.y, (int64_t(t0) + r) * a.C + ic, y);
            }
        }
    }
}

template <auto* F>
void small_launch(int64_t blocks, size_t smem, const SsmArgs& a, int tiles, int direct, cudaStream_t st) {
    static unsigned long long done;
    allow_smem((const void*)F, smem, &done);
    F<<<unsigned(blocks), SSM_THREADS, smem, st>>>(a, tiles, direct);
}

int tiles_of(const SsmArgs& a, int CB) {
    const int Cg = a.C / a.G;
    return a.G * ((Cg + CB - 1) / CB);
}

template <class E, int SPT, int P, bool FULL, int MODE>
void launch(const SsmArgs& a, cudaStream_t st) {
    constexpr int PS = SPT * P / 4;  // the small form's lanes per channel
    using S = Small<PS>;
    const int wide = tiles_of(a, Walk<SPT, P>::CB), narrow = tiles_of(a, S::CB);
    const int64_t rows = a.direct ? a.N : a.maxC;
    ProfScope ps(MODE == STATE ? KK_SSM_STATE : MODE == OUT ? KK_SSM_OUT : KK_SSM_RSTATE, st);
    // the walk once it has blocks enough for the 152 multiprocessors; where the small form ends, both
    // measured (us, C = 1024 .. 4096, T = 1024 .. 4096): out 22.6 / 24.6 at 128 walk blocks, 39 / 29 at
    // 256; state 26.7 / 26.7 at 512, 49 / 43 at 1024; rstate 51 / 59 at 1024, 94 / 96 at 2048
    constexpr int limit = MODE == OUT ? 160 : MODE == STATE ? 512 : 2048;
    if (a.direct || a.maxC * wide < limit)
        small_launch<k_ssm_small<E, PS, FULL, MODE>>(rows * narrow, S::floats * sizeof(float), a, narrow, a.direct, st);
    else
        k_ssm_walk<E, SPT, P, FULL, MODE><<<unsigned(a.maxC * wide), SSM_THREADS, 0, st>>>(a, wide);
}

template <class E, int MODE>
void by_states(const SsmArgs& a, cudaStream_t st) {
    switch (a.S) {  // the usual state counts fill their lanes; others are padded to the next one
        case 4: return launch<E, 4, 1, true, MODE>(a, st);
        case 8: return launch<E, 8, 1, true, MODE>(a, st);
        case 16: return launch<E, 16, 1, true, MODE>(a, st);
        case 32: return launch<E, 16, 2, true, MODE>(a, st);
        case 64: return launch<E, 16, 4, true, MODE>(a, st);
        default: break;
    }
    if (a.S < 8) return launch<E, 8, 1, false, MODE>(a, st);
    if (a.S < 16) return launch<E, 16, 1, false, MODE>(a, st);
    if (a.S < 32) return launch<E, 16, 2, false, MODE>(a, st);
    return launch<E, 16, 4, false, MODE>(a, st);
}

template <int MODE>
void by_type(const SsmArgs& a, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) by_states<__nv_bfloat16, MODE>(a, st);
    else if (dtype == KDA_DT_FP16) by_states<__half, MODE>(a, st);
    else by_states<float, MODE>(a, st);
}

}  // namespace

void launch_ssm_scan(const SsmArgs& a, int dtype, cudaStream_t st) {
    if (a.T > CH) by_type<STATE>(a, dtype, st);  // at most one chunk of tokens: no chunk has a successor
    if (!a.direct) {
        ProfScope ps(KK_SSM_CARRY, st);
        const int64_t CS = int64_t(a.C) * a.S;
        const int bpd = int((CS + CARRY_THREADS - 1) / CARRY_THREADS);
        k_ssm_carry<<<unsigned(int64_t(bpd) * a.N), CARRY_THREADS, 0, st>>>(a, bpd);
    }
    by_type<OUT>(a, dtype, st);
}

void launch_ssm_rstate(const SsmArgs& a, int dtype, cudaStream_t st) {
    if (a.T > CH) by_type<RSTATE>(a, dtype, st);
}

}  // namespace kda
