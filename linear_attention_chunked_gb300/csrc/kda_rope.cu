// Norm of every head's queries and keys and their rotation to positions, forward and backward.
//
//   xh = x / sqrt(sum_c x_c^2 / D + eps),  n = xh w             (norm; else n = x)
//   y  = scale R(pos freq) n on the first R channels, in pairs, n on the others
//   backward:  d = the turn undone on dy (scale kept),  dw = sum_rows d xh,  g = d w
//              dx = (g - xh sum_c(g xh) / D) / sqrt(..)          (norm; else dx = d)
//
// Bound by HBM: forward 2, backward 3 (2 without the norm) row transfers.  A row of D channels belongs to a
// group of lanes that each hold four pairs (two vectors of four elements; both members of a pair lie in one
// lane, so the turn needs no exchange), the norm's sum is one exchange over the group.  A group takes one
// token's heads in turn, several rows in flight: the token's cosines and sines are computed once for them.
//
// Angles.  A position times a frequency in fp32 is off by a thousandth of a turn at position 10^4 already.
// Here a frequency is a 64-bit fraction of a turn per token, F = freq / (2 pi) 2^64 mod 2^64, so pos F mod
// 2^64 is the angle's fraction of a turn, exact for any 32-bit position but for F's own rounding (below
// 2^-53 freq / 2 pi a token: 10^-10 turns at position 10^6); its upper 32 bits go through sincospif.
#include <math.h>

#include "kda_ssm.cuh"

namespace kda {

namespace {

struct RopeArgs {
    int64_t T;
    int Hq, Hk, D, R, norm;
    float eps, scale, inv_d;
    const void *q, *k, *gq, *gk;  // inputs; gradients of the outputs (backward)
    void *oq, *ok;
    const int* pos;
    const double* freq;
    const float *wq, *wk;
    int64_t ldq, ldk;    // token strides of q, k
    int64_t ldgq, ldgk;  // of gq, gk
    int64_t ldoq, ldok;  // of the outputs
    int split, per;      // parts that a token's heads are cut into, heads of a part
    float* part;         // [blocks][2][D] partial dwq, dwk
    float *dwq, *dwk;
    int blocks;
};

constexpr int RP_THREADS = 256;
constexpr int RP_MAXD = 256;

// freq / (2 pi) as a 64-bit fraction of a turn.  freq = M 2^(E - 63) with a 64-bit M, 1 / (2 pi) = C 2^-66:
// their product's upper half times 2^(E - 1) is the fraction (whole turns fall out at the top).
__device__ __forceinline__ unsigned long long turns_per_token(double freq) {
    const unsigned long long b = (unsigned long long)__double_as_longlong(freq);
    const int ex = int(b >> 52) & 0x7ff;
    if (ex == 0) return 0;  // zero (or below 1e-307)
    const unsigned long long M = (b << 11) | (1ull << 63);
    constexpr unsigned long long C = (unsigned long long)(0.63661977236758134 * 18446744073709551616.0);  // 2 / pi
    const unsigned long long hi = __umul64hi(M, C);
    const int E = ex - 1023 - 1;
    const unsigned long long F = E >= 64 || E <= -64 ? 0 : E >= 0 ? hi << E : hi >> -E;
    return b >> 63 ? 0ull - F : F;
}

__device__ __forceinline__ void cos_sin(int pos, unsigned long long F, float scale, float& c, float& s) {
    const unsigned long long turn = (unsigned long long)(long long)pos * F;
    sincospif(float(int(turn >> 32)) * 4.656612873077392578125e-10f, &s, &c);  // 2^-31: half turns
    c *= scale;
    s *= scale;
}

template <class E> struct alignas(4 * sizeof(E)) Quad { E e[4]; };
template <class E> __device__ __forceinline__ E rp_cast(float v);
template <> __device__ __forceinline__ float rp_cast<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rp_cast<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rp_cast<__half>(float v) { return __float2half_rn(v); }

// Channels of pair p of a row (p >= R / 2: channels that are not turned, two by two)
__device__ __forceinline__ void pair_at(int p, int R, bool pairs, int& a, int& b) {
    if (p < R / 2 && !pairs) a = p, b = R / 2 + p;
    else a = 2 * p, b = 2 * p + 1;
}

// A lane's row values: NP pairs (x[i], y[i])
template <int NP> struct Row { float x[NP], y[NP]; };

// The channels of a lane.  VEC: one unit of eight channels, two quads at o0 and o1 (halves: the members of
// four pairs; otherwise eight neighbours).  Else up to NP single pairs.
template <class E, int NP, bool PAIRS, bool VEC>
struct Lane {
    // VEC: NP = 4
    int o0, o1;       // VEC: the quads' channels
    int l, D, R, G;   // otherwise pair i is l + i G
    bool on, neighbours;
    __device__ __forceinline__ Lane(int lane, int D_, int R_, int G_) : l(lane), D(D_), R(R_), G(G_) {
        if (VEC) {
            on = 8 * l < D;
            neighbours = PAIRS || 8 * l >= R;
            o0 = neighbours ? 8 * l : 4 * l;
            o1 = neighbours ? 8 * l + 4 : R / 2 + 4 * l;
        } else {
            on = true;
        }
    }
    __device__ __forceinline__ bool has(int i) const { return VEC ? on : l + i * G < D / 2; }
    __device__ __forceinline__ bool turns(int i) const { return VEC ? 8 * l < R : l + i * G < R / 2; }
    __device__ __forceinline__ int pair(int i) const { return VEC ? 4 * l + i : l + i * G; }
    // the raw elements of a row, to be kept while others load
    struct Raw { Quad<E> a, b; };
    __device__ __forceinline__ Raw load(const void* base, int64_t at) const {
        Raw r;
        const E* p = static_cast<const E*>(base) + at;
        if constexpr (VEC) {
            if (on) {
                r.a = *reinterpret_cast<const Quad<E>*>(p + o0);
                r.b = *reinterpret_cast<const Quad<E>*>(p + o1);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) r.a.e[i] = r.b.e[i] = rp_cast<E>(0.f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                r.a.e[i] = r.b.e[i] = rp_cast<E>(0.f);
                if (has(i)) {
                    int ca, cb;
                    pair_at(l + i * G, R, PAIRS, ca, cb);
                    r.a.e[i] = p[ca];
                    r.b.e[i] = p[cb];
                }
            }
        }
        return r;
    }
    __device__ __forceinline__ void store(void* base, int64_t at, const Row<NP>& v) const {
        E* p = static_cast<E*>(base) + at;
        if constexpr (VEC) {
            if (!on) return;
            Quad<E> a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // neighbours: pair i is channels 2 i, 2 i + 1 of the eight
                if (neighbours) {
                    (i < 2 ? a : b).e[2 * (i & 1)] = rp_cast<E>(v.x[i]);
                    (i < 2 ? a : b).e[2 * (i & 1) + 1] = rp_cast<E>(v.y[i]);
                } else {
                    a.e[i] = rp_cast<E>(v.x[i]);
                    b.e[i] = rp_cast<E>(v.y[i]);
                }
            }
            *reinterpret_cast<Quad<E>*>(p + o0) = a;
            *reinterpret_cast<Quad<E>*>(p + o1) = b;
        } else {
#pragma unroll
            for (int i = 0; i < NP; ++i)
                if (has(i)) {
                    int ca, cb;
                    pair_at(l + i * G, R, PAIRS, ca, cb);
                    p[ca] = rp_cast<E>(v.x[i]);
                    p[cb] = rp_cast<E>(v.y[i]);
                }
        }
    }
    __device__ __forceinline__ Row<NP> values(const Raw& r) const {
        Row<NP> v;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (VEC && neighbours) {
                v.x[i] = ssm_f<E>((i < 2 ? r.a : r.b).e[2 * (i & 1)]);
                v.y[i] = ssm_f<E>((i < 2 ? r.a : r.b).e[2 * (i & 1) + 1]);
            } else {
                v.x[i] = ssm_f<E>(r.a.e[i]);
                v.y[i] = ssm_f<E>(r.b.e[i]);
            }
        }
        return v;
    }
    // fp32 parameters of the lane's channels (w null: ones)
    __device__ __forceinline__ Row<NP> weights(const float* w) const {
        Row<NP> v;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            v.x[i] = v.y[i] = 1.f;
            int ca, cb;
            pair_at(pair(i), R, PAIRS, ca, cb);
            if (w && has(i)) v.x[i] = w[ca], v.y[i] = w[cb];
        }
        return v;
    }
};

__device__ __forceinline__ float group_sum(float v, int G) {
    for (int o = G >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr int RP_ROWS = 4;  // rows of a group in flight

// BWD: q, k and the gradients in, gradients out; otherwise q, k in, turned out.  A work unit is one part
// of one token's heads (q's heads, then k's).
template <class E, int NP, bool PAIRS, bool VEC, bool BWD>
__global__ void __launch_bounds__(RP_THREADS) k_rope(RopeArgs a, int G) {
    const int tid = threadIdx.x, lane = tid & (G - 1), groups = RP_THREADS / G;
    const Lane<E, NP, PAIRS, VEC> L(lane, a.D, a.R, G);
    unsigned long long F[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) F[i] = L.has(i) && L.turns(i) ? turns_per_token(a.freq[L.pair(i)]) : 0;
    const Row<NP> wq = L.weights(a.norm ? a.wq : nullptr), wk = L.weights(a.norm ? a.wk : nullptr);
    Row<NP> sq, sk;  // sums of dwq, dwk
#pragma unroll
    for (int i = 0; i < NP; ++i) sq.x[i] = sq.y[i] = sk.x[i] = sk.y[i] = 0.f;
    const int H = a.Hq + a.Hk;
    const int64_t units = a.T * a.split, per_wave = int64_t(gridDim.x) * groups;
    // the lanes of a warp run the same number of rounds (exchanges over the group are warp-wide)
    const int64_t rounds = (units + per_wave - 1) / per_wave;
    for (int64_t round = 0; round < rounds; ++round) {
        const int64_t u = round * per_wave + int64_t(blockIdx.x) * groups + tid / G;
        const bool live = u < units;
        const int64_t t = live ? u / a.split : 0;
        const int h0 = live ? int(u % a.split) * a.per : 0, h1 = live ? min(h0 + a.per, H) : 0;
        float c[NP], s[NP];
        const int pos = live ? a.pos[t] : 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            c[i] = 1.f, s[i] = 0.f;
            if (L.has(i) && L.turns(i)) cos_sin(pos, F[i], a.scale, c[i], s[i]);
        }
        for (int hb = 0; hb < a.per; hb += RP_ROWS) {
            typename Lane<E, NP, PAIRS, VEC>::Raw x[RP_ROWS], g[RP_ROWS];
#pragma unroll
            for (int r = 0; r < RP_ROWS; ++r) {
                const int h = h0 + hb + r;
                if (h >= h1) continue;
                const bool isq = h < a.Hq;
                const int hh = isq ? h : h - a.Hq;
                if (!BWD || a.norm) x[r] = L.load(isq ? a.q : a.k, t * (isq ? a.ldq : a.ldk) + int64_t(hh) * a.D);
                if (BWD) g[r] = L.load(isq ? a.gq : a.gk, t * (isq ? a.ldgq : a.ldgk) + int64_t(hh) * a.D);
            }
#pragma unroll
            for (int r = 0; r < RP_ROWS; ++r) {
                const int h = h0 + hb + r;
                const bool use = h < h1;
                const bool isq = h < a.Hq;
                const int hh = isq ? h : h - a.Hq;
                const Row<NP>& w = isq ? wq : wk;
                Row<NP> v;
                float rs = 1.f;
                if (a.norm) {
                    float ss = 0.f;
                    if (use) {
                        v = L.values(x[r]);
#pragma unroll
                        for (int i = 0; i < NP; ++i) ss = fmaf(v.x[i], v.x[i], fmaf(v.y[i], v.y[i], ss));
                    }
                    rs = 1.f / sqrtf(fmaf(group_sum(ss, G), a.inv_d, a.eps));
                } else if (!BWD && use) {
                    v = L.values(x[r]);
                }
                if (!BWD) {
                    if (!use) continue;
                    Row<NP> y;
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        float p = v.x[i], z = v.y[i];
                        if (a.norm) p *= rs * w.x[i], z *= rs * w.y[i];
                        y.x[i] = L.turns(i) ? fmaf(p, c[i], -(z * s[i])) : p;
                        y.y[i] = L.turns(i) ? fmaf(p, s[i], z * c[i]) : z;
                    }
                    L.store(isq ? a.oq : a.ok, t * (isq ? a.ldoq : a.ldok) + int64_t(hh) * a.D, y);
                } else {
                    Row<NP> d;
                    float dot = 0.f;
                    if (use) {
                        const Row<NP> y = L.values(g[r]);
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            d.x[i] = L.turns(i) ? fmaf(y.x[i], c[i], y.y[i] * s[i]) : y.x[i];
                            d.y[i] = L.turns(i) ? fmaf(y.y[i], c[i], -(y.x[i] * s[i])) : y.y[i];
                            if (a.norm) {
                                v.x[i] *= rs, v.y[i] *= rs;
                                Row<NP>& sw = isq ? sq : sk;
                                sw.x[i] = fmaf(d.x[i], v.x[i], sw.x[i]);
                                sw.y[i] = fmaf(d.y[i], v.y[i], sw.y[i]);
                                d.x[i] *= w.x[i], d.y[i] *= w.y[i];
                                dot = fmaf(d.x[i], v.x[i], fmaf(d.y[i], v.y[i], dot));
                            }
                        }
                    }
                    if (a.norm) dot = group_sum(dot, G) * a.inv_d;
                    if (!use) continue;
                    if (a.norm)
#pragma unroll
                        for (int i = 0; i < NP; ++i) {
                            d.x[i] = rs * fmaf(-v.x[i], dot, d.x[i]);
                            d.y[i] = rs * fmaf(-v.y[i], dot, d.y[i]);
                        }
                    L.store(isq ? a.oq : a.ok, t * (isq ? a.ldoq : a.ldok) + int64_t(hh) * a.D, d);
                }
            }
        }
    }
    if (BWD && a.part) {  // the groups' sums, added in their order
        __shared__ float red[2][RP_MAXD];
        for (int gi = 0; gi < groups; ++gi) {
            if (tid / G == gi) {
#pragma unroll
                for (int i = 0; i < NP; ++i)
                    if (L.has(i)) {
                        int ca, cb;
                        pair_at(L.pair(i), a.R, PAIRS, ca, cb);
                        red[0][ca] = gi ? red[0][ca] + sq.x[i] : sq.x[i];
                        red[0][cb] = gi ? red[0][cb] + sq.y[i] : sq.y[i];
                        red[1][ca] = gi ? red[1][ca] + sk.x[i] : sk.x[i];
                        red[1][cb] = gi ? red[1][cb] + sk.y[i] : sk.y[i];
                    }
            }
            __syncthreads();
        }
        for (int i = tid; i < 2 * a.D; i += RP_THREADS)
            a.part[int64_t(blockIdx.x) * 2 * a.D + i] = red[i / a.D][i % a.D];
    }
}

// dwq and dwk: the blocks' sums, one warp per channel, in an order that depends on their number alone
__global__ void __launch_bounds__(256) k_rope_reduce(RopeArgs a) {
    const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (c >= 2 * a.D) return;
    float v = 0.f;
    for (int b = lane; b < a.blocks; b += 32) v += a.part[int64_t(b) * 2 * a.D + c];
    v = warp_sum(v);
    float* out = c < a.D ? a.dwq : a.dwk;
    if (lane == 0 && out) out[c % a.D] = v;
}

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t esize(int dtype) { return dtype == KDA_DT_FP32 ? 4 : 2; }
int64_t ld_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

constexpr int RP_BWD_BLOCKS = 152 * 4;  // most blocks of a backward that sums dw

kda_status check_problem(const kda_rope_problem* p) {
    if (!p || p->T < 0 || p->T > INT32_MAX || p->Hq < 0 || p->Hq > 65535 || p->Hk < 0 || p->Hk > 65535 ||
        p->Hq + p->Hk < 1 || p->D < 2 || p->D % 2 || p->R < 0 || p->R % 2 || p->R > p->D)
        return KDA_ERR_INVALID_ARG;
    if (p->D > RP_MAXD) return KDA_ERR_UNSUPPORTED;
    if (p->layout != KDA_ROPE_HALF && p->layout != KDA_ROPE_PAIRS) return KDA_ERR_INVALID_ARG;
    if (p->norm != 0 && p->norm != 1) return KDA_ERR_INVALID_ARG;
    if (p->norm && !(p->eps >= 0.f)) return KDA_ERR_INVALID_ARG;
    if (p->dtype != KDA_DT_BF16 && p->dtype != KDA_DT_FP16 && p->dtype != KDA_DT_FP32) return KDA_ERR_INVALID_ARG;
    const int64_t q = int64_t(p->Hq) * p->D, k = int64_t(p->Hk) * p->D;
    if (ld_or(p->ld_q, q) < q || ld_or(p->ld_k, k) < k || ld_or(p->ld_qo, q) < q || ld_or(p->ld_ko, k) < k)
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

template <class E, bool BWD>
void launch(RopeArgs a, int layout, cudaStream_t st) {
    const bool pairs = layout == KDA_ROPE_PAIRS;
    // four pairs a lane where the channels and every row allow quads, else one pair at a time
    auto wide = [&](const void* p, int64_t ld) { return !p || (al(p, 4 * sizeof(E)) && ld % 4 == 0); };
    const bool vec = a.D % 8 == 0 && a.R % 8 == 0 && wide(a.q, a.ldq) && wide(a.k, a.ldk) && wide(a.gq, a.ldgq) &&
                     wide(a.gk, a.ldgk) && wide(a.oq, a.ldoq) && wide(a.ok, a.ldok);
    int G = 1;
    while (G < 32 && G * (vec ? 8 : 2) < a.D) G *= 2;
    const int groups = RP_THREADS / G, H = a.Hq + a.Hk;
    // a group takes 16 heads of a token, fewer where that leaves too few groups
    a.per = 16;
    while (a.per > RP_ROWS && a.T * ((H + a.per - 1) / a.per) < int64_t(152) * 8 * groups) a.per /= 2;
    a.split = (H + a.per - 1) / a.per;
    const int64_t blocks = (a.T * a.split + groups - 1) / groups;
    const int64_t most = BWD && a.part ? RP_BWD_BLOCKS : 152 * 8;
    a.blocks = int(blocks < most ? blocks : most);
    {
        ProfScope ps(BWD ? KK_ROPE_BWD : KK_ROPE_FWD, st);
        if (vec) {
            if (pairs) k_rope<E, 4, true, true, BWD><<<a.blocks, RP_THREADS, 0, st>>>(a, G);
            else k_rope<E, 4, false, true, BWD><<<a.blocks, RP_THREADS, 0, st>>>(a, G);
        } else {
            if (pairs) k_rope<E, 4, true, false, BWD><<<a.blocks, RP_THREADS, 0, st>>>(a, G);
            else k_rope<E, 4, false, false, BWD><<<a.blocks, RP_THREADS, 0, st>>>(a, G);
        }
    }
    if (BWD && a.part) {
        ProfScope ps(KK_ROPE_REDUCE, st);
        k_rope_reduce<<<(2 * a.D + 7) / 8, 256, 0, st>>>(a);
    }
}

template <bool BWD>
void launch_any(const RopeArgs& a, int layout, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) launch<__nv_bfloat16, BWD>(a, layout, st);
    else if (dtype == KDA_DT_FP16) launch<__half, BWD>(a, layout, st);
    else launch<float, BWD>(a, layout, st);
}

RopeArgs make_args(const kda_rope_problem* p, const int32_t* pos, const double* freq, const float* wq, const float* wk) {
    RopeArgs a{};
    a.T = p->T, a.Hq = p->Hq, a.Hk = p->Hk, a.D = p->D, a.R = p->R, a.norm = p->norm;
    a.eps = p->eps, a.scale = p->scale, a.inv_d = 1.f / float(p->D);
    a.pos = pos, a.freq = freq, a.wq = wq, a.wk = wk;
    const int64_t q = int64_t(p->Hq) * p->D, k = int64_t(p->Hk) * p->D;
    a.ldq = ld_or(p->ld_q, q), a.ldk = ld_or(p->ld_k, k);
    return a;
}

// q, k, pos, freq and the norm's weights of a call with tokens
bool inputs_ok(const kda_rope_problem* p, const int32_t* pos, const double* freq, const float* wq, const float* wk) {
    return pos && al(pos, 4) && (p->R == 0 || freq) && al(freq, 8) && al(wq, 4) && al(wk, 4);
}
bool rows_ok(const kda_rope_problem* p, const void* q, const void* k) {
    const size_t e = esize(p->dtype);
    return (p->Hq == 0 || (q && al(q, e))) && (p->Hk == 0 || (k && al(k, e)));
}

size_t part_bytes(const kda_rope_problem* p) {
    return p->norm ? size_t(RP_BWD_BLOCKS) * 2 * size_t(p->D) * 4 : 0;
}

kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_rope_workspace_size(const kda_rope_problem* p, size_t* ws_bytes) {
    if (kda_status s = check_problem(p)) return s;
    if (ws_bytes) *ws_bytes = part_bytes(p);
    return KDA_OK;
}

kda_status kda_rope_fwd(const kda_rope_problem* p, const void* q, const void* k, const int32_t* pos,
                        const double* freq, const float* wq, const float* wk, void* q_out, void* k_out,
                        kda_stream_t stream) {
    if (kda_status s = check_problem(p)) return s;
    if (p->T == 0) return KDA_OK;
    if (!inputs_ok(p, pos, freq, wq, wk) || !rows_ok(p, q, k) || !rows_ok(p, q_out, k_out)) return KDA_ERR_INVALID_ARG;
    RopeArgs a = make_args(p, pos, freq, wq, wk);
    a.q = p->Hq ? q : nullptr, a.k = p->Hk ? k : nullptr;
    a.oq = p->Hq ? q_out : nullptr, a.ok = p->Hk ? k_out : nullptr;
    a.ldoq = ld_or(p->ld_qo, int64_t(p->Hq) * p->D), a.ldok = ld_or(p->ld_ko, int64_t(p->Hk) * p->D);
    launch_any<false>(a, p->layout, p->dtype, reinterpret_cast<cudaStream_t>(stream));
    return launched();
}

kda_status kda_rope_bwd(const kda_rope_problem* p, const void* q, const void* k, const int32_t* pos,
                        const double* freq, const float* wq, const float* wk, const void* dq_out, const void* dk_out,
                        void* dq, void* dk, float* dwq, float* dwk, void* ws, size_t ws_bytes, kda_stream_t stream) {
    if (kda_status s = check_problem(p)) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool sums = p->norm && (dwq || dwk);
    if (p->T == 0) {
        if (sums && ((dwq && cudaMemsetAsync(dwq, 0, size_t(p->D) * 4, st) != cudaSuccess) ||
                     (dwk && cudaMemsetAsync(dwk, 0, size_t(p->D) * 4, st) != cudaSuccess)))
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    if (!inputs_ok(p, pos, freq, wq, wk) || (p->norm && !rows_ok(p, q, k)) || !rows_ok(p, dq_out, dk_out) ||
        !rows_ok(p, dq, dk) || !al(dwq, 4) || !al(dwk, 4))
        return KDA_ERR_INVALID_ARG;
    if (sums && (!ws || !al(ws, 16))) return KDA_ERR_INVALID_ARG;
    if (sums && ws_bytes < part_bytes(p)) return KDA_ERR_WORKSPACE;
    RopeArgs a = make_args(p, pos, freq, wq, wk);
    const int64_t dense_q = int64_t(p->Hq) * p->D, dense_k = int64_t(p->Hk) * p->D;
    if (p->norm) a.q = p->Hq ? q : nullptr, a.k = p->Hk ? k : nullptr;
    a.gq = p->Hq ? dq_out : nullptr, a.gk = p->Hk ? dk_out : nullptr;
    a.ldgq = ld_or(p->ld_qo, dense_q), a.ldgk = ld_or(p->ld_ko, dense_k);
    a.oq = p->Hq ? dq : nullptr, a.ok = p->Hk ? dk : nullptr;
    a.ldoq = dense_q, a.ldok = dense_k;
    if (sums) a.part = static_cast<float*>(ws);
    a.dwq = dwq, a.dwk = dwk;
    launch_any<true>(a, p->layout, p->dtype, st);
    return launched();
}

kda_status kda_rope_frequencies(int32_t R, double base, int scaling, double factor, double trained, double slow,
                                double fast, double* freq, float* scale) {
    if (R < 0 || R % 2 || R > RP_MAXD || !(base > 0.0) || !isfinite(base) || (R > 0 && !freq)) return KDA_ERR_INVALID_ARG;
    if (scaling < KDA_ROPE_PLAIN || scaling > KDA_ROPE_RAMP) return KDA_ERR_INVALID_ARG;
    if (scaling != KDA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return KDA_ERR_INVALID_ARG;
    if (scaling == KDA_ROPE_RAMP && (!(trained > 0.0) || !(slow >= 0.0) || !(fast > slow))) return KDA_ERR_INVALID_ARG;
    if (scaling == KDA_ROPE_BASE) base *= pow(factor, double(R) / double(R > 2 ? R - 2 : 1));
    const double two_pi = 6.283185307179586;
    for (int i = 0; i < R / 2; ++i) {
        double f = pow(base, -2.0 * i / R);
        if (scaling == KDA_ROPE_LINEAR) f /= factor;
        if (scaling == KDA_ROPE_RAMP) {
            const double keep = fmin(fmax((trained * f / two_pi - slow) / (fast - slow), 0.0), 1.0);
            f = f * keep + f / factor * (1.0 - keep);
        }
        freq[i] = f;
    }
    if (scale) *scale = scaling == KDA_ROPE_RAMP ? float(0.1 * log(factor) + 1.0) : 1.f;
    return KDA_OK;
}

}  // extern "C"
