// Norm of every head's queries and keys and their rotation to positions, forward and backward.
//
//   xh = x / sqrt(sum_c x_c^2 / D + eps),  n = xh w             (norm; else n = x)
//   y  = scale R(pos freq) n on the first R channels, in pairs, n on the others
//   backward:  d = the turn undone on dy (scale kept),  dw = sum_rows d xh,  g = d w
//              dx = (g - xh sum_c(g xh) / D) / sqrt(..)          (norm; else dx = d)
//   sum x^2 and sum g x go through one exchange: dx = rs (g - xh rs sum(g x) / D) with rs = 1 / sqrt(..) (rs^3 leaves fp32 where
//   rs, xh and the gradient do not)
//
// Bound by HBM: forward 2, backward 3 (2 without the norm) row transfers.  A row of D channels belongs to a
// group of lanes that each hold 8 pairs (4 of fp32) as two 16-byte accesses; both members of a pair lie in one lane, so
// the turn needs no exchange, and the norm's sum is one exchange over the group.  A block takes a tile of tokens of
// one of the two tensors: its threads compute the tile's cosines and sines once, a group keeps those of one
// token and the weights in registers and walks the token's heads.  The rows come through a ring in shared memory that
// cp.async fills ahead, over the ends of tiles too; a thread copies exactly the bytes that it reads, so the ring needs no
// barrier.
// 16384 tokens x 2 x 64 heads of 128 channels, bf16: forward and backward 466 us, 5.7 TB/s, 85% of the measured HBM peak:
// what is left is instructions, 16 warps a multiprocessor at 120 registers.  In a loop on the same tensors (16384 x 2 x 64 heads,
// forward / backward in shares of that peak): 128 channels 81 / 81%, half of them turned 82 / 83%, fp32 84 / 85%, 96 channels 85 / 61%
// (6 of a group's 8 lanes), 80 70 / 51%, 144 65 / 48%, 52 of 80 (8-byte packs) 51 / 33%, single pairs picked out of words
// 126 41 / 28% (neighbours 54 / 40%), 50 34 / 21% (44 / 31%), 130 25 / 18% (33 / 26%: 65 of 128 places).
//
// Angles.  A position times a frequency in fp32 is off by a thousandth of a turn at position 10^4 already.
// Here a frequency is a 64-bit fraction of a turn per token, F = freq / (2 pi) 2^64 mod 2^64, so pos F mod
// 2^64 is the angle's fraction of a turn, exact for any 32-bit position but for F's own rounding (below
// 2^-53 freq / 2 pi a token: 10^-10 turns at position 10^6); its upper 32 bits go through sincospif.
#include <math.h>

#include "kda_ssm.cuh"

namespace kda {

namespace {

// One tensor: q or k
struct RopeSide {
    const void *x, *g;  // input; gradient of the output (backward)
    void* out;
    const float* w;
    float* dw;
    int64_t ldx, ldg, ldo;  // token strides
    int H;
    int per_token;      // groups of a block that share a token's heads
    int blocks;         // of the launch
    float* part;        // [blocks][D] partial dw
};
struct RopeArgs {
    int64_t T;
    int D, R, norm;
    float eps, scale, inv_d;
    const int* pos;
    const double* freq;
    RopeSide side[2];
};

constexpr int RP_THREADS = 256;
constexpr int RP_MAXD = 256;
constexpr int RP_TOKENS = 16;  // most tokens of a tile

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

template <class E> __device__ __forceinline__ E rp_cast(float v);
template <> __device__ __forceinline__ float rp_cast<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rp_cast<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rp_cast<__half>(float v) { return __float2half_rn(v); }
// Two neighbours of a 16-bit type as the word that they are, one instruction each way (element by element it is three)
template <class E> __device__ __forceinline__ float word_lo(uint32_t w);
template <class E> __device__ __forceinline__ float word_hi(uint32_t w);
template <class E> __device__ __forceinline__ uint32_t word_of(float lo, float hi);
template <> __device__ __forceinline__ float word_lo<__nv_bfloat16>(uint32_t w) { return __uint_as_float(w << 16); }
template <> __device__ __forceinline__ float word_hi<__nv_bfloat16>(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
template <> __device__ __forceinline__ uint32_t word_of<__nv_bfloat16>(float lo, float hi) { return pack2(lo, hi); }
__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
template <> __device__ __forceinline__ float word_lo<__half>(uint32_t w) { return __low2float(as_half2(w)); }
template <> __device__ __forceinline__ float word_hi<__half>(uint32_t w) { return __high2float(as_half2(w)); }
template <> __device__ __forceinline__ uint32_t word_of<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// N consecutive elements: words where they fill them
template <class E, int N> struct alignas(N * sizeof(E)) Pack { uint32_t w[N * sizeof(E) / 4]; };
template <> struct alignas(2) Pack<__nv_bfloat16, 1> { __nv_bfloat16 e; };
template <> struct alignas(2) Pack<__half, 1> { __half e; };
template <class E, int N>
__device__ __forceinline__ float pack_get(const Pack<E, N>& p, int i) {
    if constexpr (sizeof(E) == 4) return __uint_as_float(p.w[i]);
    else if constexpr (N == 1) return ssm_f<E>(p.e);
    else return i & 1 ? word_hi<E>(p.w[i / 2]) : word_lo<E>(p.w[i / 2]);
}
// elements i and i + 1
template <class E, int N>
__device__ __forceinline__ void pack_put2(Pack<E, N>& p, int i, float a, float b) {
    if constexpr (sizeof(E) == 4) p.w[i] = __float_as_uint(a), p.w[i + 1] = __float_as_uint(b);
    else p.w[i / 2] = word_of<E>(a, b);
}
template <class E>
__device__ __forceinline__ Pack<E, 1> pack_one(float a) {
    Pack<E, 1> p;
    if constexpr (sizeof(E) == 4) p.w[0] = __float_as_uint(a);
    else p.e = rp_cast<E>(a);
    return p;
}

// Channels of pair p of a row (p >= R / 2: channels that are not turned, two by two)
__device__ __forceinline__ void pair_at(int p, int R, bool pairs, int& a, int& b) {
    if (p < R / 2 && !pairs) a = p, b = R / 2 + p;
    else a = 2 * p, b = 2 * p + 1;
}

// A lane's row: NP pairs (x, y), two to a register pair
template <int NP> struct Row { f2 x[NP / 2], y[NP / 2]; };

// The channels of a lane: U units, unit u the (l + u G)-th of its row, of two packs of N channels each, so that
// neighbouring lanes' packs are neighbours in memory.  Halves: the first and the second members of N pairs (units past
// R: channels of each half of the rest, which is not turned).  Pairs: the pairs of N channels in each half of the row.
// N = 1: one pair, wherever its members lie.
template <class E, int N, int U, bool PAIRS>
struct Lane {
    static constexpr int NP = N * U;  // pairs of a lane
    int o0[U], o1[U];
    int l, D, R, G;
    __device__ __forceinline__ Lane(int lane, int D_, int R_, int G_) : l(lane), D(D_), R(R_), G(G_) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = l + u * G;
            if (N == 1) {
                pair_at(j, R, PAIRS, o0[u], o1[u]);
            } else {
                const bool turned = 2 * N * j < R;
                o0[u] = PAIRS || turned ? N * j : R + N * j - R / 2;
                o1[u] = PAIRS ? D / 2 + N * j : turned ? R / 2 + N * j : R + (D - R) / 2 + N * j - R / 2;
            }
        }
    }
    __device__ __forceinline__ bool on(int u) const { return 2 * N * (l + u * G) < D; }
    __device__ __forceinline__ bool has(int i) const { return on(i / N); }
    // the pair of the rotation that pair i of the lane is (where it turns)
    __device__ __forceinline__ int pair(int i) const {
        const int u = i / N, e = i % N;
        if (N == 1 || !PAIRS) return N * (l + u * G) + e;
        return (2 * e < N ? o0[u] : o1[u]) / 2 + e % (N / 2 > 0 ? N / 2 : 1);
    }
    __device__ __forceinline__ bool turns(int i) const {
        const int u = i / N, e = i % N;
        if (N == 1 || !PAIRS) return 2 * N * (l + u * G) < R;
        return (2 * e < N ? o0[u] : o1[u]) < R;
    }
    // of pairs 2 i and 2 i + 1 of narrow packs: turned where they turn, else plain
    __device__ __forceinline__ f2 pick(int i, f2 turned, f2 plain) const {
        float t0, t1, p0, p1;
        up2(turned, t0, t1);
        up2(plain, p0, p1);
        return pk2(turns(2 * i) ? t0 : p0, turns(2 * i + 1) ? t1 : p1);
    }
    // the channels of pair i's members
    __device__ __forceinline__ void channels(int i, int& a, int& b) const {
        const int u = i / N, e = i % N;
        if (N == 1) a = o0[u], b = o1[u];
        else if (!PAIRS) a = o0[u] + e, b = o1[u] + e;
        else a = (2 * e < N ? o0[u] : o1[u]) + 2 * (e % (N / 2 > 0 ? N / 2 : 1)), b = a + 1;
    }
    struct Raw { Pack<E, N> a[U], b[U]; };
    // straight from memory (single pairs)
    __device__ __forceinline__ Raw load(const void* base, int64_t at, bool use) const {
        Raw r;
        const E* p = static_cast<const E*>(base) + at;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            r.a[u] = r.b[u] = Pack<E, N>{};
            if (on(u) && use) {
                r.a[u] = *reinterpret_cast<const Pack<E, N>*>(p + o0[u]);
                r.b[u] = *reinterpret_cast<const Pack<E, N>*>(p + o1[u]);
            }
        }
        return r;
    }
    __device__ __forceinline__ Row<NP> values(const Raw& r) const {
        Row<NP> v;
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            const int u = 2 * i / N, e = 2 * i % N;
            if constexpr (N == 1) {
                v.x[i] = pk2(pack_get<E, N>(r.a[2 * i], 0), pack_get<E, N>(r.a[2 * i + 1], 0));
                v.y[i] = pk2(pack_get<E, N>(r.b[2 * i], 0), pack_get<E, N>(r.b[2 * i + 1], 0));
            } else if constexpr (PAIRS && N == 2) {  // one pair a pack
                v.x[i] = pk2(pack_get<E, N>(r.a[u], 0), pack_get<E, N>(r.b[u], 0));
                v.y[i] = pk2(pack_get<E, N>(r.a[u], 1), pack_get<E, N>(r.b[u], 1));
            } else if constexpr (PAIRS) {
                const Pack<E, N>& n = 2 * e < N ? r.a[u] : r.b[u];
                const int k = 2 * e % N;
                v.x[i] = pk2(pack_get<E, N>(n, k), pack_get<E, N>(n, k + 2));
                v.y[i] = pk2(pack_get<E, N>(n, k + 1), pack_get<E, N>(n, k + 3));
            } else {
                v.x[i] = pk2(pack_get<E, N>(r.a[u], e), pack_get<E, N>(r.a[u], e + 1));
                v.y[i] = pk2(pack_get<E, N>(r.b[u], e), pack_get<E, N>(r.b[u], e + 1));
            }
        }
        return v;
    }
    __device__ __forceinline__ void store(void* base, int64_t at, const Row<NP>& v) const {
        E* p = static_cast<E*>(base) + at;
        float x[NP], y[NP];
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            up2(v.x[i], x[2 * i], x[2 * i + 1]);
            up2(v.y[i], y[2 * i], y[2 * i + 1]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!on(u)) continue;
            Pack<E, N> a, b;
            if constexpr (N == 1) {
                a = pack_one<E>(x[u]), b = pack_one<E>(y[u]);
            } else {
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    const int i = u * N + e, k = u * N + e / 2;
                    if (PAIRS) {
                        pack_put2<E, N>(a, e, x[k], y[k]);
                        pack_put2<E, N>(b, e, x[k + N / 2], y[k + N / 2]);
                    } else {
                        pack_put2<E, N>(a, e, x[i], x[i + 1]);
                        pack_put2<E, N>(b, e, y[i], y[i + 1]);
                    }
                }
            }
            *reinterpret_cast<Pack<E, N>*>(p + o0[u]) = a;
            *reinterpret_cast<Pack<E, N>*>(p + o1[u]) = b;
        }
    }
    // fp32 parameters of the lane's channels (w null: ones)
    __device__ __forceinline__ Row<NP> weights(const float* w) const {
        Row<NP> v;
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            float t[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int ca, cb;
                channels(2 * i + e, ca, cb);
                if (w && has(2 * i + e)) t[e] = w[ca], t[2 + e] = w[cb];
            }
            v.x[i] = pk2(t[0], t[1]);
            v.y[i] = pk2(t[2], t[3]);
        }
        return v;
    }
};

template <int BYTES>
__device__ __forceinline__ void cp_bytes(void* smem, const void* gmem) {
    if constexpr (BYTES == 16) cp16(smem, gmem);
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(smem_u32(smem)), "l"(gmem), "n"(BYTES));
}

template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int G) {
    for (int o = G >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
__device__ __forceinline__ float both_sum(f2 v) {
    float a, b;
    up2(v, a, b);
    return a + b;
}
__device__ __forceinline__ f2 twice(float x) { return pk2(x, x); }

// Rows ahead in the ring, and blocks of a multiprocessor that its shared memory is sized for
template <bool BWD> constexpr int rp_depth() { return BWD ? 4 : 8; }
constexpr int RP_OCCUPANCY = 2;
// words of a lane's single pairs, and one more that keeps the groups' rows in banks of their own
template <class E, int U> constexpr int rp_words() { return U * int(sizeof(E)) / 2; }
template <bool BWD> constexpr size_t rp_smem(int row_bytes) {  // bytes of both packs of a lane's units
    return size_t(rp_depth<BWD>()) * (BWD ? 2 : 1) * row_bytes * RP_THREADS;
}

// BWD: inputs and gradients in, gradients out; otherwise inputs in, turned out.  The first side[0].blocks blocks do q, the
// others k.  tokens = groups / per_token tokens a tile.
// STAY (wide packs): some channels do not turn.  They are passed on, not turned by 1 and 0, which would take 0 times an infinity into
// another channel of no pair with it.  Wide packs turn as a whole or not at all; where all turn, the test would cost 5% of the
// backward.  Narrow packs pick member by member.
// AHEAD: rows come through the ring, for N = 1 as whole words of which a group's lanes then pick their pairs, and go out as
// words too; else (rows that no word fits) element by element.
template <class E, int N, int U, bool PAIRS, bool BWD, bool AHEAD, bool STAY>
__global__ void __launch_bounds__(RP_THREADS, RP_OCCUPANCY) k_rope(RopeArgs a, int G) {
    using P = Pack<E, N>;
    constexpr int NP = N * U;
    constexpr bool RING = AHEAD && N > 1, WORDS = AHEAD && N == 1;
    constexpr int WU = rp_words<E, U>();
    constexpr int DEPTH = rp_depth<BWD>(), ROWS = BWD ? 1 : 2;  // ROWS rows of a group are worked on together
    extern __shared__ __align__(16) unsigned char ring_raw[];
    P* ring = reinterpret_cast<P*>(ring_raw);  // [DEPTH][x, then g: two packs of every unit][thread]
    __shared__ __align__(16) float cs[RP_TOKENS][RP_MAXD];  // cosines of R / 2 pairs, then sines
    __shared__ unsigned long long turn[RP_MAXD / 2];        // turns_per_token of the pairs
    __shared__ int place[RP_TOKENS];                        // the tile's positions
    const int tid = threadIdx.x, lane = tid & (G - 1), groups = RP_THREADS / G, group = tid / G;
    const int which = int(blockIdx.x) >= a.side[0].blocks;
    const RopeSide& sd = a.side[which];
    const int block = int(blockIdx.x) - (which ? a.side[0].blocks : 0);
    const Lane<E, N, U, PAIRS> L(lane, a.D, a.R, G);
    const int half = a.R / 2, tokens = groups / sd.per_token;
    const int own = group / sd.per_token, first = group - own * sd.per_token;
    const int rows = (sd.H + ROWS * sd.per_token - 1) / (ROWS * sd.per_token) * ROWS;  // of a group in a tile
    const Row<NP> w = L.weights(a.norm ? sd.w : nullptr);
    Row<NP> sum;  // of dw
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) sum.x[i] = sum.y[i] = twice(0.f);
    const int64_t tiles = (a.T + tokens - 1) / tokens;
    const bool some_stay = N <= 2 && a.R < a.D;
    auto slot = [&](int d, int k, int u) { return ring + ((d * (BWD ? 4 : 2) + k) * U + u) * RP_THREADS + tid; };
    // WORDS: [DEPTH][x, then g][group][word], then a row of every group on its way out
    const int row_words = a.D * int(sizeof(E)) / 4;
    auto words = [&](int d, int k) {
        return reinterpret_cast<uint32_t*>(ring_raw) + ((d * (BWD ? 2 : 1) + k) * groups + group) * (G * (WU + 1));
    };
    // the next row to be copied (its tile, place in the tile, head and addresses), and its place in the ring
    const int step = sd.per_token * a.D;  // elements from a group's row to its next
    int64_t ahead = block;
    int ahead_row = 0, ahead_at = 0;
    const E *ahead_x = nullptr, *ahead_g = nullptr;
    int ahead_heads = 0;  // rows that the group has in the tile
    auto copy_next = [&]() {
        if constexpr (AHEAD) {
            if (ahead_row == 0) {
                const int64_t t = ahead * tokens + own;
                ahead_heads = ahead < tiles && t < a.T ? (sd.H - first + sd.per_token - 1) / sd.per_token : 0;
                if (!BWD || a.norm) ahead_x = static_cast<const E*>(sd.x) + t * sd.ldx + int64_t(first) * a.D;
                if (BWD) ahead_g = static_cast<const E*>(sd.g) + t * sd.ldg + int64_t(first) * a.D;
            }
            if (ahead_row < ahead_heads) {
                const E *x = ahead_x, *g = ahead_g;
                if constexpr (WORDS) {
#pragma unroll
                    for (int i = 0; i < WU; ++i) {
                        const int k = lane + i * G;
                        if (k < row_words) {
                            if (!BWD || a.norm) cp_bytes<4>(words(ahead_at, 0) + k, reinterpret_cast<const uint32_t*>(x) + k);
                            if constexpr (BWD) cp_bytes<4>(words(ahead_at, 1) + k, reinterpret_cast<const uint32_t*>(g) + k);
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (RING && L.on(u)) {
                        if (!BWD || a.norm) {
                            cp_bytes<sizeof(P)>(slot(ahead_at, 0, u), x + L.o0[u]);
                            cp_bytes<sizeof(P)>(slot(ahead_at, 1, u), x + L.o1[u]);
                        }
                        if constexpr (BWD) {
                            cp_bytes<sizeof(P)>(slot(ahead_at, 2, u), g + L.o0[u]);
                            cp_bytes<sizeof(P)>(slot(ahead_at, 3, u), g + L.o1[u]);
                        }
                    }
            }
            cp_commit();
            ahead_at = ahead_at + 1 == DEPTH ? 0 : ahead_at + 1;
            ahead_x += step;
            ahead_g += step;
            if (++ahead_row == rows) ahead_row = 0, ahead += sd.blocks;
        }
    };
    for (int d = 0; d < DEPTH; ++d) copy_next();
    int at = 0;
    // positions are read a tile ahead: the cosines and sines of a tile wait for no load
    auto position = [&](int64_t tile) { return tid < tokens && tile * tokens + tid < a.T ? a.pos[tile * tokens + tid] : 0; };
    int bad = 0;
    for (int i = tid; i < half; i += RP_THREADS) {
        const double f = a.freq[i];
        turn[i] = turns_per_token(f);
        bad |= !isfinite(f);
    }
    const bool broken = __syncthreads_or(bad);  // no number among the frequencies: its pairs' angles are none
    int next = position(block);
    for (int64_t tile = block; tile < tiles; tile += sd.blocks) {
        if (tid < tokens) place[tid] = next;
        __syncthreads();
        for (int i = tid; i < tokens * half; i += RP_THREADS) {
            const int t = i / half, k = i - t * half;
            cos_sin(place[t], turn[k], a.scale, cs[t][k], cs[t][half + k]);
        }
        if (broken)
            for (int i = tid; i < tokens * half; i += RP_THREADS) {
                const int t = i / half, k = i - t * half;
                if (!isfinite(a.freq[k])) cs[t][k] = cs[t][half + k] = __int_as_float(0x7fffffff);
            }
        next = position(tile + sd.blocks);
        __syncthreads();
        const int64_t t = tile * tokens + own;
        const bool live = t < a.T;
        f2 c[NP / 2], s[NP / 2];
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
            float u[4] = {1.f, 1.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (L.has(2 * i + e) && L.turns(2 * i + e))
                    u[e] = cs[own][L.pair(2 * i + e)], u[2 + e] = cs[own][half + L.pair(2 * i + e)];
            c[i] = pk2(u[0], u[1]);
            s[i] = pk2(u[2], u[3]);
        }
        const int64_t x0 = t * sd.ldx, g0 = t * sd.ldg;
        E* out = static_cast<E*>(sd.out) + t * sd.ldo + int64_t(first) * a.D;  // of the next row
        // (every lane of a warp runs every round: the exchanges are warp-wide)
        for (int r0 = 0; r0 < rows; r0 += ROWS) {
            typename Lane<E, N, U, PAIRS>::Raw x[ROWS], g[ROWS];
            if constexpr (AHEAD) cp_wait<DEPTH - ROWS>();
            if constexpr (WORDS) __syncwarp();  // the other lanes' words
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int h = (r0 + r) * sd.per_token + first;
                const bool use = live && h < sd.H;
                if constexpr (RING) {
                    const P none{};
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool full = use && L.on(u);  // (else what the ring holds is of no row)
                        if (!BWD || a.norm) x[r].a[u] = full ? *slot(at, 0, u) : none, x[r].b[u] = full ? *slot(at, 1, u) : none;
                        if constexpr (BWD) g[r].a[u] = full ? *slot(at, 2, u) : none, g[r].b[u] = full ? *slot(at, 3, u) : none;
                    }
                    at = at + 1 == DEPTH ? 0 : at + 1;
                } else if constexpr (WORDS) {
                    const P *px = reinterpret_cast<const P*>(words(at, 0)), *pg = reinterpret_cast<const P*>(words(at, BWD ? 1 : 0));
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const bool full = use && L.on(u);
                        const P none{};
                        x[r].a[u] = x[r].b[u] = none;
                        if (full && (!BWD || a.norm)) x[r].a[u] = px[L.o0[u]], x[r].b[u] = px[L.o1[u]];
                        if constexpr (BWD) {
                            g[r].a[u] = g[r].b[u] = none;
                            if (full) g[r].a[u] = pg[L.o0[u]], g[r].b[u] = pg[L.o1[u]];
                        }
                    }
                    at = at + 1 == DEPTH ? 0 : at + 1;
                } else {
                    if (!BWD || a.norm) x[r] = L.load(sd.x, x0 + int64_t(h) * a.D, use);
                    if (BWD) g[r] = L.load(sd.g, g0 + int64_t(h) * a.D, use);
                }
            }
            if constexpr (WORDS) __syncwarp();  // read by every lane, before the places are filled again
            Row<NP> v[ROWS], o[ROWS];
            float all[2 * ROWS];  // the rows' sums over channels: x^2, and g x (backward)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                if (!BWD || a.norm) v[r] = L.values(x[r]);
                f2 xx = twice(0.f), gx = twice(0.f);
                if (a.norm)
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) xx = fma2(v[r].x[i], v[r].x[i], fma2(v[r].y[i], v[r].y[i], xx));
                if constexpr (BWD) {  // the turn undone
                    o[r] = L.values(g[r]);
                    auto undo = [&](int i) {
                        const f2 p = o[r].x[i], z = o[r].y[i];
                        o[r].x[i] = fma2(p, c[i], mul2(z, s[i]));
                        o[r].y[i] = fma2(mul2(p, s[i]), twice(-1.f), mul2(z, c[i]));
                        if (some_stay) o[r].x[i] = L.pick(i, o[r].x[i], p), o[r].y[i] = L.pick(i, o[r].y[i], z);
                    };
                    if constexpr (STAY) {
#pragma unroll
                        for (int i = 0; i < NP / 2; ++i)
                            if (L.turns(2 * i)) undo(i);
                    }
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) {
                        if (!STAY) undo(i);
                        if (a.norm) gx = fma2(mul2(o[r].x[i], w.x[i]), v[r].x[i], fma2(mul2(o[r].y[i], w.y[i]), v[r].y[i], gx));
                    }
                }
                all[r] = both_sum(xx);
                all[ROWS + r] = BWD ? both_sum(gx) : 0.f;
            }
            if (a.norm) {
                if constexpr (BWD) {
                    group_sums<2 * ROWS>(all, G);
                } else {
                    float xx[ROWS];
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) xx[r] = all[r];
                    group_sums<ROWS>(xx, G);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) all[r] = xx[r];
                }
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int h = (r0 + r) * sd.per_token + first;
                const bool use = live && h < sd.H;
                // (no row, no part in dw: without an eps its 1 / sqrt(0) would be one)
                const float rs = !BWD || use ? rsqrtf(fmaf(all[r], a.inv_d, a.eps)) : 0.f;
                const f2 rs2 = twice(rs);
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) {
                        f2 p = v[r].x[i], z = v[r].y[i];
                        if (a.norm) p = mul2(p, mul2(w.x[i], rs2)), z = mul2(z, mul2(w.y[i], rs2));
                        o[r].x[i] = p;
                        o[r].y[i] = z;
                        if (!STAY || L.turns(2 * i)) {
                            o[r].x[i] = fma2(p, c[i], mul2(mul2(z, s[i]), twice(-1.f)));
                            o[r].y[i] = fma2(p, s[i], mul2(z, c[i]));
                        }
                        if (some_stay) o[r].x[i] = L.pick(i, o[r].x[i], p), o[r].y[i] = L.pick(i, o[r].y[i], z);
                    }
                } else if (a.norm) {
                    const f2 k = twice(-rs * all[ROWS + r] * a.inv_d);
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) {
                        const f2 xh = mul2(v[r].x[i], rs2), yh = mul2(v[r].y[i], rs2);
                        sum.x[i] = fma2(o[r].x[i], xh, sum.x[i]);
                        sum.y[i] = fma2(o[r].y[i], yh, sum.y[i]);
                        o[r].x[i] = mul2(fma2(xh, k, mul2(o[r].x[i], w.x[i])), rs2);
                        o[r].y[i] = mul2(fma2(yh, k, mul2(o[r].y[i], w.y[i])), rs2);
                    }
                }
                copy_next();  // into a place just read
                if constexpr (WORDS) {
                    uint32_t* row = words(DEPTH, 0);
                    L.store(row, 0, o[r]);
                    __syncwarp();
                    uint32_t* to = reinterpret_cast<uint32_t*>(out);
#pragma unroll
                    for (int i = 0; i < WU; ++i)
                        if (use && lane + i * G < row_words) to[lane + i * G] = row[lane + i * G];
                    __syncwarp();
                } else if (use) {
                    L.store(out, 0, o[r]);
                }
                out += step;
            }
        }
    }
    if constexpr (AHEAD) cp_wait<0>();
    if (BWD && sd.part) {  // the groups' sums, added in their order
        float* red = &cs[0][0];
        for (int gi = 0; gi < groups; ++gi) {
            __syncthreads();
            if (group == gi) {
#pragma unroll
                for (int i = 0; i < NP / 2; ++i) {
                    float u[4];
                    up2(sum.x[i], u[0], u[1]);
                    up2(sum.y[i], u[2], u[3]);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (L.has(2 * i + e)) {
                            int ca, cb;
                            L.channels(2 * i + e, ca, cb);
                            red[ca] = gi ? red[ca] + u[e] : u[e];
                            red[cb] = gi ? red[cb] + u[2 + e] : u[2 + e];
                        }
                }
            }
        }
        __syncthreads();
        for (int i = tid; i < a.D; i += RP_THREADS) sd.part[int64_t(block) * a.D + i] = red[i];
    }
}

// dwq and dwk: the blocks' sums, one warp per channel, in an order that depends on their number alone
__global__ void __launch_bounds__(256) k_rope_reduce(RopeArgs a) {
    const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const RopeSide& sd = a.side[blockIdx.y];
    if (c >= a.D || !sd.dw) return;
    float v = 0.f;
    for (int b = lane; b < sd.blocks; b += 32) v += sd.part[int64_t(b) * a.D + c];
    v = warp_sum(v);
    if (lane == 0) sd.dw[c] = v;
}

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t esize(int dtype) { return dtype == KDA_DT_FP32 ? 4 : 2; }
int64_t ld_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

constexpr int RP_SMS = 152;  // multiprocessors: a launch has one wave of blocks at most (and one more block)
constexpr int RP_MAXBLOCKS = RP_SMS * 2;

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

template <class E, int N, int U, bool BWD, bool AHEAD>
void launch_as(RopeArgs a, bool pairs, cudaStream_t st) {
    int G = 1;
    while (G < 32 && G * 2 * N * (AHEAD ? U : 1) < a.D) G *= 2;  // (straight from memory: as many lanes as there are pairs)
    const int groups = RP_THREADS / G, all = a.side[0].H + a.side[1].H;
    constexpr int most = RP_SMS * RP_OCCUPANCY;
    for (RopeSide& s : a.side) {
        // blocks in proportion to the heads
        const int64_t share = (int64_t(most) * s.H + all - 1) / all;
        // a group takes 8 heads of a token, fewer where that leaves blocks without a tile; tiles of at most RP_TOKENS tokens
        int per = 1;
        while (per < groups && (groups / per > RP_TOKENS || s.H > 8 * per)) per *= 2;
        while (per < groups && per < s.H && a.T * per < share * groups) per *= 2;
        const int64_t tiles = (a.T + groups / per - 1) / (groups / per);
        s.per_token = per;
        s.blocks = int(s.H == 0 ? 0 : share < tiles ? share : tiles);
    }
    if (a.side[1].part) a.side[1].part = a.side[0].part + size_t(a.side[0].blocks) * a.D;
    const unsigned grid = unsigned(a.side[0].blocks + a.side[1].blocks);
    {
        static unsigned long long done[4];
        const size_t smem = !AHEAD ? 0 : N > 1 ? rp_smem<BWD>(2 * U * int(sizeof(Pack<E, N>)))
                                               : rp_smem<BWD>(4 * (rp_words<E, U>() + 1)) + 4 * (rp_words<E, U>() + 1) * RP_THREADS;
        constexpr bool WIDE = N > 2;
        const bool stay = WIDE && a.R < a.D;
        auto* kernel = pairs ? (stay ? k_rope<E, N, U, true, BWD, AHEAD, WIDE> : k_rope<E, N, U, true, BWD, AHEAD, false>)
                             : (stay ? k_rope<E, N, U, false, BWD, AHEAD, WIDE> : k_rope<E, N, U, false, BWD, AHEAD, false>);
        // (the limit counts the static part too)
        allow_smem(reinterpret_cast<const void*>(kernel), smem + RP_TOKENS * RP_MAXD * sizeof(float), &done[2 * stay + pairs]);
        ProfScope ps(BWD ? KK_ROPE_BWD : KK_ROPE_FWD, st);
        kernel<<<grid, RP_THREADS, smem, st>>>(a, G);
    }
    if (BWD && a.side[0].part) {
        ProfScope ps(KK_ROPE_REDUCE, st);
        k_rope_reduce<<<dim3((a.D + 7) / 8, 2), 256, 0, st>>>(a);
    }
}

template <class E, bool BWD>
void launch(const RopeArgs& a, int layout, cudaStream_t st) {
    constexpr int V = 16 / int(sizeof(E));
    // the widest packs that the channels and every row allow: 16 bytes a lane, or several units of 8 or 4, or pairs
    // one at a time
    auto fits = [&](int n, bool whole) {  // whole: rows of words, whatever the turned part
        if (!whole && (a.D % (2 * n) || a.R % (2 * n))) return false;
        for (const RopeSide& s : a.side)
            if (s.H && (!al(s.x, n * sizeof(E)) || s.ldx % n || !al(s.g, n * sizeof(E)) || s.ldg % n ||
                        !al(s.out, n * sizeof(E)) || s.ldo % n))
                return false;
        return true;
    };
    const bool pairs = layout == KDA_ROPE_PAIRS;
    if (fits(V, false)) launch_as<E, V, 1, BWD, true>(a, pairs, st);
    else if (V == 8 && fits(4, false)) launch_as<E, 4, V / 4, BWD, true>(a, pairs, st);
    else if (fits(2, false)) launch_as<E, 2, V / 2, BWD, true>(a, pairs, st);
    else if (sizeof(E) == 4 || fits(2, true)) launch_as<E, 1, V, BWD, true>(a, pairs, st);  // (fp32 rows are words at any address)
    else if constexpr (sizeof(E) == 2) launch_as<E, 1, 4, BWD, false>(a, pairs, st);
}

template <bool BWD>
void launch_any(const RopeArgs& a, int layout, int dtype, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) launch<__nv_bfloat16, BWD>(a, layout, st);
    else if (dtype == KDA_DT_FP16) launch<__half, BWD>(a, layout, st);
    else launch<float, BWD>(a, layout, st);
}

RopeArgs make_args(const kda_rope_problem* p, const int32_t* pos, const double* freq, const float* wq, const float* wk) {
    RopeArgs a{};
    a.T = p->T, a.D = p->D, a.R = p->R, a.norm = p->norm;
    a.eps = p->eps, a.scale = p->scale, a.inv_d = 1.f / float(p->D);
    a.pos = pos, a.freq = freq;
    a.side[0].H = p->Hq, a.side[1].H = p->Hk;
    a.side[0].w = wq, a.side[1].w = wk;
    a.side[0].ldx = ld_or(p->ld_q, int64_t(p->Hq) * p->D), a.side[1].ldx = ld_or(p->ld_k, int64_t(p->Hk) * p->D);
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
    return p->norm ? size_t(RP_MAXBLOCKS + 1) * size_t(p->D) * 4 : 0;
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
    a.side[0].x = q, a.side[1].x = k;
    a.side[0].out = q_out, a.side[1].out = k_out;
    a.side[0].ldo = ld_or(p->ld_qo, int64_t(p->Hq) * p->D), a.side[1].ldo = ld_or(p->ld_ko, int64_t(p->Hk) * p->D);
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
    if (p->norm) a.side[0].x = q, a.side[1].x = k;
    else a.side[0].ldx = a.side[1].ldx = 0;  // (not read: no bar to wide accesses)
    a.side[0].g = dq_out, a.side[1].g = dk_out;
    a.side[0].ldg = ld_or(p->ld_qo, dense_q), a.side[1].ldg = ld_or(p->ld_ko, dense_k);
    a.side[0].out = dq, a.side[1].out = dk;
    a.side[0].ldo = dense_q, a.side[1].ldo = dense_k;
    if (sums) a.side[0].part = a.side[1].part = static_cast<float*>(ws);
    a.side[0].dw = dwq, a.side[1].dw = dwk;
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
