// Layer norm over rows of C channels, forward and backward.
//
//   v = x + res (rounded to the row type, as it is handed on; v = x without res)
//   mean = sum v / C,  rstd = 1 / sqrt(sum (v - mean)^2 / C + eps),  xh = (v - mean) rstd
//   y = xh w + b
//   d = dy w:  dv = rstd (d - mean(d) - xh mean(d xh)) + dsum,  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: forward 2 (4 with res) and backward 3 (4 with dsum) row transfers.  A row is held in
// the registers of a warp or of a block, so it is read once and the variance is taken about the mean
// (no cancellation).  Where there are rows enough, a block walks many of them: w and b (fp32: twice a
// bf16 row's bytes each) stay in registers, and the rows come through a ring in shared memory that
// cp.async fills ahead.  A thread copies exactly the vectors that it reads, so the ring needs no
// barrier.  Two rows at a time share the exchange of their sums, and the arithmetic runs on pairs of
// values.  The backward keeps its columns' dw and db terms in registers over the rows of its walk, and
// a second kernel adds the blocks' sums in order: results are bitwise reproducible.  Rows too long
// for the registers take kernels that read them again.
#include "kda_ssm.cuh"

namespace kda {

namespace {

struct LnArgs {
    int64_t T;
    int C;
    float eps;
    const void *x, *res, *dy, *dsum;
    const float *w, *b, *mean_in, *rstd_in;
    void *sum, *y, *dx;
    float *mean, *rstd;
    float* part;  // [parts][2][C] partial dw, db
    int parts;    // slots that the rows of a walk are dealt to
};

// V consecutive elements (one 16-byte access when V > 1)
template <class E, int V>
struct alignas(V > 1 ? 16 : sizeof(E)) Vec {
    E e[V];
};
template <class E, int V>
__device__ __forceinline__ Vec<E, V> ln_load(const void* p, int64_t i) {
    return *reinterpret_cast<const Vec<E, V>*>(static_cast<const E*>(p) + i);
}
template <class E, int V>
__device__ __forceinline__ void ln_store(void* p, int64_t i, const Vec<E, V>& r) {
    *reinterpret_cast<Vec<E, V>*>(static_cast<E*>(p) + i) = r;
}
template <class E> __device__ __forceinline__ E ln_cast(float v);
template <> __device__ __forceinline__ float ln_cast<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 ln_cast<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half ln_cast<__half>(float v) { return __float2half_rn(v); }

// Arithmetic on pairs of values (one packed instruction for two), on single values where rows are not
// whole vectors
using kda::add2;  // (the single-value forms below would hide the pairs')
using kda::fma2;
using kda::mul2;
__device__ __forceinline__ float mul2(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float add2(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float total(float v) { return v; }
__device__ __forceinline__ float total(f2 v) { return hsum2(v); }
template <int V> struct PairOf { using T = f2; };
template <> struct PairOf<1> { using T = float; };
template <int V> using Pair = typename PairOf<V>::T;
template <int V> __host__ __device__ constexpr int pairs() { return V == 1 ? 1 : V / 2; }
template <int V> __device__ __forceinline__ Pair<V> both(float x) {
    if constexpr (V == 1) return x;
    else return pk2(x, x);
}
// pair j of a vector
template <class E, int V>
__device__ __forceinline__ Pair<V> ln_get(const Vec<E, V>& v, int j) {
    if constexpr (V == 1) return ssm_f<E>(v.e[0]);
    else return pk2(ssm_f<E>(v.e[2 * j]), ssm_f<E>(v.e[2 * j + 1]));
}
template <class E, int V>
__device__ __forceinline__ void ln_put(Vec<E, V>& v, int j, Pair<V> x) {
    if constexpr (V == 1) {
        v.e[0] = ln_cast<E>(x);
    } else {
        float p, q;
        up2(x, p, q);
        v.e[2 * j] = ln_cast<E>(p);
        v.e[2 * j + 1] = ln_cast<E>(q);
    }
}
// V consecutive fp32 parameters, `none` where there are none
template <int V>
__device__ __forceinline__ void ln_par(const float* p, int c, Pair<V> (&o)[pairs<V>()], float none) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < pairs<V>(); ++j) o[j] = both<V>(none);
    } else if constexpr (V == 1) {
        o[0] = p[c];
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; j += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p + c + 2 * j);
            o[j] = t.x, o[j + 1] = t.y;
        }
    }
}

constexpr int LN_WARP_ROWS = 4;  // rows per block when a row takes one warp
template <int NT> __host__ __device__ constexpr int ln_block() { return NT == 32 ? 32 * LN_WARP_ROWS : NT; }

// Sums of N values over the threads of a row, in one exchange; `buf` is a fresh [NT / 32][N] per call
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*buf)[N]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) buf[threadIdx.x >> 5][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += buf[w][i];
    }
}

// ---- walks over many rows ----

// Walking blocks per multiprocessor (512 threads in all) and their share of the shared memory.  More
// threads with less of a row each lose at the barriers: 16384 x 8192 bf16 rows forward + backward took
// 380 us with 1024 threads of one vector a row against 315 us with 512 of two.
template <int NT> __host__ __device__ constexpr int ln_blocks() { return 512 / ln_block<NT>(); }
template <int NT> __host__ __device__ constexpr int ln_budget() { return 200 * 1024 / ln_blocks<NT>(); }
// Rows of a walk are taken R at a time (their sums cross the block together), D - 1 such steps ahead
template <int V, int K, int NT, int M> __host__ __device__ constexpr int ln_rows() {
    return V > 1 && K * V <= 16 && 4 * M * K * ln_block<NT>() * 16 <= ln_budget<NT>() ? 2 : 1;
}
template <int V, int K, int NT, int M> __host__ __device__ constexpr int ln_depth() {
    const int d = ln_budget<NT>() / (M * ln_rows<V, K, NT, M>() * K * ln_block<NT>() * 16);
    return d < 2 ? 2 : d > 4 ? 4 : d;
}
template <int V, int K, int NT, int M> constexpr size_t ln_ring_bytes() {
    return V > 1 ? size_t(ln_depth<V, K, NT, M>()) * M * ln_rows<V, K, NT, M>() * K * ln_block<NT>() * 16 : 0;
}

// A thread's vectors of M tensors' rows, step by step: step i covers rows row0 + (i R + r) stride
template <class E, int V, int K, int NT, int M>
struct Ring {
    static constexpr int R = ln_rows<V, K, NT, M>(), D = ln_depth<V, K, NT, M>();
    uint4* mine;  // this thread's first vector
    const E* src[M];
    int64_t row, stride, T;
    int C, tid, d = 0;
    __device__ __forceinline__ Ring(uint4* smem, const void* const (&t)[M], int tid_, int64_t row0, int64_t stride_,
                                    int64_t T_, int C_)
        : mine(smem + threadIdx.x), row(row0), stride(stride_), T(T_), C(C_), tid(tid_) {
#pragma unroll
        for (int m = 0; m < M; ++m) src[m] = static_cast<const E*>(t[m]);
#pragma unroll
        for (int i = 0; i < D - 1; ++i) put();
    }
    __device__ __forceinline__ uint4* at(int slot, int r, int m, int k) {
        return mine + (((slot * R + r) * M + m) * K + k) * ln_block<NT>();
    }
    __device__ __forceinline__ void put() {  // the next step into the next slot
#pragma unroll
        for (int r = 0; r < R; ++r, row += stride)
            if (row < T)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const int c = (k * NT + tid) * V;
                        if (c < C) cp16(reinterpret_cast<void*>(at(d, r, m, k)), src[m] + row * C + c);
                    }
        cp_commit();
        d = d + 1 == D ? 0 : d + 1;
    }
    // waits for the oldest step and starts the next one's copies.  D - 1 steps lie in the ring, so the
    // oldest is one behind the slot that put() fills, and stays until the next turn
    int old;
    __device__ __forceinline__ void turn() {
        cp_wait<D - 2>();
        old = d + 1 == D ? 0 : d + 1;
        put();
    }
    __device__ __forceinline__ Vec<E, V> get(int r, int m, int k) {
        return *reinterpret_cast<const Vec<E, V>*>(at(old, r, m, k));
    }
};

// Forward over the rows slot, slot + parts, .. of a slot (a block, or a warp where a row takes one)
template <class E, int V, int K, int NT, bool RES>
__global__ void __launch_bounds__(ln_block<NT>(), ln_blocks<NT>()) k_ln_fwd_walk(LnArgs a) {
    extern __shared__ __align__(16) uint4 ring_smem[];
    constexpr int M = RES ? 2 : 1, H = pairs<V>();
    using P = Pair<V>;
    using Rg = Ring<E, V, K, NT, M>;
    constexpr int R = Rg::R;
    __shared__ __align__(16) float buf[2][2][NT / 32][R];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int slot = NT == 32 ? blockIdx.x * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && slot >= a.parts) return;
    const float inv = 1.f / float(a.C);
    P w[K][H], b[K][H];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * NT + tid) * V;
        if (c < a.C) {
            ln_par<V>(a.w, c, w[k], 1.f);
            ln_par<V>(a.b, c, b[k], 0.f);
        }
    }
    const void* src[M];
    src[0] = a.x;
    if (RES) src[M - 1] = a.res;
    Rg ring(ring_smem, src, tid, slot, a.parts, a.T, a.C);
    int odd = 0;
    for (int64_t row0 = slot; row0 < a.T; row0 += int64_t(R) * a.parts, odd ^= 1) {
        ring.turn();
        P f[R][K][H];
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * int64_t(a.parts);
            P sum = both<V>(0.f);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + tid) * V;
                if (c < a.C && row < a.T) {
                    Vec<E, V> v = ring.get(r, 0, k);
                    if (RES) {
                        const Vec<E, V> q = ring.get(r, M - 1, k);
#pragma unroll
                        for (int j = 0; j < H; ++j) ln_put<E, V>(v, j, add2(ln_get<E, V>(v, j), ln_get<E, V>(q, j)));
                        if (a.sum) ln_store<E, V>(a.sum, row * a.C + c, v);
                    }
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        f[r][k][j] = ln_get<E, V>(v, j);
                        sum = add2(sum, f[r][k][j]);
                    }
                }
            }
            mean[r] = total(sum);
        }
        row_sums<NT, R>(mean, buf[odd][0]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv;
            P sq = both<V>(0.f);
            const P neg = both<V>(-mean[r]);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if ((k * NT + tid) * V < a.C)
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        f[r][k][j] = add2(f[r][k][j], neg);
                        sq = fma2(f[r][k][j], f[r][k][j], sq);
                    }
            rstd[r] = total(sq);
        }
        row_sums<NT, R>(rstd, buf[odd][1]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * int64_t(a.parts);
            if (row >= a.T) break;
            rstd[r] = rsqrtf(rstd[r] * inv + a.eps);
            if (tid == 0) {
                if (a.mean) a.mean[row] = mean[r];
                if (a.rstd) a.rstd[row] = rstd[r];
            }
            const P rs = both<V>(rstd[r]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + tid) * V;
                if (c < a.C) {
                    Vec<E, V> y;
#pragma unroll
                    for (int j = 0; j < H; ++j) ln_put<E, V>(y, j, fma2(mul2(f[r][k][j], rs), w[k][j], b[k][j]));
                    ln_store<E, V>(a.y, row * a.C + c, y);
                }
            }
        }
    }
    cp_wait<0>();
}

// Plain loads into registers in the ring's place (rows that are not whole vectors)
template <class E, int V, int K, int NT, int M>
struct Direct {
    static constexpr int R = 1;
    const E* src[M];
    Vec<E, V> v[M][K];
    int64_t row, stride;
    int C, tid;
    __device__ __forceinline__ Direct(uint4*, const void* const (&t)[M], int tid_, int64_t row0, int64_t stride_, int64_t, int C_)
        : row(row0 - stride_), stride(stride_), C(C_), tid(tid_) {
#pragma unroll
        for (int m = 0; m < M; ++m) src[m] = static_cast<const E*>(t[m]);
    }
    __device__ __forceinline__ void turn() {
        row += stride;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int k = 0; k < K; ++k)
                if ((k * NT + tid) * V < C) v[m][k] = ln_load<E, V>(src[m], row * C + (k * NT + tid) * V);
    }
    __device__ __forceinline__ Vec<E, V> get(int, int m, int k) { return v[m][k]; }
};
template <class E, int V, int K, int NT, int M> struct RowsOf { using T = Ring<E, V, K, NT, M>; };
template <class E, int K, int NT, int M> struct RowsOf<E, 1, K, NT, M> { using T = Direct<E, 1, K, NT, M>; };

// Backward over the rows of a slot.  Whole-vector rows are read from the ring twice, before and after
// the exchange of their sums, and hold no registers across it.
template <class E, int V, int K, int NT, bool DSUM>
__global__ void __launch_bounds__(ln_block<NT>(), V > 1 ? ln_blocks<NT>() : 1) k_ln_bwd(LnArgs a) {
    extern __shared__ __align__(16) uint4 ring_smem[];
    constexpr int M = DSUM ? 3 : 2, H = pairs<V>();
    using P = Pair<V>;
    using Rg = typename RowsOf<E, V, K, NT, M>::T;
    constexpr int R = Rg::R;
    constexpr bool HOLD = K * V <= 16;  // w in registers over the walk
    __shared__ __align__(16) float buf[2][NT / 32][2 * R];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int slot = NT == 32 ? blockIdx.x * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && slot >= a.parts) return;
    const float inv = 1.f / float(a.C);
    P dw[K][H], db[K][H], wh[HOLD ? K : 1][H];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < H; ++j) dw[k][j] = db[k][j] = both<V>(0.f);
    if constexpr (HOLD)
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((k * NT + tid) * V < a.C) ln_par<V>(a.w, (k * NT + tid) * V, wh[k], 1.f);
    const void* src[M];
    src[0] = a.x;
    src[1] = a.dy;
    if (DSUM) src[M - 1] = a.dsum;
    Rg rows(ring_smem, src, tid, slot, a.parts, a.T, a.C);
    float nm[R], nr[R];  // the next step's statistics
    auto stats = [&](int64_t row0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * int64_t(a.parts);
            nm[r] = row < a.T ? a.mean_in[row] : 0.f;
            nr[r] = row < a.T ? a.rstd_in[row] : 0.f;
        }
    };
    stats(slot);
    int odd = 0;
    for (int64_t row0 = slot; row0 < a.T; row0 += int64_t(R) * a.parts, odd ^= 1) {
        rows.turn();
        float m[R], rs[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) m[r] = nm[r], rs[r] = nr[r];
        stats(row0 + int64_t(R) * a.parts);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[2 * r] = s[2 * r + 1] = 0.f;
            if (row0 + r * int64_t(a.parts) >= a.T) continue;
            const P rr = both<V>(rs[r]), mr = both<V>(-m[r]);
            P s0 = both<V>(0.f), s1 = s0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + tid) * V;
                if (c < a.C) {
                    const Vec<E, V> x = rows.get(r, 0, k), g = rows.get(r, 1, k);
                    P wl[H];
                    if constexpr (!HOLD) ln_par<V>(a.w, c, wl, 1.f);
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const P xh = mul2(add2(ln_get<E, V>(x, j), mr), rr), q = ln_get<E, V>(g, j);
                        const P d = mul2(q, HOLD ? wh[HOLD ? k : 0][j] : wl[j]);
                        dw[k][j] = fma2(q, xh, dw[k][j]);
                        db[k][j] = add2(db[k][j], q);
                        s0 = add2(s0, d);
                        s1 = fma2(d, xh, s1);
                    }
                }
            }
            s[2 * r] = total(s0);
            s[2 * r + 1] = total(s1);
        }
        row_sums<NT, 2 * R>(s, buf[odd]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * int64_t(a.parts);
            if (row >= a.T) break;
            const P rr = both<V>(rs[r]), mr = both<V>(-m[r]);
            const P n0 = both<V>(-(s[2 * r] * inv)), n1 = both<V>(-(s[2 * r + 1] * inv) * rs[r]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (k * NT + tid) * V;
                if (c < a.C) {
                    const Vec<E, V> x = rows.get(r, 0, k), g = rows.get(r, 1, k);
                    Vec<E, V> e, o;
                    if (DSUM) e = rows.get(r, M - 1, k);
                    P wl[H];
                    if constexpr (!HOLD) ln_par<V>(a.w, c, wl, 1.f);
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const P xh = mul2(add2(ln_get<E, V>(x, j), mr), rr);
                        const P d = mul2(ln_get<E, V>(g, j), HOLD ? wh[HOLD ? k : 0][j] : wl[j]);
                        P t = fma2(xh, n1, mul2(add2(d, n0), rr));  // rstd (d - mean d - xh mean(d xh))
                        if (DSUM) t = add2(t, ln_get<E, V>(e, j));
                        ln_put<E, V>(o, j, t);
                    }
                    ln_store<E, V>(a.dx, row * a.C + c, o);
                }
            }
        }
    }
    if constexpr (V > 1) cp_wait<0>();
    float* p = a.part + int64_t(slot) * 2 * a.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * NT + tid) * V;
        if (c < a.C)
#pragma unroll
            for (int j = 0; j < H; ++j) {
                if constexpr (V > 1) {
                    *reinterpret_cast<P*>(p + c + 2 * j) = dw[k][j];
                    *reinterpret_cast<P*>(p + a.C + c + 2 * j) = db[k][j];
                } else {
                    p[c] = dw[k][0];
                    p[a.C + c] = db[k][0];
                }
            }
    }
}

// dw, db: column sums of the partials.  32 columns x 32 strands of parts per block; a strand's parts
// are added in order, then the strands.
__global__ void __launch_bounds__(1024) k_ln_reduce(LnArgs a, float* dw, float* db) {
    __shared__ float s[32][33];
    const int cx = threadIdx.x & 31, st = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;  // column of [2 C]
    float v = 0.f;
    if (c < 2 * a.C) {
        const float* p = a.part + c;
#pragma unroll 4
        for (int i = st; i < a.parts; i += 32) v += p[int64_t(i) * 2 * a.C];
    }
    s[st][cx] = v;
    __syncthreads();
    if (st == 0 && c < 2 * a.C) {
#pragma unroll
        for (int i = 1; i < 32; ++i) v += s[i][cx];
        if (c < a.C) { if (dw) dw[c] = v; }
        else if (db) db[c - a.C] = v;
    }
}

// ---- few rows: one per block (or warp) ----

template <class E, int V, int K, int NT>
__global__ void __launch_bounds__(ln_block<NT>()) k_ln_fwd(LnArgs a) {
    constexpr int H = pairs<V>();
    using P = Pair<V>;
    __shared__ float buf[2][NT / 32][1];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = NT == 32 ? int64_t(blockIdx.x) * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && row >= a.T) return;
    const int64_t base = row * a.C;
    const float inv = 1.f / float(a.C);
    P f[K][H], s = both<V>(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * NT + tid) * V;
        if (c < a.C) {
            Vec<E, V> x = ln_load<E, V>(a.x, base + c);
            if (a.res) {
                const Vec<E, V> r = ln_load<E, V>(a.res, base + c);
#pragma unroll
                for (int j = 0; j < H; ++j) ln_put<E, V>(x, j, add2(ln_get<E, V>(x, j), ln_get<E, V>(r, j)));
                if (a.sum) ln_store<E, V>(a.sum, base + c, x);
            }
#pragma unroll
            for (int j = 0; j < H; ++j) {
                f[k][j] = ln_get<E, V>(x, j);
                s = add2(s, f[k][j]);
            }
        }
    }
    float mean[1] = {total(s)}, rstd[1];
    row_sums<NT, 1>(mean, buf[0]);
    mean[0] *= inv;
    s = both<V>(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k)
        if ((k * NT + tid) * V < a.C)
#pragma unroll
            for (int j = 0; j < H; ++j) {
                f[k][j] = add2(f[k][j], both<V>(-mean[0]));
                s = fma2(f[k][j], f[k][j], s);
            }
    rstd[0] = total(s);
    row_sums<NT, 1>(rstd, buf[1]);
    rstd[0] = rsqrtf(rstd[0] * inv + a.eps);
    if (tid == 0) {
        if (a.mean) a.mean[row] = mean[0];
        if (a.rstd) a.rstd[row] = rstd[0];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * NT + tid) * V;
        if (c < a.C) {
            P w[H], b[H];
            ln_par<V>(a.w, c, w, 1.f);
            ln_par<V>(a.b, c, b, 0.f);
            Vec<E, V> y;
#pragma unroll
            for (int j = 0; j < H; ++j) ln_put<E, V>(y, j, fma2(mul2(f[k][j], both<V>(rstd[0])), w[j], b[j]));
            ln_store<E, V>(a.y, base + c, y);
        }
    }
}

// ---- rows of any length: re-read instead of held ----

constexpr int LONG_NT = 1024;

__device__ __forceinline__ float long_sum(float v, float (*buf)[1]) {
    float s[1] = {v};
    row_sums<LONG_NT, 1>(s, buf);
    return s[0];
}

template <class E>
__global__ void __launch_bounds__(LONG_NT) k_ln_fwd_long(LnArgs a) {
    __shared__ float buf[2][LONG_NT / 32][1];
    const int64_t row = blockIdx.x, base = row * a.C;
    const float inv = 1.f / float(a.C);
    auto val = [&](int c) {
        const float v = ssm_ld<E>(a.x, base + c);
        return a.res ? ssm_f<E>(ln_cast<E>(v + ssm_ld<E>(a.res, base + c))) : v;
    };
    float s = 0.f;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float v = val(c);
        s += v;
    }
    const float mean = long_sum(s, buf[0]) * inv;
    s = 0.f;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float v = val(c) - mean;
        s = fmaf(v, v, s);
    }
    const float rstd = rsqrtf(long_sum(s, buf[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float v = val(c);
        if (a.res && a.sum) ssm_st<E>(a.sum, base + c, v);
        ssm_st<E>(a.y, base + c, fmaf((v - mean) * rstd, a.w ? a.w[c] : 1.f, a.b ? a.b[c] : 0.f));
    }
}

template <class E>
__global__ void __launch_bounds__(LONG_NT) k_ln_bwd_long(LnArgs a) {
    __shared__ float buf[2][LONG_NT / 32][1];
    const int64_t row = blockIdx.x, base = row * a.C;
    const float inv = 1.f / float(a.C), mean = a.mean_in[row], rstd = a.rstd_in[row];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float d = __fmul_rn(ssm_ld<E>(a.dy, base + c), a.w ? a.w[c] : 1.f);
        s0 += d;
        s1 = fmaf(d, (ssm_ld<E>(a.x, base + c) - mean) * rstd, s1);
    }
    s0 = long_sum(s0, buf[0]) * inv;
    s1 = long_sum(s1, buf[1]) * inv;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float d = __fmul_rn(ssm_ld<E>(a.dy, base + c), a.w ? a.w[c] : 1.f);
        float t = rstd * (d - s0 - (ssm_ld<E>(a.x, base + c) - mean) * rstd * s1);
        if (a.dsum) t += ssm_ld<E>(a.dsum, base + c);
        ssm_st<E>(a.dx, base + c, t);
    }
}

// partial dw, db of a run of rows: one thread per column
template <class E>
__global__ void __launch_bounds__(256) k_ln_cols_long(LnArgs a) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= a.C) return;
    float dw = 0.f, db = 0.f;
    for (int64_t r = blockIdx.y; r < a.T; r += a.parts) {
        const float q = ssm_ld<E>(a.dy, r * a.C + c);
        dw = fmaf(q, (ssm_ld<E>(a.x, r * a.C + c) - a.mean_in[r]) * a.rstd_in[r], dw);
        db += q;
    }
    float* p = a.part + int64_t(blockIdx.y) * 2 * a.C;
    p[c] = dw;
    p[a.C + c] = db;
}

// ---- dispatch ----

// Threads per row and vectors per thread by the row's length in vectors: the fewest threads whose
// registers hold the row.  wide: rows are whole 16-byte vectors.  nt = 0: the re-reading kernels.  Of
// the 1024-vector rows (16384 x 8192 bf16), the forward takes 91 us with 256 threads of four vectors
// and 99 with 512 of two; the backward, whose accumulators are twice as many, 186 and 145.
struct Shape { int nt, k; bool wide; };
Shape shape_of(int C, int esize, bool back) {
    const int V = 16 / esize;
    if (C % V == 0) {
        const Shape wide[] = {{32, 1, true}, {32, 2, true}, {128, 1, true}, {128, 2, true}, {256, 2, true},
                              back ? Shape{512, 2, true} : Shape{256, 4, true}, {512, 4, true}};
        for (const Shape& s : wide)
            if (C / V <= s.nt * s.k) return s;
        return {0, 0, true};
    }
    for (int nt : {32, 128, 512})
        if (C <= nt * 16) return {nt, 16, false};
    return {0, 0, false};
}

// Slots of a walk: as many blocks as the machine's 152 multiprocessors hold at once (rows of a warp go
// four to a block), with at least two rows each
int parts_of(int64_t T, const Shape& s) {
    const int slots = s.nt ? 152 * (512 / s.nt) : 32;
    const int64_t want = s.nt ? (T + 1) / 2 : T;
    return int(want < 1 ? 1 : want < slots ? want : slots);
}

template <auto* F>
void ring_launch(unsigned blocks, int threads, size_t smem, const LnArgs& a, cudaStream_t st) {
    static unsigned long long done;
    allow_smem((const void*)F, smem, &done);
    F<<<blocks, threads, smem, st>>>(a);
}

template <class E, int V, int K, int NT>
void fwd(LnArgs a, const Shape& s, cudaStream_t st) {
    // a walk pays off from four rows per slot on; fewer rows spread one per block (or warp)
    const int parts = parts_of(a.T, s);
    if constexpr (V > 1) {
        if (a.T >= 4 * int64_t(parts)) {
            a.parts = parts;
            const unsigned blocks = unsigned(NT == 32 ? (parts + LN_WARP_ROWS - 1) / LN_WARP_ROWS : parts);
            if (a.res) ring_launch<k_ln_fwd_walk<E, V, K, NT, true>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 2>(), a, st);
            else ring_launch<k_ln_fwd_walk<E, V, K, NT, false>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 1>(), a, st);
            return;
        }
    }
    const int64_t blocks = NT == 32 ? (a.T + LN_WARP_ROWS - 1) / LN_WARP_ROWS : a.T;
    k_ln_fwd<E, V, K, NT><<<unsigned(blocks), ln_block<NT>(), 0, st>>>(a);
}
template <class E, int V, int K, int NT>
void bwd(const LnArgs& a, cudaStream_t st) {
    const unsigned blocks = unsigned(NT == 32 ? (a.parts + LN_WARP_ROWS - 1) / LN_WARP_ROWS : a.parts);
    if (a.dsum) ring_launch<k_ln_bwd<E, V, K, NT, true>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 3>(), a, st);
    else ring_launch<k_ln_bwd<E, V, K, NT, false>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 2>(), a, st);
}
template <class E, int V, int K, int NT>
void run(const LnArgs& a, const Shape& s, bool back, cudaStream_t st) {
    if (back) {
        if constexpr (NT != 256 || K != 4) bwd<E, V, K, NT>(a, st);
    } else {
        if constexpr (NT != 512 || K != 2) fwd<E, V, K, NT>(a, s, st);
    }
}
template <class E>
void by_shape(const LnArgs& a, const Shape& s, bool back, cudaStream_t st) {
    constexpr int V = 16 / sizeof(E);
    if (!s.nt) {
        if (!back) {
            k_ln_fwd_long<E><<<unsigned(a.T), LONG_NT, 0, st>>>(a);
        } else {
            k_ln_bwd_long<E><<<unsigned(a.T), LONG_NT, 0, st>>>(a);
            k_ln_cols_long<E><<<dim3(unsigned((a.C + 255) / 256), unsigned(a.parts)), 256, 0, st>>>(a);
        }
    } else if (!s.wide) {
        if (s.nt == 32) run<E, 1, 16, 32>(a, s, back, st);
        else if (s.nt == 128) run<E, 1, 16, 128>(a, s, back, st);
        else run<E, 1, 16, 512>(a, s, back, st);
    } else if (s.nt == 32) {
        s.k == 1 ? run<E, V, 1, 32>(a, s, back, st) : run<E, V, 2, 32>(a, s, back, st);
    } else if (s.nt == 128) {
        s.k == 1 ? run<E, V, 1, 128>(a, s, back, st) : run<E, V, 2, 128>(a, s, back, st);
    } else if (s.nt == 256) {
        s.k == 2 ? run<E, V, 2, 256>(a, s, back, st) : run<E, V, 4, 256>(a, s, back, st);
    } else {
        s.k == 2 ? run<E, V, 2, 512>(a, s, back, st) : run<E, V, 4, 512>(a, s, back, st);
    }
}
void by_type(const LnArgs& a, int dtype, const Shape& s, bool back, cudaStream_t st) {
    if (dtype == KDA_DT_BF16) by_shape<__nv_bfloat16>(a, s, back, st);
    else if (dtype == KDA_DT_FP16) by_shape<__half>(a, s, back, st);
    else by_shape<float>(a, s, back, st);
}

bool opt(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool req(const void* p) { return p && opt(p); }
int esize(int dtype) { return dtype == KDA_DT_FP32 ? 4 : 2; }

kda_status check(const kda_layernorm_problem* p) {
    if (!p || p->T < 0 || p->T > INT32_MAX || p->C < 1 || p->C > (1 << 24) || !(p->eps >= 0.f))
        return KDA_ERR_INVALID_ARG;
    if (p->dtype != KDA_DT_BF16 && p->dtype != KDA_DT_FP16 && p->dtype != KDA_DT_FP32) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_layernorm_workspace_size(const kda_layernorm_problem* p, size_t* ws_bytes) {
    if (kda_status s = check(p)) return s;
    if (ws_bytes) *ws_bytes = align256(size_t(parts_of(p->T, shape_of(p->C, esize(p->dtype), true))) * 2 * size_t(p->C) * 4);
    return KDA_OK;
}

kda_status kda_layernorm_fwd(const kda_layernorm_problem* p, const void* x, const void* res, const float* w,
                             const float* b, void* sum, void* y, float* mean, float* rstd, kda_stream_t stream) {
    if (kda_status s = check(p)) return s;
    if ((p->T > 0 && !(req(x) && req(y))) || !opt(x) || !opt(y) || !opt(res) || !opt(w) || !opt(b) || !opt(sum) ||
        !opt(mean) || !opt(rstd))
        return KDA_ERR_INVALID_ARG;
    if (sum && !res) return KDA_ERR_INVALID_ARG;  // the sum exists only with a residual
    if (p->T == 0) return KDA_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LnArgs a{};
    a.T = p->T, a.C = p->C, a.eps = p->eps;
    a.x = x, a.res = res, a.w = w, a.b = b, a.sum = sum, a.y = y, a.mean = mean, a.rstd = rstd;
    {
        ProfScope ps(KK_LN_FWD, st);
        by_type(a, p->dtype, shape_of(p->C, esize(p->dtype), false), false, st);
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_layernorm_bwd(const kda_layernorm_problem* p, const void* x, const float* w, const float* mean,
                             const float* rstd, const void* dy, const void* dsum, void* dx, float* dw, float* db,
                             void* ws, size_t ws_bytes, kda_stream_t stream) {
    if (kda_status s = check(p)) return s;
    if (p->T > 0 && !(req(x) && req(mean) && req(rstd) && req(dy) && req(dx))) return KDA_ERR_INVALID_ARG;
    if (!opt(w) || !opt(dsum) || !opt(dw) || !opt(db) || !req(ws)) return KDA_ERR_INVALID_ARG;
    const Shape s = shape_of(p->C, esize(p->dtype), true);
    size_t need = 0;
    kda_layernorm_workspace_size(p, &need);
    if (ws_bytes < need) return KDA_ERR_WORKSPACE;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LnArgs a{};
    a.T = p->T, a.C = p->C, a.eps = p->eps;
    a.x = x, a.w = w, a.mean_in = mean, a.rstd_in = rstd, a.dy = dy, a.dsum = dsum, a.dx = dx;
    a.part = static_cast<float*>(ws);
    a.parts = p->T > 0 ? parts_of(p->T, s) : 0;  // no rows: the sums below are zero
    if (p->T > 0) {
        ProfScope ps(KK_LN_BWD, st);
        by_type(a, p->dtype, s, true, st);
    }
    if (dw || db) {
        ProfScope ps(KK_LN_REDUCE, st);
        k_ln_reduce<<<unsigned((2 * p->C + 31) / 32), 1024, 0, st>>>(a, dw, db);
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
