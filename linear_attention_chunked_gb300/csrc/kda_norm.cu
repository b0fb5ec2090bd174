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
//
// Rows whose length is no multiple of a vector (V elements) start inside one.  They are read as the aligned
// vectors that cover them, the neighbours' elements cleared (SHIFT); a slot's rows are V apart or a
// multiple of it, so all of them start at the same place in a vector and its columns stay in its
// registers.
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

// V consecutive elements, one 16-byte access
template <class E, int V>
struct alignas(16) Vec {
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

// pair j of a vector
template <class E, int V>
__device__ __forceinline__ f2 ln_get(const Vec<E, V>& v, int j) {
    return pk2(ssm_f<E>(v.e[2 * j]), ssm_f<E>(v.e[2 * j + 1]));
}
template <class E, int V>
__device__ __forceinline__ void ln_put(Vec<E, V>& v, int j, f2 x) {
    float p, q;
    up2(x, p, q);
    v.e[2 * j] = ln_cast<E>(p);
    v.e[2 * j + 1] = ln_cast<E>(q);
}
__device__ __forceinline__ f2 both(float x) { return pk2(x, x); }
__device__ __forceinline__ f2 ln_mul_rn(f2 a, f2 b) {
    float p, q, r, t;
    up2(a, p, q);
    up2(b, r, t);
    return pk2(__fmul_rn(p, r), __fmul_rn(q, t));
}
// whether the V columns from cb (negative, or reaching past C, at a row's ends) hold a neighbour's elements
template <int V> __device__ __forceinline__ bool ln_edge(int cb, int C) { return cb < 0 || cb + V > C; }
template <class E, int V>
__device__ __forceinline__ void ln_clip(Vec<E, V>& v, int cb, int C) {
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (cb + j < 0 || cb + j >= C) v.e[j] = ln_cast<E>(0.f);
}
__device__ __forceinline__ f2 ln_inside(f2 v, int c, int C) {
    float p, q;
    up2(v, p, q);
    return pk2(c >= 0 && c < C ? p : 0.f, c + 1 >= 0 && c + 1 < C ? q : 0.f);
}
template <class E, int V, bool SHIFT>
__device__ __forceinline__ void ln_store_row(void* p, int64_t row0, int cb, int C, const Vec<E, V>& v) {
    if (SHIFT && ln_edge<V>(cb, C)) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (cb + j >= 0 && cb + j < C) static_cast<E*>(p)[row0 + cb + j] = v.e[j];
    } else {
        ln_store<E, V>(p, row0 + cb, v);
    }
}
// V fp32 parameters from column cb, `none` where there are none
template <int V, bool SHIFT>
__device__ __forceinline__ void ln_par(const float* p, int cb, int C, f2 (&o)[V / 2], float none) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) o[j] = both(none);
    } else if (SHIFT) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = cb + j >= 0 && cb + j < C ? p[cb + j] : 0.f;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) o[j] = pk2(f[2 * j], f[2 * j + 1]);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; j += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p + cb + 2 * j);
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
    return K * V <= 16 && 4 * M * K * ln_block<NT>() * 16 <= ln_budget<NT>() ? 2 : 1;
}
template <int V, int K, int NT, int M> __host__ __device__ constexpr int ln_depth() {
    const int d = ln_budget<NT>() / (M * ln_rows<V, K, NT, M>() * K * ln_block<NT>() * 16);
    return d < 2 ? 2 : d > 4 ? 4 : d;
}
template <int V, int K, int NT, int M> constexpr size_t ln_ring_bytes() {
    return size_t(ln_depth<V, K, NT, M>()) * M * ln_rows<V, K, NT, M>() * K * ln_block<NT>() * 16;
}

// Copies the vector at element i of a tensor of n; SHIFT: the last one may end past it (cleared there)
template <class E, int V, bool SHIFT>
__device__ __forceinline__ void ln_copy(uint4* smem, const E* src, int64_t i, int64_t n) {
    const int bytes = SHIFT && n - i < V ? int(n - i) * int(sizeof(E)) : 16;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(smem)), "l"(src + i), "r"(bytes) : "memory");
}

// A thread's vectors of M tensors' rows, step by step: step i covers rows row0 + (i R + r) stride
template <class E, int V, int K, int NT, int M, bool SHIFT>
struct Ring {
    static constexpr int R = ln_rows<V, K, NT, M>(), D = ln_depth<V, K, NT, M>();
    uint4* mine;  // this thread's first vector
    const E* src[M];
    int64_t row, stride, T;
    int C, tid, sh, d = 0;
    __device__ __forceinline__ Ring(uint4* smem, const void* const (&t)[M], int tid_, int64_t row0, int64_t stride_,
                                    int64_t T_, int C_, int sh_)
        : mine(smem + threadIdx.x), row(row0), stride(stride_), T(T_), C(C_), tid(tid_), sh(sh_) {
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
                        const int cb = (k * NT + tid) * V - sh;
                        if (cb < C) ln_copy<E, V, SHIFT>(at(d, r, m, k), src[m], row * C + cb, T * C);
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
template <class E, int V, int K, int NT, bool RES, bool SHIFT>
__global__ void __launch_bounds__(ln_block<NT>(), ln_blocks<NT>()) k_ln_fwd_walk(LnArgs a) {
    extern __shared__ __align__(16) uint4 ring_smem[];
    constexpr int M = RES ? 2 : 1, H = V / 2;
    using P = f2;
    using Rg = Ring<E, V, K, NT, M, SHIFT>;
    constexpr int R = Rg::R;
    __shared__ __align__(16) float buf[2][2][NT / 32][R];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int slot = NT == 32 ? blockIdx.x * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && slot >= a.parts) return;
    const float inv = 1.f / float(a.C);
    const int sh = SHIFT ? int(int64_t(slot) * a.C % V) : 0;
    P w[K][H], b[K][H];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int cb = (k * NT + tid) * V - sh;
        if (cb < a.C) {
            ln_par<V, SHIFT>(a.w, cb, a.C, w[k], 1.f);
            ln_par<V, SHIFT>(a.b, cb, a.C, b[k], 0.f);
        }
    }
    const void* src[M];
    src[0] = a.x;
    if (RES) src[M - 1] = a.res;
    Rg ring(ring_smem, src, tid, slot, a.parts, a.T, a.C, sh);
    int odd = 0;
    for (int64_t row0 = slot; row0 < a.T; row0 += int64_t(R) * a.parts, odd ^= 1) {
        ring.turn();
        P f[R][K][H];
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * int64_t(a.parts);
            P sum = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int cb = (k * NT + tid) * V - sh;
                if (cb < a.C && row < a.T) {
                    Vec<E, V> v = ring.get(r, 0, k);
                    if (RES) {
                        const Vec<E, V> q = ring.get(r, M - 1, k);
#pragma unroll
                        for (int j = 0; j < H; ++j) ln_put<E, V>(v, j, add2(ln_get<E, V>(v, j), ln_get<E, V>(q, j)));
                        if (a.sum) ln_store_row<E, V, SHIFT>(a.sum, row * a.C, cb, a.C, v);
                    }
                    if (SHIFT && ln_edge<V>(cb, a.C)) ln_clip<E, V>(v, cb, a.C);
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        f[r][k][j] = ln_get<E, V>(v, j);
                        sum = add2(sum, f[r][k][j]);
                    }
                }
            }
            mean[r] = hsum2(sum);
        }
        row_sums<NT, R>(mean, buf[odd][0]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] *= inv;
            P sq = 0;
            const P neg = both(-mean[r]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int cb = (k * NT + tid) * V - sh;
                if (cb < a.C)
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        f[r][k][j] = add2(f[r][k][j], neg);
                        if (SHIFT) f[r][k][j] = ln_inside(f[r][k][j], cb + 2 * j, a.C);
                        sq = fma2(f[r][k][j], f[r][k][j], sq);
                    }
            }
            rstd[r] = hsum2(sq);
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
            const P rs = both(rstd[r]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int cb = (k * NT + tid) * V - sh;
                if (cb < a.C) {
                    Vec<E, V> y;
#pragma unroll
                    for (int j = 0; j < H; ++j) ln_put<E, V>(y, j, fma2(mul2(f[r][k][j], rs), w[k][j], b[k][j]));
                    ln_store_row<E, V, SHIFT>(a.y, row * a.C, cb, a.C, y);
                }
            }
        }
    }
    cp_wait<0>();
}

// Backward over the rows of a slot.  The rows are read from the ring twice, before and after the exchange
// of their sums, and hold no registers across it.
template <class E, int V, int K, int NT, bool DSUM, bool SHIFT>
__global__ void __launch_bounds__(ln_block<NT>(), ln_blocks<NT>()) k_ln_bwd(LnArgs a) {
    extern __shared__ __align__(16) uint4 ring_smem[];
    constexpr int M = DSUM ? 3 : 2, H = V / 2;
    using P = f2;
    using Rg = Ring<E, V, K, NT, M, SHIFT>;
    constexpr int R = Rg::R;
    constexpr bool HOLD = K * V <= 16;  // w in registers over the walk
    __shared__ __align__(16) float buf[2][NT / 32][2 * R];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int slot = NT == 32 ? blockIdx.x * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && slot >= a.parts) return;
    const int sh = SHIFT ? int(int64_t(slot) * a.C % V) : 0;
    const float inv = 1.f / float(a.C);
    P dw[K][H], db[K][H], wh[HOLD ? K : 1][H];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < H; ++j) dw[k][j] = db[k][j] = 0;
    if constexpr (HOLD)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int cb = (k * NT + tid) * V - sh;
            if (cb < a.C) ln_par<V, SHIFT>(a.w, cb, a.C, wh[k], 1.f);
        }
    const void* src[M];
    src[0] = a.x;
    src[1] = a.dy;
    if (DSUM) src[M - 1] = a.dsum;
    Rg rows(ring_smem, src, tid, slot, a.parts, a.T, a.C, sh);
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
        // x and dy of row r, vector k (the neighbours' elements zero: they add nothing to any sum)
        auto get2 = [&](int r, int k, int cb, Vec<E, V>& x, Vec<E, V>& g) {
            x = rows.get(r, 0, k), g = rows.get(r, 1, k);
            if (SHIFT && ln_edge<V>(cb, a.C)) {
                ln_clip<E, V>(x, cb, a.C);
                ln_clip<E, V>(g, cb, a.C);
            }
        };
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[2 * r] = s[2 * r + 1] = 0.f;
            if (row0 + r * int64_t(a.parts) >= a.T) continue;
            const P rr = both(rs[r]), mr = both(-m[r]);
            P s0 = 0, s1 = 0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int cb = (k * NT + tid) * V - sh;
                if (cb < a.C) {
                    Vec<E, V> x, g;
                    get2(r, k, cb, x, g);
                    P wl[H];
                    if constexpr (!HOLD) ln_par<V, SHIFT>(a.w, cb, a.C, wl, 1.f);
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
            s[2 * r] = hsum2(s0);
            s[2 * r + 1] = hsum2(s1);
        }
        row_sums<NT, 2 * R>(s, buf[odd]);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + r * int64_t(a.parts);
            if (row >= a.T) break;
            const P rr = both(rs[r]), mr = both(-m[r]);
            const P n0 = both(-(s[2 * r] * inv)), n1 = both(-(s[2 * r + 1] * inv) * rs[r]);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int cb = (k * NT + tid) * V - sh;
                if (cb < a.C) {
                    const Vec<E, V> x = rows.get(r, 0, k), g = rows.get(r, 1, k);
                    Vec<E, V> e, o;
                    if (DSUM) e = rows.get(r, M - 1, k);
                    P wl[H];
                    if constexpr (!HOLD) ln_par<V, SHIFT>(a.w, cb, a.C, wl, 1.f);
#pragma unroll
                    for (int j = 0; j < H; ++j) {
                        const P xh = mul2(add2(ln_get<E, V>(x, j), mr), rr);
                        // SHIFT: the product as it was summed, unfused with the difference below (a row of one
                        // element has exactly no gradient)
                        const P q = ln_get<E, V>(g, j), wj = HOLD ? wh[HOLD ? k : 0][j] : wl[j];
                        const P d = SHIFT ? ln_mul_rn(q, wj) : mul2(q, wj);
                        P t = fma2(xh, n1, mul2(add2(d, n0), rr));  // rstd (d - mean d - xh mean(d xh))
                        if (DSUM) t = add2(t, ln_get<E, V>(e, j));
                        ln_put<E, V>(o, j, t);
                    }
                    ln_store_row<E, V, SHIFT>(a.dx, row * a.C, cb, a.C, o);
                }
            }
        }
    }
    cp_wait<0>();
    float* p = a.part + int64_t(slot) * 2 * a.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int cb = (k * NT + tid) * V - sh;
        if (cb < a.C)
#pragma unroll
            for (int j = 0; j < H; ++j) {
                if (SHIFT) {
                    float u[2], v[2];
                    up2(dw[k][j], u[0], u[1]);
                    up2(db[k][j], v[0], v[1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = cb + 2 * j + i;
                        if (c >= 0 && c < a.C) p[c] = u[i], p[a.C + c] = v[i];
                    }
                } else {
                    *reinterpret_cast<f2*>(p + cb + 2 * j) = dw[k][j];
                    *reinterpret_cast<f2*>(p + a.C + cb + 2 * j) = db[k][j];
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

template <class E, int V, int K, int NT, bool SHIFT>
__global__ void __launch_bounds__(ln_block<NT>()) k_ln_fwd(LnArgs a) {
    constexpr int H = V / 2;
    using P = f2;
    __shared__ float buf[2][NT / 32][1];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = NT == 32 ? int64_t(blockIdx.x) * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && row >= a.T) return;
    const int64_t base = row * a.C, all = a.T * a.C;
    const int sh = SHIFT ? int(base % V) : 0;
    const float inv = 1.f / float(a.C);
    auto load = [&](const void* p, int cb) {
        if (SHIFT && base + cb + V > all) {  // the tensor's last vector
            Vec<E, V> v;
#pragma unroll
            for (int j = 0; j < V; ++j) v.e[j] = base + cb + j < all ? static_cast<const E*>(p)[base + cb + j] : ln_cast<E>(0.f);
            return v;
        }
        return ln_load<E, V>(p, base + cb);
    };
    P f[K][H], s = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int cb = (k * NT + tid) * V - sh;
        if (cb < a.C) {
            Vec<E, V> x = load(a.x, cb);
            if (a.res) {
                const Vec<E, V> r = load(a.res, cb);
#pragma unroll
                for (int j = 0; j < H; ++j) ln_put<E, V>(x, j, add2(ln_get<E, V>(x, j), ln_get<E, V>(r, j)));
                if (a.sum) ln_store_row<E, V, SHIFT>(a.sum, base, cb, a.C, x);
            }
            if (SHIFT && ln_edge<V>(cb, a.C)) ln_clip<E, V>(x, cb, a.C);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                f[k][j] = ln_get<E, V>(x, j);
                s = add2(s, f[k][j]);
            }
        }
    }
    float mean[1] = {hsum2(s)}, rstd[1];
    row_sums<NT, 1>(mean, buf[0]);
    mean[0] *= inv;
    s = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int cb = (k * NT + tid) * V - sh;
        if (cb < a.C)
#pragma unroll
            for (int j = 0; j < H; ++j) {
                f[k][j] = add2(f[k][j], both(-mean[0]));
                if (SHIFT) f[k][j] = ln_inside(f[k][j], cb + 2 * j, a.C);
                s = fma2(f[k][j], f[k][j], s);
            }
    }
    rstd[0] = hsum2(s);
    row_sums<NT, 1>(rstd, buf[1]);
    rstd[0] = rsqrtf(rstd[0] * inv + a.eps);
    if (tid == 0) {
        if (a.mean) a.mean[row] = mean[0];
        if (a.rstd) a.rstd[row] = rstd[0];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int cb = (k * NT + tid) * V - sh;
        if (cb < a.C) {
            P w[H], b[H];
            ln_par<V, SHIFT>(a.w, cb, a.C, w, 1.f);
            ln_par<V, SHIFT>(a.b, cb, a.C, b, 0.f);
            Vec<E, V> y;
#pragma unroll
            for (int j = 0; j < H; ++j) ln_put<E, V>(y, j, fma2(mul2(f[k][j], both(rstd[0])), w[j], b[j]));
            ln_store_row<E, V, SHIFT>(a.y, base, cb, a.C, y);
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
// registers hold the row.  shift: rows start inside vectors (up to V - 1 elements in, so that one
// more may be needed).  nt = 0: the re-reading kernels.  Of the 1024-vector rows (16384 x 8192 bf16), the
// forward takes 91 us with 256 threads of four vectors and 99 with 512 of two; the backward, whose
// accumulators are twice as many, 186 and 145.
struct Shape { int nt, k; bool shift; };
Shape shape_of(int C, int esize, bool back) {
    const int V = 16 / esize;
    const bool shift = C % V != 0;
    const int n = shift ? (C + V - 1 + V - 1) / V : C / V;
    const int shapes[][2] = {{32, 1}, {32, 2}, {128, 1}, {128, 2}, {256, 2}, {back ? 512 : 256, back ? 2 : 4}, {512, 4}};
    for (const auto& s : shapes)
        if (n <= s[0] * s[1]) return {s[0], s[1], shift};
    return {0, 0, shift};
}

// Slots of a walk: as many blocks as the machine's 152 multiprocessors hold at once (rows of a warp go
// four to a block), with at least two rows each; a multiple of 8, the largest V, so that a slot's rows
// start alike
int parts_of(int64_t T, const Shape& s) {
    const int slots = s.nt ? 152 * (512 / s.nt) : 32;
    const int64_t want = s.nt ? (T + 1) / 2 : T;
    const int parts = int(want < 1 ? 1 : want < slots ? want : slots);
    return s.nt && s.shift ? (parts + 7) / 8 * 8 : parts;
}

template <auto* F>
void ring_launch(unsigned blocks, int threads, size_t smem, const LnArgs& a, cudaStream_t st) {
    static unsigned long long done;
    allow_smem((const void*)F, smem, &done);
    F<<<blocks, threads, smem, st>>>(a);
}

template <class E, int V, int K, int NT, bool SHIFT>
void fwd(LnArgs a, const Shape& s, cudaStream_t st) {
    // a walk pays off from four rows per slot on; fewer rows spread one per block (or warp)
    const int parts = parts_of(a.T, s);
    if (a.T >= 4 * int64_t(parts)) {
        a.parts = parts;
        const unsigned blocks = unsigned(NT == 32 ? (parts + LN_WARP_ROWS - 1) / LN_WARP_ROWS : parts);
        if (a.res) ring_launch<k_ln_fwd_walk<E, V, K, NT, true, SHIFT>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 2>(), a, st);
        else ring_launch<k_ln_fwd_walk<E, V, K, NT, false, SHIFT>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 1>(), a, st);
        return;
    }
    const int64_t blocks = NT == 32 ? (a.T + LN_WARP_ROWS - 1) / LN_WARP_ROWS : a.T;
    k_ln_fwd<E, V, K, NT, SHIFT><<<unsigned(blocks), ln_block<NT>(), 0, st>>>(a);
}
template <class E, int V, int K, int NT, bool SHIFT>
void bwd(const LnArgs& a, cudaStream_t st) {
    const unsigned blocks = unsigned(NT == 32 ? (a.parts + LN_WARP_ROWS - 1) / LN_WARP_ROWS : a.parts);
    if (a.dsum) ring_launch<k_ln_bwd<E, V, K, NT, true, SHIFT>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 3>(), a, st);
    else ring_launch<k_ln_bwd<E, V, K, NT, false, SHIFT>>(blocks, ln_block<NT>(), ln_ring_bytes<V, K, NT, 2>(), a, st);
}
template <class E, int V, int K, int NT>
void run(const LnArgs& a, const Shape& s, bool back, cudaStream_t st) {
    if (back) {
        if constexpr (NT != 256 || K != 4) s.shift ? bwd<E, V, K, NT, true>(a, st) : bwd<E, V, K, NT, false>(a, st);
    } else {
        if constexpr (NT != 512 || K != 2) s.shift ? fwd<E, V, K, NT, true>(a, s, st) : fwd<E, V, K, NT, false>(a, s, st);
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
