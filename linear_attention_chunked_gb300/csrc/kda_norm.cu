// Layer norm over rows of C channels, forward and backward.
//
//   v = x + res (rounded to the row type, as it is handed on; v = x without res)
//   mean = sum v / C,  rstd = 1 / sqrt(sum (v - mean)^2 / C + eps),  xh = (v - mean) rstd
//   y = xh w + b
//   d = dy w:  dv = rstd (d - mean(d) - xh mean(d xh)) + dsum,  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by HBM: forward 2 (4 with res) and backward 3 (4 with dsum) row transfers.  A row is held in
// the registers of a warp, four warps or sixteen, so it is read once and the variance is taken
// about the mean (no cancellation).  The backward keeps its columns' dw and db terms in registers
// over the rows a block walks, and a second kernel adds the blocks' sums in order: results are
// bitwise reproducible.  Rows too long for the registers take kernels that read them again.
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
    float* part;  // [blocks][2][C] partial dw, db
    int parts;
};

// V consecutive elements (one 16-byte access when V > 1)
template <class E, int V>
struct Vec {
    E e[V];
};
template <class E, int V>
__device__ __forceinline__ Vec<E, V> ln_load(const void* p, int64_t i) {
    Vec<E, V> r;
    if constexpr (V > 1) *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(static_cast<const E*>(p) + i);
    else r.e[0] = static_cast<const E*>(p)[i];
    return r;
}
template <class E, int V>
__device__ __forceinline__ void ln_store(void* p, int64_t i, const Vec<E, V>& r) {
    if constexpr (V > 1) *reinterpret_cast<uint4*>(static_cast<E*>(p) + i) = *reinterpret_cast<const uint4*>(&r);
    else static_cast<E*>(p)[i] = r.e[0];
}
template <class E> __device__ __forceinline__ E ln_cast(float v);
template <> __device__ __forceinline__ float ln_cast<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 ln_cast<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half ln_cast<__half>(float v) { return __float2half_rn(v); }
template <class E> __device__ __forceinline__ float ln_f(E v) { return ssm_ld<E>(&v, 0); }

// V consecutive fp32 parameters
template <int V>
__device__ __forceinline__ void ln_par(const float* p, int c, float (&f)[V], float none) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = none;
    } else if constexpr (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 t = *reinterpret_cast<const float4*>(p + c + j);
            f[j] = t.x, f[j + 1] = t.y, f[j + 2] = t.z, f[j + 3] = t.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = p[c + j];
    }
}

// Sum over the NT threads of a row; `buf` is a fresh slot of NT / 32 floats per call and row
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if constexpr (NT > 32) {
        const int w = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[w] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) v += buf[i];
    }
    return v;
}

constexpr int LN_WARP_ROWS = 4;  // rows per block when a row takes one warp
template <int NT> __host__ __device__ constexpr int ln_block() { return NT == 32 ? 32 * LN_WARP_ROWS : NT; }

// K vectors of V elements per thread, NT threads per row
template <class E, int V, int K, int NT>
__global__ void __launch_bounds__(ln_block<NT>()) k_ln_fwd(LnArgs a) {
    __shared__ float buf[2][NT / 32];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = NT == 32 ? int64_t(blockIdx.x) * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    if (NT == 32 && row >= a.T) return;
    const int64_t base = row * a.C;
    const float inv = 1.f / float(a.C);
    float f[K][V];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * NT + tid) * V;
        if (c < a.C) {
            Vec<E, V> x = ln_load<E, V>(a.x, base + c);
            if (a.res) {
                const Vec<E, V> r = ln_load<E, V>(a.res, base + c);
#pragma unroll
                for (int j = 0; j < V; ++j) x.e[j] = ln_cast<E>(ln_f<E>(x.e[j]) + ln_f<E>(r.e[j]));
                if (a.sum) ln_store<E, V>(a.sum, base + c, x);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) s += f[k][j] = ln_f<E>(x.e[j]);
        }
    }
    const float mean = row_sum<NT>(s, buf[0]) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        if ((k * NT + tid) * V < a.C)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                f[k][j] -= mean;
                s = fmaf(f[k][j], f[k][j], s);
            }
    const float rstd = rsqrtf(row_sum<NT>(s, buf[1]) * inv + a.eps);
    if (tid == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (k * NT + tid) * V;
        if (c < a.C) {
            float w[V], b[V];
            ln_par<V>(a.w, c, w, 1.f);
            ln_par<V>(a.b, c, b, 0.f);
            Vec<E, V> y;
#pragma unroll
            for (int j = 0; j < V; ++j) y.e[j] = ln_cast<E>(fmaf(f[k][j] * rstd, w[j], b[j]));
            ln_store<E, V>(a.y, base + c, y);
        }
    }
}

// The rows r = slot, slot + slots, .. of a slot (a block, or a warp where a row takes one)
template <class E, int V, int K, int NT>
__global__ void __launch_bounds__(ln_block<NT>()) k_ln_bwd(LnArgs a) {
    __shared__ float buf[2][2][NT / 32];
    const int tid = NT == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int slot = NT == 32 ? blockIdx.x * LN_WARP_ROWS + (threadIdx.x >> 5) : blockIdx.x;
    const float inv = 1.f / float(a.C);
    float dw[K][V], db[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] = db[k][j] = 0.f;
    // the next row's loads start before the current row's sums, while the registers hold both
    constexpr bool AHEAD = K * V <= 16;
    Vec<E, V> x[K], g[K], nx[K], ng[K];
    float mean = 0.f, rstd = 0.f;
    auto load = [&](Vec<E, V>(&vx)[K], Vec<E, V>(&vg)[K], int64_t row) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * NT + tid) * V;
            if (c < a.C) {
                vx[k] = ln_load<E, V>(a.x, row * a.C + c);
                vg[k] = ln_load<E, V>(a.dy, row * a.C + c);
            }
        }
        mean = a.mean_in[row];
        rstd = a.rstd_in[row];
    };
    const int64_t T = slot < a.parts ? a.T : 0;  // (a block of warps may reach past the slots)
    if (AHEAD && slot < T) load(nx, ng, slot);
    int odd = 0;
    for (int64_t row = slot; row < T; row += a.parts, odd ^= 1) {
        if (!AHEAD) load(nx, ng, row);
#pragma unroll
        for (int k = 0; k < K; ++k) x[k] = nx[k], g[k] = ng[k];
        const float m = mean, r = rstd;
        if (AHEAD && row + a.parts < T) load(nx, ng, row + a.parts);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * NT + tid) * V;
            if (c < a.C) {
                float w[V];
                ln_par<V>(a.w, c, w, 1.f);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (ln_f<E>(x[k].e[j]) - m) * r, q = ln_f<E>(g[k].e[j]), d = __fmul_rn(q, w[j]);
                    dw[k][j] = fmaf(q, xh, dw[k][j]);
                    db[k][j] += q;
                    s0 += d;
                    s1 = fmaf(d, xh, s1);
                }
            }
        }
        s0 = row_sum<NT>(s0, buf[odd][0]) * inv;
        s1 = row_sum<NT>(s1, buf[odd][1]) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * NT + tid) * V;
            if (c < a.C) {
                float w[V];
                ln_par<V>(a.w, c, w, 1.f);
                Vec<E, V> o, e;
                if (a.dsum) e = ln_load<E, V>(a.dsum, row * a.C + c);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float xh = (ln_f<E>(x[k].e[j]) - m) * r;
                    float t = r * (__fmul_rn(ln_f<E>(g[k].e[j]), w[j]) - s0 - xh * s1);  // d as it was summed
                    if (a.dsum) t += ln_f<E>(e.e[j]);
                    o.e[j] = ln_cast<E>(t);
                }
                ln_store<E, V>(a.dx, row * a.C + c, o);
            }
        }
    }
    if (slot < a.parts) {
        float* p = a.part + int64_t(slot) * 2 * a.C;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (k * NT + tid) * V;
            if (c < a.C)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    p[c + j] = dw[k][j];
                    p[a.C + c + j] = db[k][j];
                }
        }
    }
}

// dw, db: column sums of the partials.  32 columns x 8 strands of parts per block; a strand's parts
// are added in order, then the strands.
__global__ void k_ln_reduce(LnArgs a, float* dw, float* db) {
    __shared__ float s[8][33];
    const int cx = threadIdx.x & 31, st = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;  // column of [2 C]
    float v = 0.f;
    if (c < 2 * a.C) {
        const float* p = a.part + c;
#pragma unroll 4
        for (int i = st; i < a.parts; i += 8) v += p[int64_t(i) * 2 * a.C];
    }
    s[st][cx] = v;
    __syncthreads();
    if (st == 0 && c < 2 * a.C) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][cx];
        if (c < a.C) { if (dw) dw[c] = v; }
        else if (db) db[c - a.C] = v;
    }
}

// ---- rows of any length: re-read instead of held ----

constexpr int LONG_NT = 1024;

template <class E>
__global__ void __launch_bounds__(LONG_NT) k_ln_fwd_long(LnArgs a) {
    __shared__ float buf[2][LONG_NT / 32];
    const int64_t row = blockIdx.x, base = row * a.C;
    const float inv = 1.f / float(a.C);
    auto val = [&](int c) {
        const float v = ssm_ld<E>(a.x, base + c);
        return a.res ? ln_f<E>(ln_cast<E>(v + ssm_ld<E>(a.res, base + c))) : v;
    };
    float s = 0.f;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float v = val(c);
        s += v;
    }
    const float mean = row_sum<LONG_NT>(s, buf[0]) * inv;
    s = 0.f;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float v = val(c) - mean;
        s = fmaf(v, v, s);
    }
    const float rstd = rsqrtf(row_sum<LONG_NT>(s, buf[1]) * inv + a.eps);
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
    __shared__ float buf[2][LONG_NT / 32];
    const int64_t row = blockIdx.x, base = row * a.C;
    const float inv = 1.f / float(a.C), mean = a.mean_in[row], rstd = a.rstd_in[row];
    float s0 = 0.f, s1 = 0.f;
    for (int c = threadIdx.x; c < a.C; c += LONG_NT) {
        const float d = __fmul_rn(ssm_ld<E>(a.dy, base + c), a.w ? a.w[c] : 1.f);
        s0 += d;
        s1 = fmaf(d, (ssm_ld<E>(a.x, base + c) - mean) * rstd, s1);
    }
    s0 = row_sum<LONG_NT>(s0, buf[0]) * inv;
    s1 = row_sum<LONG_NT>(s1, buf[1]) * inv;
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
// registers hold the row (a warp up to 4 vectors a lane, then 128, then 512 threads).  wide: rows
// are whole 16-byte vectors.  nt = 0: the re-reading kernels.
struct Shape { int nt, k; bool wide; };
Shape shape_of(int C, int esize) {
    const int V = 16 / esize;
    if (C % V == 0) {
        const int n = C / V;
        for (int nt : {32, 128, 512})
            for (int k : {1, 2, 4})
                if (n <= nt * k) return {nt, k, true};
        return {0, 0, true};
    }
    for (int nt : {32, 128, 512})
        if (C <= nt * 16) return {nt, 16, false};
    return {0, 0, false};
}

// Partial sums of the backward: rows are dealt to this many slots (two blocks of 512 threads per
// multiprocessor or the same number of threads in smaller blocks)
int parts_of(int64_t T, const Shape& s) {
    const int slots = s.nt == 512 ? 304 : s.nt == 128 ? 1216 : s.nt == 32 ? 2432 : 32;
    // a slot walks at least two rows where there are rows enough: fewer partial sums to add
    const int64_t want = s.nt ? (T + 1) / 2 : T;
    return int(want < 1 ? 1 : want < slots ? want : slots);
}

template <class E, int V, int K, int NT>
void fwd(const LnArgs& a, cudaStream_t st) {
    const int64_t blocks = NT == 32 ? (a.T + LN_WARP_ROWS - 1) / LN_WARP_ROWS : a.T;
    k_ln_fwd<E, V, K, NT><<<unsigned(blocks), ln_block<NT>(), 0, st>>>(a);
}
template <class E, int V, int K, int NT>
void bwd(const LnArgs& a, cudaStream_t st) {
    const int blocks = NT == 32 ? (a.parts + LN_WARP_ROWS - 1) / LN_WARP_ROWS : a.parts;
    k_ln_bwd<E, V, K, NT><<<unsigned(blocks), ln_block<NT>(), 0, st>>>(a);
}
template <class E, int V, int K>
void by_threads(const LnArgs& a, const Shape& s, bool back, cudaStream_t st) {
    if (s.nt == 32) back ? bwd<E, V, K, 32>(a, st) : fwd<E, V, K, 32>(a, st);
    else if (s.nt == 128) back ? bwd<E, V, K, 128>(a, st) : fwd<E, V, K, 128>(a, st);
    else back ? bwd<E, V, K, 512>(a, st) : fwd<E, V, K, 512>(a, st);
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
    } else if (!s.wide) by_threads<E, 1, 16>(a, s, back, st);
    else if (s.k == 1) by_threads<E, V, 1>(a, s, back, st);
    else if (s.k == 2) by_threads<E, V, 2>(a, s, back, st);
    else by_threads<E, V, 4>(a, s, back, st);
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
    if (ws_bytes) *ws_bytes = align256(size_t(parts_of(p->T, shape_of(p->C, esize(p->dtype)))) * 2 * size_t(p->C) * 4);
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
        by_type(a, p->dtype, shape_of(p->C, esize(p->dtype)), false, st);
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_layernorm_bwd(const kda_layernorm_problem* p, const void* x, const float* w, const float* mean,
                             const float* rstd, const void* dy, const void* dsum, void* dx, float* dw, float* db,
                             void* ws, size_t ws_bytes, kda_stream_t stream) {
    if (kda_status s = check(p)) return s;
    if (p->T > 0 && !(req(x) && req(mean) && req(rstd) && req(dy) && req(dx))) return KDA_ERR_INVALID_ARG;
    if (!opt(w) || !opt(dsum) || !opt(dw) || !opt(db) || !req(ws)) return KDA_ERR_INVALID_ARG;
    const Shape s = shape_of(p->C, esize(p->dtype));
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
        k_ln_reduce<<<unsigned((2 * p->C + 31) / 32), 256, 0, st>>>(a, dw, db);
    }
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
