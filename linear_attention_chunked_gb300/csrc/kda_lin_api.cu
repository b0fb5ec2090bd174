// Host side of the linear attention's entry points: validation, workspace, launches.
#include <mutex>

#include "kda_lin.cuh"

using namespace kda;

namespace {

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool req(const void* p) { return p && al(p, 16); }
bool opt(const void* p) { return al(p, 16); }
int64_t ld_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

std::mutex g_mu;
bool g_ready[128];

// Once per device: that it is an sm_103 part, and the walks' shared memory limits.
kda_status setup_lin() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
    if (dev < 0 || dev >= 128) return KDA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_ready[dev]) return KDA_OK;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (major != 10 || minor != 3) return KDA_ERR_UNSUPPORTED;
    if (lin_setup() != cudaSuccess) return KDA_ERR_CUDA;
    g_ready[dev] = true;
    return KDA_OK;
}

// cuTensorMapEncodeTiled, looked up once through the runtime (no link-time libcuda dependency).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// Whether long documents are cut into segments, and the tokens of one (a power of two).  This depends on the heads
// alone: a document's results must not depend on the pack.  A walk takes 2.4 us a chunk where its block does not wait for
// HBM, so a document of 16384 tokens takes 0.305 ms uncut, whatever the heads up to the multiprocessors' number; cut, its
// states between segments cost a second pass over two of the rows: forward 0.094 ms at 16 heads, 0.171 at 32, 0.248 at 48,
// 0.34 at 64.  A backward walks three times as many heads: cut 0.183 ms at 16, uncut 0.306 at 24 to 48.  Segments of
// 2048 tokens make one wave of blocks of 16384 tokens and 16 heads; fewer heads take shorter ones.
bool cuts(int H, bool back) { return H < (back ? 24 : 64); }
int segment(int H) {
    int s = 512;
    while (s < 128 * H && s < LIN_WHOLE) s *= 2;
    return s;
}
// Segments that a document set may have, and slots between them
int64_t max_segments(const kda_linattn_problem* p) { return p->T / segment(p->H) + p->N; }
size_t slot_bytes(const kda_linattn_problem* p, bool back) {
    return cuts(p->H, back) && p->T > LIN_WHOLE ? size_t(p->T / segment(p->H)) * size_t(p->H) * D * D * 4 : 0;
}

kda_status check_sizes(const kda_linattn_problem* p) {
    if (!p || p->T < 0 || p->T > INT32_MAX - 8192 || p->N < 1 || p->N > 65535 || p->H < 1 || p->H > 65535 ||
        p->Hk < 1 || p->H % p->Hk)
        return KDA_ERR_INVALID_ARG;
    if (p->dtype != KDA_DT_BF16 && p->dtype != KDA_DT_FP16 && p->dtype != KDA_DT_FP32) return KDA_ERR_INVALID_ARG;
    if (p->d != D || p->dtype != KDA_DT_BF16) return KDA_ERR_UNSUPPORTED;
    const int64_t dk = int64_t(p->Hk) * D, dv = int64_t(p->H) * D;
    for (int64_t ld : {p->ld_q, p->ld_k, p->ld_v})
        if (ld % 8) return KDA_ERR_INVALID_ARG;
    if (ld_or(p->ld_q, dk) < dk || ld_or(p->ld_k, dk) < dk || ld_or(p->ld_v, dv) < dv) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

kda_status check_problem(const kda_linattn_problem* p) {
    if (kda_status s = check_sizes(p)) return s;
    if (!p->cu_seqlens || !al(p->cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    // one-dimensional grids
    if (max_segments(p) * p->H > INT32_MAX / 16 || p->T * p->Hk / 8 >= INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

struct Regions {
    size_t status, tab, multi, counts, front, back, share_q, share_k;  // inside the workspace
    size_t fwd, bwd_saved, bwd_replay;
    size_t kept, saved;  // inside the saved set: the slots behind its header
};

Regions regions(const kda_linattn_problem* p) {
    Regions r{};
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
    r.status = take(256);
    r.counts = take(2 * sizeof(int));
    r.tab = take(size_t(max_segments(p)) * sizeof(int4));
    r.multi = take(size_t(p->T / LIN_WHOLE) * sizeof(int4));
    const size_t plan = o, kept = slot_bytes(p, true);  // the backward reads the forward's slots where it cuts
    r.front = take(slot_bytes(p, false));
    r.fwd = o;
    o = plan;
    r.back = take(kept);
    if (p->Hk < p->H) {  // each head's part of dq and dk
        r.share_q = take(size_t(p->T) * p->H * D * 4);
        r.share_k = take(size_t(p->T) * p->H * D * 4);
    }
    r.bwd_saved = o;
    r.bwd_replay = o + kept;
    r.kept = 256;
    r.saved = 256 + kept;
    return r;
}

LinArgs make_args(const kda_linattn_problem* p, const Regions& r, bool back, const float* slope, void* ws) {
    LinArgs a{};
    char* w = static_cast<char*>(ws);
    a.T = p->T;
    a.N = p->N;
    a.H = p->H;
    a.seg = segment(p->H);
    a.direct = !cuts(p->H, back) || p->T <= LIN_WHOLE;
    a.cu = p->cu_seqlens;
    a.slope = slope;
    a.status = static_cast<int*>(ws);
    a.sizes = make_int4(int(p->T), p->N, p->H, p->Hk);
    a.plan = {reinterpret_cast<int4*>(w + r.tab), reinterpret_cast<int4*>(w + r.multi), reinterpret_cast<int*>(w + r.counts)};
    return a;
}

using bf = __nv_bfloat16;

// The rows of a call, in the order of LinMaps
enum { IN_Q, IN_K, IN_V, IN_DO, OUT_O, OUT_DV, OUT_DK, OUT_DQ = OUT_O };

// share: heads that share a row of q and k
LinPass make_pass(int query, int key, int value, int share, int store, void* out, int out_fp32, const float* s0,
                  float* s_end, int trans, int back, float in, float by) {
    auto per = [&](int t) { return t == IN_Q || t == IN_K ? share : 1; };
    return {query, key, value, store, per(query), per(key), per(value), out, out_fp32, s0, s_end, trans, back, in, by};
}

struct Rows {
    const void* p;
    int heads;
    int64_t ld;  // 0: dense
};
kda_status make_maps(int64_t T, const Rows (&rows)[7], LinMaps* tm) {
    if (T == 0) return KDA_OK;  // no row is read
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return KDA_ERR_CUDA;
    for (int i = 0; i < 7; ++i) {
        const Rows& r = rows[i];
        if (!r.p) continue;
        const cuuint64_t dims[4] = {64, cuuint64_t(T), 2, cuuint64_t(r.heads)};
        const cuuint64_t strides[3] = {cuuint64_t(ld_or(r.ld, int64_t(r.heads) * D)) * 2, 128, D * 2};
        const cuuint32_t box[4] = {64, LC, 2, 1}, one[4] = {1, 1, 1, 1};
        if (enc(&tm->m[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(r.p), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

// dq and dk of a shared head: the sum of its heads' parts, in head order, rounded once.
__global__ void __launch_bounds__(256) k_lin_share(const float* pq, const float* pk, bf* dq, bf* dk, int64_t rows,
                                                   int share, const int* status) {
    if (*status != KDA_OK) return;
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= rows * D) return;
    const float* p = blockIdx.y ? pk : pq;
    const int64_t row = i / D, c = i % D;  // row: token * Hk + head
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < share; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(p + (row * share + j) * D + c);
        s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    *reinterpret_cast<uint2*>((blockIdx.y ? dk : dq) + i) = make_uint2(pack2(s.x, s.y), pack2(s.z, s.w));
}

kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

kda_status kda_linattn_workspace_size(const kda_linattn_problem* p, int op, size_t* ws_bytes, size_t* saved_bytes) {
    if (kda_status s = check_problem(p)) return s;
    const Regions r = regions(p);
    size_t w = 0;
    if (op == KDA_OP_FWD) w = r.fwd;
    else if (op == KDA_OP_BWD_SAVED) w = r.bwd_saved;
    else if (op == KDA_OP_BWD_REPLAY) w = r.bwd_replay;
    else return KDA_ERR_INVALID_ARG;
    if (ws_bytes) *ws_bytes = w;
    if (saved_bytes) *saved_bytes = r.saved;
    return KDA_OK;
}

kda_status kda_linattn_fwd(const kda_linattn_problem* p, const void* q, const void* k, const void* v,
                           const float* slope, const float* h0, void* o, float* ht, void* saved, void* ws,
                           size_t ws_bytes, kda_stream_t stream) {
    if (kda_status s = check_problem(p)) return s;
    if (p->T > 0 && !(req(q) && req(k) && req(v) && req(o))) return KDA_ERR_INVALID_ARG;
    if (!req(slope) || !opt(h0) || !opt(ht) || !opt(saved) || !req(ws)) return KDA_ERR_INVALID_ARG;
    const Regions r = regions(p);
    if (ws_bytes < r.fwd) return KDA_ERR_WORKSPACE;
    if (ht && ht == h0) return KDA_ERR_INVALID_ARG;  // blocks of a document's ends read the one and write the other
    if (kda_status s = setup_lin()) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LinArgs a = make_args(p, r, false, slope, ws);
    LinMaps tm{};
    const Rows rows[7] = {{q, p->Hk, p->ld_q}, {k, p->Hk, p->ld_k}, {v, p->H, p->ld_v}, {}, {o, p->H, 0}};
    if (kda_status s = make_maps(p->T, rows, &tm)) return s;
    a.made_for = static_cast<int4*>(saved);
    a.front = reinterpret_cast<float*>(saved && cuts(p->H, true) ? static_cast<char*>(saved) + r.kept
                                                                 : static_cast<char*>(ws) + r.front);
    a.passes = 1;
    a.pass[0] = make_pass(IN_Q, IN_K, IN_V, p->H / p->Hk, OUT_O, o, 0, h0, ht, 0, 0, 1.f, p->scale);
    if (a.direct) {
        if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    } else {
        launch_lin_plan(a, st);
        launch_lin_states(a, tm, 0, st);
    }
    launch_lin_walk(a, tm, st);
    return launched();
}

kda_status kda_linattn_bwd(const kda_linattn_problem* p, const void* q, const void* k, const void* v,
                           const float* slope, const float* h0, const void* dO, const float* dht, const void* saved,
                           void* dq, void* dk, void* dv, float* dh0, void* ws, size_t ws_bytes,
                           kda_stream_t stream) {
    if (kda_status s = check_problem(p)) return s;
    if (p->T > 0 && !(req(q) && req(k) && req(v) && req(dO) && req(dq) && req(dk) && req(dv)))
        return KDA_ERR_INVALID_ARG;
    if (!req(slope) || !opt(h0) || !opt(dht) || !opt(saved) || !opt(dh0) || !req(ws)) return KDA_ERR_INVALID_ARG;
    const Regions r = regions(p);
    if (ws_bytes < (saved ? r.bwd_saved : r.bwd_replay)) return KDA_ERR_WORKSPACE;
    // three walks read the inputs side by side while they write the outputs
    if (dh0 && (dh0 == h0 || dh0 == dht)) return KDA_ERR_INVALID_ARG;
    for (const void* out : {dq, dk, dv})
        if (p->T > 0 && (out == q || out == k || out == v || out == dO)) return KDA_ERR_INVALID_ARG;
    if (kda_status s = setup_lin()) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LinArgs a = make_args(p, r, true, slope, ws);
    LinMaps tm{};
    char* w = static_cast<char*>(ws);
    const int share = p->H / p->Hk, part = share > 1;
    const Rows none{};
    const Rows rows[7] = {{q, p->Hk, p->ld_q}, {k, p->Hk, p->ld_k}, {v, p->H, p->ld_v}, {dO, p->H, 0},
                          part ? none : Rows{dq, p->H, 0}, {dv, p->H, 0}, part ? none : Rows{dk, p->H, 0}};
    if (kda_status s = make_maps(p->T, rows, &tm)) return s;
    float* pq = reinterpret_cast<float*>(w + r.share_q);
    float* pk = reinterpret_cast<float*>(w + r.share_k);
    a.expected = static_cast<const int4*>(saved);
    a.front = reinterpret_cast<float*>(saved ? const_cast<char*>(static_cast<const char*>(saved)) + r.kept : w + r.bwd_saved);
    a.back = reinterpret_cast<float*>(w + r.back);
    if (a.direct) {
        if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    } else {
        launch_lin_plan(a, st);
        if (!saved) {  // the states between segments, as the forward's
            a.pass[0] = make_pass(IN_Q, IN_K, IN_V, share, 0, nullptr, 0, h0, nullptr, 0, 0, 1.f, p->scale);
            launch_lin_states(a, tm, 0, st);
        }
        a.pass[0] = make_pass(IN_K, IN_Q, IN_DO, share, 0, nullptr, 0, dht, nullptr, 0, 1, p->scale, 1.f);
        launch_lin_states(a, tm, 0, st);
    }
    a.passes = 3;
    a.pass[0] = make_pass(IN_DO, IN_V, IN_K, share, OUT_DQ, part ? static_cast<void*>(pq) : dq, part, h0, nullptr, 1, 0, 1.f, p->scale);
    a.pass[1] = make_pass(IN_K, IN_Q, IN_DO, share, OUT_DV, dv, 0, dht, dh0, 0, 1, p->scale, 1.f);
    a.pass[2] = make_pass(IN_V, IN_DO, IN_Q, share, OUT_DK, part ? static_cast<void*>(pk) : dk, part, dht, nullptr, 1, 1, p->scale, 1.f);
    launch_lin_walk(a, tm, st);
    if (part && p->T > 0) {
        const int64_t rows = p->T * p->Hk;
        ProfScope ps(KK_LIN_SHARE, st);
        k_lin_share<<<dim3(unsigned((rows * D / 4 + 255) / 256), 2), 256, 0, st>>>(
            pq, pk, static_cast<bf*>(dq), static_cast<bf*>(dk), rows, share, a.status);
    }
    return launched();
}

kda_status kda_linattn_step(const kda_linattn_problem* p, const void* q, const void* k, const void* v,
                            const float* slope, const int32_t* slots, int64_t n_slots, const float* h_in,
                            float* h_out, void* o, void* ws, kda_stream_t stream) {
    if (!p) return KDA_ERR_INVALID_ARG;
    kda_linattn_problem pr = *p;
    pr.T = pr.N;  // one token per sequence; T and cu_seqlens are not read
    if (kda_status s = check_sizes(&pr)) return s;
    if (int64_t(pr.N) * pr.H > INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (!req(q) || !req(k) || !req(v) || !req(slope) || !req(h_in) || !req(h_out) || !req(o) || !al(slots, 4) ||
        !opt(ws) || n_slots < 1 || (!slots && n_slots < pr.N))
        return KDA_ERR_INVALID_ARG;
    const int64_t dk = int64_t(pr.Hk) * D, dv = int64_t(pr.H) * D;
    const LinStepArgs a{pr.N, pr.H, pr.H / pr.Hk, ld_or(pr.ld_q, dk), ld_or(pr.ld_k, dk), ld_or(pr.ld_v, dv), n_slots,
                        pr.scale, static_cast<const bf*>(q), static_cast<const bf*>(k), static_cast<const bf*>(v), slope,
                        h_in, slots, h_out, static_cast<bf*>(o), static_cast<int*>(ws)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    launch_lin_step(a, st);
    return launched();
}

}  // extern "C"
