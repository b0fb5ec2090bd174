// Host side of the linear attention's entry points: validation, workspace, launches.
#include "kda_lin.cuh"

using namespace kda;

namespace {

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool req(const void* p) { return p && al(p, 16); }
bool opt(const void* p) { return al(p, 16); }
int64_t ld_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

// Once per device and process: that it is an sm_103 part.
kda_status setup_lin() {
    static unsigned long long ready[2];
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
    if (dev < 0 || dev >= 128) return KDA_ERR_UNSUPPORTED;
    const unsigned long long bit = 1ull << (dev & 63);
    if (__atomic_load_n(&ready[dev >> 6], __ATOMIC_ACQUIRE) & bit) return KDA_OK;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (major != 10 || minor != 3) return KDA_ERR_UNSUPPORTED;
    __atomic_fetch_or(&ready[dev >> 6], bit, __ATOMIC_RELEASE);
    return KDA_OK;
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
    if (int64_t(p->N) * p->H > INT32_MAX / 3 || p->T * p->Hk / 8 >= INT32_MAX) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

struct Regions {
    size_t status, share_q, share_k;  // inside the workspace
    size_t fwd, bwd;
    size_t saved;
};

Regions regions(const kda_linattn_problem* p) {
    Regions r{};
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
    r.status = take(256);
    r.fwd = o;
    if (p->Hk < p->H) {  // each head's part of dq and dk
        r.share_q = take(size_t(p->T) * p->H * D * 4);
        r.share_k = take(size_t(p->T) * p->H * D * 4);
    }
    r.bwd = o;
    r.saved = 256;
    return r;
}

LinArgs make_args(const kda_linattn_problem* p, const float* slope, void* ws) {
    LinArgs a{};
    a.T = p->T;
    a.N = p->N;
    a.H = p->H;
    a.cu = p->cu_seqlens;
    a.slope = slope;
    a.status = static_cast<int*>(ws);
    a.sizes = make_int4(int(p->T), p->N, p->H, p->Hk);
    return a;
}

using bf = __nv_bfloat16;

// q, k, v and dO as a walk's rows
struct Rows {
    const bf* p;
    int64_t ld;
    int share;
};
struct Inputs {
    Rows q, k, v, dO;
    Inputs(const kda_linattn_problem* p, const void* q_, const void* k_, const void* v_, const void* dO_) {
        const int64_t dk = int64_t(p->Hk) * D, dv = int64_t(p->H) * D;
        const int share = p->H / p->Hk;
        q = {static_cast<const bf*>(q_), ld_or(p->ld_q, dk), share};
        k = {static_cast<const bf*>(k_), ld_or(p->ld_k, dk), share};
        v = {static_cast<const bf*>(v_), ld_or(p->ld_v, dv), 1};
        dO = {static_cast<const bf*>(dO_), dv, 1};
    }
};

LinPass make_pass(const Rows& query, const Rows& key, const Rows& value, void* out, int out_fp32, const float* s0,
                  float* s_end, int trans, int back, float in, float by) {
    return {query.p, key.p, value.p, query.ld, key.ld, value.ld, query.share, key.share, value.share,
            out, out_fp32, s0, s_end, trans, back, in, by};
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
    else if (op == KDA_OP_BWD_SAVED) w = r.bwd;
    else if (op == KDA_OP_BWD_REPLAY) w = r.bwd;
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
    if (kda_status s = setup_lin()) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LinArgs a = make_args(p, slope, ws);
    const Inputs in(p, q, k, v, nullptr);
    if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    a.made_for = static_cast<int4*>(saved);
    a.passes = 1;
    a.pass[0] = make_pass(in.q, in.k, in.v, o, 0, h0, ht, 0, 0, 1.f, p->scale);
    launch_lin_walk(a, st);
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
    if (ws_bytes < r.bwd) return KDA_ERR_WORKSPACE;
    if (kda_status s = setup_lin()) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    LinArgs a = make_args(p, slope, ws);
    const Inputs in(p, q, k, v, dO);
    const int part = p->Hk < p->H;
    float* pq = reinterpret_cast<float*>(static_cast<char*>(ws) + r.share_q);
    float* pk = reinterpret_cast<float*>(static_cast<char*>(ws) + r.share_k);
    if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    a.expected = static_cast<const int4*>(saved);
    a.passes = 3;
    a.pass[0] = make_pass(in.dO, in.v, in.k, part ? static_cast<void*>(pq) : dq, part, h0, nullptr, 1, 0, 1.f, p->scale);
    a.pass[1] = make_pass(in.k, in.q, in.dO, dv, 0, dht, dh0, 0, 1, p->scale, 1.f);
    a.pass[2] = make_pass(in.v, in.dO, in.q, part ? static_cast<void*>(pk) : dk, part, dht, nullptr, 1, 1, p->scale, 1.f);
    launch_lin_walk(a, st);
    if (part && p->T > 0) {
        const int64_t rows = p->T * p->Hk;
        ProfScope ps(KK_LIN_SHARE, st);
        k_lin_share<<<dim3(unsigned((rows * D / 4 + 255) / 256), 2), 256, 0, st>>>(
            pq, pk, static_cast<bf*>(dq), static_cast<bf*>(dk), rows, p->H / p->Hk, a.status);
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
    const Inputs in(&pr, q, k, v, nullptr);
    const LinStepArgs a{pr.N, pr.H, pr.H / pr.Hk, in.q.ld, in.k.ld, in.v.ld, n_slots, pr.scale, in.q.p, in.k.p,
                        in.v.p, slope, h_in, slots, h_out, static_cast<bf*>(o), static_cast<int*>(ws)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    launch_lin_step(a, st);
    return launched();
}

}  // extern "C"
