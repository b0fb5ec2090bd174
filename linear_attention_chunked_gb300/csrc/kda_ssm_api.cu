// Host side of the selective state-space scan's entry points: validation, workspace, launches.
#include <mutex>

#include "kda_ssm.cuh"
#include "kda_ssm_launch.cuh"

using namespace kda;

namespace {

std::mutex g_mu;
bool g_ready[128];

// Once per device: shared memory limits of the backward kernels.
kda_status setup_ssm() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return KDA_ERR_CUDA;
    if (dev < 0 || dev >= 128) return KDA_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_ready[dev]) return KDA_OK;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (major != 10 || minor != 3) return KDA_ERR_UNSUPPORTED;
    if (ssm_bwd_setup() != cudaSuccess) return KDA_ERR_CUDA;
    g_ready[dev] = true;
    return KDA_OK;
}

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool req(const void* p) { return p && al(p, 16); }
bool opt(const void* p) { return al(p, 16); }
size_t esize(int dtype) { return dtype == KDA_DT_FP32 ? 4 : 2; }
int64_t ld_or(int64_t ld, int64_t dense) { return ld ? ld : dense; }

kda_status check_sizes(const kda_ssm_problem* p) {
    if (!p || p->T < 0 || p->T > INT32_MAX - 1024 || p->N < 1 || p->N > 65535 || p->C < 1 || p->C > (1 << 20) ||
        p->S < 1 || p->G < 1 || p->C % p->G)
        return KDA_ERR_INVALID_ARG;
    if (p->S > SSM_MAXS) return KDA_ERR_UNSUPPORTED;
    if (p->dtype != KDA_DT_BF16 && p->dtype != KDA_DT_FP16 && p->dtype != KDA_DT_FP32) return KDA_ERR_INVALID_ARG;
    if (p->dt_softplus != 0 && p->dt_softplus != 1) return KDA_ERR_INVALID_ARG;
    const int64_t GS = int64_t(p->G) * p->S;
    if (ld_or(p->ld_u, p->C) < p->C || ld_or(p->ld_dt, p->C) < p->C || ld_or(p->ld_z, p->C) < p->C ||
        ld_or(p->ld_b, GS) < GS || ld_or(p->ld_c, GS) < GS)
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

int64_t max_chunks(const kda_ssm_problem* p) { return (p->T + CH - 1) / CH + p->N; }

kda_status check_problem(const kda_ssm_problem* p) {
    if (kda_status s = check_sizes(p)) return s;
    if (!p->cu_seqlens || !al(p->cu_seqlens, 4)) return KDA_ERR_INVALID_ARG;
    // one-dimensional grids: blocks of at least 8 channels per chunk or of 128 states per document
    const int64_t tiles = int64_t(p->G) * ((p->C / p->G + 7) / 8);
    if (max_chunks(p) * tiles > INT32_MAX || (int64_t(p->C) * p->S + 127) / 128 * p->N > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// The chunk plan (its bytes first in a saved set, or in the workspace), and what follows.
struct Regions {
    size_t status, made_for, nchunks, doc_off, doc_order, chunk_tab, plan;  // inside the plan; its size
    size_t sumdt, hs, gs, pBC, pA;                                // inside the workspace
    size_t head, fwd, bwd_saved, bwd_replay, states, saved;
};

Regions regions(const kda_ssm_problem* p) {
    Regions r{};
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = align256(o + bytes); return at; };
    const size_t nc = size_t(max_chunks(p)), CS = size_t(p->C) * p->S;
    const SsmBwdPlan pl = ssm_bwd_plan(int64_t(nc), p->C, p->S, p->G);
    r.status = take(256);
    r.made_for = r.status + sizeof(int4);  // in the status word's 256 bytes
    r.nchunks = take(sizeof(int));
    r.doc_off = take(sizeof(int) * size_t(p->N + 1));
    r.doc_order = take(sizeof(int) * size_t(p->N));
    r.chunk_tab = take(sizeof(int4) * nc);
    r.plan = o;
    r.sumdt = take(nc * p->C * 4);
    r.head = o;
    r.states = align256(nc * SSM_SUB * CS * 4);
    r.saved = r.plan + r.states;
    r.fwd = r.head + align256(nc * CS * 4);  // without a saved set the chunks' states lie behind the header
    r.gs = take(nc * CS * 4);
    r.pBC = take(size_t(p->G) * pl.splits * size_t(p->T) * 2 * p->S * 4);
    r.pA = take(nc * p->C * size_t(p->S + 2) * 4);
    r.bwd_saved = o;
    r.hs = take(r.states);  // replay's
    r.bwd_replay = o;
    return r;
}

// the chunk plan at `base`
void use_plan(SsmArgs& a, const Regions& r, char* base) {
    a.status = reinterpret_cast<int*>(base + r.status);
    a.nchunks = reinterpret_cast<int*>(base + r.nchunks);
    a.doc_off = reinterpret_cast<int*>(base + r.doc_off);
    a.chunk_tab = reinterpret_cast<int4*>(base + r.chunk_tab);
}

SsmArgs make_args(const kda_ssm_problem* p, const Regions& r, void* ws) {
    SsmArgs a{};
    a.T = p->T;
    a.maxC = max_chunks(p);
    a.N = p->N;
    a.C = p->C;
    a.S = p->S;
    a.G = p->G;
    a.softplus = p->dt_softplus;
    const int64_t GS = int64_t(p->G) * p->S;
    a.ldu = ld_or(p->ld_u, p->C);
    a.lddt = ld_or(p->ld_dt, p->C);
    a.ldz = ld_or(p->ld_z, p->C);
    a.ldb = ld_or(p->ld_b, GS);
    a.ldc = ld_or(p->ld_c, GS);
    a.sizes = make_int4(int(p->T), p->N | p->S << 16, p->C, p->G);
    a.cu = p->cu_seqlens;
    char* w = static_cast<char*>(ws);
    a.call_status = static_cast<int*>(ws);
    use_plan(a, r, w);
    a.sumdt = reinterpret_cast<float*>(w + r.sumdt);
    a.gs = reinterpret_cast<float*>(w + r.gs);
    a.pBC = reinterpret_cast<float*>(w + r.pBC);
    a.pA = reinterpret_cast<float*>(w + r.pA);
    return a;
}

// u, dt, B, C and z are views of the caller's projections: element alignment is enough
kda_status check_inputs(const kda_ssm_problem* p, const void* u, const void* dt, const float* A, const void* B,
                        const void* Cm, const float* Dk, const float* bias, const void* z, const float* h0) {
    const size_t e = esize(p->dtype);
    if (!req(A) || !opt(Dk) || !opt(bias) || !opt(h0) || !al(z, e)) return KDA_ERR_INVALID_ARG;
    if (p->T > 0 && !(u && al(u, e) && dt && al(dt, e) && B && al(B, e) && Cm && al(Cm, e))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

void launch_plan(const SsmArgs& a, const Regions& r, cudaStream_t st) {
    Params q{};
    q.T = a.T;
    q.N = a.N;
    q.cu = a.cu;
    q.maxC = a.maxC;
    q.status = a.status;
    q.nchunks = a.nchunks;
    q.doc_off = a.doc_off;
    q.doc_order = reinterpret_cast<int*>(reinterpret_cast<char*>(a.status) - r.status + r.doc_order);
    q.chunk_tab = a.chunk_tab;
    ProfScope ps(KK_PLAN, st);
    k_plan<<<1, NTHR, 0, st>>>(q);
}

kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

kda_status kda_ssm_workspace_size(const kda_ssm_problem* p, int op, size_t* ws_bytes, size_t* saved_bytes) {
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

kda_status kda_ssm_fwd(const kda_ssm_problem* p, const void* u, const void* dt, const float* A, const void* B,
                       const void* Cm, const float* D_, const float* dt_bias, const void* z, const float* h0,
                       void* y, float* ht, void* saved, void* ws, size_t ws_bytes, kda_stream_t stream) {
    if (kda_status s = check_problem(p)) return s;
    if (kda_status s = check_inputs(p, u, dt, A, B, Cm, D_, dt_bias, z, h0)) return s;
    if ((p->T > 0 && !req(y)) || !opt(y) || !opt(ht) || !opt(saved) || !req(ws)) return KDA_ERR_INVALID_ARG;
    const Regions r = regions(p);
    if (ws_bytes < (saved ? r.head : r.fwd)) return KDA_ERR_WORKSPACE;
    if (kda_status s = setup_ssm()) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    SsmArgs a = make_args(p, r, ws);
    a.u = u, a.dt = dt, a.A = A, a.B = B, a.Cm = Cm, a.D = D_, a.bias = dt_bias, a.z = z, a.h0 = h0;
    a.y = y;
    a.ht = ht;
    // a saved set holds the plan and the states of every 16th token
    a.hs = reinterpret_cast<float*>(saved ? static_cast<char*>(saved) + r.plan : static_cast<char*>(ws) + r.head);
    if (saved) {
        use_plan(a, r, static_cast<char*>(saved));
        a.made_for = reinterpret_cast<int4*>(static_cast<char*>(saved) + r.made_for);
    }
    a.sub = saved ? SSM_SUB : 1;
    // a short prompt (every document within one chunk, few of them): one launch, no plan, no carry
    a.direct = !saved && a.T <= CH && a.N <= 64;
    if (!a.direct) launch_plan(a, r, st);
    launch_ssm_scan(a, p->dtype, st);
    return launched();
}

kda_status kda_ssm_bwd(const kda_ssm_problem* p, const void* u, const void* dt, const float* A, const void* B,
                       const void* Cm, const float* D_, const float* dt_bias, const void* z, const float* h0,
                       const void* dy, const float* dht, const void* saved, void* du, void* ddt, float* dA,
                       void* dB, void* dC, float* dD, float* ddt_bias, void* dz, float* dh0, void* ws,
                       size_t ws_bytes, kda_stream_t stream) {
    if (kda_status s = check_problem(p)) return s;
    if (kda_status s = check_inputs(p, u, dt, A, B, Cm, D_, dt_bias, z, h0)) return s;
    if (p->T > 0 && !(req(dy) && req(du) && req(ddt) && req(dB) && req(dC) && (z ? req(dz) : opt(dz))))
        return KDA_ERR_INVALID_ARG;
    if (!req(dA) || !opt(dht) || !opt(saved) || !opt(dD) || !opt(ddt_bias) || !opt(dh0) || !req(ws))
        return KDA_ERR_INVALID_ARG;
    const Regions r = regions(p);
    if (ws_bytes < (saved ? r.bwd_saved : r.bwd_replay)) return KDA_ERR_WORKSPACE;
    if (kda_status s = setup_ssm()) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    SsmArgs a = make_args(p, r, ws);
    a.u = u, a.dt = dt, a.A = A, a.B = B, a.Cm = Cm, a.D = D_, a.bias = dt_bias, a.z = z, a.h0 = h0;
    a.sub = SSM_SUB;
    if (saved) {
        char* set = static_cast<char*>(const_cast<void*>(saved));
        use_plan(a, r, set);
        a.made_for = reinterpret_cast<int4*>(set + r.made_for);
        a.from_saved = 1;
        a.hs = reinterpret_cast<float*>(set + r.plan);
    } else {  // recompute the states (no y, no final state)
        launch_plan(a, r, st);
        a.hs = reinterpret_cast<float*>(static_cast<char*>(ws) + r.hs);
        launch_ssm_scan(a, p->dtype, st);
    }
    a.dy = dy, a.dht = dht;
    a.du = du, a.ddt = ddt, a.dA = dA, a.dB = dB, a.dC = dC, a.dD = dD, a.dbias = ddt_bias, a.dz = dz, a.dh0 = dh0;
    launch_ssm_bwd(a, p->dtype, st);
    return launched();
}

kda_status kda_ssm_step(const kda_ssm_problem* p, const void* u, const void* dt, const float* A, const void* B,
                        const void* Cm, const float* D_, const float* dt_bias, const void* z,
                        const int32_t* slots, int64_t n_slots, const float* h_in, float* h_out, void* y, void* ws,
                        kda_stream_t stream) {
    if (!p) return KDA_ERR_INVALID_ARG;
    kda_ssm_problem q = *p;
    q.T = q.N;  // one token per sequence; T and cu_seqlens are not read
    if (kda_status s = check_sizes(&q)) return s;
    if (kda_status s = check_inputs(&q, u, dt, A, B, Cm, D_, dt_bias, z, nullptr)) return s;
    if (!req(h_in) || !req(h_out) || !req(y) || !al(slots, 4) || !opt(ws) || n_slots < 1 ||
        (!slots && n_slots < q.N))
        return KDA_ERR_INVALID_ARG;
    const Regions none{};
    const SsmArgs t = make_args(&q, none, ws);
    SsmStepArgs a{q.N, q.C, q.S, q.G, q.dt_softplus, t.ldu, t.lddt, t.ldb, t.ldc, t.ldz, n_slots,
                  u, dt, B, Cm, z, A, D_, dt_bias, h_in, slots, h_out, y, static_cast<int*>(ws)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!clear_status(ws, st)) return KDA_ERR_CUDA;
    launch_ssm_step(a, q.dtype, st);
    return launched();
}

}  // extern "C"
