// Linear attention with a decay for each head: the walk over packed documents.
#include "kda_lin.cuh"

namespace kda {

namespace {

constexpr int LIN_ROWS = 16;  // tokens staged together

// One block per document, head and pass; thread j holds column j of the state.
__global__ void __launch_bounds__(128) k_lin_recur(LinArgs a) {
    __shared__ float sq[LIN_ROWS][D], sk[LIN_ROWS][D];
    const int j = threadIdx.x;
    const int ps = int(blockIdx.x % unsigned(a.passes)), rest = int(blockIdx.x / unsigned(a.passes));
    const int h = rest % a.H, n = rest / a.H;
    const LinPass& p = a.pass[ps];
    if (a.expected) {
        const int4 m = *a.expected;
        if (m.x != a.sizes.x || m.y != a.sizes.y || m.z != a.sizes.z || m.w != a.sizes.w) {
            if (j == 0) *a.status = KDA_ERR_DEVICE_CHECK;
            return;
        }
    }
    if (a.made_for && blockIdx.x == 0 && j == 0) *a.made_for = a.sizes;
    const int c0 = a.cu[n], c1 = a.cu[n + 1];
    if (c0 < 0 || c1 < c0 || c1 > a.T || (n == 0 && c0 != 0) || (n == a.N - 1 && c1 != a.T)) {
        if (j == 0) *a.status = KDA_ERR_DEVICE_CHECK;
        return;
    }
    const float lam = expf(a.slope[h]), pre = p.back ? 1.f : lam, post = p.back ? lam : 1.f;
    const size_t sn = (size_t(n) * a.H + h) * D * D;
    float S[D];
#pragma unroll
    for (int i = 0; i < D; ++i) S[i] = p.s0 ? p.s0[sn + (p.trans ? j * D + i : i * D + j)] : 0.f;
    const int len = c1 - c0;
    for (int r0 = 0; r0 < len; r0 += LIN_ROWS) {
        const int m = min(LIN_ROWS, len - r0);
        __syncthreads();
        for (int r = 0; r < m; ++r) {
            const int64_t t = p.back ? c1 - 1 - (r0 + r) : c0 + r0 + r;
            sq[r][j] = bf2f(p.query[t * p.ldq + (h / p.rq) * D + j]);
            sk[r][j] = bf2f(p.key[t * p.ldk + (h / p.rk) * D + j]);
        }
        __syncthreads();
        for (int r = 0; r < m; ++r) {
            const int64_t t = p.back ? c1 - 1 - (r0 + r) : c0 + r0 + r;
            const float v = p.in * bf2f(p.value[t * p.ldv + (h / p.rv) * D + j]);
            float o = 0.f;
#pragma unroll
            for (int i = 0; i < D; ++i) {
                S[i] = fmaf(S[i], pre, sk[r][i] * v);
                o = fmaf(sq[r][i], S[i], o);
                S[i] *= post;
            }
            store_out(p.out, (size_t(t) * a.H + h) * D + j, p.by * o, p.out_fp32);
        }
    }
    if (p.s_end)
#pragma unroll
        for (int i = 0; i < D; ++i) p.s_end[sn + (p.trans ? j * D + i : i * D + j)] = S[i];
}

}  // namespace

void launch_lin_walk(const LinArgs& a, cudaStream_t st) {
    ProfScope ps(KK_LIN_WALK, st);
    k_lin_recur<<<unsigned(a.N) * unsigned(a.H) * unsigned(a.passes), 128, 0, st>>>(a);
}

}  // namespace kda
