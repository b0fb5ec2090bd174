// Segments of the linear attention's documents, and the states between them.  One block's scan (5 us) and a pass over the
// slots (64 KB each, read and written once: 8 us for 16 heads of 16384 tokens) stand before a walk that is cut.
#include "kda_lin.cuh"

namespace kda {

namespace {

constexpr int PLAN_THREADS = 256;

// One block: each thread counts the segments of a run of documents, a scan gives the runs' first
// segments, warps write the entries.  Malformed offsets, or a saved set of other sizes, set the status word and
// leave no segments, so the call's later kernels do nothing.
__global__ void __launch_bounds__(PLAN_THREADS) k_lin_plan(LinArgs a) {
    constexpr int NW = PLAN_THREADS / 32;
    __shared__ long long wseg[NW], wmul[NW];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, L = a.seg;
    const int per = (a.N + PLAN_THREADS - 1) / PLAN_THREADS;
    const int n0 = min(tid * per, a.N), n1 = min(n0 + per, a.N);
    int bad = 0;
    long long segs = 0, muls = 0;  // 64-bit: malformed offsets cannot wrap the sums
    for (int n = n0; n < n1; ++n) {
        const long long len = (long long)a.cu[n + 1] - a.cu[n];
        bad |= len < 0;
        segs += len > LIN_WHOLE ? (len + L - 1) / L : 1;
        muls += len > LIN_WHOLE;
    }
    if (tid == 0) {
        bad |= a.cu[0] != 0 || int64_t(a.cu[a.N]) != a.T;
        if (a.expected) {
            const int4 m = *a.expected;
            bad |= m.x != a.sizes.x || m.y != a.sizes.y || m.z != a.sizes.z || m.w != a.sizes.w;
        }
    }
    long long s = segs, m = muls;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ys = __shfl_up_sync(0xffffffffu, s, o), ym = __shfl_up_sync(0xffffffffu, m, o);
        if (lane >= o) s += ys, m += ym;
    }
    if (lane == 31) wseg[w] = s, wmul[w] = m;
    bad = __syncthreads_or(bad);
    long long total_s = 0, total_m = 0;
    s -= segs, m -= muls;
    for (int i = 0; i < NW; ++i) {
        if (i < w) s += wseg[i], m += wmul[i];
        total_s += wseg[i], total_m += wmul[i];
    }
    if (tid == 0) {
        a.status[0] = bad ? KDA_ERR_DEVICE_CHECK : KDA_OK;
        a.plan.counts[0] = bad ? 0 : int(total_s);
        a.plan.counts[1] = bad ? 0 : int(total_m);
        if (a.made_for) *a.made_for = a.sizes;
    }
    if (bad) return;
    for (int n = n0; n < n1; ++n) {
        const int at = a.cu[n], len = a.cu[n + 1] - at, k = len > LIN_WHOLE ? (len + L - 1) / L : 1, l = k > 1 ? L : len;
        const int base = int(s) - n;  // slots in front: one less than its segments for every document
        if (k > 1) a.plan.multi[m++] = make_int4(n, base, k, len);
        for (int j = 0; j < k; ++j)
            a.plan.tab[s + j] = make_int4(n, at + j * l, min(l, len - j * l) | (j == 0) << 16 | (j == k - 1) << 17, base + j);
        s += k;
    }
}

// The slots of a document: forwards, slot j holds what segment j adds and receives the state behind it; backwards
// the same from the other end.  A thread walks four elements of a state.
__global__ void __launch_bounds__(256) k_lin_carry(LinArgs a, int back, const float* s0, float* slots) {
    constexpr int BLOCKS = D * D / 1024;
    const int part = int(blockIdx.x % BLOCKS), rest = int(blockIdx.x / BLOCKS), h = rest % a.H, i = rest / a.H;
    if (i >= a.plan.counts[1]) return;
    const int4 doc = a.plan.multi[i];
    const size_t e = size_t(part) * 1024 + threadIdx.x * 4, one = size_t(a.H) * D * D;
    const float slope = a.slope[h];
    const float full = expf(slope * float(a.seg)), rest_len = expf(slope * float(doc.w - (doc.z - 1) * a.seg));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s0) x = *reinterpret_cast<const float4*>(s0 + (size_t(doc.x) * a.H + h) * D * D + e);
    float* p = slots + (size_t(doc.y + (back ? doc.z - 2 : 0)) * a.H + h) * D * D + e;
    const ptrdiff_t step = back ? -ptrdiff_t(one) : ptrdiff_t(one);
    constexpr int AHEAD = 4;
    for (int j = 0; j < doc.z - 1; j += AHEAD) {
        float4 add[AHEAD];
#pragma unroll
        for (int r = 0; r < AHEAD; ++r)
            if (j + r < doc.z - 1) add[r] = *reinterpret_cast<const float4*>(p + r * step);
#pragma unroll
        for (int r = 0; r < AHEAD; ++r)
            if (j + r < doc.z - 1) {
                const float f = back && j + r == 0 ? rest_len : full;
                x.x = fmaf(f, x.x, add[r].x), x.y = fmaf(f, x.y, add[r].y);
                x.z = fmaf(f, x.z, add[r].z), x.w = fmaf(f, x.w, add[r].w);
                *reinterpret_cast<float4*>(p + r * step) = x;
            }
        p += AHEAD * step;
    }
}

}  // namespace

void launch_lin_plan(const LinArgs& a, cudaStream_t st) {
    ProfScope ps(KK_LIN_PLAN, st);
    k_lin_plan<<<1, PLAN_THREADS, 0, st>>>(a);
}

void launch_lin_carry(const LinArgs& a, int pass, cudaStream_t st) {
    const LinPass& p = a.pass[pass];
    ProfScope ps(KK_LIN_CARRY, st);
    // at most T / LIN_WHOLE documents have more than one segment
    k_lin_carry<<<unsigned(a.T / LIN_WHOLE) * unsigned(a.H) * (D * D / 1024), 256, 0, st>>>(a, p.back, p.s0,
                                                                                   p.back ? a.back : a.front);
}

}  // namespace kda
