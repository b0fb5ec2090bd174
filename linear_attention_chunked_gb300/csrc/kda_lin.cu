// Linear attention with a decay for each head: the chunked walk over packed documents on tcgen05 tensor cores.
//
// Chunks of 128 tokens.  Per segment of a document (kda_lin_plan.cu), head and pass, chunk after chunk, with the
// state X [128 key channels][128 value channels] in fp32 (forwards; n tokens in the chunk, i, j < n):
//     P    = Query Key^T                              [i][j]
//     P'   = P lambda^(i - j) for j <= i, else 0      rounded to bf16
//     Out  = by (P' Value + lambda^(i + 1) Query X)   X as an operand rounded to bf16
//     X   <- lambda^n X + (in lambda^(n - 1 - j) Value_j)^T Key_j, summed
// Backwards (the state is Y, see kda_lin.cuh) the mask is j >= i with lambda^(j - i), Query Y takes lambda^(n - 1 - i)
// and Value_j takes lambda^(j + 1).
//
// What bounds it: a token and head is 1 KB of rows, 2.9 us of a multiprocessor's share of HBM for a chunk, and 40 to 48
// products of 128 x 128 x 16, some 3550 to 4200 clocks.  One block per multiprocessor holds a state and works on
// successive chunks: 16384 tokens (9000 / 5000 / 2384) x 64 heads take 199 us, 5.4 TB/s (80% of the measured 6.77), the
// last third of it on the 64 blocks of the longest document; one document of 16384 x 64 (64 blocks) 305 to 340 us from card to
// card, 2.4 us a chunk and more, bound by the chain of its own steps.  Of those 2.4 us the products alone take 1.9 and the
// hand-overs alone 1.3.
//
// The state stays in tensor memory as X^T (lane = value channel); the scaled values are the state product's left operand
// in tensor memory, split into bf16 planes, so that with three of them (8 + 8 + 8 bits: exact) the state's products are fp32
// products.  The scores and the state are rounded to bf16 as operands of products whose sums are rounded to bf16 rows:
// each adds as much as the output's own rounding: 0.0023 of a row's length from 64 bits in all, where one rounding is 0.0017.
// (The delta rule's triangular inverse multiplies such errors, so KDA's products carry hi and lo operands.  Here nothing
// does; second planes of scores and state would be 16 products more beside a chunk's 40 to 48, and shared memory holds one
// plane of the state.)  Query, Key and Value come by TMA and are read where they land:
//     P      A = Query [tokens][keys],    B = Key [tokens][keys]
//     QX     A = Query,                   B = X^T in shared memory, bf16 [values][keys]
//     P'V    A = P' (tensor memory),      B = Value [tokens][values] read across
//     state  A = values^T (tensor memory), B = Key read across
// Four groups of warps work at once: A (two groups) scales and splits the values, B masks and rounds the scores and
// hands the output to TMA, C rounds and decays the state and scales Query X's rows; three warps issue loads, products
// and stores.  The chunk's tiles go through a ring of five, each taken again as soon as its last product has read it.
// Rows behind a document's end (another's) are cleared in K and V, so nothing of them, were it not finite, is multiplied.
//
// Measured beside it, one document of 16384 x 64 (305 us): one column factor for scores and state where the decay is mild,
// without the pass over Query X's rows: 326; eight warps in B: 312; the output stored from registers: 508; lane 0 polling
// for its warp: 471; products issued by one thread in one piece: 342.
#include <limits.h>

#include "kda_lin.cuh"
#include "kda_ssm.cuh"
#include "kda_tc.cuh"

namespace kda {

void launch_lin_carry(const LinArgs& a, int pass, cudaStream_t st);

namespace {

constexpr uint32_t TILE = LC * D * 2;  // bytes of one chunk's rows of one head

// lambda^n = exp(slope n), 1 for n = 0 whatever the slope
__device__ __forceinline__ float decay(float slope, int n) { return n == 0 ? 1.f : expf(slope * float(n)); }

// ---- tensor memory, packed words ----
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 16 lanes x 8 columns: lane i holds row i / 4 of column 4 j + i % 4 in word 2 j and row 8 + i / 4 in word 2 j + 1
__device__ __forceinline__ void tmem_st_16x8(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem], issued by one thread: A's row i is lane i, its 16-bit elements 2 c and 2 c + 1 lie in
// column c.
__device__ __forceinline__ void mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}
// True in one lane of a warp, always the same.  Products issued under it take their operands from uniform registers:
// 76 clocks each (left operand in tensor memory; 108 in shared memory), where a branch on the thread's number costs 106.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tma_store4(const CUtensorMap* map, int x, int y, int z, int u, const void* src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(u), "r"(smem_u32(src))
                 : "memory");
}

// A wait gives up after about a second.  (The roles' code has to share the instruction cache: with the clock read in the
// wait's loop the walk takes 8% longer.)
constexpr uint32_t WAIT_TRIES = 250000;
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival for a warp whose lanes have all finished their part
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    tc::fence_before_sync();
    __syncwarp();
    asm volatile("{\n .reg .pred p;\n setp.eq.s32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar), "r"(lane) : "memory");
}

// 128-byte-swizzled tile pair [2 blocks of 64 channels][128 tokens][128 bytes]: clears the rows from n on.  128 threads.
__device__ __forceinline__ void clear_rows(unsigned char* tile, int n, int tid) {
    for (int i = tid; i < 2 * (LC - n) * 8; i += 128) {
        const int c = i & 7, r = n + ((i >> 3) % (LC - n)), b = (i >> 3) / (LC - n);
        *reinterpret_cast<uint4*>(tile + b * (TILE / 2) + r * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// A piece (16 tokens) of a chunk's values, times the tokens' factors f (shared memory) and `all`, split into bf16 planes
// as the left operand of a product in tensor memory: lane = channel, token pairs in the columns taddr.. of hi, mid and
// lo, 8 each.  Three planes are cut off (8 bits each: exact), two are rounded (the rest of the first, at most 2^-8, to 8 bits:
// off by 2^-17 at most, 2.5e-6 in the 2-norm).  A warp does its 32 channels; 8 x 8 blocks are transposed as they are loaded,
// which gives a lane the pairs that a 16-lane store takes.
constexpr int PIECES = LC / 16;
constexpr uint32_t PLANES = 24;  // columns of a piece
template <int N>
__device__ __forceinline__ void split_piece(const unsigned char* tile, int piece, int w, int lane, const float* f, float all,
                                            uint32_t taddr) {
    const int m = lane >> 3, r = lane & 7;
    const unsigned char* base = tile + ((w & 3) >> 1) * (TILE / 2) + (16 * piece + (m >> 1) * 8 + r) * 128;
    const int c8 = (w & 1) * 4 + (m & 1);
    uint32_t x[2][4];
    ldsm4t(x[0], base + ((c8 ^ r) << 4));
    ldsm4t(x[1], base + (((c8 + 2) ^ r) << 4));
    const f2 all2 = pk2(all, all);
    f2 fw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        fw[i] = mul2(*reinterpret_cast<const f2*>(f + 16 * piece + 8 * i + 2 * (lane & 3)), all2);
    constexpr uint32_t mask = 0xffff0000u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // 16 channels
        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f2 y = mul2(fw[j >> 1], pk2(__uint_as_float(x[h][j] << 16), __uint_as_float(x[h][j] & mask)));
            const f2 minus = pk2(-1.f, -1.f);
            float y0, y1, r0, r1;
            up2(y, y0, y1);
            if (N == 2) {
                hi[j] = pack2(y0, y1);
                up2(fma2(pk2(__uint_as_float(hi[j] << 16), __uint_as_float(hi[j] & mask)), minus, y), r0, r1);
                mid[j] = pack2(r0, r1);
            } else {
                hi[j] = __byte_perm(__float_as_uint(y0), __float_as_uint(y1), 0x7632);
                const f2 rest = fma2(pk2(__uint_as_float(__float_as_uint(y0) & mask), __uint_as_float(__float_as_uint(y1) & mask)), minus, y);
                up2(rest, r0, r1);
                mid[j] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
                up2(fma2(pk2(__uint_as_float(__float_as_uint(r0) & mask), __uint_as_float(__float_as_uint(r1) & mask)), minus, rest), r0, r1);
                lo[j] = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
            }
        }
        const uint32_t at = taddr + (uint32_t(16 * h) << 16);
        tmem_st_16x8(at, hi);
        tmem_st_16x8(at + 8, mid);
        if (N == 3) tmem_st_16x8(at + 16, lo);
    }
    tmem_wait_st();
}
// The products of a piece: D += planes * rows 16 piece.. of the key tile, read across
__device__ __forceinline__ void piece_products(uint32_t d, uint32_t planes, uint64_t key, int piece, uint32_t idesc, bool first,
                                               bool three) {
    const uint64_t b = key + uint64_t((piece * 2048) >> 4);
    if (three) mma_ta(d, planes + 16, b, idesc, !first);
    mma_ta(d, planes + 8, b, idesc, three || !first);
    mma_ta(d, planes, b, idesc, 1u);
}

// The segment of a block: {document, first token, length, flags as in LinPlan, w}; false: none (or malformed offsets)
struct Seg {
    int doc, t0, len, w;
    bool first, last;
};
__device__ __forceinline__ bool lin_segment(const LinArgs& a, int i, Seg& s) {
    if (!a.direct) {
        if (i >= a.plan.counts[0]) return false;
        const int4 e = a.plan.tab[i];
        s.doc = e.x, s.t0 = e.y, s.len = e.z & 0xffff, s.w = e.w;
        s.first = e.z >> 16 & 1, s.last = e.z >> 17 & 1;
        return true;
    }
    // a document for every i: the longest first, by a warp's lanes, where they have a lane each.  (More of them are taken in the
    // pack's order: a rank is a shuffle a document in every block, and no form that keeps it once was built.)
    if (a.N > 1 && a.N <= 32) {
        const int lane = threadIdx.x & 31;
        const int own = lane < a.N ? a.cu[lane + 1] - a.cu[lane] : INT_MIN;
        int rank = 0;
        for (int k = 0; k < a.N; ++k) {
            const int x = __shfl_sync(0xffffffffu, own, k);
            rank += x > own || (x == own && k < lane);
        }
        i = __ffs(__ballot_sync(0xffffffffu, lane < a.N && rank == i)) - 1;
    }
    const int c0 = a.cu[i], c1 = a.cu[i + 1];
    bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.T && (i > 0 || c0 == 0) && (i < a.N - 1 || c1 == a.T);
    if (a.expected) {
        const int4 m = *a.expected;
        ok = ok && m.x == a.sizes.x && m.y == a.sizes.y && m.z == a.sizes.z && m.w == a.sizes.w;
    }
    if (!ok) {
        if (threadIdx.x == 0) *a.status = KDA_ERR_DEVICE_CHECK;
        return false;
    }
    if (a.made_for && blockIdx.x == 0 && threadIdx.x == 0) *a.made_for = a.sizes;
    s = {i, c0, c1 - c0, 0, true, true};
    return true;
}

// ---- the walk ----

// A: warps 0-7, B: 8-11, C: 12-15, loads: 16, products: 17, stores: 18
constexpr int WALK_THREADS = 608;
constexpr int W_TILES = 5;                         // ring of chunk tiles: Query, Key, Value of chunk 0, of chunk 1, ..
constexpr int W_X = W_TILES * int(TILE);           // the state as an operand
constexpr int W_OUT = W_X + int(TILE);             // an output on its way
constexpr int W_TAB = W_OUT + int(TILE);           // state factors of a full and of the short chunk [128], score factors [32], [64]
constexpr int W_BAR = W_TAB + (128 + 128 + 32 + 64) * 4;
constexpr size_t WALK_SMEM = W_BAR + 320 + 1024;
static_assert(WALK_SMEM <= 232448, "walk: shared memory above the opt-in limit");

// tensor memory columns: scores (their rounded form in the first half), output, state, pieces of split values
constexpr uint32_t C_P = 0, C_O = 128, C_X = 256, C_V = 384;
constexpr int W_PIECES = 4;
static_assert(C_V + W_PIECES * PLANES <= 512, "walk: tensor memory");

// By tile: it has landed, it may be loaded again.  By piece: it is split, its columns may be written again.
enum WalkBar {
    B_FULL = 0, B_FREE = W_TILES, B_A = 2 * W_TILES, B_AFREE = B_A + W_PIECES,
    B_P = B_AFREE + W_PIECES, B_QX, B_B, B_SCALED, B_S, B_C, B_O, B_OFREE, B_STAGED, B_STORED, B_FIX, B_X0, B_SPARE, B_END
};
static_assert(8 * B_END + 8 <= 320, "walk: barriers");

__global__ void __launch_bounds__(WALK_THREADS, 1) k_lin_walk(LinArgs a, const __grid_constant__ LinMaps tm) {
    extern __shared__ unsigned char smraw[];
    unsigned char* sm = tc::align1024(smraw);
    const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int ps = int(blockIdx.x % unsigned(a.passes)), rest = int(blockIdx.x / unsigned(a.passes));
    const int hd = rest % a.H;
    const LinPass& p = a.pass[ps];
    Seg g;
    if (!lin_segment(a, rest / a.H, g)) return;
    const bool back = p.back;
    const size_t doc_state = (size_t(g.doc) * a.H + hd) * D * D;
    // the state that the walk starts from, and where the document's last one goes
    const bool starts = back ? g.last : g.first, ends = back ? g.first : g.last;
    // (a walk that starts from zero leaves Query X of its first chunk out, and its first product clears the state)
    const float* x0 = starts ? (p.s0 ? p.s0 + doc_state : nullptr)
                             : (back ? a.back + (size_t(g.w) * a.H + hd) * D * D
                                     : a.front + (size_t(g.w - 1) * a.H + hd) * D * D);
    float* x1 = ends && p.s_end ? p.s_end + doc_state : nullptr;
    const int nc = (g.len + LC - 1) / LC;
    if (nc == 0) {  // an empty document keeps its state
        if (x1)
            for (int i = tid; i < D * D; i += WALK_THREADS) x1[i] = x0 ? x0[i] : 0.f;
        return;
    }
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + W_BAR);
    const uint32_t sbar = smem_u32(bar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + W_BAR + 8 * B_END);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + W_BAR + 8 * B_END + 4);
    float* fs = reinterpret_cast<float*>(sm + W_TAB);  // a full chunk's state factors
    float* fshort = fs + 128;                          // the short chunk's (of at most one)
    float* fn = fshort + 128;                          // score factors in a block off the diagonal, by column
    float* fd = fn + 32;                               // and in it: [31 + row - column]
    const float slope = a.slope[hd];
    // chunk c of the walk: its place in the segment and its tokens
    auto place = [&](int c) { return back ? nc - 1 - c : c; };
    auto tokens = [&](int c) { return min(LC, g.len - LC * place(c)); };
    auto tile = [&](int i) { return sm + (i % W_TILES) * TILE; };  // tile 3 c: Query of chunk c, then Key, Value
    auto load = [&](int i) {  // by one thread
        const int b = i % W_TILES, c = i / 3, which = i - 3 * c;
        tc::mbar_expect_tx(&bar[B_FULL + b], TILE);
        tc::tma4(tile(i), &tm.m[which == 0 ? p.query : which == 1 ? p.key : p.value], 0, g.t0 + LC * place(c), 0,
                 hd / (which == 0 ? p.rq : which == 1 ? p.rk : p.rv), &bar[B_FULL + b]);
    };
    if (w == 16) {  // the first rows are on their way while the rest is set up
        if (elect()) {
            for (int i = 0; i < B_SPARE; ++i) {
                const bool four = (i >= B_A && i < B_AFREE) || i == B_B || i == B_SCALED || i == B_C || i == B_OFREE || i == B_STAGED;
                tc::mbar_init(&bar[i], i == B_X0 ? 12 : i == B_FIX ? 8 : four ? 4 : 1);
            }
            *abort_flag = 0;
            tc::fence_mbar_init();
            tc::fence_async_smem();
            for (int i = 0; i < min(W_TILES, 3 * nc); ++i) load(i);
        }
        __syncwarp();
    }
    if (w == 0) tc::tmem_alloc(tslot, 512);
    if (tid < LC) {
        fs[tid] = p.in * decay(slope, back ? tid + 1 : LC - 1 - tid);
        const int m = g.len - LC * (nc - 1);
        fshort[tid] = tid < m ? p.in * decay(slope, back ? tid + 1 : m - 1 - tid) : 0.f;
    } else if (tid < LC + 32) {
        // lambda^(31 - i), times lambda^(row - the block's last column); backwards lambda^i, times lambda^(its first - row)
        fn[tid - LC] = p.in * p.by * decay(slope, back ? tid - LC : LC + 31 - tid);
    } else if (tid < LC + 96) {
        const int d = (tid - LC - 32 - 31) * (back ? -1 : 1);
        fd[tid - LC - 32] = d >= 0 ? p.in * p.by * decay(slope, d) : 0.f;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    const uint32_t tl = tbase + (uint32_t(32 * (w & 3)) << 16);  // this warp's lanes
    const int row = 32 * (w & 3) + lane;

    // whether chunk c's values still reach a state that is read; whether its output leaves by TMA
    auto adds = [&](int c) { return c + 1 < nc || x1; };
    // The state that a document ends in is an fp32 output: the values that still weigh more than 1/64 in it are split into three
    // planes, exactly; those before them get two, which is off by 2^-23 of what they were at their time (three everywhere: 5%
    // of a forward), and so does a state that only bf16 rows are made of.
    auto three = [&](int c) {
        const int beyond = back ? LC * place(c) : max(g.len - LC * (c + 1), 0);  // tokens that the walk still meets
        return x1 && (beyond == 0 || slope * float(beyond) > -4.16f);
    };
    auto staged = [&](int c) { return !p.out_fp32 && tokens(c) == LC; };
    // Waits for the turn-th completion of barrier b.  A wait that runs out of tries ends the warp's part; every other
    // wait runs out too, and the block reports and ends, when nothing of its copies and products is in flight any more.
    bool ok = true;  // the same in a warp's lanes
    int loaded = 0;  // tiles (warp 16)
    auto wait = [&](int b, int turn) {
        ok = ok && tc::warp_wait<WAIT_TRIES>(sbar + 8 * b, uint32_t(turn) & 1u);
        tc::fence_after_sync();
        return ok;
    };
    // 32 columns of the state that the walk starts from
    auto start_block = [&](int j) {
        float v[32];
        if (p.trans) {
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(x0 + row * D + 32 * j + i);
                v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = x0[(32 * j + i) * D + row];
        }
        tc::tmem_st32(tl + C_X + 32 * j, v);
    };
    auto landed = [&](int i) { return wait(B_FULL + i % W_TILES, i / W_TILES); };
    auto arrive = [&](int b) { warp_arrive(sbar + 8 * b, lane); };
    // the groups share the blocks
    const bool blank = !x0;
    if (w < 16 && !blank) {
        start_block(w >> 2);
        if (w < 12) arrive(B_X0);
    }

    if (w < 8) {
        // ---- A: the values, scaled and split, a piece at a time ----
        for (int c = 0; c < nc; ++c) {
            const int n = tokens(c);
            if (!landed(3 * c + 2)) break;
            if (n < LC) {  // the rows of other documents: cleared before any product reads them (one chunk of a walk)
                if (!landed(3 * c + 1)) break;
                clear_rows(tile(3 * c + 1 + (w >> 2)), n, tid & 127);
                tc::fence_async_smem();
                arrive(B_FIX);
                if (!wait(B_FIX, 0)) break;
            }
            if (!adds(c)) break;
            const float* f = n < LC ? fshort : fs;
            const bool exact = three(c);
            for (int i = PIECES * c + (w >> 2); i < PIECES * (c + 1); i += 2) {
                const int b = i % W_PIECES;
                if (i >= W_PIECES && !wait(B_AFREE + b, i / W_PIECES - 1)) break;
                if (exact) split_piece<3>(tile(3 * c + 2), i % PIECES, w, lane, f, 1.f, tl + C_V + PLANES * b);
                else split_piece<2>(tile(3 * c + 2), i % PIECES, w, lane, f, 1.f, tl + C_V + PLANES * b);
                arrive(B_A + b);
            }
            if (!ok) break;
        }
    } else if (w < 12) {
        // ---- B: the scores; the output ----
        const int q = w & 3;
        float e[3];  // the second factor of block j (back: j + 1)
#pragma unroll
        for (int j = 0; j < 3; ++j) e[j] = decay(slope, max(back ? 32 * (j + 1) - row : row - 32 * j - 31, 0));
        const float* fr = fd + 31 + lane;
        unsigned char* ot = sm + W_OUT;
        for (int c = 0; c <= nc; ++c) {
            if (c > 0) {
                const int d = c - 1;  // the chunk whose output is ready
                if (!wait(B_O, d)) break;
                const int n = tokens(d);
                if (staged(d)) {
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t o[2][16];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float v[32];
                            tc::tmem_ld32(tl + C_O + 64 * h + 32 * j, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[j][i] = pack2(v[2 * i], v[2 * i + 1]);
                        }
                        if (h == 1) arrive(B_OFREE);
                        else if (d > 0 && !wait(B_STORED, d - 1)) break;
                        tc::st_sw128(ot + h * (TILE / 2), row, 0, o[0]);
                        tc::st_sw128(ot + h * (TILE / 2), row, 32, o[1]);
                    }
                    if (!ok) break;
                    tc::fence_async_smem();
                } else {
                    const int even = row & ~1;
                    const size_t off = (size_t(g.t0 + LC * place(d) + row) * a.H + hd) * D, ld = size_t(a.H) * D;
#pragma unroll 1
                    for (int j = 0; j < 4; ++j) {
                        float v[32];
                        tc::tmem_ld32(tl + C_O + 32 * j, v);
                        if (p.out_fp32) {
                            tc::st_rows_paired_f32<32>(static_cast<float*>(p.out) + off + 32 * j, ld, v, lane, even < n, even + 1 < n);
                        } else {
                            uint4 x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[i] = make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                                                  pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
                            tc::st_rows_paired<4>(reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + off + 32 * j),
                                                  ld / 2, x, lane, even < n, even + 1 < n);
                        }
                    }
                    arrive(B_OFREE);
                    if (d > 0 && !wait(B_STORED, d - 1)) break;
                }
                arrive(B_STAGED);
            }
            if (c == nc) break;
            const int n = tokens(c);
            if (!wait(B_P, c)) break;
            // a block is read, scaled and written back packed, into columns that were read before
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                uint32_t o[16];
                if (back ? j >= q : j <= q) {
                    float v[32];
                    tc::tmem_ld32(tl + C_P + 32 * j, v);
                    if (j != q) {
                        const int k = back ? j - 1 : j;
                        const float ej = k == 0 ? e[0] : k == 1 ? e[1] : e[2];
                        const f2 e2 = pk2(ej, ej);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const f2 y = mul2(pk2(v[2 * i], v[2 * i + 1]), mul2(*reinterpret_cast<const f2*>(fn + 2 * i), e2));
                            up2(y, v[2 * i], v[2 * i + 1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= fr[-i];
                    }
                    if (n < LC)  // (a growing state's factors may be infinite there)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * j + i >= n) v[i] = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = pack2(v[2 * i], v[2 * i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0u;
                }
                tmem_st16u(tl + C_P + 16 * j, o);
            }
            tmem_wait_st();
            arrive(B_B);
        }
    } else if (w < 16) {
        // ---- C: the state as an operand, its decay; Query X's rows ----
        unsigned char* xt = sm + W_X;
        for (int c = 0; c < nc; ++c) {
            const int n = tokens(c);
            const float fx = decay(slope, n), fo = p.by * decay(slope, back ? max(n - 1 - row, 0) : row + 1);
            if (c == 0 && blank) {
                arrive(B_C);
                arrive(B_SCALED);
                continue;
            }
            if (!(c > 0 ? wait(B_S, c - 1) : wait(B_X0, 0))) break;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float v[32];
                tc::tmem_ld32(tl + C_X + 32 * j, v);
                uint32_t b[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) b[i] = pack2(v[2 * i], v[2 * i + 1]);
                tc::st_sw128(xt + (j >> 1) * (TILE / 2), row, 32 * (j & 1), b);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= fx;
                tc::tmem_st32(tl + C_X + 32 * j, v);
            }
            tc::fence_async_smem();
            arrive(B_C);
            if (!wait(B_QX, c)) break;
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float v[32];
                tc::tmem_ld32(tl + C_O + 32 * j, v);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= fo;
                tc::tmem_st32(tl + C_O + 32 * j, v);
            }
            arrive(B_SCALED);
        }
        if (x1 && wait(B_S, nc - 1)) {
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float v[32];
                tc::tmem_ld32(tl + C_X + 32 * j, v);
                if (p.trans) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(x1 + row * D + 32 * j + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x1[(32 * j + i) * D + row] = v[i];
                }
            }
        }
    } else if (w == 16) {
        // ---- loads ----
        int i = min(W_TILES, 3 * nc);
        for (; i < 3 * nc; ++i) {
            if (!wait(B_FREE + i % W_TILES, i / W_TILES - 1)) break;
            if (elect()) load(i);
            __syncwarp();
        }
        loaded = i;
    } else if (w == 17) {
        // ---- products ----
        const uint32_t ID = tc::idesc_bf16(128, 128, false, false), IDt = tc::idesc_bf16(128, 128, false, true);
        const uint64_t dX = tc::sdesc(smem_u32(sm + W_X), 16, 1024);
        auto kstep = [](int s) { return uint64_t(((s >> 2) * int(TILE / 2) + (s & 3) * 32) >> 4); };  // along the channels
        auto tstep = [](int s) { return uint64_t((s * 2048) >> 4); };                                 // along the tokens
        auto spent = [&](int i) { tc::mma_commit(&bar[B_FREE + i % W_TILES]); };
        for (int c = -1; c < nc; ++c) {
            if (c >= 0) {
                if (!wait(B_C, c) || (c > 0 && !wait(B_OFREE, c - 1))) break;
                const bool first = c == 0 && blank;
                if (elect()) {
                    const uint64_t dq = tc::sdesc(smem_u32(tile(3 * c)), 16, 1024);
                    if (!first) {
#pragma unroll
                        for (int s = 0; s < 8; ++s) tc::mma(tbase + C_O, dq + kstep(s), dX + kstep(s), ID, s > 0);
                    }
                    tc::mma_commit(&bar[B_QX]);
                    spent(3 * c);
                }
                __syncwarp();
                if (adds(c)) {
                    const uint64_t dk = tc::sdesc(smem_u32(tile(3 * c + 1)), TILE / 2, 1024);
                    const bool exact = three(c);
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) {
                        const int b = i % W_PIECES;
                        if (!wait(B_A + b, c * (PIECES / W_PIECES) + i / W_PIECES)) break;
                        if (elect()) {
                            piece_products(tbase + C_X, tbase + C_V + PLANES * b, dk, i, IDt, first && i == 0, exact);
                            tc::mma_commit(&bar[B_AFREE + b]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (elect()) tc::mma_commit(&bar[B_S]);
                    __syncwarp();
                }
                if (!landed(3 * c + 2) || !wait(B_B, c) || !wait(B_SCALED, c)) break;
                if (elect()) {
                    const uint64_t dv = tc::sdesc(smem_u32(tile(3 * c + 2)), TILE / 2, 1024);
                    spent(3 * c + 1);
#pragma unroll
                    for (int s = 0; s < 8; ++s) mma_ta(tbase + C_O, tbase + C_P + 8 * s, dv + tstep(s), IDt, !first || s > 0);
                    spent(3 * c + 2);
                    tc::mma_commit(&bar[B_O]);
                }
                __syncwarp();
            }
            if (c + 1 < nc) {
                const int d = c + 1;
                if (!landed(3 * d) || !landed(3 * d + 1)) break;
                if (tokens(d) < LC && !wait(B_FIX, 0)) break;
                if (elect()) {
                    const uint64_t dq = tc::sdesc(smem_u32(tile(3 * d)), 16, 1024), dk = tc::sdesc(smem_u32(tile(3 * d + 1)), 16, 1024);
#pragma unroll
                    for (int s = 0; s < 8; ++s) tc::mma(tbase + C_P, dq + kstep(s), dk + kstep(s), ID, s > 0);
                    tc::mma_commit(&bar[B_P]);
                }
                __syncwarp();
            }
        }
    } else {
        // ---- stores ----
        for (int c = 0; c < nc; ++c) {
            if (!wait(B_STAGED, c)) break;
            if (elect()) {
                if (staged(c)) {
                    tma_store4(&tm.m[p.store], 0, g.t0 + LC * place(c), 0, hd, sm + W_OUT);
                    tc::bulk_commit();
                    tc::bulk_wait_read0();
                }
                mbar_arrive(sbar + 8 * B_STORED);
            }
            __syncwarp();
        }
    }
    if (!ok) *abort_flag = 1;
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (*abort_flag) {  // whichever warp gave up
        if (tid == 0) *a.status = KDA_ERR_TIMEOUT;
        if (w == 16)
            for (int k = max(loaded - W_TILES, 0); k < loaded; ++k)
                tc::mbar_wait(&bar[B_FULL + k % W_TILES], (k / W_TILES) & 1, 100000000ull);
        if (w == 17 && elect()) tc::drain_mmas(&bar[B_SPARE], 100000000ull);
        __syncthreads();
    }
    if (w == 0) tc::tmem_dealloc(tbase, 512);
}

// ---- what a segment adds to the state ----

constexpr int STATE_THREADS = 320;  // two groups of four warps take the pieces in turn; loads: warp 8, products: 9
constexpr int S_STAGES = 3;
constexpr int S_BUFS = PIECES;      // pieces of split values in tensor memory: a chunk's
constexpr int S_TAB = S_STAGES * 2 * int(TILE);
constexpr int S_BAR = S_TAB + 128 * 4;
constexpr size_t STATE_SMEM = S_BAR + 256 + 1024;
enum StateBar {
    SB_FULL = 0, SB_EMPTY = S_STAGES, SB_READY = 2 * S_STAGES, SB_FREE = SB_READY + S_BUFS, SB_DONE = SB_FREE + S_BUFS, SB_FIX,
    SB_SPARE, SB_END
};

// No decay of the state between chunks: a token's factor reaches to the segment's end, the products add up.
// Bound by HBM on paper (512 B a token and head; 24 products a chunk, half its time); 16384 tokens x 16 heads: 35 us,
// 3.4 TB/s: one wave of 112 blocks that work (144 are launched), a sixth of whose time is their start and the store of the state.
__global__ void __launch_bounds__(STATE_THREADS, 1) k_lin_state(LinArgs a, int ps, const __grid_constant__ LinMaps tm) {
    extern __shared__ unsigned char smraw[];
    unsigned char* sm = tc::align1024(smraw);
    const int tid = threadIdx.x, w = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int hd = int(blockIdx.x % unsigned(a.H));
    const LinPass& p = a.pass[ps];
    Seg g;
    if (!lin_segment(a, int(blockIdx.x / unsigned(a.H)), g)) return;
    const bool back = p.back;
    if (back ? g.first : g.last) return;  // nothing walks on from here
    float* out = back ? a.back + (size_t(g.w - 1) * a.H + hd) * D * D : a.front + (size_t(g.w) * a.H + hd) * D * D;
    const int nc = (g.len + LC - 1) / LC;
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S_BAR);
    const uint32_t sbar = smem_u32(bar);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + S_BAR + 8 * SB_END);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S_BAR + 8 * SB_END + 4);
    float* fs = reinterpret_cast<float*>(sm + S_TAB);
    const float slope = a.slope[hd];
    if (tid == 0) {
        for (int i = 0; i < SB_SPARE; ++i)
            tc::mbar_init(&bar[i], (i >= SB_READY && i < SB_FREE) || i == SB_FIX ? 4 : 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (w == 0) tc::tmem_alloc(tslot, 512);
    if (w == 8 && lane < 2) tc::tma_prefetch_map(&tm.m[lane ? p.value : p.key]);
    if (tid < LC) fs[tid] = p.in * decay(slope, back ? tid + 1 : LC - 1 - tid);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = *tslot;
    const uint32_t tl = tbase + (uint32_t(32 * (w & 3)) << 16);
    const int row = 32 * (w & 3) + lane;
    auto tile = [&](int c, int which) { return sm + ((c % S_STAGES) * 2 + which) * TILE; };
    bool ok = true;  // waits as in the walk
    int loaded = 0;  // chunks (warp 8)
    auto wait = [&](int b, int turn) {
        ok = ok && tc::warp_wait<WAIT_TRIES>(sbar + 8 * b, uint32_t(turn) & 1u);
        tc::fence_after_sync();
        return ok;
    };
    auto arrive = [&](int b) { warp_arrive(sbar + 8 * b, lane); };
    constexpr uint32_t C_V = 128;  // columns: state 0, then the pieces of split values

    if (w < 8) {
        const int grp = w >> 2;
        for (int c = 0; c < nc; ++c) {
            const int n = min(LC, g.len - LC * c);
            if (!wait(SB_FULL + c % S_STAGES, c / S_STAGES)) break;
            if (n < LC) {
                if (grp == 0) {
                    clear_rows(tile(c, 0), n, tid);
                    clear_rows(tile(c, 1), n, tid);
                    tc::fence_async_smem();
                    arrive(SB_FIX);
                }
                if (!wait(SB_FIX, 0)) break;
            }
            // forwards only full chunks come here (the last segment adds to nothing)
            const float all = decay(slope, back ? LC * c : g.len - LC * (c + 1));
            for (int i = grp; i < PIECES; i += 2) {
                if (c > 0 && !wait(SB_FREE + i, c - 1)) break;
                split_piece<3>(tile(c, 1), i, w, lane, fs, all, tl + C_V + PLANES * i);
                arrive(SB_READY + i);
            }
            if (!ok) break;
        }
        if (w < 4 && wait(SB_DONE, 0)) {
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                float x[32];
                tc::tmem_ld32(tl + 32 * j, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) out[(32 * j + i) * D + row] = x[i];
            }
        }
    } else if (w == 8) {
        const CUtensorMap *mk = &tm.m[p.key], *mv = &tm.m[p.value];
        for (int c = 0; c < nc; ++c) {
            const int s = c % S_STAGES, t = g.t0 + LC * c;
            if (c >= S_STAGES && !wait(SB_EMPTY + s, c / S_STAGES - 1)) break;
            if (elect()) {
                tc::mbar_expect_tx(&bar[SB_FULL + s], 2 * TILE);
                tc::tma4(tile(c, 1), mv, 0, t, 0, hd / p.rv, &bar[SB_FULL + s]);
                tc::tma4(tile(c, 0), mk, 0, t, 0, hd / p.rk, &bar[SB_FULL + s]);
            }
            __syncwarp();
            loaded = c + 1;
        }
    } else {
        const uint32_t IDt = tc::idesc_bf16(128, 128, false, true);
        for (int c = 0; c < nc; ++c) {
            const uint64_t dk = tc::sdesc(smem_u32(tile(c, 0)), TILE / 2, 1024);
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                if (!wait(SB_READY + i, c)) break;
                if (elect()) {
                    piece_products(tbase, tbase + C_V + PLANES * i, dk, i, IDt, c == 0 && i == 0, true);
                    tc::mma_commit(&bar[SB_FREE + i]);
                    if (i == PIECES - 1) tc::mma_commit(&bar[SB_EMPTY + c % S_STAGES]);
                    if (i == PIECES - 1 && c == nc - 1) tc::mma_commit(&bar[SB_DONE]);
                }
                __syncwarp();
            }
            if (!ok) break;
        }
    }
    if (!ok) *abort_flag = 1;
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (*abort_flag) {
        if (tid == 0) *a.status = KDA_ERR_TIMEOUT;
        if (w == 8)
            for (int c = max(loaded - S_STAGES, 0); c < loaded; ++c)
                tc::mbar_wait(&bar[SB_FULL + c % S_STAGES], (c / S_STAGES) & 1, 100000000ull);
        if (w == 9 && elect()) tc::drain_mmas(&bar[SB_SPARE], 100000000ull);
        __syncthreads();
    }
    if (w == 0) tc::tmem_dealloc(tbase, 512);
}

}  // namespace

cudaError_t lin_setup() {
    cudaError_t e = cudaFuncSetAttribute(k_lin_walk, cudaFuncAttributeMaxDynamicSharedMemorySize, int(WALK_SMEM));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(k_lin_state, cudaFuncAttributeMaxDynamicSharedMemorySize, int(STATE_SMEM));
}

// segments that the call may have
static unsigned lin_segments(const LinArgs& a) { return unsigned(a.direct ? a.N : a.T / a.seg + a.N); }

void launch_lin_states(const LinArgs& a, const LinMaps& tm, int pass, cudaStream_t st) {
    {
        ProfScope ps(KK_LIN_STATE, st);
        k_lin_state<<<lin_segments(a) * unsigned(a.H), STATE_THREADS, STATE_SMEM, st>>>(a, pass, tm);
    }
    launch_lin_carry(a, pass, st);
}

void launch_lin_walk(const LinArgs& a, const LinMaps& tm, cudaStream_t st) {
    ProfScope ps(KK_LIN_WALK, st);
    k_lin_walk<<<lin_segments(a) * unsigned(a.H) * unsigned(a.passes), WALK_THREADS, WALK_SMEM, st>>>(a, tm);
}

}  // namespace kda
