// delta_chunk.cu -- the gated delta rule over prompts, 32 rows at a time.
//
// A key row is k_i = r_i K_i, K_i with its largest element in [1, 2) and r_i what is left
// of its size (over its norm, where rows are normalized).  With G_i the running sum of
// the log decays inside a chunk, a_i = e^{G_i}, b_i = beta_i r_i, W_i what row i adds to
// the state along K_i, and S the state before it, the rows of a chunk are
//   W = T diag(b) (V - diag(a r) K S),  T = (I + L)^-1,
//   L_ij = b_i r_i e^{G_i - G_j} K_i.K_j  (j < i),
//   O = diag(a) Q S + A W,  A_ij = e^{G_i - G_j} Q_i.K_j  (j <= i),
//   S <- e^{G_C} S + K^T diag(e^{G_C - G_j}) W.
// The sizes of keys stay in b and r, which are fp32 numbers: W has the state's size, and
// T and A have none.
// T and A depend on the rows alone, so helper warps prepare them (and the
// tiles) four to six chunks ahead; what is serial is the chain over S.  The columns
// of S are independent: a chain warp owns 16 of them and keeps S^T [16][k_dim] in
// fp32 accumulator registers (with 32 columns a CTA, two warps with half of k_dim
// each).  Every product takes its left operand from registers that the product
// before it left there (S^T K^T, Y^T T^T, W^T K).
//
// Precision: the tensor cores multiply 16-bit floats.  K and Q rows are bf16 and
// become fp16 exactly up to a power of two per row; S, Y, W, T and A are split
// into two fp16 parts each (22 bits; 11 + 11), two products where the other
// operand is exact, three where both are split.  The answers need both parts too: a
// row that overwrites what the state held has Q S and A W cancel, and what is left
// of 11 bits of each can be all wrong.  fp16's range is covered by a power of two per
// state column that follows the column's size; an element of K or Q below 2^-14 of its
// row's largest, and a product's operand below 2^-11 of its column's size, is off by up
// to 2^-25 of that size instead of 2^-24 of itself.  Two kinds of parts of a chunk would
// leave fp16's range and are taken row by row in fp32, by the same warps on the same
// registers: rows that stretch the state (b r |K|^2 past 2.25, or an entry of T past 64,
// or a growing "decay"), and columns whose size changes too far within the part (a row
// that finds far less than the state the part began with, or than what is written later).
// 32 rows then take 15 to 18 us instead of 1.9 to 4.
//
// Bound by the chain: 4096 rows of one sequence, 32 heads of 128 x 128, take 247 us
// (1.9 us a chunk; its mma.sync instructions alone 0.3 us of it, the rest what each
// of them waits for), 8 sequences of 1 to 1024 rows 129 us, the 1024 rows being the
// longest chain (4.0 us a chunk of 128 columns, 1.6 us of tensor time).  Tried and
// slower: the state's update fused with the next chunk's K S (415 us: spills), rows
// brought in by bulk copies (96 small ones a chunk), helpers with unrolled loops
// (their code pushes the chain's out of the instruction cache: 267 to 320 us).
#include <climits>

#include "seq.cuh"
#include "tc5.cuh"

namespace gattn {

namespace {

constexpr int kC = 32;             // rows of a chunk
constexpr int kTS = 40;            // row stride of T and A (halves): conflict-free ldmatrix
constexpr int kLS = 16;            // row stride of L's diagonal blocks (floats)
constexpr float kMinG = -200.f;    // e^-200 is 0 in fp32
// Parts with more than this go row by row.  A row's map I - b r K K^T does not stretch
// the state up to 2, and then no entry of T passes |K_j| / |K_i| * 2 < 46.  Sums of
// 32 products of such T, K and S in [0.5, 32] stay below fp16's 65504
constexpr float kGain = 2.25f, kTopT = 64.f, kGrowth = 1.f / 256;
// A column's unit is the state's, or that of what a part writes where that is more than
// kMost of the state's.  An operand is off by up to 2^-25 of the unit: a part goes row by
// row where a row finds less than kLeast of it, in what is left of the state the part
// began with (0.5 to 32 in its own unit) and in what has been written by then.  For a row
// that writes nothing, only answers in 8 bits, an eighth of that is enough
constexpr float kMost = 4096.f, kLeast = 1.f / 2048;

// Every array starts on a 16-byte boundary: they are read in 16-byte vectors.
template <int DK, int NCW>
struct alignas(16) Stage {
    alignas(16) __half k[kC][DK + 8];              // first bf16, then fp16 in place
    alignas(16) __half q[kC][DK + 8];
    alignas(16) __nv_bfloat16 v[kC][16 * NCW + 8];
    alignas(16) __half t_hi[kC][kTS];              // T^T: [j][i]
    alignas(16) __half t_lo[kC][kTS];
    alignas(16) __half a_hi[kC][kTS];              // A^T: [j][i]
    alignas(16) __half a_lo[kC][kTS];
    alignas(16) float ar[kC];                      // per row: a r, b, e^{G_C - G}, a, scale of q
    alignas(16) float b[kC];
    alignas(16) float c[kC];
    alignas(16) float a[kC];
    alignas(16) float sq[kC];
    alignas(16) float r[kC];                       // for rows one by one: r, e^g
    alignas(16) float d[kC];
    alignas(16) float found[kC];                   // |b v| a row finds written, over the part's largest; negative
                                                   // before any b.  While T and A are made: low parts of G
    // the helper's own
    alignas(16) float lt[kC][kLS];                 // diagonal blocks of L^T: [j][i - j - 1]
    alignas(16) float gh[kC];
    alignas(16) float br[kC];                      // b r
    float gamma;                                   // decay of the part
    float most;                                    // largest |b v|, infinite for `alone`
    float low[2][NCW];                             // smallest_writes(): with and without empty columns
    int lo, hi, more;                              // rows of the chunk this is for; more of it follow
    int alone;                                     // row by row
};

// The warps of a CTA: a chain warp per 16 of its NCW * 16 state columns, and helper
// warps with a stage each.  With two such groups of columns the serial chain gets
// all that shortens it: two warps per group, half of the state's rows each, that
// add up their shares of K S, and an output warp per group for Q S and A W.
template <int NCW>
struct Roles {
    static constexpr bool SPLIT = NCW == 2;
    static constexpr int KH = SPLIT ? 2 : 1;       // chain warps per group of columns
    static constexpr int CHAIN = NCW * KH;
    static constexpr int OUT = SPLIT ? NCW : 0;
    static constexpr int HELP = SPLIT ? 6 : 4;
    static constexpr int THREADS = (CHAIN + OUT + HELP) * 32;
};

// What chain warps hand their output warp: S in parts, as operands, and W.
template <int DK>
struct alignas(16) Handed {
    uint4 s[DK / 16][2][32];
    float4 w[4][32];
    float2 unit[32];
};

// What a chain warp hands the other one of its columns: its share of K S and of the
// columns' largest elements.
struct alignas(16) Share {
    float4 x[4][32];
    float2 top[32];
};

template <int DK, int NCW>
struct alignas(16) Shared {
    using R = Roles<NCW>;
    Stage<DK, NCW> st[R::HELP];
    Handed<DK> to[R::SPLIT ? NCW : 1];
    Share share[R::SPLIT ? NCW : 1][R::KH];
    uint64_t full[R::HELP], empty[R::HELP];
    uint64_t s_full[2], w_full[2], taken[2], shared[2][2], read[2][2];
    int abort;
};
static_assert((kTS * 2) % 16 == 0 && (kLS * 4) % 16 == 0 && sizeof(Stage<128, 2>) % 16 == 0 &&
                  sizeof(Stage<64, 8>) % 16 == 0,
              "vectors of 16 bytes");

// Stores four 8x8 fragments transposed: memory rows are the fragments' columns.
__device__ __forceinline__ void stsm_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a),
                 "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void cp16_zfill(void *dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// (x0, x1) as hi + lo fp16 pairs
__device__ __forceinline__ void split_h2(float x0, float x1, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = pack_h2(x0 - f.x, x1 - f.y);
}

// A fragments (hi, lo) of one k16 step from two neighbouring accumulator tiles
__device__ __forceinline__ void split_frag(const float (&c0)[4], const float (&c1)[4], uint32_t (&hi)[4],
                                           uint32_t (&lo)[4])
{
    split_h2(c0[0], c0[1], hi[0], lo[0]);
    split_h2(c0[2], c0[3], hi[1], lo[1]);
    split_h2(c1[0], c1[1], hi[2], lo[2]);
    split_h2(c1[2], c1[3], hi[3], lo[3]);
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    mma_f16(d, a, b0, b1, d);
}

// 2^(hi + lo), lo below a unit in the last place of hi
__device__ __forceinline__ float ex2_pair(float hi, float lo) { return ex2(hi) * fmaf(lo, 0.693147181f, 1.f); }

// Largest magnitude (bf16 bits) of a row of 16-byte units.
template <int U>
__device__ __forceinline__ unsigned row_top(const void *row)
{
    const uint4 *p = static_cast<const uint4 *>(row);
    unsigned top = 0;
#pragma unroll 4
    for (int i = 0; i < U; ++i) {
        const uint4 u = p[i];
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                                     __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
    }
    return max(top & 0xFFFFu, top >> 16);
}

// A bf16 row of K and one of Q in shared memory become fp16 with their largest
// elements brought to [1, 2): returns the powers of two multiplied by and the sums of
// squares of the result.  A lane per pair of rows; topk, topq: the largest
// magnitudes.
template <int DK>
__device__ __forceinline__ float4 rows_to_half(__half *krow, __half *qrow, unsigned topk, unsigned topq)
{
    uint4 *kp = reinterpret_cast<uint4 *>(krow), *qp = reinterpret_cast<uint4 *>(qrow);
    int ek = (int)(topk >> 7), eq = (int)(topq >> 7);
    ek = ek == 255 ? 127 : min(max(ek, 1), 253);     // infinities and NaN pass as they are
    eq = eq == 255 ? 127 : min(max(eq, 1), 253);
    const float fk = __int_as_float((254 - ek) << 23), fq = __int_as_float((254 - eq) << 23);
    float kk[2] = {0.f, 0.f}, qq[2] = {0.f, 0.f};
    auto half_pair = [](uint32_t u, float f, float (&sum)[2]) {
        const uint32_t h = pack_h2(bf16_lo(u) * f, bf16_hi(u) * f);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        sum[0] = fmaf(x.x, x.x, sum[0]);
        sum[1] = fmaf(x.y, x.y, sum[1]);
        return h;
    };
#pragma unroll 1
    for (int i = 0; i < DK / 8; ++i) {
        const uint4 u = kp[i], w = qp[i];
        kp[i] = make_uint4(half_pair(u.x, fk, kk), half_pair(u.y, fk, kk), half_pair(u.z, fk, kk),
                           half_pair(u.w, fk, kk));
        qp[i] = make_uint4(half_pair(w.x, fq, qq), half_pair(w.y, fq, qq), half_pair(w.z, fq, qq),
                           half_pair(w.w, fq, qq));
    }
    return make_float4(fk, fq, kk[0] + kk[1], qq[0] + qq[1]);
}

// For each chain warp's columns what tells it when to look closer: at most the smallest
// of the columns' largest |b v| (by every fourth row and to 2^-7), by `least`, what rows
// find of it at their least (infinite: of no interest).  Columns nothing is written to
// are left out; if the state may fade in one of them, low[0] is 0.
template <int DK, int NCW>
__device__ __forceinline__ void smallest_writes(Stage<DK, NCW> &s, float least)
{
    // lanes side by side on pairs of columns, two rows at once where pairs are few
    constexpr int PAIRS = 8 * NCW, SIDE = PAIRS < 32 ? PAIRS : 32, PER = PAIRS / SIDE, STEP = 32 / SIDE;
    const int lane = threadIdx.x & 31;
    unsigned top[PER];
    auto row = [&](int r) {
        const __nv_bfloat162 b = __float2bfloat162_rn(s.b[r]);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const __nv_bfloat162 v =
                __habs2(__hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&s.v[r][2 * (lane % SIDE + 32 * p)]), b));
            top[p] = __vmaxu2(top[p], *reinterpret_cast<const unsigned *>(&v));
        }
    };
    auto join = [&] {
        bool none = false;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
#pragma unroll
            for (int o = SIDE; o < 32; o <<= 1)
                top[p] = __vmaxu2(top[p], __shfl_xor_sync(0xffffffffu, top[p], o));
            none |= (top[p] & 0xFFFFu) == 0 || top[p] >> 16 == 0;
        }
        return none;
    };
#pragma unroll
    for (int p = 0; p < PER; ++p)
        top[p] = 0;
#pragma unroll
    for (int r = 3; r < kC; r += 4 * STEP)
        row(r + 4 * (lane / SIDE));
    if (__any_sync(0xffffffffu, join())) {
#pragma unroll 1
        for (int r = lane / SIDE; r < kC; r += STEP)
            row(r);
        join();
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const unsigned x = __vsub2(top[p], 0x00010001u);               // zeros go to the top
        unsigned low = min(x & 0xFFFFu, x >> 16), high = max(x & 0xFFFFu, x >> 16);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            low = min(low, __shfl_xor_sync(0xffffffffu, low, o));
            high = max(high, __shfl_xor_sync(0xffffffffu, high, o));
        }
        const float f = __uint_as_float(low << 16);                     // NaN: none is written to
        if (lane < SIDE && lane % 8 == 0) {
            const int group = lane / 8 + 4 * p;
            s.low[0][group] = high == 0xFFFFu && least < INFINITY ? 0.f : f * least;
            s.low[1][group] = f * fminf(least, 1.f);
        }
    }
}

// Everything of rows [lo, hi) of the chunk at t0 that does not depend on the
// state, by one warp; the chunk's other rows count as absent.  A row whose key,
// value, decay or strength is not finite has to be the first of its part: 0 * NaN
// would carry it to the rows before it.  When there is one in between, nothing is
// prepared and its index is returned, else hi.
template <int DK, int NCW>
__device__ __forceinline__ int prepare_rows(const DeltaArgs &a, Stage<DK, NCW> &s, int t0, int lo, int hi, int h,
                                            int hk, int col0)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr int KU = DK / 8, VU = 2 * NCW;      // 16-byte units of a row
    {
        const __nv_bfloat16 *kp = a.k + hk * a.ks.head, *qp = a.q + hk * a.qs.head;
        const int c = (lane % KU) * 8;
#pragma unroll 2
        for (int r = lane / KU; r < kC; r += 32 / KU) {
            const bool ok = r >= lo && r < hi;
            const long long row = t0 + (ok ? r : lo);
            cp16_zfill(&s.k[r][c], kp + row * a.ks.tok + c, ok);
            cp16_zfill(&s.q[r][c], qp + row * a.qs.tok + c, ok);
        }
        const __nv_bfloat16 *vp = a.v + h * a.vs.head + col0;
        const int cv = (lane % VU) * 8;
#pragma unroll 1
        for (int r = lane / VU; r < kC; r += 32 / VU) {
            const bool ok = r >= lo && r < hi;
            cp16_zfill(&s.v[r][cv], vp + (t0 + (ok ? r : lo)) * a.vs.tok + cv, ok);
        }
    }
    const bool on = lane >= lo && lane < hi;
    const float beta = on ? a.beta[(long long)(t0 + lane) * a.bt + h] : 0.f;
    float gr = on ? a.g[(long long)(t0 + lane) * a.gt + h] : 0.f;
    gr = gr < kMinG ? kMinG : gr;
    // the sums in units of log2 e and as float pairs: differences of far sums stay exact
    float gh = gr * 1.44269502f, gl = fmaf(gr, 1.44269502f, -gh) + gr * 1.92596299e-8f;
    s.d[lane] = expf(gr);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float h2 = __shfl_up_sync(0xffffffffu, gh, o), l2 = __shfl_up_sync(0xffffffffu, gl, o);
        if (lane >= o) {
            const float sum = gh + h2, b = sum - gh;
            gl += l2 + ((gh - (sum - b)) + (h2 - b));
            gh = sum;
        }
    }
    const float gch = __shfl_sync(0xffffffffu, gh, 31), gcl = __shfl_sync(0xffffffffu, gl, 31);
    s.gh[lane] = gh;
    s.found[lane] = gl;
    const float ai = ex2_pair(gh, gl), ci = ex2((gch - gh) + (gcl - gl));
    cp_async_wait_all();
    __syncwarp();
    const unsigned topk = row_top<KU>(&s.k[lane][0]);
    const unsigned topv = row_top<VU>(&s.v[lane][0]);
    const bool bad = lane > lo && lane < hi &&
                     (topk >= 0x7F80u || topv >= 0x7F80u ||
                      !(fabsf(gr) < INFINITY) || !(fabsf(beta) < INFINITY));
    const unsigned bads = __ballot_sync(0xffffffffu, bad);
    if (bads)
        return __ffs(bads) - 1;
    const float4 row = rows_to_half<DK>(&s.k[lane][0], &s.q[lane][0], topk, row_top<KU>(&s.q[lane][0]));
    // r of k = K 2^-e / sqrt(4^-e sum + eps), 2^e at hand; beside an eps 4^e past fp32 the
    // sum of a row below 2^-50 counts for nothing
    auto power = [](float inv) { return __int_as_float((254 << 23) - __float_as_int(inv)); };
    auto norm = [&](float inv, float sum) {
        const float e = a.l2_eps * inv * inv;
        return !a.l2norm ? power(inv) : e < INFINITY ? rsqrtf(sum + e) : power(inv) * rsqrtf(a.l2_eps);
    };
    const float r = on ? norm(row.x, row.z) : 0.f, rq = on ? norm(row.y, row.w) : 0.f;
    s.r[lane] = r;
    s.br[lane] = beta * r * r;
    const bool stretch = !(fabsf(beta * r * r) * row.z <= kGain) || gr > kGrowth;
    s.b[lane] = beta * r;
    s.a[lane] = ai;
    s.ar[lane] = ai * r;
    s.c[lane] = ci;
    s.sq[lane] = a.scale * rq;
    // the largest |b v|; as bits: order of non-negative floats, with NaN on top
    const float write = fabsf(beta * r) * __uint_as_float(topv << 16);
    const unsigned wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(write));
    // what a row finds written, to a power of two: the largest so far with its decay
    const int at = __float2int_rn(gh);
    int size = write > 0.f ? (__float_as_int(write) >> 23) - at : INT_MIN / 2;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int s2 = __shfl_up_sync(0xffffffffu, size, o);
        if (lane >= o)
            size = max(size, s2);
    }
    const int most = __reduce_max_sync(0xffffffffu, on ? size + at : INT_MIN / 2);
    const unsigned acts = __ballot_sync(0xffffffffu, on && beta != 0.f);
    const bool still = (acts & ((2u << lane) - 1)) == 0;           // as if the state only decayed
    const float answers = acts >> lane & 1 ? 1.f : 8.f;
    const float found = still ? -1.f : ex2((float)(size + at - most)) * answers;
    // where little is left of the state: the least that is found written
    const unsigned least = __reduce_min_sync(
        0xffffffffu, __float_as_uint(on && !still && ai * answers < 2.f * kLeast ? found : INFINITY));
    if (lane == 31) {
        s.gamma = ai;
        s.most = __uint_as_float(wtop);
    }
    __syncwarp();
    smallest_writes(s, __uint_as_float(least));
    // The 16 x 8 tiles of K K^T and K Q^T (row j, column i) that hold some i >= j, and
    // from each its part of L and of A.  A loop that stays rolled: with it the code of
    // all roles stays small enough for the SM's instruction cache
    uint32_t bh[2][2], bl[2][2];       // L of rows 16-31, columns 0-15, as a B operand
    const int ar = (lane & 7) + ((lane >> 3) & 1) * 8, ac = (lane >> 4) * 8;
    const __half *brow = (lane < 16 ? &s.k[0][0] : &s.q[0][0]) + (lane & 7) * (DK + 8) + ((lane >> 3) & 1) * 8;
#pragma unroll 1
    for (int tile = 0; tile < 6; ++tile) {
        const int mt = tile >> 2, nt = tile - 2 * mt;
        float kk[4] = {}, kq[4] = {};
        const uint32_t pa = smem_u32(&s.k[mt * 16 + ar][ac]), pb = smem_u32(brow + nt * 8 * (DK + 8));
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks) {
            uint32_t fa[4], fb[4];
            ldsm_x4(fa, pa + ks * 32);
            ldsm_x4(fb, pb + ks * 32);
            mma(kk, fa, fb[0], fb[1]);
            mma(kq, fa, fb[2], fb[3]);
        }
        const int i0 = nt * 8 + 2 * t;
        const float2 ghi = *reinterpret_cast<const float2 *>(&s.gh[i0]);
        const float2 gli = *reinterpret_cast<const float2 *>(&s.found[i0]);
        const float2 bi = *reinterpret_cast<const float2 *>(&s.br[i0]);
        uint32_t vh[2], vl[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int j = mt * 16 + g + half * 8;
            const float ghj = s.gh[j], glj = s.found[j];
            const float d0 = i0 >= j ? ex2((ghi.x - ghj) + (gli.x - glj)) : 0.f;
            const float d1 = i0 + 1 >= j ? ex2((ghi.y - ghj) + (gli.y - glj)) : 0.f;
            const float l0 = d0 * bi.x * kk[half * 2];
            const float l1 = d1 * bi.y * kk[half * 2 + 1];
            if (tile != 2 && tile != 3) {      // a diagonal block's: column j from its row j + 1 on
                float *lt = &s.lt[j][i0 - j - 1];
                if (i0 > j)
                    lt[0] = l0;
                if (i0 + 1 > j)
                    lt[1] = l1;
            } else
                split_h2(l0, l1, vh[half], vl[half]);
            uint32_t wh, wl;
            split_h2(i0 >= j ? d0 * kq[half * 2] : 0.f, i0 + 1 >= j ? d1 * kq[half * 2 + 1] : 0.f, wh, wl);
            *reinterpret_cast<uint32_t *>(&s.a_hi[j][i0]) = wh;
            *reinterpret_cast<uint32_t *>(&s.a_lo[j][i0]) = wl;
        }
        if (tile == 2) {
            bh[0][0] = vh[0], bl[0][0] = vl[0];
            bh[1][0] = vh[1], bl[1][0] = vl[1];
        } else if (tile == 3) {
            bh[0][1] = vh[0], bl[0][1] = vl[0];
            bh[1][1] = vh[1], bl[1][1] = vl[1];
        }
    }
    __syncwarp();
    s.found[lane] = found;             // the tiles are done with G
    float top = 0.f;                   // T's largest entry
    // T = (I + L)^-1.  Its two 16 x 16 diagonal blocks by forward substitution, a
    // column per lane: x[0] is the next unknown, taken out of every later row while
    // those move up by one.  Rows past the block's last are never used
    {
        const int base = lane & 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = i == (lane & 15) ? 1.f : 0.f;
#pragma unroll
        for (int m = 0; m < 16; m += 2) {
            float xm[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                xm[e] = x[0];
#pragma unroll
                for (int i4 = 0; i4 < 4; ++i4) {
                    const float4 l = *reinterpret_cast<const float4 *>(&s.lt[base + m + e][i4 * 4]);
                    const float lv[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (i4 * 4 + k < 15)
                            x[i4 * 4 + k] = fmaf(-lv[k], xm[e], x[i4 * 4 + k + 1]);
                }
            }
            top = fmaxf(top, fmaxf(fabsf(xm[0]), fabsf(xm[1])));
            uint32_t xh, xl;
            split_h2(xm[0], xm[1], xh, xl);
            *reinterpret_cast<uint32_t *>(&s.t_hi[lane][base + m]) = xh;
            *reinterpret_cast<uint32_t *>(&s.t_lo[lane][base + m]) = xl;
        }
    }
    __syncwarp();
    // the block below them: T21 = -T22 (L21 T11), associated as (T22 L21) T11
    {
        const int pr = (lane & 7) + (lane >> 4) * 8, pc = ((lane >> 3) & 1) * 8;
        uint32_t fh[4], fl[4];
        // T22 [i][n] from its transpose
        ldsm_x4_trans(fh, smem_u32(&s.t_hi[16 + pr][16 + pc]));
        ldsm_x4_trans(fl, smem_u32(&s.t_lo[16 + pr][16 + pc]));
        float p[2][4] = {}, q[2][4] = {};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            mma(p[n], fh, bh[n][0], bh[n][1]);
            mma(p[n], fl, bh[n][0], bh[n][1]);
            mma(p[n], fh, bl[n][0], bl[n][1]);
        }
        split_frag(p[0], p[1], fh, fl);
        uint32_t th[4], tl[4];
        ldsm_x4(th, smem_u32(&s.t_hi[pr][pc]));
        ldsm_x4(tl, smem_u32(&s.t_lo[pr][pc]));
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            mma(q[n], fh, th[2 * n], th[2 * n + 1]);
            mma(q[n], fl, th[2 * n], th[2 * n + 1]);
            mma(q[n], fh, tl[2 * n], tl[2 * n + 1]);
        }
        // q [i][j], stored as T^T [j][16 + i]
        uint32_t xh[4], xl[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top = fmaxf(top, fmaxf(fabsf(q[n][2 * half]), fabsf(q[n][2 * half + 1])));
                split_h2(-q[n][2 * half], -q[n][2 * half + 1], xh[2 * n + half], xl[2 * n + half]);
            }
        stsm_x4_trans(smem_u32(&s.t_hi[pr][16 + pc]), xh[0], xh[1], xh[2], xh[3]);
        stsm_x4_trans(smem_u32(&s.t_lo[pr][16 + pc]), xl[0], xl[1], xl[2], xl[3]);
    }
    const bool alone = __any_sync(0xffffffffu, (on && stretch) || !(top <= kTopT));
    if (lane == 0) {
        s.alone = alone;
        if (alone)
            s.most = INFINITY;
    }
    return hi;
}

// The sequence of a rank, longest first where a warp can sort them (up to 64).
__device__ __forceinline__ int ranked_seq(const SeqArgs &q, int rank)
{
    if (!q.cu || q.n > 64)
        return rank;
    const int lane = threadIdx.x & 31;
    int r0, len[2], above[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        len[k] = -1;
        if (lane + 32 * k < q.n)
            seq_rows(q, lane + 32 * k, r0, len[k]);
    }
    for (int i = 0; i < q.n; ++i) {
        const int li = __shfl_sync(0xffffffffu, i < 32 ? len[0] : len[1], i & 31);
#pragma unroll
        for (int k = 0; k < 2; ++k)
            above[k] += li > len[k] || (li == len[k] && i < lane + 32 * k);
    }
    const unsigned m0 = __ballot_sync(0xffffffffu, lane < q.n && above[0] == rank);
    const unsigned m1 = __ballot_sync(0xffffffffu, lane + 32 < q.n && above[1] == rank);
    return m0 ? __ffs(m0) - 1 : 31 + __ffs(m1);
}

template <int DK, int NCW>
__global__ void __launch_bounds__(Roles<NCW>::THREADS, 1)
delta_chunk_kernel(const __grid_constant__ DeltaArgs a)
{
    using R = Roles<NCW>;
    extern __shared__ __align__(128) uint8_t raw[];
    auto &sh = *reinterpret_cast<Shared<DK, NCW> *>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int parts = a.dv / (16 * NCW);
    const int part = blockIdx.x % parts, h = (blockIdx.x / parts) % a.Hv;
    const int s = ranked_seq(a.sq, blockIdx.x / parts / a.Hv);
    const int hk = h / (a.Hv / a.Hk), col0 = part * 16 * NCW;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    if (slot < 0) {
        if (threadIdx.x == 0)
            seq_flag(a.sq, GATTN_STATUS_RANGE);
        __nv_bfloat16 *out = a.out + (long long)h * a.os.head + col0;
        for (long long i = threadIdx.x; i < (long long)len * 2 * NCW; i += blockDim.x)
            *reinterpret_cast<uint4 *>(out + (r0 + i / (2 * NCW)) * a.os.tok + (i % (2 * NCW)) * 8) =
                make_uint4(0, 0, 0, 0);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < R::HELP; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], R::CHAIN + R::OUT);
        }
        for (int i = 0; i < R::OUT; ++i) {
            mbar_init(&sh.s_full[i], R::KH);
            mbar_init(&sh.w_full[i], 1);
            mbar_init(&sh.taken[i], 1);
            for (int k = 0; k < 2; ++k) {
                mbar_init(&sh.shared[i][k], 1);
                mbar_init(&sh.read[i][k], 1);
            }
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    volatile int *abort = &sh.abort;
    const int chunks = (len + kC - 1) / kC;
    if (warp >= R::CHAIN + R::OUT) {
        const int w = warp - R::CHAIN - R::OUT;
        Stage<DK, NCW> &st = sh.st[w];
        int use = 0, lo = 0, hi = 0;
        for (int c = w; c < chunks;) {
            // a part of the chunk: all of it, but for rows that are not finite
            const int rows = min(kC, len - c * kC);
            if (hi <= lo) {
                hi = rows;
                if (use > 0 && !__all_sync(0xffffffffu, tc5_wait(&sh.empty[w], (use - 1) & 1, abort)))
                    break;
            }
            const int end = prepare_rows<DK, NCW>(a, st, r0 + c * kC, lo, hi, h, hk, col0);
            if (end < hi) {
                __syncwarp();
                hi = end;
                continue;
            }
            if (lane == 0) {
                st.lo = lo;
                st.hi = hi;
                st.more = hi < rows;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.full[w]);
            ++use;
            lo = hi < rows ? hi : 0;
            hi = 0;
            c += lo ? 0 : R::HELP;
        }
        return;
    }
    // ldmatrix lane addresses: rows of a tile pair (plain), k rows of one step (trans)
    const int pr = (lane & 7) + (lane >> 4) * 8, pc = ((lane >> 3) & 1) * 8;
    const int tr = (lane & 7) + ((lane >> 3) & 1) * 8, tc = (lane >> 4) * 8;
    const int cw = warp % NCW;             // whose 16 columns
    __nv_bfloat16 *out = a.out + (long long)(r0 + lane) * a.os.tok + (long long)h * a.os.head + col0 + cw * 16;
    // one k16 step of (16 columns of S) x (32 rows of K or Q), and its operand
    auto load_rows = [&](uint32_t (&b)[2][4], const __half (*rows)[DK + 8], int ks) {
#pragma unroll
        for (int n2 = 0; n2 < 2; ++n2)
            ldsm_x4(b[n2], smem_u32(&rows[n2 * 16 + pr][ks * 16 + pc]));
    };
    auto times_rows = [&](float (&D)[4][4], float (&E)[4][4], const uint32_t (&hi)[4], const uint32_t (&lo)[4],
                          const uint32_t (&b)[2][4]) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            mma(D[nt], hi, b[nt / 2][(nt & 1) * 2], b[nt / 2][(nt & 1) * 2 + 1]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            mma(E[nt], lo, b[nt / 2][(nt & 1) * 2], b[nt / 2][(nt & 1) * 2 + 1]);
    };
    // D += X M^T for a lower triangular M [i][j], held transposed in two parts: its
    // rows 0-15 need the first k16 step only
    auto times_lower = [&](float (&D)[4][4], const float (&X)[4][4], const __half (*mh)[kTS],
                           const __half (*ml)[kTS]) {
        uint32_t hi[2][4], lo[2][4];
        split_frag(X[0], X[1], hi[0], lo[0]);
        split_frag(X[2], X[3], hi[1], lo[1]);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int n2 = kk; n2 < 2; ++n2) {
                uint32_t th[4], tl[4];
                ldsm_x4_trans(th, smem_u32(&mh[kk * 16 + tr][n2 * 16 + tc]));
                ldsm_x4_trans(tl, smem_u32(&ml[kk * 16 + tr][n2 * 16 + tc]));
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma(D[n2 * 2 + n], hi[kk], th[2 * n], th[2 * n + 1]);
                    mma(D[n2 * 2 + n], lo[kk], th[2 * n], th[2 * n + 1]);
                    mma(D[n2 * 2 + n], hi[kk], tl[2 * n], tl[2 * n + 1]);
                }
            }
    };
    // a part's rows on their way out, from where their values were: a row of 16
    // columns per lane
    auto rows_out = [&](Stage<DK, NCW> &st, int c) {
        __syncwarp();
        if (lane >= st.lo && lane < st.hi) {
            const uint4 *src = reinterpret_cast<const uint4 *>(&st.v[lane][cw * 16]);
            uint4 *dst = reinterpret_cast<uint4 *>(out + (long long)c * kC * a.os.tok);
            dst[0] = src[0];
            dst[1] = src[1];
        }
    };
    // O = scale (a Q S + A W), O holding Q S
    auto finish_rows = [&](float (&O)[4][4], float (&W)[4][4], Stage<DK, NCW> &st, int c, float u0, float u1) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            const float2 aa = *reinterpret_cast<const float2 *>(&st.a[nt * 8 + 2 * t]);
            O[nt][0] *= aa.x;
            O[nt][1] *= aa.y;
            O[nt][2] *= aa.x;
            O[nt][3] *= aa.y;
        }
        float top = 0.f;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            top = fmaxf(top, fmaxf(fmaxf(fabsf(W[nt][0]), fabsf(W[nt][1])), fmaxf(fabsf(W[nt][2]), fabsf(W[nt][3]))));
        if (__any_sync(0xffffffffu, top > 32768.f)) {      // past fp16's range: in larger units
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    O[nt][e] *= 0x1p-12f;
                    W[nt][e] *= 0x1p-12f;
                }
            u0 *= 0x1p12f;
            u1 *= 0x1p12f;
        }
        times_lower(O, W, st.a_hi, st.a_lo);
#pragma unroll
        for (int n2 = 0; n2 < 2; ++n2) {
            uint32_t x[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const int nt = n2 * 2 + n;
                const float2 f = *reinterpret_cast<const float2 *>(&st.sq[nt * 8 + 2 * t]);
                x[n * 2] = pack_bf16x2(O[nt][0] * f.x * u0, O[nt][1] * f.y * u0);
                x[n * 2 + 1] = pack_bf16x2(O[nt][2] * f.x * u1, O[nt][3] * f.y * u1);
            }
            stsm_x4_trans(smem_u32(&st.v[n2 * 16 + pr][cw * 16 + pc]), x[0], x[1], x[2], x[3]);
        }
        rows_out(st, c);
    };
    bool ok = true;
    unsigned phase = 0;                    // per stage
    if (R::SPLIT && warp >= R::CHAIN) {
        // ------------------------------------------------ output warps
        Handed<DK> &from = sh.to[R::SPLIT ? cw : 0];
        for (int c = 0, turn = 0; c < chunks; turn ^= 1) {
            const int w = c % R::HELP;
            ok = __all_sync(0xffffffffu, tc5_wait(&sh.full[w], phase >> w & 1, abort) &&
                                             tc5_wait(&sh.s_full[cw & 1], turn, abort));
            if (!ok)
                break;
            phase ^= 1u << w;
            Stage<DK, NCW> &st = sh.st[w];
            float O[4][4] = {}, W[4][4];
#pragma unroll 2
            for (int ks = 0; ks < DK / 16; ++ks) {
                const uint4 uh = from.s[ks][0][lane], ul = from.s[ks][1][lane];
                const uint32_t hi[4] = {uh.x, uh.y, uh.z, uh.w}, lo[4] = {ul.x, ul.y, ul.z, ul.w};
                uint32_t b[2][4];
                load_rows(b, st.q, ks);
                times_rows(O, O, hi, lo, b);
            }
            ok = __all_sync(0xffffffffu, tc5_wait(&sh.w_full[cw & 1], turn, abort));
            if (!ok)
                break;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float4 x = from.w[nt][lane];
                W[nt][0] = x.x;
                W[nt][1] = x.y;
                W[nt][2] = x.z;
                W[nt][3] = x.w;
            }
            const float2 u = from.unit[lane];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.taken[cw & 1]);
            if (u.x > 0.f)                 // else the chain wrote them row by row
                finish_rows(O, W, st, c, u.x, u.y);
            c += st.more ? 0 : 1;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[w]);
        }
        return;
    }
    // ------------------------------------------------------------------- the chain
    // accumulator tile j holds S^T: rows (columns of S) g and g + 8, k-elements
    // 8 j + 2 t and the next
    constexpr int ROWS = DK / R::KH;       // of the state, in this warp
    const int half = warp / NCW;           // which of them
    float S[ROWS / 8][4];
    const long long so = slot * a.state_stride + ((long long)h * DK + half * ROWS) * a.dv + col0 + cw * 16 + g;
#pragma unroll
    for (int j = 0; j < ROWS / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[j][e] = a.state ? a.state[so + (long long)(8 * j + 2 * t + (e & 1)) * a.dv + (e >> 1) * 8] : 0.f;
    // rows g and g + 8 of S are held in units of a power of two each, so that the
    // parts fit fp16
    float unit[2] = {1.f, 1.f}, inv_unit[2] = {1.f, 1.f};
    // the exponent that takes m into [8, 16), within limits that keep units finite; 0 for
    // 0, infinities and NaN
    auto steps = [&](int hf, float m) {
        const int e = m > 0.f && m < INFINITY ? min(max((__float_as_int(m) >> 23) - 130, -120), 120) : 0;
        const int ue = (__float_as_int(unit[hf]) >> 23) - 127;
        return min(max(e, -100 - ue), 120 - ue);
    };
    auto refit = [&](int hf, int e) {
        const int ue = (__float_as_int(unit[hf]) >> 23) - 127;
        unit[hf] = __int_as_float((127 + ue + e) << 23);
        inv_unit[hf] = __int_as_float((127 - ue - e) << 23);
        return __int_as_float((127 - e) << 23);
    };
    auto scale_rows = [&](float f0, float f1) {
#pragma unroll
        for (int j = 0; j < ROWS / 8; ++j) {
            S[j][0] *= f0;
            S[j][1] *= f0;
            S[j][2] *= f1;
            S[j][3] *= f1;
        }
    };
    auto quad_max = [&](float m) {
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    };
    float top0[2];                     // sizes of the columns, while `first` holds
    auto column_tops = [&] {
        top0[0] = top0[1] = 0.f;
#pragma unroll
        for (int j = 0; j < ROWS / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                top0[e >> 1] = fmaxf(top0[e >> 1], fabsf(S[j][e]));
    };
    column_tops();
    // X and top of the column's two halves together; false if the wait ran out
    int turns = 0;
    auto add_shares = [&](float (&X)[4][4], float (&top)[2]) {
        Share &mine = sh.share[R::SPLIT ? cw : 0][R::SPLIT ? half : 0];
        Share &other = sh.share[R::SPLIT ? cw : 0][R::SPLIT ? half ^ 1 : 0];
        if (turns > 0 && !__all_sync(0xffffffffu, tc5_wait(&sh.read[cw & 1][half], (turns - 1) & 1, abort)))
            return false;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            mine.x[nt][lane] = make_float4(X[nt][0], X[nt][1], X[nt][2], X[nt][3]);
        mine.top[lane] = make_float2(top[0], top[1]);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.shared[cw & 1][half ^ 1]);
        if (!__all_sync(0xffffffffu, tc5_wait(&sh.shared[cw & 1][half], turns & 1, abort)))
            return false;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            const float4 x = other.x[nt][lane];
            X[nt][0] += x.x;
            X[nt][1] += x.y;
            X[nt][2] += x.z;
            X[nt][3] += x.w;
        }
        top[0] = fmaxf(top[0], other.top[lane].x);
        top[1] = fmaxf(top[1], other.top[lane].y);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.read[cw & 1][half ^ 1]);
        ++turns;
        return true;
    };
    // top0 from this warp's own elements to the column's
    auto join_tops = [&] {
        if (R::SPLIT) {
            float none[4][4] = {};
            if (!add_shares(none, top0))
                return false;
        }
        top0[0] = quad_max(top0[0]);
        top0[1] = quad_max(top0[1]);
        return true;
    };
    ok = join_tops();
    // A part row by row, in fp32:
    //   S <- e^g S + K w,  w = b (v - r e^g S^T K),  out = scale (e^g S^T Q + (Q.K) w).
    // S leaves it in units of 1, with its sizes in top0
    auto row_by_row = [&](Stage<DK, NCW> &st, int c) {
        scale_rows(unit[0], unit[1]);
        unit[0] = unit[1] = inv_unit[0] = inv_unit[1] = 1.f;
        const int col = cw * 16 + g, k0 = half * ROWS + 2 * t;
#pragma unroll 1
        for (int i = st.lo; i < st.hi; ++i) {
            // this lane's elements of S^T K, S^T Q (columns g and g + 8) and Q.K
            float x[4][4] = {}, none[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < ROWS / 8; ++j) {
                const float2 k = __half22float2(*reinterpret_cast<const __half2 *>(&st.k[i][k0 + 8 * j]));
                const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&st.q[i][k0 + 8 * j]));
                x[0][0] = fmaf(S[j][0], k.x, fmaf(S[j][1], k.y, x[0][0]));
                x[0][1] = fmaf(S[j][2], k.x, fmaf(S[j][3], k.y, x[0][1]));
                x[0][2] = fmaf(S[j][0], q.x, fmaf(S[j][1], q.y, x[0][2]));
                x[0][3] = fmaf(S[j][2], q.x, fmaf(S[j][3], q.y, x[0][3]));
                x[1][0] = fmaf(k.x, q.x, fmaf(k.y, q.y, x[1][0]));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[0][e] += __shfl_xor_sync(0xffffffffu, x[0][e], o);
                x[1][0] += __shfl_xor_sync(0xffffffffu, x[1][0], o);
            }
            const float v0 = __bfloat162float(st.v[i][col]), v1 = __bfloat162float(st.v[i][col + 8]);
            if (R::SPLIT && !add_shares(x, none))
                return false;
            const float d = st.d[i], b = st.b[i], dr = d * st.r[i], sc = st.sq[i];
            const float w0 = b * (v0 - dr * x[0][0]), w1 = b * (v1 - dr * x[0][1]);
#pragma unroll
            for (int j = 0; j < ROWS / 8; ++j) {
                const float2 k = __half22float2(*reinterpret_cast<const __half2 *>(&st.k[i][k0 + 8 * j]));
                S[j][0] = fmaf(k.x, w0, d * S[j][0]);
                S[j][1] = fmaf(k.y, w0, d * S[j][1]);
                S[j][2] = fmaf(k.x, w1, d * S[j][2]);
                S[j][3] = fmaf(k.y, w1, d * S[j][3]);
            }
            __syncwarp();                  // the row's values have been read
            if (half == 0 && t == 0) {
                st.v[i][col] = __float2bfloat16(sc * fmaf(x[1][0], w0, d * x[0][2]));
                st.v[i][col + 8] = __float2bfloat16(sc * fmaf(x[1][0], w1, d * x[0][3]));
            }
        }
        if (half == 0)
            rows_out(st, c);
        column_tops();
        return join_tops();
    };
    bool first = true;
    Handed<DK> &to = sh.to[R::SPLIT ? cw : 0];
    auto load_values = [&](float (&v)[4][4], const Stage<DK, NCW> &st) {
#pragma unroll
        for (int n2 = 0; n2 < 2; ++n2) {
            uint32_t x[4];
            // rows of the tile are packed rows, its columns ours: transposed
            ldsm_x4_trans(x, smem_u32(&st.v[n2 * 16 + pr][cw * 16 + pc]));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int nt = n2 * 2 + (e >> 1), hf = e & 1;
                v[nt][hf * 2] = bf16_lo(x[e]);
                v[nt][hf * 2 + 1] = bf16_hi(x[e]);
            }
        }
    };
    auto pow2 = [](int e) { return __int_as_float((127 + e) << 23); };
    bool looked = false;
    int bare = 0, empty = 0;               // a column of the warp, which of the lane's, without a state
    for (int c = 0, use = 0; ok && c < chunks;) {
        // the loop proper, until a part wants a closer look: what that takes stands
        // behind it, so that its registers and code are not in the way
        bool apart = false;
        for (; ok && c < chunks; ++use) {
            const int w = c % R::HELP, turn = use & 1;
            ok = __all_sync(0xffffffffu, tc5_wait(&sh.full[w], phase >> w & 1, abort));
            if (!ok)
                break;
            Stage<DK, NCW> &st = sh.st[w];
            float v[4][4];
            load_values(v, st);
            if (__any_sync(0xffffffffu, first || !(st.most * fmaxf(inv_unit[0], inv_unit[1]) <= kMost) ||
                                            st.low[bare][cw] * fminf(inv_unit[0], inv_unit[1]) <
                                                (bare ? 1.f / 1024 : 1.25f * kLeast)) &&
                !looked) {
                apart = true;
                break;
            }
            looked = false;
            phase ^= 1u << w;
            // K S (and Q S)
            float X[4][4] = {}, O[4][4] = {};
            __half2 top[2] = {__half2half2(__ushort_as_half(0)), __half2half2(__ushort_as_half(0))};
            if (R::SPLIT && use > 0) {
                ok = __all_sync(0xffffffffu, tc5_wait(&sh.taken[cw & 1], turn ^ 1, abort));
                if (!ok)
                    break;
            }
            uint32_t bk[2][2][4], bq[2][4];
            float X2[4][4] = {};               // the low parts' sums, apart: shorter chains
            const int ks0 = half * (ROWS / 16);
            load_rows(bk[0], st.k, ks0);
#pragma unroll
            for (int ks = 0; ks < ROWS / 16; ++ks) {
                uint32_t hi[4], lo[4];
                if (ks + 1 < ROWS / 16)
                    load_rows(bk[(ks + 1) & 1], st.k, ks0 + ks + 1);
                if (!R::SPLIT)
                    load_rows(bq, st.q, ks);
                split_frag(S[2 * ks], S[2 * ks + 1], hi, lo);
                if (R::SPLIT) {
                    to.s[ks0 + ks][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    to.s[ks0 + ks][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top[e & 1] = __hmax2(top[e & 1], __habs2(*reinterpret_cast<const __half2 *>(&hi[e])));
                if (R::SPLIT)
                    times_rows(X, X2, hi, lo, bk[ks & 1]);
                else
                    times_rows(X, X, hi, lo, bk[ks & 1]);
                if (!R::SPLIT)
                    times_rows(O, O, hi, lo, bq);
            }
            if (R::SPLIT)
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        X[nt][e] += X2[nt][e];
            float m[2];                        // the columns' largest elements
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const float2 th = __half22float2(top[hf]);
                m[hf] = fmaxf(th.x, th.y);
            }
            if (R::SPLIT) {
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.s_full[cw & 1]);
                ok = add_shares(X, m);
                if (!ok)
                    break;
            }
            // Y = b (V - a r K S), then W = T Y
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float2 ar = *reinterpret_cast<const float2 *>(&st.ar[nt * 8 + 2 * t]);
                const float2 be = *reinterpret_cast<const float2 *>(&st.b[nt * 8 + 2 * t]);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    X[nt][2 * hf] = be.x * (v[nt][2 * hf] * inv_unit[hf] - ar.x * X[nt][2 * hf]);
                    X[nt][2 * hf + 1] = be.y * (v[nt][2 * hf + 1] * inv_unit[hf] - ar.y * X[nt][2 * hf + 1]);
                }
            }
            float W[4][4] = {};
            times_lower(W, X, st.t_hi, st.t_lo);
            if (R::SPLIT && half == 0) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
                    to.w[nt][lane] = make_float4(W[nt][0], W[nt][1], W[nt][2], W[nt][3]);
                to.unit[lane] = make_float2(unit[0], unit[1]);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.w_full[cw & 1]);
            }
            // S <- gamma S + (c W)^T K
            float ounit[2];
            {
                float P[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    const float2 cc = *reinterpret_cast<const float2 *>(&st.c[nt * 8 + 2 * t]);
                    P[nt][0] = W[nt][0] * cc.x;
                    P[nt][1] = W[nt][1] * cc.y;
                    P[nt][2] = W[nt][2] * cc.x;
                    P[nt][3] = W[nt][3] * cc.y;
                }
                // what S will hold: its decayed size, or what is written now
                const float gamma = st.gamma;
                float f[2];
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    m[hf] *= gamma;
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
                        m[hf] = fmaxf(m[hf], fmaxf(fabsf(P[nt][2 * hf]), fabsf(P[nt][2 * hf + 1])));
                    m[hf] = quad_max(m[hf]);
                    f[hf] = gamma;
                }
                ounit[0] = unit[0];
                ounit[1] = unit[1];
                auto out_of = [](float x) { return !(x >= 0.5f && x <= 32.f); };
                bare = empty = 0;
                if (__any_sync(0xffffffffu, out_of(m[0]) || out_of(m[1]))) {
                    empty = (m[0] == 0.f) + 2 * (m[1] == 0.f);
                    bare = __any_sync(0xffffffffu, empty);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        // left with nothing: a unit for what the other columns take
                        const float size = m[hf] == 0.f ? st.most * inv_unit[hf] : m[hf];
                        const float x = refit(hf, steps(hf, out_of(size) ? size : 0.f));
                        f[hf] *= x;
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt) {
                            P[nt][2 * hf] *= x;
                            P[nt][2 * hf + 1] *= x;
                        }
                    }
                }
                uint32_t hi[2][4], lo[2][4];
                split_frag(P[0], P[1], hi[0], lo[0]);
                split_frag(P[2], P[3], hi[1], lo[1]);
                scale_rows(f[0], f[1]);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int j2 = 0; j2 < ROWS / 16; ++j2) {
                        uint32_t b[4];
                        ldsm_x4_trans(b, smem_u32(&st.k[kk * 16 + tr][half * ROWS + j2 * 16 + tc]));
                        mma(S[2 * j2], hi[kk], b[0], b[1]);
                        mma(S[2 * j2 + 1], hi[kk], b[2], b[3]);
                        mma(S[2 * j2], lo[kk], b[0], b[1]);
                        mma(S[2 * j2 + 1], lo[kk], b[2], b[3]);
                    }
            }
            if (!R::SPLIT)
                finish_rows(O, W, st, c, ounit[0], ounit[1]);
            c += st.more ? 0 : 1;
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.empty[w]);
        }
        if (!apart)
            break;
        const int w = c % R::HELP, turn = use & 1;
        Stage<DK, NCW> &st = sh.st[w];
        {
            // what is written to each column, in its unit
            float v[4][4], m[2] = {0.f, 0.f};
            int e[2];
            bool far = st.alone;
            load_values(v, st);
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const float2 be = *reinterpret_cast<const float2 *>(&st.b[nt * 8 + 2 * t]);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    m[hf] = fmaxf(m[hf], fmaxf(fabsf(be.x * v[nt][2 * hf]), fabsf(be.y * v[nt][2 * hf + 1])));
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                m[hf] = quad_max(m[hf]) * inv_unit[hf];
                // its state at the least; what fp32 may hold for good below 2^-118 is none
                float state = !first ? (empty >> hf & 1 ? 0.f : 0.5f) : top0[hf];
                state = first && state * unit[hf] < 0x1p-118f ? 0.f : state;
                e[hf] = first ? steps(hf, state) : 0;
                // far above the state, or all there is: the unit is theirs
                if (m[hf] * pow2(-e[hf]) > kMost || !(state > 0.f))
                    e[hf] = steps(hf, m[hf]);
                m[hf] *= pow2(-e[hf]);
                state *= pow2(-e[hf]);
                far |= !(m[hf] <= kMost);
                // the rows of this lane's quarter of the part
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        const int i = nt * 8 + 2 * t + o;
                        const float found = st.found[i];
                        const float x = fmaxf(st.a[i] * state * (st.b[i] == 0.f ? 8.f : 1.f), m[hf] * found);
                        far |= i >= st.lo && i < st.hi && found >= 0.f && x < kLeast && (x > 0.f || state > 0.f);
                    }
            }
            if (!__any_sync(0xffffffffu, far)) {
                scale_rows(refit(0, e[0]), refit(1, e[1]));
                if (first)
                    bare = empty = 0;
                first = false;
                looked = true;
                continue;
            }
        }
        phase ^= 1u << w;
        if (R::SPLIT) {
            // nothing for the output warp this time: a unit of 0 says so
            ok = use == 0 || __all_sync(0xffffffffu, tc5_wait(&sh.taken[cw & 1], turn ^ 1, abort));
            if (!ok)
                break;
            if (half == 0)
                to.unit[lane] = make_float2(0.f, 0.f);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.s_full[cw & 1]);
                if (half == 0)
                    mbar_arrive(&sh.w_full[cw & 1]);
            }
        }
        ok = row_by_row(st, c);
        if (!ok)
            break;
        first = true;
        c += st.more ? 0 : 1;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.empty[w]);
        ++use;
    }
    if (!ok) {
        if (lane == 0)
            seq_flag(a.sq, GATTN_STATUS_TIMEOUT);
        return;
    }
    if (a.state_out && (len > 0 || a.state_out != a.state))
#pragma unroll
        for (int j = 0; j < ROWS / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                a.state_out[so + (long long)(8 * j + 2 * t + (e & 1)) * a.dv + (e >> 1) * 8] =
                    S[j][e] * unit[e >> 1];
}

template <int DK, int NCW>
cudaError_t launch(const DeltaArgs &a, cudaStream_t s)
{
    auto *fn = delta_chunk_kernel<DK, NCW>;
    constexpr int smem = sizeof(Shared<DK, NCW>);
    static_assert(smem <= 227 * 1024, "shared memory");
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(fn, smem, done);
    if (e != cudaSuccess)
        return e;
    const long long grid = (long long)a.sq.n * a.Hv * (a.dv / (16 * NCW));
    if (grid > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Roles<NCW>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

template <int DK>
cudaError_t launch_dk(const DeltaArgs &a, cudaStream_t s)
{
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    // columns per CTA: as many as keep every SM busy, since a CTA's helpers do the
    // same work for any number of them.  Sequences of 1024 rows with 32 heads of 128 x
    // 128, by 32, 64 and 128 columns: one 70, 86 and 125 us; two 140, 86 and 125; four
    // 277, 175 and 128; sixteen 982, 608 and 507
    const long long cols = (long long)a.sq.n * a.Hv * a.dv;
    if (a.dv % 128 == 0 && cols / 64 > sms)
        return launch<DK, 8>(a, s);
    if (a.dv % 64 == 0 && cols / 32 > sms)
        return launch<DK, 4>(a, s);
    return launch<DK, 2>(a, s);
}

}  // namespace

cudaError_t launch_delta_prompt(const DeltaArgs &a, cudaStream_t s)
{
    return a.dk == 64 ? launch_dk<64>(a, s) : launch_dk<128>(a, s);
}

}  // namespace gattn
