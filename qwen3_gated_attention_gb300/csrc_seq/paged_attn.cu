// paged_attn.cu -- causal attention of one to a few new rows of each sequence over a
// key-value cache in pages, with grouped heads and the sigmoid output gate.
//
//   out = sum_j p_j v_j / sum_j p_j * sigmoid(gate),  p_j = 2^(c q . k_j - m)
//
// over the positions j that a row sees.  Bound by memory: every key and value is read
// once for all rows and heads that share it.  See paged_ring.cuh for how the work is cut;
// a segment that falls into several CTAs leaves (m, sum, O) of each part in the workspace,
// and a second kernel joins them.
//
// Within a CTA the units of a part go round NS groups of warps, each with its own
// running maximum and sum; a warp of a group has eight of the tile's rows.  Warps wait for
// units only, never for each other: at a part's end each leaves (m, sum, O) in shared
// memory for other warps that join, divide, gate and write them, and goes on with the next.
// Tiles are of 8, 16 or 64 rows.  The eight warps of a wide one form as many groups as a
// part's rows leave (four for a token of twelve heads beside drafts of other sequences: 42
// us instead of 50), and join among themselves.
//
// The matrix instructions run with the cache as their first operand (16 positions, or
// 16 elements of the values) and the rows as their second, eight wide: one token's
// heads of a group are mostly eight or fewer, and the other way round they would fill a
// quarter of 16 rows and hold twice the registers (128 for O with heads of 256: every
// load then waited for a free one, and four drafted rows of twelve heads took 102 us).  The
// scores stay in registers; turned over, eight by eight, they are what the product with
// the values takes.  p goes into that product as two bf16 numbers, 16 bits of it: 8 bits
// alone would be an error of the size of the output's own rounding, and the matrix units
// have the time.  The reference m of a row moves only when the maximum outgrows it by 2^8.
//
// Measured, kernel and join together: 32 sequences of up to 15000 positions, 32 heads of
// 256 over 8: 176 us, 6.6 TB/s, 98 % of the copy rate.  One sequence of 131072, 24 heads
// over 2: 51 us, of which the join takes 6 and the start 3.  64 sequences of 211 to 4200,
// 16 heads of 64 over 8, in pages of 16: 52 us, 5.0 TB/s (2 KB a copy; CTAs whose copies
// are slow end 10 us after the others).  Eight sequences of four drafted rows, 24 heads over
// 2: 47 us for 20 us of bytes: 48 rows are six warps of eight, two of them on one scheduler;
// for 32 positions its matrix instructions take 1536 cycles, and so do the reads of keys and
// values that every warp makes from shared memory (rows loaded anew for each unit instead
// of kept in registers change nothing).  One token
// over 1004 positions: 9.6 us, two launches and five dependent loads.  Chunks of 30 to 500 rows
// of 16 heads over 4, behind 256 to 30000 positions: 618 us for 61 us of products.
#include <cudaTypedefs.h>

#include "paged_ring.cuh"

namespace gattn {

using namespace paged;

namespace {

// RT: tiles of eight rows.
template <int D, int RT>
struct Cfg {
    // warps: consumers, joining ones (WIDE: none, the consumers join), producers; twelve
    // have 168 registers each
    static constexpr bool WIDE = RT == 8;
    static constexpr int M = 8 * RT, CW = RT == 1 ? 4 : 8, NS = CW / RT, NE = WIDE ? 0 : RT == 1 ? 4 : 2;
    static constexpr int NP = RT == 2 ? 2 : 4;
    static constexpr int THREADS = (CW + NE + NP) * 32;
    // columns that are handed over at once: what leaves the ring enough slots
    static constexpr int DR = WIDE ? 64 : D, ROUNDS = D / DR;
    static constexpr int XROW = DR + 4;                // floats of a row: two rows 8 banks apart
    static constexpr int XB = CW * 8 * XROW * 4;
    static constexpr int ER = NE ? M / NE : 8;         // rows of a warp that finishes them
    static constexpr int ITEMS = ER * (DR / 4) / 32;   // of its lanes, four columns each
    static constexpr int U = kUnit<D> * (WIDE ? 2 : 1), UNIT = U * D * 4;
    static constexpr int FIXED = 2 * M * D * 2 + XB + 4096 + 1024;
    static constexpr int FIT = (227 * 1024 - FIXED) / UNIT, STEP = NS > NP ? NS : NP;
    static constexpr int SLOTS = (FIT > 12 ? 12 : FIT) / STEP * STEP;
    static constexpr int SMEM = SLOTS * UNIT + 2 * M * D * 2 + XB + 1024;
    using R = Ring<D, U, M, true, SLOTS, NP, NS, RT, CW + NE>;
    static_assert(SMEM + 4096 <= 227 * 1024 && SLOTS >= 4 / (U / kUnit<D>) && DR * ROUNDS == D && XROW % 16 == 4 &&
                      ITEMS * 32 == ER * (DR / 4), "");
};

// Floats of a partial result: rows, then their m and sums.
template <int D, int M>
constexpr int kPartial = M * (D + 2);

// What the join needs to know of a CTA's last segment.
struct Rec {
    int live, slot, last, r0, rowf, hf, nrows, hk;
};

// Four columns of a row's gate before its sigmoid, as they are in memory.
__device__ __forceinline__ uint4 gate4(const PagedAttnArgs &a, long long at)
{
    if (a.gate_f32)
        return *reinterpret_cast<const uint4 *>(static_cast<const float *>(a.gate) + at);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.gate) + at);
    return make_uint4(w.x, w.y, 0, 0);
}

// Four finished columns of a row: divided, gated, rounded once.
__device__ __forceinline__ void finish4(const PagedAttnArgs &a, long long to, float4 o, float l, const uint4 &raw)
{
    const float inv = l == 0.f ? 0.f : 1.f / l;        // no position seen: zeros
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    // a row that saw nothing stays zero whatever its gate holds
    if (a.gate && l != 0.f) {
        const float4 g = a.gate_f32 ? make_float4(__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z),
                                                  __uint_as_float(raw.w))
                                    : make_float4(bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y));
        o.x /= 1.f + __expf(-g.x), o.y /= 1.f + __expf(-g.y);
        o.z /= 1.f + __expf(-g.z), o.w /= 1.f + __expf(-g.w);
    }
    *reinterpret_cast<uint2 *>(a.out + to) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

// The rows of skipped sequences, by every thread of the grid.
__device__ __noinline__ void zero_skipped(const PagedAttnArgs &a)
{
    if (blockIdx.x == 0 && threadIdx.x == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    const int ch = a.d / 8, row16 = a.H * ch;           // 16-byte pieces of a head and a row
    each_skipped(a, [&](int r0, int len) {
        const long long step = (long long)gridDim.x * blockDim.x;
        for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < (long long)len * row16; i += step) {
            const long long row = r0 + i / row16;
            const int x = (int)(i % row16), h = x / ch, c = x % ch;
            *reinterpret_cast<uint4 *>(a.out + row * a.os.tok + h * a.os.head + c * 8) = make_uint4(0, 0, 0, 0);
            if (c == 0 && a.lse)
                a.lse[row * a.H + h] = -INFINITY;
        }
    });
}

template <int D, int RT>
__global__ void __launch_bounds__(Cfg<D, RT>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, int min_units)
{
    using C = Cfg<D, RT>;
    using R = typename C::R;
    constexpr int M = C::M, NS = C::NS, CW = C::CW, NE = C::NE, U = C::U, DR = C::DR;
    constexpr bool WIDE = C::WIDE;
    extern __shared__ uint8_t raw[];
    __shared__ R ring;
    __shared__ float red_m[CW * 8], red_l[CW * 8];   // of the consumers' rows
    __shared__ float fac[CW * 8], row_l[M];            // what the joining warps make of them
    __shared__ long long row_out[M], row_gate[M], row_lse[M];   // where their rows are
    __shared__ uint64_t xfull, xempty;                 // the hand-over buffer
    uint8_t *units = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = units + C::SLOTS * C::UNIT;
    float *const xb = reinterpret_cast<float *>(qbuf + 2 * M * D * 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.H / a.Hk;
    if (threadIdx.x == 0) {
        mbar_init(&xfull, CW);
        mbar_init(&xempty, WIDE ? CW : NE);
        ring.init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    // (no early start for the join: its blocks would sit on the SMs that are done first, 1 us
    // more for a verify step)
    pdl_wait();
    // (the barriers of the plan make the ring's known)
    const Run run = plan_run<C::THREADS, M, U>(a, group, min_units);
    if (run.bad)
        zero_skipped(a);
    Rec *const recs = reinterpret_cast<Rec *>(static_cast<float *>(a.ws) + 2ll * kMaxCtas * kPartial<D, M>);
    if (run.x0 >= run.x1) {
        if (threadIdx.x == 0)
            recs[blockIdx.x].live = 0;
        return;
    }
    if (warp >= CW + NE) {
        Rec rec{};
        produce(a, ring, units, qbuf, &kmap, &vmap, run, group, warp - CW - NE, [&](const Part &p, int last) {
            rec = {1, p.slot, last, p.r0, p.rowf, p.hf, p.nrows, p.hk};
        });
        if (warp == CW + NE && lane == 0)
            recs[blockIdx.x] = rec;
        return;
    }
    // The finished rows of a part: `er` of them (C::ER, or fewer in a wide tile) by one warp
    // from row e0 on, DR columns at a time: places() first, then gates() before, sums() and
    // columns() after they are in xb, where `ns` groups have left `rows` rows each.  What a
    // warp keeps of its rows is its own: in a wide tile the next part's rows are others.
    constexpr int ITEMS = C::ITEMS;
    const int mine = WIDE ? warp * 8 : (warp - CW) * C::ER;            // its first place
    auto places = [&](const Part &p, int e0, int er) {
        const int h = p.hf + e0 + lane, head = p.hk * group + h % group;        // a lane a row
        const long long to = p.r0 + p.rowf + h / group;
        if (lane < er) {
            row_out[mine + lane] = to * a.os.tok + head * a.os.head;
            row_gate[mine + lane] = to * a.gs.tok + head * a.gs.head;
            row_lse[mine + lane] = to * a.H + head;
        }
        __syncwarp();
    };
    auto gates = [&](const Part &p, int e0, int er, int r, uint4 (&gate)[ITEMS]) {
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const int i = q * 32 + lane, row = e0 + i / (DR / 4);
            gate[q] = make_uint4(0, 0, 0, 0);
            if (p.whole && a.gate && row < p.nrows && i < er * (DR / 4))
                gate[q] = gate4(a, row_gate[mine + row - e0] + r * DR + i % (DR / 4) * 4);
        }
    };
    auto sums = [&](const Part &p, int e0, int er, int ns, int rows) {
        if (lane < er) {
            float *const slot = static_cast<float *>(a.ws) + (2ll * blockIdx.x + p.slot) * kPartial<D, M>;
            const int row = e0 + lane;
            float top = -INFINITY, sum = 0.f;
            for (int q = 0; q < ns; ++q)
                top = fmaxf(top, red_m[q * rows + row]);
            for (int q = 0; q < ns; ++q) {
                const float f = red_m[q * rows + row] == top ? 1.f : exp2f(red_m[q * rows + row] - top);
                sum = fmaf(f, red_l[q * rows + row], sum);
                fac[mine + q * (WIDE ? er : M) + lane] = f;
            }
            row_l[mine + lane] = sum;
            if (!p.whole) {
                slot[M * D + row] = top;
                slot[M * D + M + row] = sum;
            } else if (a.lse && row < p.nrows) {
                a.lse[row_lse[mine + lane]] = lse_of(top, sum);
            }
        }
        __syncwarp();
    };
    auto columns = [&](const Part &p, int e0, int er, int ns, int rows, int r, const uint4 (&gate)[ITEMS]) {
        float *const slot = static_cast<float *>(a.ws) + (2ll * blockIdx.x + p.slot) * kPartial<D, M>;
        // all sums before the first store, which the loads might not pass
        float4 sum[ITEMS];
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const int i = q * 32 + lane, row = e0 + i / (DR / 4), c = i % (DR / 4) * 4;
            sum[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < er * (DR / 4))
#pragma unroll
                for (int n = 0; n < (WIDE ? CW : NS); ++n) {
                    if (WIDE && n >= ns)
                        break;
                    const float4 v = *reinterpret_cast<const float4 *>(xb + (n * rows + row) * C::XROW + c);
                    const float f = fac[mine + n * (WIDE ? er : M) + row - e0];
                    sum[q].x = fmaf(f, v.x, sum[q].x), sum[q].y = fmaf(f, v.y, sum[q].y);
                    sum[q].z = fmaf(f, v.z, sum[q].z), sum[q].w = fmaf(f, v.w, sum[q].w);
                }
        }
#pragma unroll
        for (int q = 0; q < ITEMS; ++q) {
            const int i = q * 32 + lane, row = e0 + i / (DR / 4), c = i % (DR / 4) * 4;
            if (row < p.nrows && i < er * (DR / 4)) {
                if (p.whole)
                    finish4(a, row_out[mine + row - e0] + r * DR + c, sum[q], row_l[mine + row - e0], gate[q]);
                else
                    *reinterpret_cast<float4 *>(slot + row * D + r * DR + c) = sum[q];
            }
        }
        __syncwarp();
    };
    if (NE && warp >= CW) {
        // ------------------------------------------------------- the joining warps
        const int e0 = (warp - CW) * C::ER;
        uint32_t xr = 0;                                // hand-overs so far
        for (int parts = 0;; ++parts) {
            const int b = parts & 1;
            if (!ring_wait(&ring.qfull[b], (uint32_t)((parts >> 1) & 1), &ring.abort, a.sq))
                return;
            const Part p = ring.part[b];
            if (!p.live)
                break;
            places(p, e0, C::ER);
#pragma unroll 1
            for (int r = 0; r < C::ROUNDS; ++r, ++xr) {
                uint4 gate[ITEMS];                      // come while the consumers work
                gates(p, e0, C::ER, r, gate);
                if (!ring_wait(&xfull, xr & 1, &ring.abort, a.sq))
                    return;
                if (r == 0)
                    sums(p, e0, C::ER, NS, M);
                columns(p, e0, C::ER, NS, M, r, gate);
                if (lane == 0)
                    mbar_arrive(&xempty);
            }
            if (lane == 0)
                mbar_arrive(&ring.qempty[b]);
        }
        return;
    }
    // --------------------------------------------------------------- consumers
    // warps of a group: in a wide tile as many as the part's rows need, two for a token of
    // 12 heads
    auto tiles_of = [](const Part &p) { return !WIDE ? RT : p.nrows <= 8 ? 1 : p.nrows <= 16 ? 2 : p.nrows <= 32 ? 4 : 8; };
    const int g = lane >> 2, cq = lane & 3;
    const int btl = box_log2(a.pg.page, U), box = (1 << btl) * D * 2, dbs = (1 << btl) * 128;
    // a lane's position (of 16) and 16-byte piece in a load of keys and of values
    const int ka = (lane & 15) * 128, kc = lane >> 4;
    const int va = ((lane & 7) + 8 * (lane >> 4)) * 128, vc = (lane >> 3) & 1;
    int it = 0;                                         // units of the CTA before this part, modulo NS
    int slot = warp / RT, phase = 0;                    // of this group's next unit
    uint32_t xr = 0;                                    // hand-overs so far
    for (int parts = 0;; ++parts) {
        const int b = parts & 1;
        if (!ring_wait(&ring.qfull[b], (uint32_t)((parts >> 1) & 1), &ring.abort, a.sq))
            return;
        const Part p = ring.part[b];
        if (!p.live)
            break;
        const int row0 = warp % tiles_of(p) * 8;        // this warp's rows
        // units that it takes, by their index modulo 8 (a wide tile's groups change: every
        // warp sees every unit) or all that it sees
        unsigned take = row0 < p.nrows ? 0xffu : 0u;
        if (WIDE)
            for (int i = 0; i < 8; ++i)
                if ((i & (CW / tiles_of(p) - 1)) != warp / tiles_of(p))
                    take &= ~(1u << i);
        const int first_row = p.p0 + p.rowf;            // the last position that every row sees
        const int last_row = p.p0 + p.rowf + (p.hf + p.nrows - 1) / group;
        int lim[2];                                     // of this lane's rows, 2 cq and the next
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = row0 + 2 * cq + e;
            lim[e] = i < p.nrows ? first_row + (p.hf + i) / group : -1;
        }
        uint32_t qf[D / 16][2];                         // the rows, as the products take them
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            uint32_t r[4];
            ldsm_x4(r, smem_u32(qbuf) + b * R::QB + (row0 + (lane & 7)) * (D * 2) +
                           (((4 * k + (lane >> 3)) ^ (lane & 7)) << 4));
            qf[2 * k][0] = r[0], qf[2 * k][1] = r[1];
            qf[2 * k + 1][0] = r[2], qf[2 * k + 1][1] = r[3];
        }
        // O[j]: elements 16 j + g and 8 on, of rows 2 cq and the next
        float O[D / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                O[j][e] = 0.f;
        // the gates of rows that this warp finishes: into L2 meanwhile
        if (WIDE && p.whole && a.gate)
            for (int i = lane; i < tiles_of(p) * (D / 64); i += 32) {
                const int row = warp * tiles_of(p) + i / (D / 64), h = p.hf + row;
                if (row < p.nrows)
                    prefetch_l2(static_cast<const char *>(a.gate) +
                                ((p.r0 + p.rowf + h / group) * a.gs.tok + (p.hk * group + h % group) * a.gs.head + i % (D / 64) * 64) *
                                    (a.gate_f32 ? 4 : 2));
            }
        const int count = max(p.u1 - p.u0, 0);
        // units of index warp / RT modulo NS within the CTA (NS is 1 in a wide tile)
        for (int n = (warp / RT - it) & (NS - 1); n < count; n += NS) {
            if (!ring_wait(&ring.full[slot], phase, &ring.abort, a.sq))
                return;
            const uint32_t ks = smem_u32(units) + slot * C::UNIT, vs = ks + R::PLANE;
            const int t0 = (p.u0 + n) * U;
            if (take >> (WIDE ? n & 7 : 0) & 1u) {
                const unsigned there = ring.ok[slot];
                // ---- scores: positions g and 8 on of each 16, rows 2 cq and the next
                constexpr int CHAINS = U < 64 ? 64 / U : 1;  // sums of independent products
                float sc[CHAINS][U / 16][4];
#pragma unroll
                for (int c = 0; c < CHAINS; ++c)
#pragma unroll
                    for (int q = 0; q < U / 16; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[c][q][e] = 0.f;
                // step i: 16 elements k of 16 positions q; four loads ahead of their products
                constexpr int STEPS = D / 16 * (U / 16), AHEAD = 4;
                uint32_t ak[2][AHEAD][4];
                auto keys = [&](int i, uint32_t (&r)[4]) {
                    const int k = i / (U / 16), q = i % (U / 16);
                    ldsm_x4(r, ks + ((q * 16) >> btl) * box + (k >> 2) * dbs + ((q * 16) & ((1 << btl) - 1)) * 128 + ka +
                                   ((((2 * k + kc) & 7) ^ (lane & 7)) << 4));
                };
#pragma unroll
                for (int x = 0; x < AHEAD; ++x)
                    keys(x, ak[0][x]);
#pragma unroll
                for (int i = 0; i < STEPS; i += AHEAD) {
                    if (i + AHEAD < STEPS)
#pragma unroll
                        for (int x = 0; x < AHEAD; ++x)
                            keys(i + AHEAD + x, ak[(i / AHEAD + 1) & 1][x]);
#pragma unroll
                    for (int x = 0; x < AHEAD; ++x) {
                        const int k = (i + x) / (U / 16), q = (i + x) % (U / 16);
                        mma(sc[k % CHAINS][q], ak[(i / AHEAD) & 1][x], qf[k][0], qf[k][1]);
                    }
                }
#pragma unroll
                for (int q = 0; q < U / 16; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (CHAINS == 4)
                            sc[0][q][e] = (sc[0][q][e] + sc[1 % CHAINS][q][e]) + (sc[2 % CHAINS][q][e] + sc[3 % CHAINS][q][e]);
                        else if constexpr (CHAINS == 2)
                            sc[0][q][e] += sc[1 % CHAINS][q][e];
                        sc[0][q][e] *= a.scale_log2;
                    }
                // ---- what a row does not see
                const bool part = t0 + U - 1 > first_row;
                if (part || there != (1u << (U >> btl)) - 1u) {
#pragma unroll
                    for (int q = 0; q < U / 16; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = q * 16 + g + 8 * (e >> 1);
                            if (t0 + t > lim[e & 1] || !((there >> (t >> btl)) & 1u))
                                sc[0][q][e] = -INFINITY;
                        }
                }
                // ---- the reference: lanes that share a row look for scores 2^8 above it, and
                //      agree on a new one only then
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int q = 0; q < U / 16; ++q)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        mx[e] = fmaxf(mx[e], fmaxf(sc[0][q][e], sc[0][q][2 + e]));
                if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o *= 2)
                            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
                        const float to = fmaxf(m[e], mx[e]), f = to == m[e] ? 1.f : exp2f(m[e] - to);
                        m[e] = to;
                        l[e] *= f;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            O[j][e] *= f;
                            O[j][2 + e] *= f;
                        }
                    }
                }
                // p, in place of the scores; hi + lo are its first 16 bits
                uint32_t hi[U / 16][2], lo[U / 16][2];
                const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
                for (int q = 0; q < U / 16; ++q)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = exp2_approx(sc[0][q][2 * x] - base[0]), p1 = exp2_approx(sc[0][q][2 * x + 1] - base[1]);
                        l[0] += p0;
                        l[1] += p1;
                        sc[0][q][2 * x] = p0;
                        sc[0][q][2 * x + 1] = p1;
                        const uint32_t h = pack_bf16x2(p0, p1);
                        hi[q][x] = turned(h);
                        lo[q][x] = turned(pack_bf16x2(p0 - bf16_lo(h), p1 - bf16_hi(h)));
                    }
                // ---- values that no row of the tile sees are stale: zeros (every warp of the
                //      group writes them); of those that some rows see, look for what is not
                //      finite: it must not meet the others' zeros
                bool odd = false;
                if (part) {
                    const int dead = max(last_row + 1 - t0, 0), some = max(first_row + 1 - t0, 0);
                    for (int i = lane; i < (U - dead) * (D / 8); i += 32) {
                        const int t = dead + i / (D / 8), c = i % (D / 8);
                        sts_v4(vs + (t >> btl) * box + (c >> 3) * dbs + (t & ((1 << btl) - 1)) * 128 + (c & 7) * 16, 0, 0, 0, 0);
                    }
                    for (int i = lane; i < (min(dead, U) - some) * (D / 8); i += 32) {
                        const int t = some + i / (D / 8), c = i % (D / 8);
                        const uint4 v = lds_v4(vs + (t >> btl) * box + (c >> 3) * dbs + (t & ((1 << btl) - 1)) * 128 + (c & 7) * 16);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            odd |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
                    }
                    __syncwarp();
                    odd = __any_sync(0xffffffffu, odd);
                }
                // ---- O += V p, four loads ahead of their products
                if (!odd) {
                    // step i: 16 positions q, 16 elements j
                    auto values = [&](int i, uint32_t (&r)[4]) {
                        const int q = i / (D / 16), j = i % (D / 16);
                        ldsm_x4_trans(r, vs + ((q * 16) >> btl) * box + (j >> 2) * dbs + ((q * 16) & ((1 << btl) - 1)) * 128 + va +
                                             ((((2 * j + vc) & 7) ^ (lane & 7)) << 4));
                    };
#pragma unroll
                    for (int x = 0; x < AHEAD; ++x)
                        values(x, ak[0][x]);
#pragma unroll
                    for (int i = 0; i < STEPS; i += AHEAD) {
                        if (i + AHEAD < STEPS)
#pragma unroll
                            for (int x = 0; x < AHEAD; ++x)
                                values(i + AHEAD + x, ak[(i / AHEAD + 1) & 1][x]);
#pragma unroll
                        for (int x = 0; x < AHEAD; ++x) {
                            const int q = (i + x) / (D / 16);
                            mma(O[(i + x) % (D / 16)], ak[(i / AHEAD) & 1][x], hi[q][0], hi[q][1]);
                        }
#pragma unroll
                        for (int x = 0; x < AHEAD; ++x) {
                            const int q = (i + x) / (D / 16);
                            mma(O[(i + x) % (D / 16)], ak[(i / AHEAD) & 1][x], lo[q][0], lo[q][1]);
                        }
                    }
                } else {
                    // position by position, each row only what it sees
#pragma unroll 1
                    for (int t = 0; t < U; ++t) {
                        float pt[2] = {0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < U / 16; ++q)
                            if (q == t >> 4)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    pt[e] = t & 8 ? sc[0][q][2 + e] : sc[0][q][e];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            pt[e] = __shfl_sync(0xffffffffu, pt[e], (t & 7) * 4 + cq);
                            if (t0 + t > lim[e] || !((there >> (t >> btl)) & 1u))
                                pt[e] = -1.f;            // not seen
                        }
                        const uint32_t vrow = vs + (t >> btl) * box + (t & ((1 << btl) - 1)) * 128;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t at = vrow + (j >> 2) * dbs + ((((2 * j + x) & 7) ^ (t & 7)) << 4) + g * 2;
                                const float v = __uint_as_float(lds_u16(at) << 16);
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!(pt[e] < 0.f))
                                        O[j][2 * x + e] = fmaf(pt[e], v, O[j][2 * x + e]);
                            }
                    }
                }
                if (part)
                    fence_proxy_async_smem();           // zeros before the next copy into this slot
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ring.empty[slot]);
            slot += NS;
            if (slot >= R::SLOTS) {
                slot -= R::SLOTS;
                phase ^= 1;
            }
        }
        it = (it + count) & (NS - 1);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&ring.qempty[b]);
        // ---- hand over
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
        }
        float *const own = xb + (warp * 8 + 2 * cq) * C::XROW + g;
        const int tiles = tiles_of(p), groups = WIDE ? CW / tiles : NS;
        if (WIDE)
            places(p, warp * tiles, tiles);
#pragma unroll
        for (int r = 0; r < C::ROUNDS; ++r) {
            uint4 gate[ITEMS];
            if (WIDE)
                gates(p, warp * tiles, tiles, r, gate);
            // (one group: every warp finishes its own rows, but others may still read what it
            // left them of the part before)
            if ((!WIDE || groups > 1 || r == 0) && !ring_wait(&xempty, (xr & 1) ^ 1u, &ring.abort, a.sq))
                return;
            if (r == 0 && g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    red_m[warp * 8 + 2 * cq + e] = m[e];
                    red_l[warp * 8 + 2 * cq + e] = l[e];
                }
            }
#pragma unroll
            for (int j = 0; j < DR / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    own[(e & 1) * C::XROW + j * 16 + 8 * (e >> 1)] = O[r * (DR / 16) + j][e];
            __syncwarp();
            if (!WIDE || groups > 1) {
                if (lane == 0)
                    mbar_arrive(&xfull);
                if (WIDE && !ring_wait(&xfull, xr & 1, &ring.abort, a.sq))
                    return;
                ++xr;
            }
            if (WIDE) {
                if (r == 0)
                    sums(p, warp * tiles, tiles, groups, tiles * 8);
                columns(p, warp * tiles, tiles, groups, tiles * 8, r, gate);
                if (groups > 1 && lane == 0)
                    mbar_arrive(&xempty);
            }
        }
    }
}

// Joins the parts of the segment that begins in CTA blockIdx.x's run and goes on behind
// it: ROWS rows a block, the parts dealt to the warps of a row, kFly of them on their
// way at a time.  Bound by three dependent loads (the record, the parts, and what the
// launch itself takes).
constexpr int kJoin = 256;

template <int M>
constexpr int kJoinRows = M > 16 ? M / 16 : 1;
template <int M>
constexpr int kFlying = M > 32 ? 10 : 5;               // two warps a row, or four and eight

template <int D, int M>
__global__ void __launch_bounds__(kJoin) paged_join_kernel(const __grid_constant__ PagedAttnArgs a)
{
    constexpr int ROWS = kJoinRows<M>, kFly = kFlying<M>, W = kJoin / 32 / ROWS, N4 = (D + 127) / 128;
    static_assert(W * 32 >= D / 4, "a thread finishes four columns");
    __shared__ float red_m[kJoin / 32], red_l[kJoin / 32];
    __shared__ float4 sums[kJoin / 32][D / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rl = warp / W, w = warp % W;
    const float *const ws = static_cast<const float *>(a.ws);
    pdl_wait();
    pdl_launch_dependents();
    const Rec rec = reinterpret_cast<const Rec *>(ws + 2ll * kMaxCtas * kPartial<D, M>)[blockIdx.x];
    const int i = blockIdx.y * ROWS + rl;
    if (!rec.live || blockIdx.y * ROWS >= rec.nrows)
        return;
    const int first = blockIdx.x, parts = rec.last - first + 1;
    const int group = a.H / a.Hk, h = rec.hf + i, head = rec.hk * group + h % group;
    const long long row = rec.r0 + rec.rowf + h / group;
    const int col = (w * 32 + lane) * 4;               // of the thread at the end
    const bool mine = i < rec.nrows && col < D;
    const uint4 gate = mine && a.gate ? gate4(a, row * a.gs.tok + head * a.gs.head + col) : make_uint4(0, 0, 0, 0);
    float top = -INFINITY, sum = 0.f;
    float4 o[N4];
#pragma unroll
    for (int c = 0; c < N4; ++c)
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = w; k0 < parts; k0 += W * kFly) {
        float m[kFly], l[kFly];
        float4 v[kFly][N4];
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int k = k0 + f * W;
            m[f] = -INFINITY;
            l[f] = 0.f;
            const float *const from = ws + (2ll * (first + k) + (k ? 0 : rec.slot)) * kPartial<D, M>;
            if (k < parts) {
                m[f] = from[M * D + i];
                l[f] = from[M * D + M + i];
            }
#pragma unroll
            for (int c = 0; c < N4; ++c) {
                v[f][c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < parts && c * 128 + lane * 4 < D)
                    v[f][c] = *reinterpret_cast<const float4 *>(from + i * D + c * 128 + lane * 4);
            }
        }
        float to = top;
#pragma unroll
        for (int f = 0; f < kFly; ++f)
            to = fmaxf(to, m[f]);
        const float keep = to == top ? 1.f : exp2f(top - to);
        top = to;
        sum *= keep;
#pragma unroll
        for (int c = 0; c < N4; ++c)
            o[c].x *= keep, o[c].y *= keep, o[c].z *= keep, o[c].w *= keep;
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const float x = m[f] == to ? 1.f : exp2f(m[f] - to);
            sum = fmaf(x, l[f], sum);
#pragma unroll
            for (int c = 0; c < N4; ++c) {
                o[c].x = fmaf(x, v[f][c].x, o[c].x), o[c].y = fmaf(x, v[f][c].y, o[c].y);
                o[c].z = fmaf(x, v[f][c].z, o[c].z), o[c].w = fmaf(x, v[f][c].w, o[c].w);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < N4; ++c)
        if (c * 128 + lane * 4 < D)
            sums[warp][c * 32 + lane] = o[c];
    if (lane == 0) {
        red_m[warp] = top;
        red_l[warp] = sum;
    }
    __syncthreads();
    if (!mine)
        return;
    top = -INFINITY;
#pragma unroll
    for (int q = 0; q < W; ++q)
        top = fmaxf(top, red_m[rl * W + q]);
    sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < W; ++q) {
        const float mq = red_m[rl * W + q], x = mq == top ? 1.f : exp2f(mq - top);
        sum = fmaf(x, red_l[rl * W + q], sum);
        const float4 p = sums[rl * W + q][col / 4];
        v.x = fmaf(x, p.x, v.x), v.y = fmaf(x, p.y, v.y), v.z = fmaf(x, p.z, v.z), v.w = fmaf(x, p.w, v.w);
    }
    if (col == 0 && a.lse)
        a.lse[row * a.H + head] = lse_of(top, sum);
    finish4(a, row * a.os.tok + head * a.os.head + col, v, sum, gate);
}

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeFn encoder()
{
    static EncodeFn fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Tiles of eight rows, 1, 2 or 8 by the rows of an average sequence.  A larger tile than a
// sequence needs costs shared memory, a smaller one meets its keys again.  Eight sequences
// of 256 to 30000 positions, heads of 256, by 1, 2 and 8 tiles, in us:
//    8 rows (32 heads over 4)   47.3   48.2   60.9
//   12 rows (24 over 2)         46.4   32.4   39.2
//   16 rows (32 over 8)        159.0   88.6  109.9
//   24 rows (24 over 2)         63.6   49.5   41.1
//   32 rows (32 over 8)        304.8  164.3  123.9
//   48 rows (24 over 2)        116.6   66.4   55.8
// One tile and two are equal up to four rows (84 us).  Heads of 64 shift the second bound
// a little: 20 rows 18.6, 19.1 and 21.5 us, 48 rows 59.6, 44.5 and 39.9.
// The rule cannot see the lengths: of uneven drafts, 1 to 6 tokens of 12 heads, it takes
// 8 tiles (42.2 us) where 2 would do (35.0).
int row_tiles(int group, int n, int total)
{
    const long long rows = ((long long)total + n - 1) / n * group;
    return rows <= 8 ? 1 : rows <= 16 ? 2 : 8;
}

template <int D, int RT>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t s)
{
    using C = Cfg<D, RT>;
    auto *fn = paged_attn_kernel<D, RT>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(fn, C::SMEM, done);
    if (e != cudaSuccess)
        return e;
    int sms = 0;
    e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    CUtensorMap km, vm;
    const int box = 1 << box_log2(a.pg.page, C::U);
    if (!encode_pages(&km, a.pg, false, a.Hk, D, box) || !encode_pages(&vm, a.pg, true, a.Hk, D, box))
        return cudaErrorInvalidValue;
    const int grid = sms < kMaxCtas ? sms : kMaxCtas;
    e = launch_paged(fn, dim3(grid), dim3(C::THREADS), C::SMEM, s, a, km, vm, 4);
    if (e != cudaSuccess)
        return e;
    return launch_paged(paged_join_kernel<D, C::M>, dim3(grid, C::M / kJoinRows<C::M>), dim3(kJoin), 0, s, a);
}

template <int D>
cudaError_t launch_d(const PagedAttnArgs &a, cudaStream_t s)
{
    switch (row_tiles(a.H / a.Hk, a.sq.n, a.sq.total)) {
    case 1: return launch<D, 1>(a, s);
    case 2: return launch<D, 2>(a, s);
    default: return launch<D, 8>(a, s);
    }
}

}  // namespace

// The tensor map of a pool: {64 elements, positions, blocks of 64, heads, pages}.
bool encode_pages(CUtensorMap *m, const Pages &pg, bool v, int Hk, int d, int box)
{
    if (!encoder())
        return false;
    const PageStride &st = v ? pg.v : pg.k;
    const cuuint64_t dims[5] = {64, (cuuint64_t)pg.page, (cuuint64_t)(d / 64), (cuuint64_t)Hk, (cuuint64_t)pg.pages};
    const cuuint64_t strides[4] = {(cuuint64_t)st.tok * 2, 128, (cuuint64_t)st.head * 2, (cuuint64_t)st.page * 2};
    const cuuint32_t b[5] = {64, (cuuint32_t)box, (cuuint32_t)(d / 64), 1, 1}, es[5] = {1, 1, 1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, v ? pg.vp : pg.kp, dims, strides, b, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

long long paged_attn_workspace(int d, int group, int n, int total)
{
    const int M = n > 0 ? 8 * row_tiles(group, n, total) : 8;
    return 2ll * kMaxCtas * M * (d + 2) * 4 + kMaxCtas * (long long)sizeof(Rec);
}

cudaError_t launch_paged_attn(const PagedAttnArgs &a, cudaStream_t s)
{
    switch (a.d) {
    case 64: return launch_d<64>(a, s);
    case 128: return launch_d<128>(a, s);
    case 192: return launch_d<192>(a, s);
    default: return launch_d<256>(a, s);
    }
}

}  // namespace gattn
