// paged_ring.cuh -- how the kernels that read pages share out and fetch their work.
//
// The work of a call is a line of units: U consecutive positions of one sequence and KV
// head, met by a tile of up to M query rows (a segment: all units of one sequence, head
// and tile).  Every CTA takes an equal run of the line, wherever it begins or ends, so
// that the lengths of the sequences do not matter.  NP warps of a CTA (producers) walk the
// run: they look up pages and copy units by turns into a ring of shared memory by TMA, the
// first one the segments' query rows and descriptions into two buffers too; the other
// warps consume.  (One producer takes 700 cycles a unit and 90 more for every box beyond
// two: as much as 16 KB take to arrive at an SM, twice that with boxes of 16 positions.)
// A part costs a CTA some time whatever its length, so every segment counts kHead units
// more than it has when the line is shared out, and units that meet many rows count double.
//
// Every slot of the ring belongs to one producer and one group of consumers: SLOTS is
// divided by the number of either.  A wait is for a phase's parity, so that it must never
// be two phases ahead; copies land in any order, and only the slot's own users are known
// to have seen its last phase.
#pragma once

#include "paged.cuh"

namespace gattn {
namespace paged {

// Positions of a unit: 16 KB of keys and values (12 KB for heads of 192); kernels may
// take twice as many.
template <int D>
constexpr int kUnit = D >= 192 ? 16 : D == 128 ? 32 : 64;

constexpr int kMaxCtas = 160, kHead = 10;

// A segment's part within a CTA, as the consumers get it.
struct Part {
    int live;              // 0: no more parts
    int s, hk, r0, p0, len;
    int rowf, hf, nrows;   // query row i: row rowf + (hf + i) / group, head (hf + i) % group
    int u0, u1;            // units that some row sees
    int whole, slot;       // the segment's only part, or where the part goes
    int pass;              // of the weights' blocks of rows
};

struct SeqUnits {
    int r0, len, p0, units;
    int tiles;             // of rows
    int cost;              // of a unit: more than four eighths of a tile of 64 rows count double
    // what a segment takes of the line, and the sequence
    __device__ __forceinline__ int length() const { return (units + kHead) * cost; }
    __device__ __forceinline__ long long all(int Hk) const { return units ? (long long)tiles * Hk * length() : 0; }
    // units in front of a place in the segment
    __device__ __forceinline__ int units_at(int v) const { return max(v / cost - kHead, 0); }
};

// `bad`: rows whose positions do not fit the table
__device__ __forceinline__ SeqUnits seq_units(const PagedAttnArgs &a, int s, int group, int M, int U, bool &bad)
{
    SeqUnits u;
    seq_rows(a.sq, s, u.r0, u.len);
    u.p0 = a.pos[s];
    bad = u.len > 0 && (u.p0 < 0 || (long long)u.p0 + u.len > a.cap);
    const bool on = u.len > 0 && !bad;
    u.units = on ? (u.p0 + u.len + U - 1) / U : 0;
    // (rows times heads fit 31 bits)
    u.tiles = on ? M ? (int)(((unsigned)u.len * group + M - 1) / M) : 1 : 0;
    u.cost = M == 64 && (unsigned)u.len * group > 32 ? 2 : 1;
    return u;
}

// A CTA's run of the line and where it begins.
struct Run {
    long long x0, x1, quota;
    long long at;          // where sequence s begins
    int s;
    bool bad;              // some sequence does not fit its table
};

// Called by every thread of the block (NT of them).  M: rows of a tile; 0: all rows
// of a sequence are one tile.
template <int NT, int M, int U>
__device__ __forceinline__ Run plan_run(const PagedAttnArgs &a, int group, int min_units)
{
    __shared__ long long sums[32];
    __shared__ long long found_at;
    __shared__ int found;
    constexpr int NW = NT / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = a.sq.n;
    Run r;
    // its share of a line of this length
    auto share = [&](long long total) {
        r.quota = total <= 0x7fffffff ? (long long)(((unsigned)total + gridDim.x - 1) / gridDim.x)
                                      : (total + gridDim.x - 1) / gridDim.x;
        r.quota = r.quota > min_units ? r.quota : min_units;
        r.x0 = r.quota * blockIdx.x;
        r.x1 = r.x0 + r.quota < total ? r.x0 + r.quota : total;
        r.s = 0;
        r.at = 0;
    };
    if (n <= 32) {
        // every warp by itself, a lane a sequence
        long long u = 0;
        bool bad = false;
        if (lane < n) {
            u = seq_units(a, lane, group, M, U, bad).all(a.Hk);
        }
        r.bad = __any_sync(0xffffffffu, bad);
        long long incl = u;
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        share(__shfl_sync(0xffffffffu, incl, 31));
        __syncthreads();                // (what the caller set up)
        if (r.x0 < r.x1) {
            r.s = __ffs(__ballot_sync(0xffffffffu, r.x0 < incl)) - 1;
            r.at = __shfl_sync(0xffffffffu, incl - u, r.s);
        }
        return r;
    }
    long long mine = 0, first = 0;
    bool any = false;
    for (int s = tid; s < n; s += NT) {
        bool bad;
        mine += seq_units(a, s, group, M, U, bad).all(a.Hk);
        any |= bad;
        if (s == tid)
            first = mine;
    }
    for (int o = 16; o; o >>= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0)
        sums[warp] = mine;
    if (tid == 0)
        found = -1;
    r.bad = __syncthreads_or(any);
    long long total = 0;
    for (int w = 0; w < NW; ++w)
        total += sums[w];
    share(total);
    if (r.x0 >= r.x1)
        return r;                       // the whole block
    long long before = 0;
    for (int base = 0; base < n; base += NT) {
        const int s = base + tid;
        long long u = 0;
        if (base == 0)
            u = first;
        else if (s < n) {
            bool bad;
            u = seq_units(a, s, group, M, U, bad).all(a.Hk);
        }
        long long incl = u;
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += v;
        }
        __syncthreads();
        if (lane == 31)
            sums[warp] = incl;
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < NW; ++w) {
            if (w < warp)
                incl += sums[w];
            all += sums[w];
        }
        incl += before;
        if (u > 0 && r.x0 >= incl - u && r.x0 < incl) {
            found = s;
            found_at = incl - u;
        }
        before += all;
        if (r.x0 < before)
            break;                      // uniform
    }
    __syncthreads();
    r.s = found;
    r.at = found_at;
    return r;
}

// Calls f(first row, rows) for the sequences that do not fit their tables, whole warps.
template <class F>
__device__ __forceinline__ void each_skipped(const PagedAttnArgs &a, F f)
{
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < a.sq.n; base += 32) {
        SeqUnits u{};
        bool bad = false;
        if (base + lane < a.sq.n)
            u = seq_units(a, base + lane, 1, 1, 1, bad);
        for (unsigned m = __ballot_sync(0xffffffffu, bad); m; m &= m - 1) {
            const int l = __ffs(m) - 1;
            f(__shfl_sync(0xffffffffu, u.r0, l), __shfl_sync(0xffffffffu, u.len, l));
        }
    }
}

// ------------------------------------------------------------------ waiting

// Waits for a phase, for two seconds at most; then (or once another wait of the CTA has
// given up) false.
__device__ __forceinline__ bool ring_wait(uint64_t *bar, uint32_t parity, volatile int *abort, const SeqArgs &q)
{
    if (mbar_try(bar, parity))
        return true;
    const unsigned long long t0 = global_ns();
    while (true) {
        if (mbar_try(bar, parity))
            return true;
        if (*abort)
            return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            seq_flag(q, GATTN_STATUS_TIMEOUT);
            return false;
        }
    }
}

// 5-D tiled copy global -> shared: element, position in the page, block of 64
// elements, head, page.
__device__ __forceinline__ void box_g2s(uint32_t dst, const CUtensorMap *map, int y, int hk, int page, uint32_t bar,
                                        uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(0), "r"(hk), "r"(page), "r"(bar),
                 "l"(policy)
                 : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// 16 bytes to shared memory without waiting; zeros where !on
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// an arrival once the thread's copies so far have landed
__device__ __forceinline__ void cp_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The ring and the two row buffers of a CTA.
// NS groups of READERS warps take the units; ROWREADERS warps read the rows' buffers.
template <int D, int U_, int M_, bool V_, int SLOTS_, int NP_, int NS, int READERS, int ROWREADERS>
struct Ring {
    static constexpr int U = U_, DB = D / 64, M = M_, SLOTS = SLOTS_, NP = NP_;
    static_assert(SLOTS > 0 && SLOTS % NP == 0 && SLOTS % NS == 0, "");
    static constexpr bool V = V_;                      // values too
    static constexpr int PLANE = U * D * 2, UNIT = V ? 2 * PLANE : PLANE;
    static constexpr int QB = M * D * 2;               // query rows, 16-byte pieces swizzled by row
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t qfull[2], qempty[2];
    Part part[2];
    float lse[2][V ? 1 : M];
    unsigned ok[SLOTS];                                // boxes of a unit whose page exists
    volatile int abort;

    __device__ __forceinline__ void init()
    {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], READERS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 64);
            mbar_init(&qempty[i], ROWREADERS);
        }
        abort = 0;
        fence_mbar_init();
    }
};

// Positions of a box: what divides the page and the unit.
__host__ __device__ inline int box_log2(int page, int U)
{
    int l = 4;
    while (l < 6 && (2 << l) <= U && page % (2 << l) == 0)
        ++l;
    return l;
}

// The query rows and the description of a part, by one warp.
template <class R>
__device__ __forceinline__ void put_rows(const PagedAttnArgs &a, R &ring, uint8_t *qbuf, const Part &p, int b, int group)
{
    constexpr int D = R::DB * 64, M = R::M;
    const int lane = threadIdx.x & 31;
    const uint32_t qdst = smem_u32(qbuf) + b * R::QB;
    constexpr int CH = D / 8, RPI = 32 / CH > 0 ? 32 / CH : 1;          // rows of an iteration
    const int rows = (p.nrows + 7) & ~7;                // what the products take: zeros behind the last
#pragma unroll
    for (int i0 = 0; i0 < M; i0 += 32) {
        // a lane a row
        const int h = p.hf + min(i0 + lane, p.nrows - 1);
        const long long off = (long long)(p.r0 + p.rowf + h / group) * a.qs.tok + (p.hk * group + h % group) * a.qs.head;
        for (int i = i0; i < min(rows, i0 + 32); i += RPI) {
            const int row = i + (RPI > 1 ? lane / CH : 0);
            const __nv_bfloat16 *src = a.q + __shfl_sync(0xffffffffu, off, row & 31);
            const int c = RPI > 1 ? lane % CH : lane;
            if (c < CH)
                cp16(qdst + row * (D * 2) + ((c ^ (row & 7)) << 4), src + c * 8, row < p.nrows);
        }
    }
    if constexpr (!R::V)
        for (int i = lane; i < M; i += 32) {
            float v = -INFINITY;
            if (i < p.nrows)
                v = a.lse[(long long)(p.r0 + p.rowf + (p.hf + i) / group) * a.H + p.hk * group + (p.hf + i) % group];
            // 2^(score - v): a row that saw nothing gives nothing
            ring.lse[b][i] = v == -INFINITY ? INFINITY : v * 1.44269504f;
        }
    if (lane == 0)
        ring.part[b] = p;
    cp_arrive(&ring.qfull[b]);
    mbar_arrive(&ring.qfull[b]);
}

// Producer warp `pw` of R::NP.  `units`: the ring's memory (1024-byte aligned), `qbuf` that of the
// row buffers.  `seen` is told of the last segment, if it begins in this run and goes on
// behind it: (part, CTA of its last unit).
template <class R, class F>
__device__ __forceinline__ void produce(const PagedAttnArgs &a, R &ring, uint8_t *units, uint8_t *qbuf,
                                        const CUtensorMap *kmap, const CUtensorMap *vmap, const Run &run, int group,
                                        int pw, F seen)
{
    constexpr int U = R::U, D = R::U > 0 ? R::DB * 64 : 0, M = R::M;
    const int lane = threadIdx.x & 31;
    const int btl = box_log2(a.pg.page, U), BT = 1 << btl, NB = U >> btl;
    const uint32_t box_bytes = BT * D * 2;
    const uint64_t pol = l2_evict_first_policy();
    int it = 0;                        // units so far, modulo NP
    int slot = pw, phase = 0;          // of this warp's next unit
    int issued = 0;                    // units of its own
    int parts = 0;
    bool stop = false;
    int s = run.s;
    bool bad;
    SeqUnits u = seq_units(a, s, group, R::V ? M : 0, U, bad);
    // first segment, and place in it, its head counted
    const long long off = run.x0 - run.at;
    const unsigned length = u.length();
    int seg = off >> 32 ? (int)(off / length) : (int)((unsigned)off / length);
    int v0 = (int)(off - (long long)seg * length);
    // pages of 32 boxes of sequence tab_s, one a lane; not looked at before they are used,
    // so that the load is on its way meanwhile
    int tab_s = -1, tab_b = 0, tab_page = 0, tab_y = 0;
    auto window = [&](int b0) {
        if (tab_s == s && b0 >= tab_b && b0 < tab_b + 32)
            return;
        tab_s = s;
        tab_b = b0 & ~31;
        const int t = (tab_b + lane) << btl;
        tab_page = -1;
        if (t < u.p0 + u.len)
            tab_page = a.pg.table[s * a.pg.table_stride + t / a.pg.page];
        tab_y = t % a.pg.page;
    };
    for (long long x = run.x0; x < run.x1 && !stop;) {
        if (seg >= u.tiles * a.Hk) {
            do
                u = seq_units(a, ++s, group, R::V ? M : 0, U, bad);
            while (u.units == 0 && s + 1 < a.sq.n);
            seg = 0;
            v0 = 0;
            if (u.units == 0)
                break;                 // lengths that changed meanwhile
        }
        // (rounded down: whoever has a segment's last place has its last unit)
        const int v1 = (int)min(run.x1 - x + v0, (long long)u.length());
        const int u0 = u.units_at(v0), u1 = u.units_at(v1);
        const int hk = u.tiles == 1 ? seg : seg / u.tiles;
        const bool whole = u0 == 0 && u1 == u.units;
        const int passes = u1 <= u0 ? 0 : R::V ? 1 : (int)(((unsigned)u.len * group + M - 1) / M);
        for (int pass = 0; pass < passes && !stop; ++pass, ++parts) {
            // ---- the rows and the description
            const int b = parts & 1;
            Part p;
            p.live = 1;
            p.s = s;
            p.hk = hk;
            p.r0 = u.r0;
            p.p0 = u.p0;
            p.len = u.len;
            const int i0 = (R::V ? seg - hk * u.tiles : pass) * M;
            p.rowf = i0 / group;
            p.hf = i0 - p.rowf * group;
            p.nrows = min(u.len * group - i0, M);
            const int last = u.p0 + p.rowf + (p.hf + p.nrows - 1) / group;     // position the tile sees last
            p.u0 = u0;
            p.u1 = R::V ? min(u1, last / U + 1) : u1;
            p.whole = whole;
            p.slot = x == run.x0 ? 0 : 1;
            p.pass = min(pass, 1);
            const int n0 = p.u0 + ((pw - it) & (R::NP - 1));            // this warp's first unit
            if (n0 < p.u1)
                window(n0 * NB);
            if (pw == 0) {
                if (!ring_wait(&ring.qempty[b], (uint32_t)((parts >> 1) & 1) ^ 1u, &ring.abort, a.sq))
                    stop = true;
                stop = __any_sync(0xffffffffu, stop);
                if (stop)
                    break;
                put_rows(a, ring, qbuf, p, b, group);
            }
            // ---- this warp's units
            const int count = max(p.u1 - p.u0, 0);
            for (int n = n0; n < p.u1; n += R::NP) {
                const int b0 = n * NB;
                window(b0);
                if (lane == 0 && !ring_wait(&ring.empty[slot], phase ^ 1, &ring.abort, a.sq))
                    stop = true;
                stop = __any_sync(0xffffffffu, stop);
                if (stop)
                    break;
                // boxes that hold positions of the sequence
                const int nb = min(NB, ((u.p0 + u.len - n * U) + BT - 1) >> btl);
                const unsigned there = __ballot_sync(0xffffffffu, (unsigned)tab_page < (unsigned)a.pg.pages);
                const unsigned ok = (there >> (b0 - tab_b)) & ((1u << nb) - 1u);
                // a lane a box; a page that does not exist is one behind the last: zeros
                const int from = b0 - tab_b + lane;
                const int page = __shfl_sync(0xffffffffu, tab_page, from & 31);
                const int y = __shfl_sync(0xffffffffu, tab_y, from & 31);
                if (lane == 0) {
                    ring.ok[slot] = ok;
                    if (ok != (1u << nb) - 1u)
                        seq_flag(a.sq, GATTN_STATUS_RANGE);
                    mbar_arrive_expect_tx(&ring.full[slot], nb * box_bytes * (R::V ? 2 : 1));
                }
                __syncwarp();
                if (lane < nb) {
                    const uint32_t dst = smem_u32(units) + slot * R::UNIT + lane * box_bytes;
                    const uint32_t bar = smem_u32(&ring.full[slot]);
                    const int from_page = ok >> lane & 1u ? page : a.pg.pages;
                    box_g2s(dst, kmap, y, hk, from_page, bar, pol);
                    if (R::V)
                        box_g2s(dst + R::PLANE, vmap, y, hk, from_page, bar, pol);
                }
                ++issued;
                slot += R::NP;
                if (slot >= R::SLOTS) {
                    slot -= R::SLOTS;
                    phase ^= 1;
                }
            }
            it = (it + count) & (R::NP - 1);
            if (pw == 0 && lane == 0 && u0 == 0 && u1 < u.units)
                seen(p, (int)((x - v0 + u.length() - 1) / run.quota));
        }
        x += v1 - v0;
        v0 = 0;
        ++seg;
    }
    if (!stop && pw == 0) {
        const int b = parts & 1;
        stop = !ring_wait(&ring.qempty[b], (uint32_t)((parts >> 1) & 1) ^ 1u, &ring.abort, a.sq);
        stop = __any_sync(0xffffffffu, stop);
        if (!stop) {
            if (lane == 0)
                ring.part[b].live = 0;
            cp_arrive(&ring.qfull[b]);
            mbar_arrive(&ring.qfull[b]);
        }
    }
    // no copy may be on its way when the block ends (where consumers gave up): the last
    // round of this warp's slots, from the newest back
    cp_async_wait_all();
    if (lane == 0)
        for (int i = 0; i < R::SLOTS / R::NP && i < issued; ++i) {
            slot -= R::NP;
            if (slot < 0) {
                slot += R::SLOTS;
                phase ^= 1;
            }
            const unsigned long long t0 = global_ns();
            while (!mbar_try(&ring.full[slot], phase) && global_ns() - t0 < kWaitLimitNs) {
            }
        }
    __syncwarp();
}

// --------------------------------------------------------------- the products

// m16n8k16 of bf16 operands into fp32; free to be scheduled between the loads
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// an 8 x 8 matrix of 16-bit elements, as the matrix instructions hold it, turned over
__device__ __forceinline__ uint32_t turned(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

}  // namespace paged

bool encode_pages(CUtensorMap *m, const Pages &pg, bool v, int Hk, int d, int box);

}  // namespace gattn
