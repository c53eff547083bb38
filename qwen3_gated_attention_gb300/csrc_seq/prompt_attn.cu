// prompt_attn.cu -- causal attention of packed prompt rows with grouped heads and
// the sigmoid output gate, on the tensor cores.
//
// A pair of CTAs (cta_group::2) owns 256 query rows, 128 each: consecutive tokens
// of one sequence times hp query heads of one KV group (hp: the power of two in the
// group's size), so that a tile of keys serves every head it can.  The pair walks
// the keys it sees in blocks of 128 with the running maximum m and sum l of the
// softmax (base 2):
//   S = Q K^T,  p = 2^(c (s - m)),  l <- l a + sum p,  O <- O a + P V,
// a = 2^(c (m_old - m)).  S and O stay in tensor memory; P goes back into S's
// columns as bf16 and is the A operand of P V: the tensor cores take no wider operand
// beside bf16 values at this rate.  l sums the rounded p, so that they add up to one.
// Each CTA loads half of a block: 64 of its keys, and half of the value columns.
// That halves what one SM reads from L2 and from its own shared memory per MMA
// (with one CTA a tile, M = 128, the MMAs waited for their operands: a block took
// 3800 cycles instead of the 2048 of its products at head_dim 256).
// The reference m of a row only moves when its maximum has grown by more than 2^8
// (p <= 256 keeps its relative precision in bf16 and in the fp32 sums), so O is
// rescaled a few times per row instead of once per block.
//
// The grid is persistent, one CTA per SM; tiles are dealt longest first.  Per CTA:
// warps 0-7 softmax and epilogue (a thread per row and half of the columns), 8
// copies, 9 issues the MMAs (of the pair, in the even CTA), 10 stores, 11 finds tiles.
// The gate tile comes through the ring like the keys and values; the rows take its
// place and leave from there, so that no thread reads or writes scattered rows.
//
// Blocks that some row sees only part of: a value that is not finite would spoil
// rows that do not see it (0 * NaN).  The softmax warps look through the values of
// such a block before its product, put zero in such a value's place, and the rows
// that do see it get it back at the end.
//
// Few rows over many keys: clusters of 2, 4 or 8 CTAs, each pair taking a share of
// the blocks; the partial (m, l, O) are joined through distributed shared memory.
//
// Measured: one prompt of 8192 rows, 16 heads of 256 over 4: 385 us, 1430 TFLOP/s, 75 % of
// the library's matrix rate (a block takes 3000 cycles, 2048 of them its products: the
// rest is the hand-over between scores, softmax and values, which two score buffers
// cover only in part).  Eight prompts of 1 to 1500 rows, 24 heads over 2: 77 us, 682
// TFLOP/s of visible products; 4.4 blocks a tile, against an epilogue of 6800 cycles
// (gates, exponentials, rows out) per tile.  Heads of 64: 41.5 us for 3960 rows of 16 heads
// over 8, bound by the softmax (1800 of 2775 cycles a block).
#include <algorithm>
#include <cmath>

#include <cudaTypedefs.h>

#include "seq.cuh"
#include "tc5.cuh"

namespace gattn {

namespace {

constexpr int kSoft = 8;                    // softmax warps
constexpr int kWarps = kSoft + 4;
constexpr int kThreads = kWarps * 32;
constexpr int kM = 128;                     // query rows of a CTA
constexpr int kN = 128;                     // keys of a block
constexpr int kSlot = 16384;                // bytes of a ring slot
constexpr int kCols = 512;                  // TMEM columns: two score buffers and O
constexpr int kOCol = 2 * kN;
constexpr float kGrow = 8.f;                // log2 growth of a row's maximum that moves its reference

// A tile as one CTA of the pair sees it.
struct Tile {
    int s;                                  // sequence, or -1: no more tiles
    int row0, rows;                         // packed row of its first token, tokens it owns
    int slot, kv0;                          // batch row and first key row of the sequence
    int seen0;                              // keys its first token sees (may be <= 0)
    int b0, nb;                             // first key block and blocks (this CTA pair's share)
    int part0;                              // from this block on some row of the pair sees only part
    int level;
};

template <int D>
struct Cfg {
    static constexpr int CH = D / 64;               // 64-element chunks of a head
    static constexpr int KS = (CH + 1) / 2;         // slots of a block's 64 keys: two chunks each
    static constexpr int CV = (D / 2 + 63) / 64;    // chunks of the CTA's value columns
    static constexpr int VK = kN / CV;              // keys per value slot
    static constexpr int VS = CV;                   // value slots per block
    static constexpr int QB = kM * D * 2;
    static constexpr int SLOTS = D == 256 ? 9 : 10;
    static constexpr int HC = D / 2;                // O columns per softmax thread
    static constexpr int ST = D + 4;                // row stride of staged partial sums (floats)
    struct alignas(16) Tables {                     // behind the ring
        uint64_t full[SLOTS], empty[SLOTS];
        uint64_t part[SLOTS];                       // loads that the softmax warps read
        uint64_t q_full, q_free, s_full[2], p_ready[2], pv_done, o_done, o_free, out_ready, t_full[2], t_empty[2];
        float mx[2][2][kM];                         // block parity, column half, row
        float lsum[2][2][kM];                       // tile parity, column half, row
        Tile tile[2];
        uint32_t tmem;
        int abort;
        int fixes[2];                               // per tile parity
        // per value column, first key (from part0 on) that holds NaN, +inf, -inf;
        // 0xFFFF: none
        uint16_t fix_at[2][3][D];
    };
    static constexpr int SMEM = QB + SLOTS * kSlot + (int)sizeof(Tables);
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(kM * ST * 4 <= SLOTS * kSlot, "partial sums fit the ring");
    static_assert(kOCol + D <= kCols, "TMEM");
};

// What the order of the tiles needs of a sequence.  All of it fits 32 bits: counts of
// at most 2^30 rows and keys.  A tile of a pair has tp = 1 << tl tokens.
struct SeqKeys {
    int r0, len, slot, kv0;
    int past;                   // keys before its first row (negative: rows that see none)
    bool ok;
    __device__ __forceinline__ int tiles(int tl) const { return (len + (1 << tl) - 1) >> tl; }
    // key blocks of its last tile
    __device__ __forceinline__ int most() const { return past + len > 0 ? (past + len + kN - 1) / kN : 0; }
    // tiles with at least x key blocks: the last ones
    __device__ __forceinline__ int at_least(int x, int tl) const
    {
        const int n = tiles(tl);
        if (x == 0 || n == 0)
            return n;
        const int keys = (x - 1) * kN + 1;              // that reach x blocks
        if (past + len < keys)
            return 0;
        const int need = keys - past;                   // tokens that see so many: at most len
        return n - min(need <= 0 ? 0 : ((need + (1 << tl) - 1) >> tl) - 1, n - 1);
    }
};

__device__ __forceinline__ SeqKeys seq_keys(const PromptAttnArgs &a, int s)
{
    SeqKeys q;
    long long past, kv0 = 0;
    q.slot = 0;
    if (a.pos) {
        seq_rows(a.sq, s, q.r0, q.len);
        q.slot = a.sq.slots ? a.sq.slots[s] : s;
        past = a.pos[s];
        q.ok = q.slot >= 0 && q.slot < a.kv_batch && past >= 0 && past + q.len <= a.kv_rows;
    } else {
        kv0 = a.cu_kv[s];
        const long long kv1 = a.cu_kv[s + 1];
        seq_rows(a.sq, s, q.r0, q.len);
        past = kv1 - kv0 - q.len;
        q.ok = kv0 >= 0 && kv1 >= kv0 && kv1 <= a.kv_rows;
    }
    q.past = q.ok ? (int)past : -q.len;                 // a skipped sequence sees nothing
    q.kv0 = (int)kv0;
    return q;
}

// Deals the tiles out by rank; called by one whole warp with rising ranks.
struct Dealer {
    SeqKeys mine;               // up to 32 sequences: the lane's own
    int base;                   // more: the lane's sequences are base + lane, ...
    int before;                 // ... with this many tiles before them

    __device__ __forceinline__ void start(const PromptAttnArgs &a)
    {
        base = before = 0;
        mine = seq_keys(a, min((int)(threadIdx.x & 31), a.sq.n - 1));
        if ((threadIdx.x & 31) >= a.sq.n)
            mine.len = 0;
    }
    // Sequence and level (tile within it) of the rank-th tile; false: none.  Up to
    // 32 sequences in order of falling key blocks, more in their own order.
    __device__ __forceinline__ bool find(const PromptAttnArgs &a, int tl, int rank, SeqKeys &q, int &s, int &level)
    {
        const int lane = threadIdx.x & 31, n = a.sq.n;
        const unsigned all = 0xffffffffu;
        auto scan = [&](int c) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(all, c, o);
                if (lane >= o)
                    c += x;
            }
            return c;
        };
        if (n <= 32) {
            auto count = [&](int x) { return (int)__reduce_add_sync(all, mine.at_least(x, tl)); };
            if (rank >= count(0))
                return false;
            int lo = 0, hi = __reduce_max_sync(all, mine.len > 0 ? mine.most() : 0);   // count(lo) > rank
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (count(mid) > rank)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            // tiles of exactly lo blocks, by lane
            const int over = mine.at_least(lo + 1, tl), here = mine.at_least(lo, tl);
            const int idx = rank - (int)__reduce_add_sync(all, over);
            const int sum = scan(here - over);
            s = __ffs(__ballot_sync(all, idx < sum)) - 1;
            level = __shfl_sync(all, mine.tiles(tl) - here + idx - (sum - (here - over)), s);
            q.r0 = __shfl_sync(all, mine.r0, s);
            q.len = __shfl_sync(all, mine.len, s);
            q.slot = __shfl_sync(all, mine.slot, s);
            q.kv0 = __shfl_sync(all, mine.kv0, s);
            q.past = __shfl_sync(all, mine.past, s);
            q.ok = __shfl_sync(all, (int)mine.ok, s);
            return true;
        }
        for (;;) {
            if (base >= n)
                return false;
            int r0, len = 0;
            if (base + lane < n)
                seq_rows(a.sq, base + lane, r0, len);
            const int sum = scan((len + (1 << tl) - 1) >> tl);
            const int total = __shfl_sync(all, sum, 31);
            if (rank - before < total) {
                const int idx = rank - before;
                const int l = __ffs(__ballot_sync(all, idx < sum)) - 1;
                level = __shfl_sync(all, sum - 1 - idx, l);     // its longest rows first
                s = base + l;
                q = seq_keys(a, s);
                return true;
            }
            before += total;
            base += 32;
        }
    }
};

// 16-bit minimum in the shared memory of a CTA of the cluster (no such atomic exists)
__device__ void atomic_min16(uint32_t addr, uint32_t v)
{
    const uint32_t w = addr & ~3u;
    const int sh = (addr & 2) * 8;
    unsigned old;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(old) : "r"(w) : "memory");
    while (((old >> sh) & 0xFFFFu) > v) {
        const unsigned next = (old & ~(0xFFFFu << sh)) | (v << sh);
        unsigned got;
        asm volatile("atom.relaxed.cluster.shared::cluster.cas.b32 %0, [%1], %2, %3;"
                     : "=r"(got)
                     : "r"(w), "r"(old), "r"(next)
                     : "memory");
        if (got == old)
            break;
        old = got;
    }
}

__device__ __forceinline__ bool not_finite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

__device__ __forceinline__ float4 ld_dsmem_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// Whether `ok` holds in all `threads` of named barrier `id`.
__device__ __forceinline__ bool named_bar_and(int id, int threads, bool ok)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
                 "barrier.cta.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)ok), "r"(id), "r"(threads)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-g)
__device__ __forceinline__ float sigmoid(float g) { return rcp(1.f + ex2(-1.4426950408889634f * g)); }

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// f *= sigmoid(g) for eight values, two with one reciprocal, 1/a = b (1/(a b)).  No
// branch within but for gates below -41 or NaN, so that they overlap.
__device__ __forceinline__ void gate8(float (&f)[8], const float (&g)[8])
{
    float x[8], a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = g[i] * -1.4426950408889634f;
        a[i] = 1.f + ex2(x[i]);
    }
    // each at most 2^60: the products stay finite
    const float top = max_nan(max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3])),
                              max_nan(max_nan(x[4], x[5]), max_nan(x[6], x[7])));
    if (top <= 60.f) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float ab = rcp(a[i] * a[i + 1]);
            f[i] *= ab * a[i + 1];
            f[i + 1] *= ab * a[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] *= rcp(a[i]);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ PromptAttnArgs a, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap gmap, const __grid_constant__ CUtensorMap omap,
                   int hp_log2, int split)
{
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *const qs = smem, *const ring = smem + C::QB;
    typename C::Tables &T = *reinterpret_cast<typename C::Tables *>(smem + C::QB + C::SLOTS * kSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank(), half = rank & 1, lead = rank & ~1u;
    const uint16_t pair = (uint16_t)(3u << lead);
    const int share = (int)rank >> 1;                  // which part of the blocks
    const int hp = 1 << hp_log2, tpt = kM >> hp_log2;
    const int groups = a.H >> hp_log2;
    auto at_lead = [&](uint64_t *bar) { return dsmem_addr(bar, lead); };

    if (warp == 8 && lane == 0) {
        for (int i = 0; i < C::SLOTS; ++i) {
            mbar_init(&T.full[i], 2);                  // the producers of both CTAs
            mbar_init(&T.empty[i], 1);
            mbar_init(&T.part[i], 1);
        }
        mbar_init(&T.q_full, 2);
        mbar_init(&T.q_free, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&T.s_full[i], 1);
            mbar_init(&T.p_ready[i], 2 * kSoft);
            mbar_init(&T.t_full[i], 1);
            mbar_init(&T.t_empty[i], 3 + 2 * kSoft);   // 8, 9, 10 here, the softmax of both CTAs
            T.fixes[i] = 0;
        }
        mbar_init(&T.pv_done, 1);
        mbar_init(&T.o_done, 1);
        mbar_init(&T.o_free, 2 * kSoft);
        mbar_init(&T.out_ready, kSoft);
        T.abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    } else if (warp == 9) {
        tmem_alloc(&T.tmem, kCols);
    } else if (warp == 10) {
        for (int i = lane; i < 2 * 3 * D; i += 32)
            (&T.fix_at[0][0][0])[i] = 0xFFFF;
    }
    Dealer deal;
    if (warp == 11)
        deal.start(a);                                 // its loads pass while the CTAs meet
    tc5_fence_before();
    __syncthreads();
    cluster_sync();
    tc5_fence_after();
    const uint32_t tmem = T.tmem;
    volatile int *abort = &T.abort;
    // the it-th tile's description
    auto next_tile = [&](int it, Tile &t) {
        if (!tc5_wait(&T.t_full[it & 1], (it >> 1) & 1, abort))
            return false;
        t = T.tile[it & 1];
        return t.s >= 0;
    };

    if (warp == 11) {
        // ------------------------------------------------------------- tiles
        // dealt round by round, every other round backwards, so that nobody keeps
        // getting the longer ones
        const int tl = 8 - hp_log2, clusters = gridDim.x / (2 * split), place = blockIdx.x / (2 * split);
        for (int it = 0;; ++it) {
            const unsigned r = (unsigned)it * clusters + (it & 1 ? clusters - 1 - place : place);
            const int group = r % (unsigned)groups;
            SeqKeys q;
            Tile t;
            const bool some = (split == 1 || it == 0) && r < 0x80000000u &&
                              deal.find(a, tl, r / (unsigned)groups, q, t.s, t.level);
            if (it >= 2 && !__all_sync(0xffffffffu, tc5_wait(&T.t_empty[it & 1], ((it >> 1) - 1) & 1, abort)))
                break;
            if (some) {
                const int tok0 = t.level << tl;
                const int last = q.past + min(q.len, tok0 + (1 << tl));
                const int nb = last > 0 ? (last + kN - 1) / kN : 0;
                const int each = split == 1 ? nb : split == 2 ? (nb + 1) >> 1 : (nb + 3) >> 2;
                t.b0 = min(nb, share * each);
                t.nb = min(nb, t.b0 + each) - t.b0;
                const int seen = q.past + tok0 + 1;
                t.part0 = seen > 0 ? seen / kN : 0;
                t.row0 = q.r0 + tok0 + (int)half * tpt;
                t.rows = max(0, min(tpt, q.len - tok0 - (int)half * tpt));
                t.slot = q.slot;
                t.kv0 = q.kv0;
                t.seen0 = seen + (int)half * tpt;
                // the group of heads, beside the level
                t.level = group;
                if (!q.ok && lane == 0)
                    seq_flag(a.sq, GATTN_STATUS_RANGE);
            } else {
                t.s = -1;
            }
            if (lane == 0) {
                T.tile[it & 1] = t;
                mbar_arrive(&T.t_full[it & 1]);
            }
            __syncwarp();
            if (!some)
                break;
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------- copies
        if (lane == 0) {
            int n = 0, used = 0;                // slots filled so far, tiles that had blocks
            uint32_t in_part = 0, pphase = 0;   // per slot: its last load signals part[]; part[]'s phase
            bool go = true;
            Tile t;
            int none = 0;
            for (int it = 0; go && next_tile(it, t); ++it) {
                if (t.nb > 0) {
                    const int head0 = t.level << hp_log2, kvh = head0 / (a.H / a.Hk);
                    go = used == 0 || tc5_wait(&T.q_free, (used - 1) & 1, abort);
                    ++used;
                    if (go) {
                        if (half == 0)
                            mbar_arrive_expect_tx(&T.q_full, 2 * C::QB);
                        else
                            mbar_arrive_cluster(at_lead(&T.q_full));
                        for (int ch = 0; ch < C::CH; ++ch)
                            tma3d(smem_u32(qs) + ch * (kM * 128), &qmap, ch * 64, head0, t.row0,
                                  at_lead(&T.q_full));
                    }
                    // waits for the next slot and announces `bytes` on the barrier its load
                    // signals: the even CTA's full[], or one's own part[]
                    uint32_t bar = 0;
                    auto fill = [&](uint32_t bytes, bool part) -> uint32_t {
                        const int sl = n % C::SLOTS;
                        if (n >= C::SLOTS && !tc5_wait(&T.empty[sl], ((n / C::SLOTS) - 1) & 1, abort)) {
                            go = false;
                            return 0;
                        }
                        in_part = part ? in_part | 1u << sl : in_part & ~(1u << sl);
                        pphase ^= part ? 1u << sl : 0u;
                        if (part) {
                            // the softmax warps wait for these bytes; full[] only keeps step
                            bar = smem_u32(&T.part[sl]);
                            if (bytes)
                                mbar_arrive_expect_tx(&T.part[sl], bytes);
                            else
                                mbar_arrive(&T.part[sl]);
                            mbar_arrive_cluster(at_lead(&T.full[sl]));
                        } else {
                            bar = at_lead(&T.full[sl]);
                            if (half == 0)
                                mbar_arrive_expect_tx(&T.full[sl], 2 * bytes);
                            else
                                mbar_arrive_cluster(bar);
                        }
                        ++n;
                        return smem_u32(ring) + sl * kSlot;
                    };
                    auto load_k = [&](int b) {
                        for (int ch = 0; ch < C::CH && go; ch += 2) {
                            const int two = min(2, C::CH - ch);
                            const uint32_t p = fill(two * 8192, false);
                            for (int x = 0; x < two && go; ++x)
                                tma4d(p + x * 8192, &kmap, (ch + x) * 64,
                                      t.kv0 + (t.b0 + b) * kN + (int)half * 64, kvh, t.slot, bar);
                        }
                    };
                    auto load_v = [&](int b) {
                        for (int g = 0; g < C::VS && go; ++g) {
                            const uint32_t p = fill(C::VK * C::CV * 128, t.b0 + b >= t.part0);
                            for (int ch = 0; ch < C::CV && go; ++ch)
                                tma4d(p + ch * (C::VK * 128), &vmap, (int)half * (D / 2) + ch * 64,
                                      t.kv0 + (t.b0 + b) * kN + g * C::VK, kvh, t.slot, bar);
                        }
                    };
                    load_k(0);
                    for (int b = 1; b < t.nb && go; ++b) {
                        load_k(b);
                        load_v(b - 1);
                    }
                    load_v(t.nb - 1);
                    // the rows' way out, with the gate where it is bf16
                    const bool gate = a.gate && !a.gate_f32;
                    for (int ch = 0; ch < C::CH && go && split == 1; ++ch) {
                        const uint32_t p = fill(gate ? kM * 128 : 0, true);
                        if (go && gate)
                            tma3d(p, &gmap, ch * 64, head0, t.row0, bar);
                    }
                }
                mbar_arrive(&T.t_empty[it & 1]);
            }
            // arrivals on this CTA's barriers that MMAs still owe it
            for (int i = max(0, n - C::SLOTS); i < n && !*abort; ++i)
                tc5_wait(&T.empty[i % C::SLOTS], (i / C::SLOTS) & 1, abort);
            if (used > 0 && !*abort)
                tc5_wait(&T.q_free, (used - 1) & 1, abort);
            // every copy has landed before the shared memory is given up, also when a
            // wait ran out (the odd CTA's are seen through the even one's barriers)
            if (*abort && half == 0 && used > 0)
                tc5_wait(&T.q_full, (used - 1) & 1, &none);
            for (int i = max(0, n - C::SLOTS); i < n && *abort; ++i) {
                const int sl = i % C::SLOTS;
                if (in_part >> sl & 1)
                    tc5_wait(&T.part[sl], (pphase >> sl & 1) ^ 1, &none);
                if (half == 0)
                    tc5_wait(&T.full[sl], (i / C::SLOTS) & 1, &none);
            }
        }
    } else if (warp == 9) {
        // --------------------------------------------------------------- MMAs
        if (lane == 0) {
            constexpr uint32_t id_s = tc5_idesc(2 * kM, kN, false), id_o = tc5_idesc(2 * kM, D, true);
            int n = 0, gb = 0, used = 0;        // slots, blocks and tiles so far
            bool go = true;
            Tile t;
            for (int it = 0; go && next_tile(it, t); ++it) {
                if (half == 0 && t.nb > 0) {
                    go = tc5_wait(&T.q_full, used & 1, abort);
                    auto scores = [&](int b) {
                        const uint32_t d = tmem + ((gb + b) & 1) * kN;
                        for (int ch = 0; ch < C::CH && go; ++ch) {
                            const int sl = n % C::SLOTS;
                            if ((ch & 1) == 0)
                                go = tc5_wait(&T.full[sl], (n / C::SLOTS) & 1, abort);
                            if (!go)
                                return;
                            tc5_fence_after();
                            const uint64_t da = tc5_desc(smem_u32(qs) + ch * (kM * 128), 16, 1024);
                            const uint64_t db = tc5_desc(smem_u32(ring) + sl * kSlot + (ch & 1) * 8192, 16, 1024);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc5_mma_ss(d, da + 2 * k, db + 2 * k, id_s, ch > 0 || k > 0);
                            if ((ch & 1) || ch == C::CH - 1) {
                                tc5_commit(&T.empty[sl], pair);
                                ++n;
                            }
                        }
                        tc5_commit(&T.s_full[(gb + b) & 1], pair);
                        if (b == t.nb - 1)
                            tc5_commit(&T.q_free, pair);
                    };
                    auto values = [&](int b) {
                        const int pb = (gb + b) & 1;
                        go = go && tc5_wait(&T.p_ready[pb], ((gb + b) >> 1) & 1, abort);
                        if (b == 0 && used > 0)
                            go = go && tc5_wait(&T.o_free, (used - 1) & 1, abort);
                        if (!go)
                            return;
                        tc5_fence_after();
                        const uint32_t d = tmem + kOCol;
                        for (int g = 0; g < C::VS; ++g, ++n) {
                            const int sl = n % C::SLOTS;
                            go = tc5_wait(&T.full[sl], (n / C::SLOTS) & 1, abort);
                            if (!go)
                                return;
                            const uint64_t db = tc5_desc(smem_u32(ring) + sl * kSlot, C::VK * 128, 1024);
#pragma unroll
                            for (int k = 0; k < C::VK / 16; ++k) {
                                // probabilities of keys 0-63 stand in columns 0-31 of the
                                // buffer, those of keys 64-127 in columns 64-95
                                const int key = g * C::VK + k * 16;
                                tc5_mma_ts(d, tmem + pb * kN + (key & 64) + (key & 63) / 2,
                                           db + k * (2048 >> 4), id_o, b > 0 || g > 0 || k > 0);
                            }
                            tc5_commit(&T.empty[sl], pair);
                        }
                        // the last product has a barrier of its own: a parity does not tell
                        // phase n from n - 2
                        tc5_commit(b == t.nb - 1 ? &T.o_done : &T.pv_done, pair);
                    };
                    scores(0);
                    for (int b = 1; b < t.nb && go; ++b) {
                        scores(b);
                        values(b - 1);
                    }
                    values(t.nb - 1);
                    gb += t.nb;
                    n += split == 1 ? C::CH : 0;
                    ++used;
                }
                mbar_arrive(&T.t_empty[it & 1]);
            }
            if (*abort && half == 0) {
                // the MMAs that were issued are done before their memory is freed
                int none = 0;
                mbar_init(&T.q_free, 1);
                fence_mbar_init();
                tc5_commit(&T.q_free, (uint16_t)(1u << rank));
                tc5_wait(&T.q_free, 0, &none);
            }
        }
    } else if (warp == 10) {
        // ------------------------------------------------------------- stores
        int n0 = 0, used = 0;
        Tile t;
        for (int it = 0; split == 1; ++it) {
            if (!__all_sync(0xffffffffu, next_tile(it, t)))
                break;
            if (t.nb > 0) {
                n0 += t.nb * (C::KS + C::VS);
                const int head0 = t.level << hp_log2;
                if (!__all_sync(0xffffffffu, tc5_wait(&T.out_ready, used & 1, abort)))
                    break;
                ++used;
                if (t.rows == tpt) {
                    if (lane == 0) {
                        for (int ch = 0; ch < C::CH; ++ch)
                            tma_store3d(&omap, smem_u32(ring) + (n0 + ch) % C::SLOTS * kSlot, ch * 64, head0, t.row0);
                        tma_store_commit();
                        tma_store_wait_read();
                    }
                } else {
                    // the rows there are: a 16-byte unit per lane, eight to a row
                    const int rows = t.rows << hp_log2, un = lane & 7;
                    for (int ch = 0; ch < C::CH; ++ch) {
                        const uint8_t *from = ring + (n0 + ch) % C::SLOTS * kSlot;
                        __nv_bfloat16 *to = a.out + (long long)t.row0 * a.os.tok + (long long)head0 * a.os.head +
                                            ch * 64 + un * 8;
#pragma unroll 4
                        for (int row = lane >> 3; row < rows; row += 4)
                            *reinterpret_cast<uint4 *>(to + (row >> hp_log2) * a.os.tok +
                                                       (row & (hp - 1)) * a.os.head) =
                                *reinterpret_cast<const uint4 *>(from + row * 128 + ((un ^ (row & 7)) << 4));
                    }
                }
                __syncwarp();
                if (lane == 0)
                    for (int ch = 0; ch < C::CH; ++ch)
                        mbar_arrive(&T.empty[(n0 + ch) % C::SLOTS]);
                n0 += C::CH;
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&T.t_empty[it & 1]);
        }
        if (lane == 0)
            tma_store_wait();
    } else {
        // ---------------------- softmax: a thread per row and half of the columns
        const int row = (warp & 3) * 32 + lane, hf = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int tok = row >> hp_log2, hd = row & (hp - 1);
        const float c = a.scale_log2;
        int gb = 0, used = 0, pvs = 0;      // blocks, tiles with blocks, products but last ones
        int n0 = 0;                         // slots before this tile
        uint32_t phase = 0;                 // per slot: parity of its next part[] phase
        bool go = true;
        // values of a slot that are not finite: remembered for both CTAs, zero here
        auto look_through = [&](uint8_t *slot, int key0, int par) {
            uint4 *p = reinterpret_cast<uint4 *>(slot);
            constexpr int PER = C::VK * C::CV * 8 / (kSoft * 32);     // 16-byte units a thread
            uint4 u[PER];
            bool hit = false;
#pragma unroll
            for (int k = 0; k < PER; ++k)
                u[k] = p[threadIdx.x + k * kSoft * 32];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                // a set exponent field is largest: one packed maximum finds it
                const unsigned top = __vmaxu2(__vmaxu2(u[k].x & 0x7FFF7FFFu, u[k].y & 0x7FFF7FFFu),
                                              __vmaxu2(u[k].z & 0x7FFF7FFFu, u[k].w & 0x7FFF7FFFu));
                hit |= (top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u;
            }
            if (!hit)
                return;
#pragma unroll 1
            for (int i = threadIdx.x; i < PER * kSoft * 32; i += kSoft * 32) {
                const uint4 v = p[i];
                uint32_t x[4] = {v.x, v.y, v.z, v.w};
                // 16-byte unit i: chunk of 64 columns, key row, unit within the row,
                // swizzled by the row
                const int ch = i / (C::VK * 8), key = (i / 8) % C::VK, un = (i & 7) ^ (key & 7);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t h = (x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                    if (!not_finite16(h))
                        continue;
                    const int what = (h & 0x7F) ? 0 : (h >> 15) ? 2 : 1;
                    const int col = (int)half * (D / 2) + ch * 64 + un * 8 + e;
                    for (uint32_t to = lead; col < D && to < lead + 2; ++to)
                        atomic_min16(dsmem_addr(&T.fix_at[par][what][col], to), key0 + key);
                    x[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
                p[i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
            for (uint32_t to = lead; to < lead + 2; ++to)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(dsmem_addr(&T.fixes[par], to)), "r"(1)
                             : "memory");
            fence_proxy_async_smem();
            asm volatile("fence.acq_rel.cluster;" ::: "memory");
        };
        Tile t;
        for (int it = 0;; ++it) {
            // one decision for all, so that the barriers below are met by everybody:
            // a wait that gives up skips work, never a barrier
            go = named_bar_and(6, kSoft * 32, next_tile(it, t) && go);
            if (!go)
                break;
            const int head = (t.level << hp_log2) + hd;
            const bool mine = tok < t.rows;
            const int seen = t.seen0 + tok;           // keys this row sees
            float m = -INFINITY;                      // the row's reference
            float l = 0.f;                            // sum over this thread's columns
            for (int b = 0; b < t.nb; ++b, ++gb) {
                const int pb = gb & 1;
                const uint32_t S = tmem + lanes + pb * kN + hf * 64;
                go = __all_sync(0xffffffffu, go && tc5_wait(&T.s_full[pb], (gb >> 1) & 1, abort));
                if (!go) {
                    named_bar_sync(2 + (warp & 3), 64);
                    continue;
                }
                tc5_fence_after();
                const bool part = t.b0 + b >= t.part0;
                const int lim = part ? seen - (t.b0 + b) * kN - hf * 64 : 64;    // visible columns
                uint32_t r0[32], r1[32];
                float mx = -INFINITY;
                tmem_ld32(r0, S);
                tmem_ld32(r1, S + 32);
                tmem_wait_ld();
                if (part) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        r0[i] = i < lim ? r0[i] : 0xFF800000u;
                        r1[i] = i + 32 < lim ? r1[i] : 0xFF800000u;
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    mx = fmaxf(mx, fmaxf(__uint_as_float(r0[i]), __uint_as_float(r1[i])));
                // the row's maximum over both halves
                T.mx[pb][hf][row] = mx;
                named_bar_sync(2 + (warp & 3), 64);
                mx = fmaxf(mx, T.mx[pb][hf ^ 1][row]);
                // move the reference on the first block and when the maximum outgrows it
                float alpha = 1.f;
                const bool move = mx > m && (m == -INFINITY || (mx - m) * c > kGrow);
                if (move) {
                    alpha = m == -INFINITY ? 0.f : ex2((m - mx) * c);
                    m = mx;
                }
                if (b > 0 && __any_sync(0xffffffffu, move)) {
                    go = __all_sync(0xffffffffu, tc5_wait(&T.pv_done, (pvs + b - 1) & 1, abort));
                    if (!go)
                        continue;
                    tc5_fence_after();
                    l *= alpha;
#pragma unroll 1
                    for (int q = 0; q < C::HC / 32; ++q) {
                        uint32_t o[32];
                        tmem_ld32(o, tmem + lanes + kOCol + hf * C::HC + q * 32);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(tmem + lanes + kOCol + hf * C::HC + q * 32, o);
                    }
                }
                // a row without a visible key so far has reference -inf: against 0
                // its masked scores give p = 0
                const float ref = m == -INFINITY ? 0.f : m;
                const uint64_t nref = pack2(-ref, -ref), cc = pack2(c, c);
                uint64_t sum0 = 0, sum1 = 0;
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t x0 =
                        mul2(add2(pack2(__uint_as_float(r0[2 * i]), __uint_as_float(r0[2 * i + 1])), nref), cc);
                    const uint64_t x1 =
                        mul2(add2(pack2(__uint_as_float(r1[2 * i]), __uint_as_float(r1[2 * i + 1])), nref), cc);
                    float e0, e1, e2, e3;
                    unpack2(x0, e0, e1);
                    unpack2(x1, e2, e3);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    e2 = ex2(e2);
                    e3 = ex2(e3);
                    pk[i] = pack_bf16x2(e0, e1);
                    pk[16 + i] = pack_bf16x2(e2, e3);
                }
                tmem_st32(S, pk);
                if (part) {
                    // slots are filled in the order K0 [K1 V0] [K2 V1] ...
                    int n = n0 + min(b + 2, t.nb) * C::KS + b * C::VS;
#pragma unroll 1
                    for (int g = 0; g < C::VS; ++g, ++n) {
                        const int sl = n % C::SLOTS;
                        go = __all_sync(0xffffffffu, tc5_wait(&T.part[sl], phase >> sl & 1, abort)) && go;
                        phase ^= 1u << sl;
                        if (go)
                            look_through(ring + sl * kSlot, (t.b0 + b - t.part0) * kN + g * C::VK, it & 1);
                    }
                }
                tmem_wait_st();
                tc5_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster(at_lead(&T.p_ready[pb]));
                // the sum of what the values are multiplied by, while they are
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum0 = add2(sum0, pack2(bf16_lo(pk[i]), bf16_hi(pk[i])));
                    sum1 = add2(sum1, pack2(bf16_lo(pk[16 + i]), bf16_hi(pk[16 + i])));
                }
                float s0, s1;
                unpack2(add2(sum0, sum1), s0, s1);
                l += s0 + s1;
            }
            pvs += max(0, t.nb - 1);
            // ------------------------------------------------------------- epilogue
            const long long orow = t.row0 + tok;
            const long long go_ = orow * a.gs.tok + (long long)head * a.gs.head + hf * C::HC;
            __nv_bfloat16 *o = a.out + orow * a.os.tok + (long long)head * a.os.head + hf * C::HC;
            n0 += t.nb * (C::KS + C::VS);
            if (t.nb > 0 && split == 1) {
                // the slots that hold the gate and take the rows
#pragma unroll 1
                for (int ch = 0; ch < C::CH; ++ch) {
                    const int sl = (n0 + ch) % C::SLOTS;
                    go = __all_sync(0xffffffffu, go && tc5_wait(&T.part[sl], phase >> sl & 1, abort));
                    phase ^= 1u << sl;
                }
            }
            T.lsum[it & 1][hf][row] = l;
            named_bar_sync(2 + (warp & 3), 64);
            l += T.lsum[it & 1][hf ^ 1][row];
            if (t.nb > 0) {
                go = __all_sync(0xffffffffu, go && tc5_wait(&T.o_done, used & 1, abort));
                tc5_fence_after();
                ++used;
            }
            const float inv = seen > 0 ? 1.f / l : 0.f;
            const bool fixes = go && *(volatile int *)&T.fixes[it & 1] != 0;
            const int from = seen - t.part0 * kN;     // keys seen in the partly seen blocks
            float *const stage = reinterpret_cast<float *>(ring) + row * C::ST + hf * C::HC;
            // 32 columns at a time in a rolled loop: this code runs once a tile, and
            // unrolled it costs more in instruction fetches than it computes
            const bool gate_smem = a.gate && !a.gate_f32;
#pragma unroll 1
            for (int q = 0; q < C::HC; q += 32) {
                if (!go)
                    continue;
                float f[32];
                const int col0 = hf * C::HC + q;
                if (t.nb > 0) {
                    uint32_t nx[32];
                    tmem_ld32(nx, tmem + lanes + kOCol + col0);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        f[i] = __uint_as_float(nx[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        f[i] = 0.f;
                }
                if (fixes) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        // values that are not finite, for the rows that see them
                        if (from > T.fix_at[it & 1][0][col0 + i])
                            f[i] = __int_as_float(0x7fffffff);
                        if (from > T.fix_at[it & 1][1][col0 + i])
                            f[i] += INFINITY;
                        if (from > T.fix_at[it & 1][2][col0 + i])
                            f[i] -= INFINITY;
                    }
                }
                if (split > 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4 *>(stage + q + 4 * i) =
                            make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
                    continue;
                }
                if (t.nb == 0) {
                    if (mine)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4 *>(o + q)[e] = make_uint4(0, 0, 0, 0);
                    continue;
                }
                uint8_t *const line = ring + (n0 + (col0 >> 6)) % C::SLOTS * kSlot + row * 128;
                uint4 *unit[4];
                float g[4][8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    unit[e] = reinterpret_cast<uint4 *>(line + ((((col0 & 63) / 8 + e) ^ (row & 7)) << 4));
                    if (gate_smem) {
                        const uint4 u = *unit[e];
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            g[e][2 * i] = bf16_lo(w[i]);
                            g[e][2 * i + 1] = bf16_hi(w[i]);
                        }
                    } else {
                        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), w = u;
                        if (a.gate && mine) {
                            const float4 *gp = reinterpret_cast<const float4 *>(
                                static_cast<const float *>(a.gate) + go_ + q + e * 8);
                            u = gp[0];
                            w = gp[1];
                        }
                        g[e][0] = u.x; g[e][1] = u.y; g[e][2] = u.z; g[e][3] = u.w;
                        g[e][4] = w.x; g[e][5] = w.y; g[e][6] = w.z; g[e][7] = w.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = f[8 * e + i] * inv;
                    if (a.gate)
                        gate8(x, g[e]);
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = seen > 0 ? pack_bf16x2(x[2 * i], x[2 * i + 1]) : 0u;
                    *unit[e] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (t.nb > 0 && split == 1) {
                n0 += C::CH;
                fence_proxy_async_smem();
            }
            tc5_fence_before();
            if (named_bar_and(6, kSoft * 32, fixes)) {
                // this tile's columns again, before its successor but one uses them
                for (int i = threadIdx.x; i < 3 * D; i += kSoft * 32)
                    (&T.fix_at[it & 1][0][0])[i] = 0xFFFF;
                if (threadIdx.x == 0)
                    T.fixes[it & 1] = 0;
            }
            if (split > 1 && hf == 0) {
                T.mx[0][0][row] = m;
                T.lsum[1][0][row] = l;                // (the only tile's own have parity 0)
            }
            __syncwarp();
            if (lane == 0) {
                if (t.nb > 0) {
                    mbar_arrive_cluster(at_lead(&T.o_free));
                    mbar_arrive(&T.out_ready);
                }
                mbar_arrive_cluster(dsmem_addr(&T.t_empty[it & 1], lead));
                mbar_arrive_cluster(dsmem_addr(&T.t_empty[it & 1], lead + 1));
            }
            if (split > 1) {
                break;                                // one tile per cluster
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        // ------------------------------------------- join the shares of the blocks
        cluster_sync();
        const Tile t = T.tile[0];
        if (warp < kSoft && t.s >= 0 && !*abort) {
            // rows of this CTA's half that this share joins
            const int each = kM / split;
            for (int row = share * each + warp; row < (share + 1) * each; row += kSoft) {
                const int tok = row >> hp_log2, hd = row & (hp - 1);
                if (tok >= t.rows)
                    continue;
                const int head = (t.level << hp_log2) + hd, seen = t.seen0 + tok;
                const long long orow = t.row0 + tok;
                float top = -INFINITY, m[4], l = 0.f;
                for (int p = 0; p < split; ++p) {
                    m[p & 3] = ld_dsmem(dsmem_addr(&T.mx[0][0][row], 2 * p + half));
                    top = fmaxf(top, m[p & 3]);
                }
                const float ref = top == -INFINITY ? 0.f : top;
                for (int p = 0; p < split; ++p) {
                    m[p & 3] = ex2((m[p & 3] - ref) * a.scale_log2);
                    l += m[p & 3] * ld_dsmem(dsmem_addr(&T.lsum[1][0][row], 2 * p + half));
                }
                const float inv = 1.f / l;
                for (int j = lane * 4; j < D; j += 128) {
                    float f[4] = {};
                    for (int p = 0; p < split; ++p) {
                        const float4 x = ld_dsmem_v4(
                            dsmem_addr(reinterpret_cast<float *>(ring) + row * C::ST + j, 2 * p + half));
                        const float w = m[p & 3];
                        f[0] += w * x.x;
                        f[1] += w * x.y;
                        f[2] += w * x.z;
                        f[3] += w * x.w;
                    }
                    const long long go_ = orow * a.gs.tok + (long long)head * a.gs.head + j;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        f[i] = seen > 0 ? f[i] * inv : 0.f;
                        if (a.gate && seen > 0) {
                            const float g = a.gate_f32
                                                ? static_cast<const float *>(a.gate)[go_ + i]
                                                : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.gate)[go_ + i]);
                            f[i] *= sigmoid(g);
                        }
                    }
                    *reinterpret_cast<uint2 *>(a.out + orow * a.os.tok + (long long)head * a.os.head + j) =
                        make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
                }
            }
        }
        __syncwarp();
    }
    cluster_sync();
    tc5_fence_after();
    if (warp == 9) {
        if (*abort && lane == 0)
            seq_flag(a.sq, GATTN_STATUS_TIMEOUT);
        __syncwarp();
        tmem_free(tmem, kCols);
    }
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

bool encode(CUtensorMap *m, int rank, const void *base, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box)
{
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box,
                     es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const PromptAttnArgs &a, cudaStream_t s)
{
    using C = Cfg<D>;
    auto *fn = prompt_attn_kernel<D>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(fn, C::SMEM, done);
    if (e != cudaSuccess)
        return e;
    if (!encoder())
        return cudaErrorNotSupported;
    int sms = 0;
    e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    int hp_log2 = 0;
    while (hp_log2 < 7 && (a.H / a.Hk) % (2 << hp_log2) == 0)
        ++hp_log2;
    const int hp = 1 << hp_log2, tpt = kM >> hp_log2;
    CUtensorMap qm, km, vm, gm, om;
    const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.sq.total};
    const cuuint64_t qst[2] = {(cuuint64_t)a.qs.head * 2, (cuuint64_t)a.qs.tok * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)hp, (cuuint32_t)tpt};
    // without keys no sequence has blocks to copy: a map of one row stands in
    const bool keys = a.kv_rows > 0;
    const cuuint64_t kd[4] = {(cuuint64_t)D, keys ? (cuuint64_t)a.kv_rows : 1, keys ? (cuuint64_t)a.Hk : 1,
                              keys ? (cuuint64_t)a.kv_batch : 1};
    const cuuint64_t kst[3] = {keys ? (cuuint64_t)a.kt * 2 : 16, keys ? (cuuint64_t)a.kh * 2 : 16,
                               keys ? (cuuint64_t)a.kb * 2 : 16};
    const cuuint64_t vst[3] = {keys ? (cuuint64_t)a.vt * 2 : 16, keys ? (cuuint64_t)a.vh * 2 : 16,
                               keys ? (cuuint64_t)a.vb * 2 : 16};
    const cuuint32_t kb[4] = {64, 64, 1, 1}, vb[4] = {64, C::VK, 1, 1};
    const bool gate = a.gate && !a.gate_f32;
    const cuuint64_t gst[2] = {(cuuint64_t)a.gs.head * 2, (cuuint64_t)a.gs.tok * 2};
    const cuuint64_t ost[2] = {(cuuint64_t)a.os.head * 2, (cuuint64_t)a.os.tok * 2};
    if (!encode(&gm, 3, gate ? a.gate : a.q, qd, gate ? gst : qst, qb) || !encode(&om, 3, a.out, qd, ost, qb))
        return cudaErrorInvalidValue;
    if (!encode(&qm, 3, a.q, qd, qst, qb) || !encode(&km, 4, keys ? a.k : a.q, kd, kst, kb) ||
        !encode(&vm, 4, keys ? a.v : a.q, kd, vst, vb))
        return cudaErrorInvalidValue;
    // tiles of a pair, at most one partly filled per sequence
    const long long tiles =
        (a.sq.total / (2 * tpt) + std::min<long long>(a.sq.n, a.sq.total)) * (a.H >> hp_log2);
    const long long most = a.max_kv > 0 ? std::min(a.max_kv, a.kv_rows) : a.kv_rows;
    // Shares of the key blocks: as many as shorten the longest way through them, at
    // 256 keys a share or more.  Of clusters of 2, 4 and 8 CTAs 76, 36 and 15 fit at
    // once; later ones start where others end, so a share's time counts between its
    // waves and their whole number.  Measured with 16 heads of 256 over 4 KV heads, 8
    // rows a sequence, by 1, 2 and 4 shares: one sequence (4 tiles) over 1000 keys
    // 22.9, 20.2 and 18.0 us, over 16000 keys 206, 112 and 64 us; 8 sequences over
    // 8000 keys 111, 66 and 118 us; 16 sequences over 8000 keys 112, 129 and 196 us
    int split = 1;
    double best = 0;
    for (int x = 1; x <= 4; x *= 2) {
        const double fit = sms * (x == 1 ? 76 : x == 2 ? 36 : 15) / 152.0;
        const double waves = tiles / fit, time = (waves <= 1 ? 1 : (waves + std::ceil(waves)) / 2) / x;
        if (x == 1 || (most / x >= 256 && time < 0.92 * best)) {
            split = x;
            best = time;
        }
    }
    const long long clusters = split == 1 ? std::min<long long>(tiles, sms / 2) : tiles;
    if (tiles * 2 * split > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2 * split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(clusters * 2 * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, fn, a, qm, km, vm, gm, om, hp_log2, split);
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttnArgs &a, cudaStream_t s)
{
    switch (a.d) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    case 192: return launch<192>(a, s);
    default: return launch<256>(a, s);
    }
}

}  // namespace gattn
