// prompt_attn.cu -- causal attention of packed prompt rows with grouped heads and
// the sigmoid output gate, on the tensor cores.
//
// A CTA owns 128 query rows: 128/hp consecutive tokens of one sequence times hp
// query heads of one KV group (hp: the power of two in the group's size), so that
// a tile of keys serves every head it can.  It walks the keys it sees in blocks
// of 128 with the running maximum m and sum l of the softmax (base 2):
//   S = Q K^T,  p = 2^(c (s - m)),  l <- l a + sum p,  O <- O a + P V,
// a = 2^(c (m_old - m)).  S and O stay in tensor memory; P goes back into S's
// columns as bf16 (one rounding per probability) and is the A operand of P V.
// The reference m of a row only moves when its maximum has grown by more than 2^8
// (p <= 256 keeps its relative precision in bf16 and in the fp32 sums), so O is
// rescaled a few times per row instead of once per block.
//
// Warps 0-3 softmax and epilogue (a thread per row), 4 copies, 5 issues the MMAs,
// 6-7 look through the values of blocks that some row sees only part of: a value
// that is not finite would spoil rows that do not see it (0 * NaN), so it is
// replaced by zero there, and the rows that do see it get it back at the end.
#include <algorithm>

#include <cudaTypedefs.h>

#include "seq.cuh"
#include "tc5.cuh"

namespace gattn {

namespace {

constexpr int kThreads = 256;
constexpr int kM = 128;          // query rows of a tile
constexpr int kN = 128;          // keys of a block
constexpr int kSlot = 16384;     // bytes of a ring slot
constexpr float kGrow = 8.f;     // log2 growth of a row's maximum that moves its reference

template <int D>
struct Cfg {
    static constexpr int NS = D > 128 ? 2 : 1;               // score buffers
    static constexpr int CH = D / 64;                        // 64-element chunks of a head
    static constexpr int VK = D == 64 ? 128 : (D == 128 ? 64 : 32);   // keys per value slot
    static constexpr int NV = kN / VK;                       // value slots per block
    static constexpr int QB = kM * D * 2;
    static constexpr int SLOTS = D == 256 ? 10 : (D == 192 ? 10 : (D == 128 ? 5 : 6));
    static constexpr int COLS = D > 128 ? 512 : 256;         // TMEM columns
    static constexpr int O_COL = NS * kN;
    static_assert(O_COL + D <= COLS, "TMEM");
    struct Tables {              // behind the ring
        uint64_t full[SLOTS], empty[SLOTS];
        uint64_t part[SLOTS];    // a value slot that warps 6-7 look through has landed
        uint64_t q_full, q_done, g_full, o_done, s_full[2], p_ready[2], pv_done;
        uint32_t tmem;
        int abort, fixes;
        int s, level;            // the tile: sequence and place, or s < 0
        // per value column, first key (from the first partly seen block on) that
        // holds NaN, +inf, -inf; 0xFFFF: none
        uint16_t fix_at[3][D];
    };
    static constexpr int SMEM = QB + SLOTS * kSlot + (int)sizeof(Tables);
    // two CTAs of up to 128 elements share an SM (1 KB of each is the system's)
    static_assert(SMEM <= (D > 128 ? 227 : 113) * 1024, "shared memory");
};

// What a CTA works on.
struct Tile {
    int row0, rows;              // packed row of its first token, tokens it owns
    int slot, kv0;               // batch row and first key row of the sequence
    int seen0;                   // keys the first token sees (may be <= 0)
    int nb;                      // key blocks
};

// Sequence and level (tile within the sequence) of the rank-th tile, tiles in
// order of falling level, so that the longest causal rows start first.  Warp 0.
__device__ void find_tile(const SeqArgs &q, int tpt, long long rank, int &s_out, int &level_out)
{
    const int lane = threadIdx.x & 31;
    auto tiles = [&](int s) {
        int r0, len;
        seq_rows(q, s, r0, len);
        return (len + tpt - 1) / tpt;
    };
    const int mine = lane < q.n ? tiles(lane) : 0;      // the first 32 stay in registers
    int most = mine;
    for (int s = lane + 32; s < q.n; s += 32)
        most = max(most, tiles(s));
    most = __reduce_max_sync(0xffffffffu, most);
    // tiles at `level` or above
    auto above = [&](int level) {
        int c = max(0, mine - level);
        for (int s = lane + 32; s < q.n; s += 32)
            c += max(0, tiles(s) - level);
        return (long long)__reduce_add_sync(0xffffffffu, c);
    };
    s_out = -1;
    level_out = 0;
    if (rank >= above(0))
        return;
    int lo = 0, hi = most - 1;                          // above(lo) > rank
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (above(mid) > rank)
            lo = mid;
        else
            hi = mid - 1;
    }
    int idx = (int)(rank - above(lo + 1));
    for (int s0 = 0; s0 < q.n; s0 += 32) {
        const int s = s0 + lane;
        const bool has = s < q.n && (s0 ? tiles(s) : mine) > lo;
        const unsigned m = __ballot_sync(0xffffffffu, has);
        const int c = __popc(m);
        if (idx < c) {
            // the idx-th set bit
            unsigned x = m;
            for (int i = 0; i < idx; ++i)
                x &= x - 1;
            s_out = s0 + __ffs(x) - 1;
            level_out = lo;
            return;
        }
        idx -= c;
    }
}

// 16-bit minimum in shared memory (no such atomic exists)
__device__ void atomic_min16(uint16_t *p, uint32_t v)
{
    unsigned *w = reinterpret_cast<unsigned *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
    const int sh = (reinterpret_cast<uintptr_t>(p) & 2) * 8;
    unsigned old = *(volatile unsigned *)w;
    while (((old >> sh) & 0xFFFFu) > v) {
        const unsigned next = (old & ~(0xFFFFu << sh)) | (v << sh);
        const unsigned got = atomicCAS(w, old, next);
        if (got == old)
            break;
        old = got;
    }
}

__device__ __forceinline__ bool not_finite16(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

template <int D>
__global__ void __launch_bounds__(kThreads, D > 128 ? 1 : 2)
prompt_attn_kernel(const __grid_constant__ PromptAttnArgs a, const __grid_constant__ CUtensorMap qmap,
                   const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap gmap, int hp_log2)
{
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *const qs = smem, *const ring = smem + C::QB;
    typename C::Tables &T = *reinterpret_cast<typename C::Tables *>(smem + C::QB + C::SLOTS * kSlot);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hp = 1 << hp_log2, tpt = kM >> hp_log2;
    const int groups = a.H >> hp_log2;
    const int hg = blockIdx.x % groups;
    const long long rank = blockIdx.x / groups;
    const int head0 = hg << hp_log2, kvh = head0 / (a.H / a.Hk);

    if (warp == 0) {
        int s, level;
        find_tile(a.sq, tpt, rank, s, level);
        if (lane == 0) {
            T.s = s;
            T.level = level;
        }
    } else if (warp == 4) {
        if (lane == 0) {
            for (int i = 0; i < C::SLOTS; ++i) {
                mbar_init(&T.full[i], 1);
                mbar_init(&T.empty[i], 1);
                mbar_init(&T.part[i], 1);
            }
            mbar_init(&T.q_full, 1);
            mbar_init(&T.q_done, 1);
            mbar_init(&T.o_done, 1);
            mbar_init(&T.g_full, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&T.s_full[i], 1);
                mbar_init(&T.p_ready[i], 128);
            }
            mbar_init(&T.pv_done, 1);
            T.abort = 0;
            T.fixes = 0;
            fence_mbar_init();
            prefetch_tensormap(&qmap);
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
    } else if (warp >= 6) {
        for (int i = threadIdx.x - 192; i < 3 * D; i += 64)
            (&T.fix_at[0][0])[i] = 0xFFFF;
    }
    __syncthreads();
    const int s = T.s;
    if (s < 0)
        return;
    Tile t;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    t.row0 = r0 + T.level * tpt;
    t.rows = min(tpt, len - T.level * tpt);
    long long kv0 = 0, keys;
    bool ok;
    t.slot = 0;
    if (a.pos) {
        t.slot = a.sq.slots ? a.sq.slots[s] : s;
        const long long p0 = a.pos[s];
        keys = p0 + len;
        ok = t.slot >= 0 && t.slot < a.kv_batch && p0 >= 0 && keys <= a.kv_rows;
    } else {
        kv0 = a.cu_kv[s];
        const long long kv1 = a.cu_kv[s + 1];
        keys = kv1 - kv0;
        ok = kv0 >= 0 && kv1 >= kv0 && kv1 <= a.kv_rows;
    }
    if (!ok && threadIdx.x == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    t.kv0 = (int)kv0;
    // |keys - len| < 2^31: both are counts of rows
    t.seen0 = ok ? (int)(keys - len) + T.level * tpt + 1 : -(1 << 30);
    const int seen_last = t.seen0 + t.rows - 1;
    t.nb = seen_last > 0 ? (seen_last + kN - 1) / kN : 0;

    const int tok = threadIdx.x >> hp_log2, hd = threadIdx.x & (hp - 1);   // of warps 0-3
    if (t.nb == 0) {
        if (threadIdx.x < kM && tok < t.rows) {
            uint4 *o = reinterpret_cast<uint4 *>(a.out + (long long)(t.row0 + tok) * a.os.tok +
                                                 (long long)(head0 + hd) * a.os.head);
            for (int i = 0; i < D / 8; ++i)
                o[i] = make_uint4(0, 0, 0, 0);
        }
        return;
    }
    if (warp == 5)
        tmem_alloc(&T.tmem, C::COLS);
    __syncthreads();
    tc5_fence_after();
    const uint32_t tmem = T.tmem;
    volatile int *abort = &T.abort;
    // blocks from here on some row of the tile sees only in part
    const int part0 = t.seen0 > 0 ? t.seen0 / kN : 0;

    if (warp == 4) {
        if (lane == 0) {
            mbar_arrive_expect_tx(&T.q_full, C::QB);
            for (int c = 0; c < C::CH; ++c)
                tma3d(smem_u32(qs) + c * (kM * 128), &qmap, c * 64, head0, t.row0, &T.q_full);
            int n = 0;                 // slots filled so far
            uint32_t in_part = 0, pphase = 0;   // per slot: its last load signals part[]; part[]'s phase
            bool go = true;
            // waits for the next slot and announces `bytes` on the barrier its load signals
            auto fill = [&](uint32_t bytes, bool part, uint64_t *&bar) -> uint32_t {
                const int sl = n % C::SLOTS;
                if (n >= C::SLOTS && !tc5_wait(&T.empty[sl], ((n / C::SLOTS) - 1) & 1, abort)) {
                    go = false;
                    return 0;
                }
                bar = part ? &T.part[sl] : &T.full[sl];
                in_part = part ? in_part | 1u << sl : in_part & ~(1u << sl);
                pphase ^= part ? 1u << sl : 0u;
                mbar_arrive_expect_tx(bar, bytes);
                ++n;
                return smem_u32(ring) + sl * kSlot;
            };
            uint64_t *bar = nullptr;
            auto load_k = [&](int b) {
                for (int c = 0; c < C::CH && go; ++c) {
                    const uint32_t p = fill(kN * 128, false, bar);
                    if (go)
                        tma4d(p, &kmap, c * 64, t.kv0 + b * kN, kvh, t.slot, bar);
                }
            };
            auto load_v = [&](int b) {
                for (int g = 0; g < C::NV && go; ++g) {
                    const uint32_t p = fill(C::VK * D * 2, b >= part0, bar);
                    if (go)
                        for (int c = 0; c < C::CH; ++c)
                            tma4d(p + c * (C::VK * 128), &vmap, c * 64, t.kv0 + b * kN + g * C::VK, kvh,
                                  t.slot, bar);
                }
            };
            if (C::NS == 2) {
                load_k(0);
                for (int b = 1; b < t.nb && go; ++b) {
                    load_k(b);
                    load_v(b - 1);
                }
                load_v(t.nb - 1);
            } else {
                for (int b = 0; b < t.nb && go; ++b) {
                    load_k(b);
                    load_v(b);
                }
            }
            // a bf16 gate tile takes the queries' place once the last scores are done
            int none = 0;
            if (a.gate && !a.gate_f32 && go && tc5_wait(&T.q_done, 0, abort)) {
                mbar_arrive_expect_tx(&T.g_full, C::QB);
                for (int c = 0; c < C::CH; ++c)
                    tma3d(smem_u32(qs) + c * (kM * 128), &gmap, c * 64, head0, t.row0, &T.g_full);
                tc5_wait(&T.g_full, 0, &none);
            }
            // every copy has landed before the shared memory is given up, also when
            // a wait ran out
            {
                tc5_wait(&T.q_full, 0, &none);
                for (int i = max(0, n - C::SLOTS); i < n; ++i) {
                    const int sl = i % C::SLOTS;
                    if (in_part >> sl & 1)
                        tc5_wait(&T.part[sl], (pphase >> sl & 1) ^ 1, &none);
                    else
                        tc5_wait(&T.full[sl], (i / C::SLOTS) & 1, &none);
                }
            }
        }
    } else if (warp == 5) {
        if (lane == 0) {
            constexpr uint32_t id_s = tc5_idesc(kM, kN, false), id_o = tc5_idesc(kM, D, true);
            int n = 0;                 // slots consumed so far
            bool go = tc5_wait(&T.q_full, 0, abort);
            auto scores = [&](int b) {
                const uint32_t d = tmem + (C::NS == 2 ? (b & 1) * kN : 0);
                for (int c = 0; c < C::CH && go; ++c, ++n) {
                    const int sl = n % C::SLOTS;
                    go = tc5_wait(&T.full[sl], (n / C::SLOTS) & 1, abort);
                    if (!go)
                        break;
                    const uint64_t da = tc5_desc(smem_u32(qs) + c * (kM * 128), 16, 1024);
                    const uint64_t db = tc5_desc(smem_u32(ring) + sl * kSlot, 16, 1024);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc5_mma_ss(d, da + 2 * k, db + 2 * k, id_s, c > 0 || k > 0);
                    tc5_commit(&T.empty[sl]);
                }
                if (go)
                    tc5_commit(&T.s_full[C::NS == 2 ? b & 1 : 0]);
                if (go && b == t.nb - 1)
                    tc5_commit(&T.q_done);
            };
            auto values = [&](int b) {
                const int pb = C::NS == 2 ? b & 1 : 0;
                go = go && tc5_wait(&T.p_ready[pb], (C::NS == 2 ? b >> 1 : b) & 1, abort);
                if (!go)
                    return;
                tc5_fence_after();
                const uint32_t p = tmem + pb * kN, d = tmem + C::O_COL;
                for (int g = 0; g < C::NV; ++g, ++n) {
                    const int sl = n % C::SLOTS;
                    go = tc5_wait(&T.full[sl], (n / C::SLOTS) & 1, abort);
                    if (!go)
                        return;
                    const uint64_t db = tc5_desc(smem_u32(ring) + sl * kSlot, C::VK * 128, 1024);
#pragma unroll
                    for (int k = 0; k < C::VK / 16; ++k)
                        tc5_mma_ts(d, p + (g * C::VK + k * 16) / 2, db + k * (2048 >> 4), id_o,
                                   b > 0 || g > 0 || k > 0);
                    tc5_commit(&T.empty[sl]);
                }
                tc5_commit(b == t.nb - 1 ? &T.o_done : &T.pv_done);
            };
            if (C::NS == 2) {
                scores(0);
                for (int b = 1; b < t.nb && go; ++b) {
                    scores(b);
                    values(b - 1);
                }
                values(t.nb - 1);
            } else {
                for (int b = 0; b < t.nb && go; ++b) {
                    scores(b);
                    values(b);
                }
            }
        }
    } else if (warp >= 6) {
        // look through the values of partly seen blocks
        int n = 0;
        uint32_t phase = 0;        // per slot: parity of its next part[] phase
        const int w = warp - 6;
        // slots are filled in the order K0 [K1 V0] [K2 V1] ... (two score buffers)
        // or K0 V0 K1 V1 ...: the first value slot of block b
        for (int b = part0; b < t.nb; ++b) {
            n = C::NS == 2 ? min(b + 2, t.nb) * C::CH + b * C::NV : (b + 1) * C::CH + b * C::NV;
            for (int g = 0; g < C::NV; ++g, ++n) {
                const int sl = n % C::SLOTS;
                bool go = tc5_wait(&T.part[sl], phase >> sl & 1, abort);
                phase ^= 1u << sl;
                uint4 *p = reinterpret_cast<uint4 *>(ring + sl * kSlot);
                constexpr int UNITS = C::VK * D / 8;
                static_assert(UNITS % 256 == 0, "four units a thread and turn");
                for (int i0 = w * 32 + lane; go && i0 < UNITS; i0 += 256) {
                    uint4 u[4];
                    bool hit = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        u[k] = p[i0 + 64 * k];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // a set exponent field is largest: one packed maximum finds it
                        const unsigned top = __vmaxu2(__vmaxu2(u[k].x & 0x7FFF7FFFu, u[k].y & 0x7FFF7FFFu),
                                                      __vmaxu2(u[k].z & 0x7FFF7FFFu, u[k].w & 0x7FFF7FFFu));
                        hit |= (top & 0xFFFFu) >= 0x7F80u || top >= 0x7F800000u;
                    }
                    if (!hit)
                        continue;
#pragma unroll 1
                    for (int i = i0; i < i0 + 256; i += 64) {
                        const uint4 v = p[i];
                        uint32_t x[4] = {v.x, v.y, v.z, v.w};
                        // 16-byte unit i: chunk of 64 columns, key row, unit within the
                        // row, swizzled by the row
                        const int c = i / (C::VK * 8), key = (i / 8) % C::VK, un = (i & 7) ^ (key & 7);
                        const int kidx = (b - part0) * kN + g * C::VK + key;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t h = (x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                            if (!not_finite16(h))
                                continue;
                            const int what = (h & 0x7F) ? 0 : (h >> 15) ? 2 : 1;
                            atomic_min16(&T.fix_at[what][c * 64 + un * 8 + e], kidx);
                            x[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
                        p[i] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    *(volatile int *)&T.fixes = 1;
                }
                fence_proxy_async_smem();
                named_bar_sync(1, 64);
                if (threadIdx.x == 6 * 32)
                    mbar_arrive(&T.full[sl]);
            }
        }
    } else {
        // ------------------------------------------------ softmax: a thread per row
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        const float c = a.scale_log2;
        const int seen = t.seen0 + tok;           // keys this row sees
        float m = -INFINITY;                      // the row's reference
        float l = 0.f;
        bool go = true;
        for (int b = 0; b < t.nb; ++b) {
            const int pb = C::NS == 2 ? b & 1 : 0;
            const uint32_t S = tmem + lanes + pb * kN;
            go = tc5_wait(&T.s_full[pb], (C::NS == 2 ? b >> 1 : b) & 1, abort);
            go = __all_sync(0xffffffffu, go);
            if (!go)
                break;
            tc5_fence_after();
            const int lim = b >= part0 ? seen - b * kN : kN;    // visible columns
            uint32_t r[32];
            float mx = -INFINITY;
#pragma unroll
            for (int q = 0; q < kN / 32; ++q) {
                tmem_ld32(r, S + q * 32);
                tmem_wait_ld();
                if (b >= part0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        mx = fmaxf(mx, q * 32 + i < lim ? __uint_as_float(r[i]) : -INFINITY);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        mx = fmaxf(mx, __uint_as_float(r[i]));
                }
            }
            // move the reference on the first block and when the maximum outgrows it
            float alpha = 1.f;
            const bool move = mx > m && (m == -INFINITY || (mx - m) * c > kGrow);
            if (move) {
                alpha = m == -INFINITY ? 0.f : ex2((m - mx) * c);
                m = mx;
            }
            if (b > 0 && __any_sync(0xffffffffu, move)) {
                go = __all_sync(0xffffffffu, tc5_wait(&T.pv_done, (b - 1) & 1, abort));
                if (!go)
                    break;
                tc5_fence_after();
                l *= alpha;
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    tmem_ld32(r, tmem + lanes + C::O_COL + q * 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                    tmem_st32(tmem + lanes + C::O_COL + q * 32, r);
                }
            }
            // a row without a visible key so far has reference -inf: against 0
            // its masked scores give p = 0
            const float ref = m == -INFINITY ? 0.f : m;
            const uint64_t nref = pack2(-ref, -ref), cc = pack2(c, c);
            uint64_t sum = 0;
#pragma unroll
            for (int q = 0; q < kN / 32; ++q) {
                uint32_t pk[16];
                tmem_ld32(r, S + q * 32);
                tmem_wait_ld();
                if (b >= part0) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (q * 32 + i >= lim)
                            r[i] = 0xFF800000u;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t x = mul2(
                        add2(pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), nref), cc);
                    float e0, e1;
                    unpack2(x, e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    sum = add2(sum, pack2(e0, e1));
                    pk[i] = pack_bf16x2(e0, e1);
                }
                tmem_st16(S + q * 16, pk);
            }
            float s0, s1;
            unpack2(sum, s0, s1);
            l += s0 + s1;
            tmem_wait_st();
            tc5_fence_before();
            mbar_arrive(&T.p_ready[pb]);
        }
        // ------------------------------------------------------------- epilogue
        // a barrier of its own: by now the last phases of pv_done may both be over,
        // and a parity does not tell phase n from n - 2
        go = go && tc5_wait(&T.o_done, 0, abort);
        const bool gate_here = a.gate && !a.gate_f32;
        if (gate_here)
            go = go && tc5_wait(&T.g_full, 0, abort);
        go = __all_sync(0xffffffffu, go);
        if (go) {
            tc5_fence_after();
            const bool mine = tok < t.rows;
            const float inv = seen > 0 ? 1.f / l : 0.f;
            const bool fixes = *(volatile int *)&T.fixes != 0;
            const long long row = t.row0 + tok;
            __nv_bfloat16 *o = a.out + row * a.os.tok + (long long)(head0 + hd) * a.os.head;
            const long long go_ = row * a.gs.tok + (long long)(head0 + hd) * a.gs.head;
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
                uint32_t r[32];
                tmem_ld32(r, tmem + lanes + C::O_COL + q * 32);
                tmem_wait_ld();
                if (!mine)
                    continue;
                float f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    f[i] = seen > 0 ? __uint_as_float(r[i]) * inv : 0.f;
                if (fixes) {
                    const int from = seen - part0 * kN;   // keys seen in the partly seen blocks
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        // values that are not finite, for the rows that see them
                        if (from > T.fix_at[0][q * 32 + i])
                            f[i] = __int_as_float(0x7fffffff);
                        if (from > T.fix_at[1][q * 32 + i])
                            f[i] += INFINITY;
                        if (from > T.fix_at[2][q * 32 + i])
                            f[i] -= INFINITY;
                    }
                }
                if (a.gate && seen > 0) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float g[8];
                        if (a.gate_f32) {
                            const float4 *gp = reinterpret_cast<const float4 *>(
                                static_cast<const float *>(a.gate) + go_ + q * 32 + e * 8);
                            const float4 u = gp[0], w = gp[1];
                            g[0] = u.x; g[1] = u.y; g[2] = u.z; g[3] = u.w;
                            g[4] = w.x; g[5] = w.y; g[6] = w.z; g[7] = w.w;
                        } else {
                            // chunk of 64 elements, row, 16-byte unit swizzled by the row
                            const int r = threadIdx.x;
                            ld_bf16x8(reinterpret_cast<const __nv_bfloat16 *>(
                                          qs + (q >> 1) * (kM * 128) + r * 128 +
                                          ((((q & 1) * 4 + e) ^ (r & 7)) << 4)),
                                      g);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            f[e * 8 + i] = __fdividef(f[e * 8 + i], 1.f + __expf(-g[i]));
                    }
                }
                uint4 *ov = reinterpret_cast<uint4 *>(o + q * 32);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    ov[e] = make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                       pack_bf16x2(f[8 * e + 4], f[8 * e + 5]),
                                       pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
            }
        }
        tc5_fence_before();
    }
    __syncwarp();
    __syncthreads();
    if (warp == 5) {
        tc5_fence_after();
        if (*abort) {
            // the MMAs that were issued are done before their memory is freed
            if (lane == 0) {
                int none = 0;
                mbar_init(&T.q_full, 1);
                fence_mbar_init();
                tc5_commit(&T.q_full);
                tc5_wait(&T.q_full, 0, &none);
                seq_flag(a.sq, GATTN_STATUS_TIMEOUT);
            }
            __syncwarp();
        }
        tmem_free(tmem, C::COLS);
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
    const cudaError_t attr = allow_smem(fn, C::SMEM, done);
    if (attr != cudaSuccess)
        return attr;
    if (!encoder())
        return cudaErrorNotSupported;
    int hp_log2 = 0;
    while (hp_log2 < 7 && (a.H / a.Hk) % (2 << hp_log2) == 0)
        ++hp_log2;
    const int hp = 1 << hp_log2, tpt = kM >> hp_log2;
    CUtensorMap qm, km, vm, gm;
    const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)a.H, (cuuint64_t)a.sq.total};
    const cuuint64_t qst[2] = {(cuuint64_t)a.qs.head * 2, (cuuint64_t)a.qs.tok * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)hp, (cuuint32_t)tpt};
    const cuuint64_t kd[4] = {(cuuint64_t)D, (cuuint64_t)a.kv_rows, (cuuint64_t)a.Hk, (cuuint64_t)a.kv_batch};
    const cuuint64_t kst[3] = {(cuuint64_t)a.kt * 2, (cuuint64_t)a.kh * 2, (cuuint64_t)a.kb * 2};
    const cuuint64_t vst[3] = {(cuuint64_t)a.vt * 2, (cuuint64_t)a.vh * 2, (cuuint64_t)a.vb * 2};
    const cuuint32_t kb[4] = {64, kN, 1, 1}, vb[4] = {64, C::VK, 1, 1};
    const bool gate = a.gate && !a.gate_f32;
    const cuuint64_t gst[2] = {(cuuint64_t)a.gs.head * 2, (cuuint64_t)a.gs.tok * 2};
    if (!encode(&gm, 3, gate ? a.gate : a.q, qd, gate ? gst : qst, qb))
        return cudaErrorInvalidValue;
    if (!encode(&qm, 3, a.q, qd, qst, qb) || !encode(&km, 4, a.k, kd, kst, kb) ||
        !encode(&vm, 4, a.v, kd, vst, vb))
        return cudaErrorInvalidValue;
    // at most one partly filled tile per sequence
    const long long tiles = a.sq.total / tpt + std::min<long long>(a.sq.n, a.sq.total);
    const long long grid = tiles * (a.H >> hp_log2);
    if (grid > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, fn, a, qm, km, vm, gm, hp_log2);
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
