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
// running maximum and sum, so that no warp waits for another until the part ends; a warp
// of a group has 16 of the tile's rows.  The scores stay in registers: as the matrix
// instruction leaves them they are what the product with the values takes.  p goes into
// that product as two bf16 numbers, 16 bits of it: 8 bits alone would be an error of
// the size of the output's own rounding, and the matrix units have the time.
// The reference m of a row moves only when the maximum outgrows it by 2^8.
#include <cudaTypedefs.h>

#include "paged_ring.cuh"

namespace gattn {

using namespace paged;

namespace {

template <int D, int MT>
struct Cfg {
    static constexpr int M = 16 * MT, NS = MT == 4 ? 2 : 4, CW = NS * MT, NP = D * MT == 1024 || (D == 64 && MT == 4) ? 2 : 4, THREADS = (CW + NP) * 32;
    static constexpr int ROUNDS = CW * D >= 1024 ? CW * D / (MT == 1 ? 1024 : 512) : 1, DR = D / ROUNDS;   // columns joined at once
    static constexpr int XROW = DR + 8;                // floats of a joined row: rows 8 banks apart
    static constexpr int XB = CW * 16 * XROW * 4;
    static constexpr int U = kUnit<D>, UNIT = U * D * 4;
    static constexpr int FIXED = 2 * M * D * 2 + XB + 2048 + 1024;
    static constexpr int FIT = (227 * 1024 - FIXED) / UNIT;
    static constexpr int SLOTS = (FIT > 12 ? 12 : FIT) / (NS > NP ? NS : NP) * (NS > NP ? NS : NP);
    static constexpr int SMEM = SLOTS * UNIT + 2 * M * D * 2 + XB + 1024;
    using R = Ring<D, M, true, SLOTS, NP, MT, CW>;
    static_assert(SMEM + 2048 <= 227 * 1024 && SLOTS >= 4 && DR % 8 == 0 && DR * ROUNDS == D && XROW % 32 == 8, "");
};

// Floats of a partial result: rows, then their m and sums.
template <int D, int M>
constexpr int kPartial = M * (D + 2);

// What the join needs to know of a CTA's last segment.
struct Rec {
    int live, slot, last, r0, rowf, hf, nrows, hk;
};

// Four columns of a row's gate before its sigmoid.
__device__ __forceinline__ float4 gate4(const PagedAttnArgs &a, long long row, int head, int col)
{
    if (!a.gate)
        return make_float4(0.f, 0.f, 0.f, 0.f);
    const long long at = row * a.gs.tok + head * a.gs.head + col;
    if (a.gate_f32)
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(a.gate) + at);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(a.gate) + at);
    return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

// Four finished columns of a row: divided, gated, rounded once.
__device__ __forceinline__ void finish4(const PagedAttnArgs &a, long long row, int head, int col, float4 o, float l,
                                        const float4 &g)
{
    const float inv = l == 0.f ? 0.f : 1.f / l;        // no position seen: zeros
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    // a row that saw nothing stays zero whatever its gate holds
    if (a.gate && l != 0.f) {
        o.x /= 1.f + __expf(-g.x), o.y /= 1.f + __expf(-g.y);
        o.z /= 1.f + __expf(-g.z), o.w /= 1.f + __expf(-g.w);
    }
    *reinterpret_cast<uint2 *>(a.out + row * a.os.tok + head * a.os.head + col) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

__device__ __forceinline__ float lse_of(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718f;
}

template <int D, int MT>
__global__ void __launch_bounds__(Cfg<D, MT>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, int min_units)
{
    using C = Cfg<D, MT>;
    using R = typename C::R;
    constexpr int M = C::M, NS = C::NS, CW = C::CW, U = C::U, DR = C::DR;
    extern __shared__ uint8_t raw[];
    __shared__ R ring;
    __shared__ float red_m[CW * 16], red_l[CW * 16], row_m[M], row_l[M];
    uint8_t *units = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = units + C::SLOTS * C::UNIT;
    float *const xb = reinterpret_cast<float *>(qbuf + 2 * M * D * 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.H / a.Hk;
    if (threadIdx.x == 0) {
        ring.init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    // (the barriers of the plan make the ring's known)
    const Run run = plan_run<C::THREADS, M, U>(a, group, min_units, [&](int, const SeqUnits &u) {
        seq_flag(a.sq, GATTN_STATUS_RANGE);
        for (long long i = 0; i < (long long)u.len * a.H; ++i) {
            const long long row = u.r0 + i / a.H;
            const int h = (int)(i % a.H);
            for (int c = 0; c < D; c += 8)
                *reinterpret_cast<uint4 *>(a.out + row * a.os.tok + h * a.os.head + c) = make_uint4(0, 0, 0, 0);
            if (a.lse)
                a.lse[row * a.H + h] = -INFINITY;
        }
    });
    Rec *const recs = reinterpret_cast<Rec *>(static_cast<float *>(a.ws) + 2ll * kMaxCtas * kPartial<D, M>);
    if (run.x0 >= run.x1) {
        if (threadIdx.x == 0)
            recs[blockIdx.x].live = 0;
        return;
    }
    if (warp >= CW) {
        Rec rec{};
        produce(a, ring, units, qbuf, &kmap, &vmap, run, group, warp - CW, [&](const Part &p, int last) {
            rec = {1, p.slot, last, p.r0, p.rowf, p.hf, p.nrows, p.hk};
        });
        if (warp == CW && lane == 0)
            recs[blockIdx.x] = rec;
        return;
    }
    // --------------------------------------------------------------- consumers
    const int st = warp / MT, mt = warp % MT;           // unit group, rows
    const int g = lane >> 2, cq = lane & 3;
    const int btl = box_log2(a.pg.page, U), box = (1 << btl) * D * 2, dbs = (1 << btl) * 128;
    long long it = 0;                                   // units of the CTA before this part
    for (int parts = 0;; ++parts) {
        const int b = parts & 1;
        // one thread decides for all, so that every warp meets the same barriers
        if (threadIdx.x == 0)
            ring.go = ring_wait(&ring.qfull[b], (uint32_t)((parts >> 1) & 1), &ring.abort, a.sq) && ring.part[b].live;
        named_bar_sync(1, CW * 32);
        if (!ring.go)
            break;
        ring_wait(&ring.qfull[b], (uint32_t)((parts >> 1) & 1), &ring.abort, a.sq);
        const Part p = ring.part[b];
        const int first_row = p.p0 + p.rowf;            // the last position that every row sees
        const int last_row = p.p0 + p.rowf + (p.hf + p.nrows - 1) / group;
        int lim[2];                                     // of this lane's rows
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const int i = mt * 16 + g + 8 * hr;
            lim[hr] = i < p.nrows ? first_row + (p.hf + i) / group : -1;
        }
        float O[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                O[j][e] = 0.f;
        const int count = max(p.u1 - p.u0, 0);
        const uint32_t qrow = smem_u32(qbuf) + b * R::QB + (mt * 16 + (lane & 15)) * (D * 2);
        // this group's units: those of index st modulo NS within the CTA
        for (int n = (int)((st - it) & (NS - 1)); n < count; n += NS) {
            const long long idx = it + n;
            const int slot = (int)(idx % R::SLOTS);
            const bool ok = ring_wait(&ring.full[slot], (uint32_t)((idx / R::SLOTS) & 1), &ring.abort, a.sq);
            const uint32_t ks = smem_u32(units) + slot * C::UNIT, vs = ks + R::PLANE;
            const int t0 = (p.u0 + n) * U;
            if (ok && mt * 16 < p.nrows) {
                const unsigned there = ring.ok[slot];
                // ---- scores
                constexpr int CHAINS = U == 16 ? 2 : 1;  // sums of independent products
                float sc[CHAINS][U / 8][4];
#pragma unroll
                for (int c = 0; c < CHAINS; ++c)
#pragma unroll
                    for (int j = 0; j < U / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[c][j][e] = 0.f;
                // a lane's row of the unit for the keys (kt) and for the values (vt)
                const int kt = (lane & 7) + 8 * (lane >> 4), vt = lane & 15;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t qa[4];
                    ldsm_x4(qa, qrow + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
                    const int ch = 2 * k + ((lane >> 3) & 1);
#pragma unroll
                    for (int q = 0; q < U / 16; ++q) {
                        const int in = (q * 16) >> btl, at = (q * 16) & ((1 << btl) - 1);
                        uint32_t kb[4];
                        ldsm_x4(kb, ks + in * box + (ch >> 3) * dbs + (at + kt) * 128 + (((ch & 7) ^ (lane & 7)) << 4));
                        mma(sc[k % CHAINS][2 * q], qa, kb[0], kb[1]);
                        mma(sc[k % CHAINS][2 * q + 1], qa, kb[2], kb[3]);
                    }
                }
#pragma unroll
                for (int j = 0; j < U / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[0][j][e] = (CHAINS == 2 ? sc[0][j][e] + sc[CHAINS - 1][j][e] : sc[0][j][e]) * a.scale_log2;
                // ---- what a row does not see
                const bool part = t0 + U - 1 > first_row;
                if (part || there != (1u << (U >> btl)) - 1u) {
#pragma unroll
                    for (int j = 0; j < U / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = j * 8 + 2 * cq + (e & 1);
                            if (t0 + t > lim[e >> 1] || !((there >> (t >> btl)) & 1u))
                                sc[0][j][e] = -INFINITY;
                        }
                }
                // ---- running maximum; rows of a quad of lanes
                float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < U / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        mx[e >> 1] = fmaxf(mx[e >> 1], sc[0][j][e]);
                bool grow = false;
                float to[2];
#pragma unroll
                for (int hr = 0; hr < 2; ++hr) {
                    mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 1));
                    mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 2));
                    to[hr] = mx[hr] > m[hr] + 8.f ? mx[hr] : m[hr];
                    grow |= to[hr] != m[hr];
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int hr = 0; hr < 2; ++hr) {
                        const float f = to[hr] == m[hr] ? 1.f : exp2f(m[hr] - to[hr]);
                        m[hr] = to[hr];
                        l[hr] *= f;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            O[j][2 * hr] *= f;
                            O[j][2 * hr + 1] *= f;
                        }
                    }
                }
                const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
                // p, in place of the scores; hi + lo are its first 16 bits
                uint32_t hi[U / 8][2], lo[U / 8][2];
#pragma unroll
                for (int j = 0; j < U / 8; ++j)
#pragma unroll
                    for (int hr = 0; hr < 2; ++hr) {
                        const float p0 = exp2f(sc[0][j][2 * hr] - base[hr]), p1 = exp2f(sc[0][j][2 * hr + 1] - base[hr]);
                        l[hr] += p0 + p1;
                        sc[0][j][2 * hr] = p0;
                        sc[0][j][2 * hr + 1] = p1;
                        hi[j][hr] = pack_bf16x2(p0, p1);
                        lo[j][hr] = pack_bf16x2(p0 - bf16_lo(hi[j][hr]), p1 - bf16_hi(hi[j][hr]));
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
                // ---- O += p V
                if (!odd) {
#pragma unroll
                    for (int q = 0; q < U / 16; ++q) {
                        const uint32_t h[4] = {hi[2 * q][0], hi[2 * q][1], hi[2 * q + 1][0], hi[2 * q + 1][1]};
                        const uint32_t w[4] = {lo[2 * q][0], lo[2 * q][1], lo[2 * q + 1][0], lo[2 * q + 1][1]};
                        const int in = (q * 16) >> btl, at = (q * 16) & ((1 << btl) - 1);
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) {
                            const int ch = 2 * j + (lane >> 4);
                            uint32_t vb[4];
                            ldsm_x4_trans(vb, vs + in * box + (ch >> 3) * dbs + (at + vt) * 128 + (((ch & 7) ^ (lane & 7)) << 4));
                            mma(O[2 * j], h, vb[0], vb[1]);
                            mma(O[2 * j + 1], h, vb[2], vb[3]);
                            mma(O[2 * j], w, vb[0], vb[1]);
                            mma(O[2 * j + 1], w, vb[2], vb[3]);
                        }
                    }
                } else {
                    // position by position, each row only what it sees
#pragma unroll 1
                    for (int t = 0; t < U; ++t) {
                        float pt[2] = {0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < U / 8; ++j)
                            if (j == t >> 3)
#pragma unroll
                                for (int hr = 0; hr < 2; ++hr)
                                    pt[hr] = t & 1 ? sc[0][j][2 * hr + 1] : sc[0][j][2 * hr];
#pragma unroll
                        for (int hr = 0; hr < 2; ++hr)
                            pt[hr] = __shfl_sync(0xffffffffu, pt[hr], (lane & ~3) | ((t & 7) >> 1));
                        const uint32_t vrow = vs + (t >> btl) * box + (t & ((1 << btl) - 1)) * 128;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            uint32_t v;
                            asm volatile("ld.shared.u32 %0, [%1];"
                                         : "=r"(v)
                                         : "r"(vrow + (j >> 3) * dbs + (((j & 7) ^ (t & 7)) << 4) + cq * 4));
#pragma unroll
                            for (int hr = 0; hr < 2; ++hr)
                                if (t0 + t <= lim[hr] && ((there >> (t >> btl)) & 1u)) {
                                    O[j][2 * hr] = fmaf(pt[hr], bf16_lo(v), O[j][2 * hr]);
                                    O[j][2 * hr + 1] = fmaf(pt[hr], bf16_hi(v), O[j][2 * hr + 1]);
                                }
                        }
                    }
                }
                if (part)
                    fence_proxy_async_smem();           // zeros before the next copy into this slot
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ring.empty[slot]);
        }
        it += count;
        if (lane == 0)
            mbar_arrive(&ring.qempty[b]);
        // ---- join the groups
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
            l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
            if (cq == 0) {
                red_m[warp * 16 + g + 8 * hr] = m[hr];
                red_l[warp * 16 + g + 8 * hr] = l[hr];
            }
        }
        named_bar_sync(1, CW * 32);
        float f[2];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            float top = -INFINITY;
#pragma unroll
            for (int q = 0; q < NS; ++q)
                top = fmaxf(top, red_m[(q * MT + mt) * 16 + g + 8 * hr]);
            f[hr] = m[hr] == top ? 1.f : exp2f(m[hr] - top);
        }
        float *const slot = static_cast<float *>(a.ws) + (2ll * blockIdx.x + p.slot) * kPartial<D, M>;
        if (threadIdx.x < M) {
            const int i = threadIdx.x;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int q = 0; q < NS; ++q)
                top = fmaxf(top, red_m[(q * MT + i / 16) * 16 + i % 16]);
#pragma unroll
            for (int q = 0; q < NS; ++q) {
                const float mq = red_m[(q * MT + i / 16) * 16 + i % 16];
                sum += red_l[(q * MT + i / 16) * 16 + i % 16] * (mq == top ? 1.f : exp2f(mq - top));
            }
            row_m[i] = top;
            row_l[i] = sum;
            if (!p.whole) {
                slot[M * D + i] = top;
                slot[M * D + M + i] = sum;
            } else if (a.lse && i < p.nrows) {
                a.lse[(long long)(p.r0 + p.rowf + (p.hf + i) / group) * a.H + p.hk * group + (p.hf + i) % group] =
                    lse_of(top, sum);
            }
        }
#pragma unroll
        for (int r = 0; r < C::ROUNDS; ++r) {
            float *const own = xb + warp * 16 * C::XROW;
#pragma unroll
            for (int j = 0; j < DR / 8; ++j)
#pragma unroll
                for (int hr = 0; hr < 2; ++hr)
                    *reinterpret_cast<float2 *>(own + (g + 8 * hr) * C::XROW + j * 8 + 2 * cq) =
                        make_float2(O[r * (DR / 8) + j][2 * hr] * f[hr], O[r * (DR / 8) + j][2 * hr + 1] * f[hr]);
            named_bar_sync(1, CW * 32);
            for (int i = threadIdx.x; i < M * (DR / 4); i += CW * 32) {
                const int row = i / (DR / 4), c = (i % (DR / 4)) * 4;
                if (row >= p.nrows)
                    break;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < NS; ++q) {
                    const float4 v = *reinterpret_cast<const float4 *>(
                        xb + ((q * MT + row / 16) * 16 + row % 16) * C::XROW + c);
                    o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
                }
                if (p.whole) {
                    const long long to = p.r0 + p.rowf + (p.hf + row) / group;
                    const int head = p.hk * group + (p.hf + row) % group;
                    finish4(a, to, head, r * DR + c, o, row_l[row], gate4(a, to, head, r * DR + c));
                } else
                    *reinterpret_cast<float4 *>(slot + row * D + r * DR + c) = o;
            }
            if (r + 1 < C::ROUNDS)
                named_bar_sync(1, CW * 32);
        }
    }
    pdl_launch_dependents();
}

// Joins the parts of the segment that begins in CTA blockIdx.x's run and goes on behind
// it: M / 16 rows a block, the parts dealt to the warps of a row, kFly of them on their
// way at a time.  Bound by three dependent loads (the record, the parts, and what the
// launch itself takes).
constexpr int kJoin = 256, kFly = 5;

template <int D, int M>
__global__ void __launch_bounds__(kJoin) paged_join_kernel(const __grid_constant__ PagedAttnArgs a)
{
    constexpr int ROWS = M / 16, W = kJoin / 32 / ROWS, N4 = (D + 127) / 128;
    static_assert(W * 32 >= D / 4, "a thread finishes four columns");
    __shared__ float red_m[kJoin / 32], red_l[kJoin / 32];
    __shared__ float4 sums[kJoin / 32][D / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rl = warp / W, w = warp % W;
    const float *const ws = static_cast<const float *>(a.ws);
    pdl_wait();
    const Rec rec = reinterpret_cast<const Rec *>(ws + 2ll * kMaxCtas * kPartial<D, M>)[blockIdx.x];
    const int i = blockIdx.y * ROWS + rl;
    if (!rec.live || blockIdx.y * ROWS >= rec.nrows)
        return;
    const int first = blockIdx.x, parts = rec.last - first + 1;
    const int group = a.H / a.Hk, h = rec.hf + i, head = rec.hk * group + h % group;
    const long long row = rec.r0 + rec.rowf + h / group;
    const int col = (w * 32 + lane) * 4;               // of the thread at the end
    const bool mine = i < rec.nrows && col < D;
    const float4 gate = mine ? gate4(a, row, head, col) : make_float4(0.f, 0.f, 0.f, 0.f);
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
    finish4(a, row, head, col, v, sum, gate);
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

// Row tiles of 16: what an average sequence's rows fill (a larger tile than a
// sequence needs costs products, a smaller one reads its keys again).
int row_tiles(int group, int n, int total)
{
    const long long rows = ((long long)total + n - 1) / n * group;
    return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

template <int D, int MT>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t s)
{
    using C = Cfg<D, MT>;
    auto *fn = paged_attn_kernel<D, MT>;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    e = cudaLaunchKernelEx(&cfg, fn, a, km, vm, C::NS);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t join = {};
    join.gridDim = dim3(grid, 16);
    join.blockDim = dim3(kJoin);
    join.stream = s;
    join.attrs = at;
    join.numAttrs = 1;
    return cudaLaunchKernelEx(&join, paged_join_kernel<D, C::M>, a);
}

template <int D>
cudaError_t launch_d(const PagedAttnArgs &a, cudaStream_t s)
{
    switch (row_tiles(a.H / a.Hk, a.sq.n, a.sq.total)) {
    case 1: return launch<D, 1>(a, s);
    case 2: return launch<D, 2>(a, s);
    default: return launch<D, 4>(a, s);
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
    const int M = n > 0 ? 16 * row_tiles(group, n, total) : 16;
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
