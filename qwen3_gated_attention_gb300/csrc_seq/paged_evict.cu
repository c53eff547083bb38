// paged_evict.cu -- shortening the sequences of a paged cache: per key head the newest
// positions and, of the others, those with the most weight, moved to the front in order.
//
// One CTA per sequence and head finds the positions: the weight that the last kept one
// has by a radix select on the ordered bits of the fp32 weights (eight at a time until 256
// or fewer are alike; the first 32768 stay in shared memory; a count for every bin and
// lane, because weights fall into few bins of the first digit and lanes that meet there
// wait), then the positions above it and the first of those that equal it, in order, by
// sums within warps.  Integer counts only, so the order of the atomics does not matter.
//
// Then the rows move, bound by memory.  Into other pages, rows are independent: a warp
// takes kRows of them, all loads before the first store.  In place a row may land where
// another one that has to move still is; but never in front of it (position j takes one
// from j or behind), so a CTA walks down the kept rows in chunks, for a slice of 64
// elements alone (slices do not meet), and stores a chunk only when every thread has
// loaded it.
//
// Measured: eight sequences of 4000 to 16384 positions cut to 4096, 4 heads of 256, into other
// pages: 52 us for 40 us of bytes (each alone, under a profiler with cold caches: the
// selection 14 us on 32 SMs, the rows 45 us, 88 % of the copy rate).  One sequence of 2500
// cut to 1024: 10 us, two launches and the steps of the selection.  In place: 134 us and 27 us
// (128 rows a step, each behind three dependent loads, and none while the selection runs).
#include "paged.cuh"

namespace gattn {

namespace {

constexpr int kSel = 1024;             // threads that select
constexpr int kCached = 32768;         // weights kept in shared memory
constexpr int kBins = 256, kList = 256;
constexpr int kSmem = kCached * 4 + kBins * 32 * 4;

// Larger weights, larger numbers; a NaN counts as -infinity, both zeros as one.
__device__ __forceinline__ uint32_t order_of(float w)
{
    if (w != w)
        w = -INFINITY;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// How many positions a sequence keeps; -1 where it is skipped.
__device__ __forceinline__ int kept_of(const PagedEvictArgs &a, int len)
{
    const int m = min(len, a.keep);
    return len < 0 || len > a.cap || m > a.out_cap ? -1 : m;
}

// Whether the rows' moves take the weights along.
__device__ __forceinline__ bool weights_move(const PagedEvictArgs &a) { return a.out_table && a.w_out != a.w; }

__global__ void __launch_bounds__(kSel) paged_select_kernel(const __grid_constant__ PagedEvictArgs a)
{
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ int counts[kBins], above_of[32], equal_of[32], chosen[3], listed;
    __shared__ uint32_t list[kList];
    uint32_t *const keys = dyn, *const hist = dyn + kCached;
    // the rows' moves start meanwhile, but not before what came before this kernel has ended:
    // they move rows in front of their own wait, so that this order must stay
    pdl_wait();
    pdl_launch_dependents();
    const int hk = blockIdx.x % a.Hk, s = blockIdx.x / a.Hk, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int len = a.lengths[s], m = kept_of(a, len);
    int *const kept = a.kept + ((long long)s * a.Hk + hk) * a.keep;
    const float *const w = a.w + s * a.w_seq + hk * a.w_head;
    for (int j = max(m, 0) + tid; j < a.keep; j += kSel)
        kept[j] = -1;
    if (hk == 0 && tid == 0) {
        a.lengths_out[s] = m < 0 ? len : m;
        if (m < 0 && a.status)
            atomicOr(a.status, GATTN_STATUS_RANGE);
    }
    if (m <= 0)
        return;
    const int rec = min(a.recent, m), cand = len - rec, need = m - rec;
    auto clear = [&] {
        for (int i = tid; i < kBins * 32; i += kSel)
            hist[i] = 0;
        __syncthreads();
    };
    // the order of the candidates, sixteen loads of a thread on their way at a time, and how
    // many have which first digit
    const int cached = min(cand, kCached);
    clear();
    for (int i0 = tid; i0 < cached; i0 += kSel * 16) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e)
            v[e] = i0 + e * kSel < cached ? w[i0 + e * kSel] : 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (i0 + e * kSel < cached) {
                const uint32_t k = order_of(v[e]);
                keys[i0 + e * kSel] = k;
                atomicAdd(&hist[(k >> 24) * 32 + lane], 1u);
            }
    }
    for (int i = kCached + tid; i < cand; i += kSel)
        atomicAdd(&hist[(order_of(w[i]) >> 24) * 32 + lane], 1u);
    if (tid < 4 && cached + tid < kCached)
        keys[cached + tid] = 0u;       // orders are above zero: -infinity's is 0x7fffff
    if (tid == 0)
        listed = 0;
    __syncthreads();
    // the order of i .. i + 3, i a multiple of four; zeros behind the last candidate
    auto four = [&](int i, uint32_t (&k)[4]) {
        if (i < kCached) {
            const uint4 x = *reinterpret_cast<const uint4 *>(keys + i);
            k[0] = x.x, k[1] = x.y, k[2] = x.z, k[3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                k[e] = i + e < cand ? order_of(w[i + e]) : 0u;
        }
    };
    // calls f for this thread's candidates
    auto each = [&](auto f) {
        for (int i = tid * 4; i < cand; i += kSel * 4) {
            uint32_t k[4];
            four(i, k);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < cand)
                    f(k[e]);
        }
    };
    uint32_t edge = 0;                 // of the last kept one
    int ties = 0;                      // how many of its equals are kept
    if (need < cand && need > 0) {
        uint32_t mask = 0;
        int left = need, alike = cand; // of those with edge's first digits: to keep, and all
        for (int shift = 24; shift >= 0 && alike > kList; shift -= 8) {
            if (shift < 24) {
                clear();
                each([&](uint32_t k) {
                    if ((k & mask) == edge)
                        atomicAdd(&hist[((k >> shift) & (kBins - 1)) * 32 + lane], 1u);
                });
                __syncthreads();
            }
            // four threads a bin, from banks that differ
            const int bin = tid >> 2;
            int c = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                c += (int)hist[bin * 32 + (tid & 3) * 8 + ((i + bin) & 7)];
            c += __shfl_xor_sync(0xffffffffu, c, 1);
            c += __shfl_xor_sync(0xffffffffu, c, 2);
            if ((tid & 3) == 0)
                counts[bin] = c;
            __syncthreads();
            // from the largest digit down, eight bins a lane
            if (warp == 0) {
                const int top = kBins - 1 - 8 * lane;
                int n[8], all = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    n[i] = counts[top - i];
                    all += n[i];
                }
                int before = all;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o)
                        before += x;
                }
                before -= all;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < left && before + n[i] >= left) {
                        chosen[0] = top - i;
                        chosen[1] = left - before;
                        chosen[2] = n[i];
                    }
                    before += n[i];
                }
            }
            __syncthreads();
            edge |= (uint32_t)chosen[0] << shift;
            mask |= (uint32_t)(kBins - 1) << shift;
            left = chosen[1];
            alike = chosen[2];
        }
        if (mask != 0xffffffffu) {
            // few are left: each counts those in front of it
            each([&](uint32_t k) {
                if ((k & mask) == edge)
                    list[atomicAdd(&listed, 1)] = k;
            });
            __syncthreads();
            if (tid < alike) {
                const uint32_t k = list[tid];
                int more = 0, same = 0;
                for (int i = 0; i < alike; ++i) {
                    more += list[i] > k;
                    same += list[i] == k;
                }
                if (more < left && more + same >= left) {      // its equals write the same
                    chosen[0] = (int)k;
                    chosen[1] = left - more;
                }
            }
            __syncthreads();
            edge = (uint32_t)chosen[0];
            left = chosen[1];
        }
        ties = left;
    }
    // the kept ones of the candidates in order: a run of them for each warp, which counts
    // those above the edge and those equal to it, then writes behind the warps before it
    if (need > 0) {
        const int run = (cand + kSel * 4 - 1) / (kSel * 4) * 128, i0 = warp * run, i1 = min(cand, i0 + run);
        // all are kept: every one is above an edge of zero
        auto above = [&](uint32_t k) { return k > edge; };
        auto equal = [&](uint32_t k) { return k == edge && k != 0u; };
        int up = 0, eq = 0;
        for (int i = i0 + lane * 4; i < i1; i += 128) {
            uint32_t k[4];
            four(i, k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                up += above(k[e]);
                eq += equal(k[e]);
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            up += __shfl_xor_sync(0xffffffffu, up, o);
            eq += __shfl_xor_sync(0xffffffffu, eq, o);
        }
        if (lane == 0) {
            above_of[warp] = up;
            equal_of[warp] = eq;
        }
        __syncthreads();
        up = lane < warp ? above_of[lane] : 0;
        eq = lane < warp ? equal_of[lane] : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            up += __shfl_xor_sync(0xffffffffu, up, o);
            eq += __shfl_xor_sync(0xffffffffu, eq, o);
        }
        for (int j = i0; j < i1; j += 128) {
            const int i = j + lane * 4;
            uint32_t k[4] = {0u, 0u, 0u, 0u};
            if (i < i1)
                four(i, k);
            int c = 0;                 // above, and equal from bit 16 on
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c += above(k[e]) + (equal(k[e]) << 16);
            int at = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, at, o);
                if (lane >= o)
                    at += x;
            }
            const int all = __shfl_sync(0xffffffffu, at, 31);
            at -= c;
            if (c) {
                int u = up + (at & 0xFFFF), q = eq + (at >> 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (above(k[e]))
                        kept[min(q, ties) + u++] = i + e;
                    else if (equal(k[e])) {
                        if (q < ties)
                            kept[q + u] = i + e;
                        ++q;
                    }
                }
            }
            up += all & 0xFFFF;
            eq += all >> 16;
        }
    }
    for (int r = tid; r < rec; r += kSel)
        kept[need + r] = len - rec + r;
    // the weights follow: where rows move to other pages, with them, but for weights in
    // place.  In place a round reads all of its own before it writes, and what
    // later rounds read lies behind what it writes.
    if (!a.w_out || weights_move(a))
        return;
    float *const wo = a.w_out + s * a.wo_seq + hk * a.wo_head;
    for (int base = 0; base < m; base += kSel * 4) {
        __syncthreads();
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = base + e * kSel + tid;
            v[e] = j < m ? w[kept[j]] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = base + e * kSel + tid;
            if (j < m)
                wo[j] = v[e];
        }
    }
}

// Where position t of a table's row is: page and row in it; page -1 if there is none.
struct Place {
    int page, row;
};

__device__ __forceinline__ Place place_of(const PagedEvictArgs &a, const int *row, int t)
{
    Place p{row[t / a.pg.page], t % a.pg.page};
    if (p.page < 0 || p.page >= a.pg.pages) {
        p.page = -1;
        if (a.status)
            atomicOr(a.status, GATTN_STATUS_RANGE);
    }
    return p;
}

constexpr int kMove = 256, kRows = 8;

// Into other pages: a warp moves kRows (heads of 64 and 128: 4 or 2 times as many) rows.
// Blocks take the last rows of all sequences first: the newest positions and sequences
// that keep everything need no selection, so they move while it runs (60 us -> 52 us for
// eight sequences of 4000 to 16384 positions, a quarter of the 4096 kept ones new).
// (In front of the wait: lengths, tables, the pages and weights that are read, and those
// that are written; of these the selection reads weights, which other weights_out never
// share, and writes none.)
__global__ void __launch_bounds__(kMove) paged_move_kernel(const __grid_constant__ PagedEvictArgs a, int groups)
{
    const int lane = threadIdx.x & 31, heads = a.n * a.Hk;
    const long long job = (blockIdx.x * (long long)kMove + threadIdx.x) >> 5;
    const int sh = (int)(job % heads), group = groups - 1 - (int)(job / heads);
    const int s = sh / a.Hk, hk = sh % a.Hk;
    const int len = a.lengths[s], m = kept_of(a, len);
    const int lpr = a.d == 64 ? 8 : a.d == 128 ? 16 : 32, per = 32 / lpr;
    const int j0 = group * kRows * per;
    if (group < 0 || j0 >= m) {
        pdl_wait();
        return;
    }
    // the first row of the newest; with nothing left out all rows are where they were
    const int need = m == len ? 0 : m - min(a.recent, m);
    const bool known = j0 >= need;
    if (!known)
        pdl_wait();
    // a lane a row
    Place from{-1, 0}, to{-1, 0};
    const int mine = j0 + lane;
    if (lane < kRows * per && mine < m) {
        const int t = known ? len - m + mine : a.kept[(long long)sh * a.keep + mine];
        if ((unsigned)t < (unsigned)len) {
            from = place_of(a, a.pg.table + s * a.pg.table_stride, t);
            if (a.w_out && weights_move(a))
                a.w_out[s * a.wo_seq + hk * a.wo_head + mine] = a.w[s * a.w_seq + hk * a.w_head + t];
        }
        to = place_of(a, a.out_table + s * a.out_stride, mine);
        if (to.page < 0)
            from.page = -1;
    }
    const int c = (lane & (lpr - 1)) * 8;
    uint4 k[kRows], v[kRows];
    const __nv_bfloat16 *const kp = static_cast<const __nv_bfloat16 *>(a.pg.kp) + hk * a.pg.k.head + c;
    const __nv_bfloat16 *const vp = static_cast<const __nv_bfloat16 *>(a.pg.vp) + hk * a.pg.v.head + c;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int l = i * per + lane / lpr;
        const int page = __shfl_sync(0xffffffffu, from.page, l), row = __shfl_sync(0xffffffffu, from.row, l);
        if (page >= 0 && c < a.d) {
            k[i] = __ldcs(reinterpret_cast<const uint4 *>(kp + page * a.pg.k.page + row * a.pg.k.tok));
            v[i] = __ldcs(reinterpret_cast<const uint4 *>(vp + page * a.pg.v.page + row * a.pg.v.tok));
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int l = i * per + lane / lpr;
        const bool on = __shfl_sync(0xffffffffu, from.page, l) >= 0;
        const int page = __shfl_sync(0xffffffffu, to.page, l), row = __shfl_sync(0xffffffffu, to.row, l);
        if (on && c < a.d) {
            *reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(kp) + page * a.pg.k.page + row * a.pg.k.tok) = k[i];
            *reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(vp) + page * a.pg.v.page + row * a.pg.v.tok) = v[i];
        }
    }
    if (known)
        pdl_wait();                    // no later work starts before the selection has ended
}

// In place: a CTA has 64 elements of the keys (or values) of one sequence and head.
constexpr int kStep = 4, kChunk = kMove / 8 * kStep;

__global__ void __launch_bounds__(kMove) paged_close_kernel(const __grid_constant__ PagedEvictArgs a)
{
    pdl_wait();
    const int slices = a.d / 64;
    int x = blockIdx.x;
    const int slice = x % slices;
    x /= slices;
    const bool val = x & 1;
    const int sh = x >> 1, s = sh / a.Hk, hk = sh % a.Hk;
    const int len = a.lengths[s], m = kept_of(a, len);
    if (m <= 0 || m == len)
        return;                        // nothing moves
    const int *const row = a.pg.table + s * a.pg.table_stride, *const kept = a.kept + (long long)sh * a.keep;
    const PageStride &st = val ? a.pg.v : a.pg.k;
    __nv_bfloat16 *const base = static_cast<__nv_bfloat16 *>(val ? a.pg.vp : a.pg.kp) + hk * st.head + slice * 64 +
                                (threadIdx.x & 7) * 8;
    uint4 cur[kStep], nxt[kStep];
    __nv_bfloat16 *to[kStep], *to_n[kStep];
    auto load = [&](int j0, uint4 (&v)[kStep], __nv_bfloat16 *(&dst)[kStep]) {
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            const int j = j0 + i * (kMove / 8) + (threadIdx.x >> 3);
            dst[i] = nullptr;
            if (j >= m)
                continue;
            const int t = kept[j];
            if (t == j || (unsigned)t >= (unsigned)len)
                continue;              // stays
            const Place f = place_of(a, row, t), o = place_of(a, row, j);
            if (f.page < 0 || o.page < 0)
                continue;
            v[i] = *reinterpret_cast<const uint4 *>(base + f.page * st.page + f.row * st.tok);
            dst[i] = base + o.page * st.page + o.row * st.tok;
        }
    };
    load(0, cur, to);
    for (int j0 = 0; j0 < m; j0 += kChunk) {
        load(j0 + kChunk, nxt, to_n);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
            if (to[i])
                *reinterpret_cast<uint4 *>(to[i]) = cur[i];
            cur[i] = nxt[i];
            to[i] = to_n[i];
        }
    }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictArgs &a, cudaStream_t s)
{
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(paged_select_kernel, kSmem, done);
    if (e != cudaSuccess)
        return e;
    e = launch_paged(paged_select_kernel, dim3((unsigned)(a.n * a.Hk)), dim3(kSel), kSmem, s, a);
    if (e != cudaSuccess)
        return e;
    if (!a.out_table)
        return launch_paged(paged_close_kernel, dim3((unsigned)(a.n * a.Hk * 2 * (a.d / 64))), dim3(kMove), 0, s, a);
    // kept rows, at most
    const long long most = a.keep < a.out_cap ? a.keep : a.out_cap;
    const int per = kRows * (a.d == 64 ? 4 : a.d == 128 ? 2 : 1);
    const int groups = (int)((most + per - 1) / per);
    const long long warps = (long long)groups * a.n * a.Hk;
    return launch_paged(paged_move_kernel, dim3((unsigned)((warps + kMove / 32 - 1) / (kMove / 32))), dim3(kMove), 0, s, a,
                        groups);
}

}  // namespace gattn
