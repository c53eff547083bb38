// prompt_rows.cu -- QK RMSNorm, partial RoPE and KV append of packed prompt rows.
//
// Per head row x of d elements at position p:
//   y = x / sqrt(mean(x^2) + eps) * w,  then for i < rd/2
//   (y_i, y_{i+rd/2}) <- (y_i cos - y_{i+rd/2} sin, y_{i+rd/2} cos + y_i sin),
// angle p * theta^(-2i/rd); values are copied.  Bound by memory: every element is
// read once and written once.  A warp works alone on (a part of) one packed row, so
// nothing waits at a barrier, and always has kFly head rows on their way while it works
// on the kFly before them, from the queries through the keys to the values; the first
// set out before the row's sequence and angles are known.  8240 rows of 32 + 8 + 8 heads
// of 256 take 75 us, 5.4 TB/s or 80 % of the copy rate (a CTA per row and head with
// barriers 144 us; a warp that loads, then works 88 us; one head row at a time 188 us);
// more loads on their way or more warps cost registers: 82 us with 24 warps an SM.  37
// rows of 16 + 4 + 4 heads: 4.5 us.
#include "seq.cuh"

namespace gattn {

namespace {

constexpr int kWarps = 4;
constexpr int kFly = 4;            // head rows in flight per group of lanes

// Two runs of four elements as they come from memory.
template <bool F32>
struct Raw {
    uint32_t w[F32 ? 8 : 4];
    __device__ __forceinline__ void load(const void *base, long long off0, long long off1)
    {
        if (F32) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off0));
            const uint4 b = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off1));
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[F32 ? 4 : 0] = b.x; w[F32 ? 5 : 1] = b.y; w[F32 ? 6 : 2] = b.z; w[F32 ? 7 : 3] = b.w;
        } else {
            const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(base) + off0));
            const uint2 b = __ldcs(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(base) + off1));
            w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
        }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 8 : 4); ++i)
            w[i] = 0;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = F32 ? __uint_as_float(w[F32 ? i : 0]) : i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
};

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float a, float b, float c, float d)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// A group of d/8 lanes (padded to a power of two) per head row, eight elements a
// lane, in two runs of four.  FAST: rd/2 is a multiple of 4; the first rd/8 lanes of
// a group then take a run from each rotary half, so partners meet in a lane.
// Otherwise the runs are neighbours and partners meet in shared memory.
template <bool F32, bool FAST>
__global__ void __launch_bounds__(kWarps * 32, F32 ? 4 : 5)
prompt_rows_kernel(const __grid_constant__ PromptRowsArgs a, int parts)
{
    __shared__ float2 table[kWarps][128];
    __shared__ float swap[FAST ? 1 : kWarps][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(job / parts), part = (int)(job % parts);
    if (t >= a.sq.total)
        return;
    const int lpu = a.d == 64 ? 8 : (a.d == 128 ? 16 : 32);   // lanes per head row
    const int sub = lane & (lpu - 1), at = lane / lpu, upw = 32 / lpu;
    const int j0 = sub * 8;
    const bool act = j0 < a.d;
    const int half = a.rd / 2;
    const bool rot = FAST && j0 < a.rd;
    const int o0 = rot ? sub * 4 : j0, o1 = rot ? half + sub * 4 : j0 + 4;   // the two runs
    const int step = parts * upw, first = part * upw + at;
    // the row's own place in q, k and v
    const long long esz = F32 ? 4 : 2;
    const char *const qrow = static_cast<const char *>(a.q) + t * a.qs.tok * esz;
    const char *const krow = static_cast<const char *>(a.k) + t * a.ks.tok * esz;
    const char *const vrow = static_cast<const char *>(a.v) + t * a.vs.tok * esz;
    // the head rows on their way: always kFly ahead of the ones at work, across q, k
    // and v, the first before anything else is known of the row
    Raw<F32> nxt[kFly];
    auto fetch = [&](const void *src, long long src_head, int u0, int heads, int r0, int r1) {
        long long so = (long long)u0 * src_head;
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            nxt[f].clear();
            if (act && u0 + f * step < heads)
                nxt[f].load(src, so + r0, so + r1);
            so += step * src_head;
        }
    };
    fetch(qrow, a.qs.head, first, a.H, o0, o1);
    const int s = find_seq_warp(a.sq, t);
    if (s < 0)
        return;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    const long long p0 = a.pos[s], p = p0 + (t - r0);
    // the last two hold for any row, if the offsets do not fall
    const bool ok = slot >= 0 && p0 >= 0 && p0 + len <= a.cap && t >= r0 && t - r0 < len;
    if (!ok && lane == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    float2 *const cs = table[warp];
    for (int i = lane; i < half; i += 32) {
        // The angle p * inv_freq as an unevaluated float pair, reduced modulo
        // 2 pi in two steps: good to a few 1e-7 rad at far positions without
        // double arithmetic
        const float pos = (float)p;
        const float2 fq = a.inv_freq[i];
        const float ph = pos * fq.x;
        const float pl = fmaf(pos, fq.x, -ph) + pos * fq.y;
        const float turns = rintf(ph * 0.15915494f);
        float red = fmaf(-turns, 6.2831855f, ph);
        red = fmaf(-turns, -1.7484555e-07f, red);
        red += pl;
        float sn, c;
        __sincosf(red, &sn, &c);
        cs[i] = make_float2(c, sn);
    }
    __syncwarp();
    const float inv_d = 1.f / (float)a.d;
    float cosv[FAST ? 4 : 8], sinv[FAST ? 4 : 8];
    Raw<false> wq, wk;
    wq.clear();
    wk.clear();
    if (act) {
        wq.load(a.q_norm, o0, o1);
        wk.load(a.k_norm, o0, o1);
    }
#pragma unroll
    for (int i = 0; i < (FAST ? 4 : 8); ++i) {
        const int j = FAST ? o0 + i : j0 + i;
        if (FAST) {
            cosv[i] = rot ? cs[j].x : 1.f;
            sinv[i] = rot ? cs[j].y : 0.f;
        } else {
            cosv[i] = j < a.rd ? cs[j < half ? j : j - half].x : 1.f;
            sinv[i] = j < a.rd ? (j < half ? -cs[j].y : cs[j - half].y) : 0.f;
        }
    }
    float *const buf = FAST ? nullptr : swap[warp] + at * lpu * 8;
    // `heads` head rows from `src`, the first of them on their way, to `dst`, normed and
    // turned by weights w; `then` fetches what comes after
    auto normed = [&](const void *src, long long src_head, __nv_bfloat16 *dst, long long dst_head, int heads,
                      const Raw<false> &weight, auto then) {
        __nv_bfloat16 *to = dst + (long long)first * dst_head;
        for (int u0 = first; u0 - at < heads || u0 == first; u0 += kFly * step) {
            Raw<F32> raw[kFly];
#pragma unroll
            for (int f = 0; f < kFly; ++f) {
                raw[f] = nxt[f];
                if (!ok)
                    raw[f].clear();
            }
            if (u0 - at + kFly * step < heads)
                fetch(src, src_head, u0 + kFly * step, heads, o0, o1);
            else
                then();
#pragma unroll
            for (int f = 0; f < kFly; ++f, to += step * dst_head) {
                const int u = u0 + f * step;
                if (u - at >= heads)           // the whole warp is past the last one
                    continue;
                float x[8], y[8], w[8];
                weight.get(w);
                raw[f].get(x);
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    s0 = fmaf(x[i], x[i], s0);
                    s1 = fmaf(x[i + 1], x[i + 1], s1);
                }
                float ss = s0 + s1;
                for (int o = lpu / 2; o; o >>= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = ok ? rsqrtf(ss * inv_d + a.eps) : 0.f;   // skipped rows: zeros
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = x[i] * (inv * w[i]);
                if (FAST) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = y[i];
                    if (rot)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[i] = y[i] * cosv[i] - y[i + 4] * sinv[i];
                            x[i + 4] = y[i + 4] * cosv[i] + y[i] * sinv[i];
                        }
                } else {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        buf[j0 + i] = y[i];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = j0 + i;
                        x[i] = j < a.rd ? y[i] * cosv[FAST ? 0 : i] +
                                              buf[j < half ? j + half : j - half] * sinv[FAST ? 0 : i]
                                        : y[i];
                    }
                }
                if (act && u < heads) {
                    store4(to + o0, x[0], x[1], x[2], x[3]);
                    store4(to + o1, x[4], x[5], x[6], x[7]);
                }
            }
        }
    };
    normed(qrow, a.qs.head, a.q_out + t * a.os.tok, a.os.head, a.H, wq,
           [&] { fetch(krow, a.ks.head, first, a.Hk, o0, o1); });
    if (!ok)
        return;
    normed(krow, a.ks.head, a.kc + slot * a.kcb + p * a.kct, a.kch, a.Hk, wk,
           [&] { fetch(vrow, a.vs.head, first, a.Hk, j0, j0 + 4); });
    __nv_bfloat16 *const vc = a.vc + slot * a.vcb + p * a.vct;
    for (int u0 = first; u0 < a.Hk; u0 += kFly * step) {
        Raw<F32> raw[kFly];
#pragma unroll
        for (int f = 0; f < kFly; ++f)
            raw[f] = nxt[f];
        if (u0 + kFly * step < a.Hk)
            fetch(vrow, a.vs.head, u0 + kFly * step, a.Hk, j0, j0 + 4);
#pragma unroll
        for (int f = 0; f < kFly; ++f)
            if (act && u0 + f * step < a.Hk) {
                float x[8];
                raw[f].get(x);
                __nv_bfloat16 *to = vc + (u0 + f * step) * a.vch + j0;
                store4(to, x[0], x[1], x[2], x[3]);
                store4(to + 4, x[4], x[5], x[6], x[7]);
            }
    }
}

}  // namespace

cudaError_t launch_prompt_rows(const PromptRowsArgs &a, int x_f32, cudaStream_t s)
{
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    // Warps per row: each repeats the row's own work (its angles, its sequence), so as
    // few as fill the GPU once (20 warps an SM; fp32 rows, with more registers, 16).
    // 16 + 4 + 4 heads of 256, by 1, 2, 4 and 8 warps a row: 37 rows 10.1, 6.7, 5.1 and
    // 4.8 us; 600 rows 10.3, 7.6, 6.5 and 9.7; 1200 rows 11.3, 8.9, 11.1 and 15.1; 9600
    // rows 49.0, 50.9, 62.3 and 91.0
    int parts = 1;
    while (parts < 8 && (long long)a.sq.total * 2 * parts <= (long long)sms * (x_f32 ? 16 : 20))
        parts *= 2;
    const long long jobs = (long long)a.sq.total * parts;
    const dim3 grid((unsigned)((jobs + kWarps - 1) / kWarps)), block(kWarps * 32);
    const bool fast = (a.rd / 2) % 4 == 0;
    auto *fn = x_f32 ? (fast ? prompt_rows_kernel<true, true> : prompt_rows_kernel<true, false>)
                     : (fast ? prompt_rows_kernel<false, true> : prompt_rows_kernel<false, false>);
    return launch_seq(fn, grid, block, s, a, parts);
}

}  // namespace gattn
