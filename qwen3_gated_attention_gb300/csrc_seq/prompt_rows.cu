// prompt_rows.cu -- QK RMSNorm, partial RoPE and KV append of packed prompt rows.
//
// Per head row x of d elements at position p:
//   y = x / sqrt(mean(x^2) + eps) * w,  then for i < rd/2
//   (y_i, y_{i+rd/2}) <- (y_i cos - y_{i+rd/2} sin, y_{i+rd/2} cos + y_i sin),
// angle p * theta^(-2i/rd); values are copied.  Bound by memory: every element is
// read once and written once.  A warp works alone on (a part of) one packed row, so
// nothing waits at a barrier: it finds the row's sequence, forms the row's angles
// once, and takes kFly head rows at a time, their loads in flight together.
#include "seq.cuh"

namespace gattn {

namespace {

constexpr int kWarps = 8;
constexpr int kFly = 4;            // head rows in flight per group of lanes

// Eight elements as they come from memory.
template <bool F32>
struct Raw {
    uint4 u[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *base, long long off)
    {
        const uint4 *p = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + off)
                             : reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + off);
        u[0] = __ldcs(p);
        if (F32)
            u[F32 ? 1 : 0] = __ldcs(p + 1);
    }
    __device__ __forceinline__ void clear()
    {
        u[0] = make_uint4(0, 0, 0, 0);
        u[F32 ? 1 : 0] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        if (F32) {
            const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[F32].x, u[F32].y, u[F32].z, u[F32].w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                f[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = bf16_lo(w[i]);
                f[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
};

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8])
{
    uint4 u;
    u.x = pack_bf16x2(f[0], f[1]);
    u.y = pack_bf16x2(f[2], f[3]);
    u.z = pack_bf16x2(f[4], f[5]);
    u.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4 *>(p) = u;
}

// A group of d/8 lanes (padded to a power of two) per head row, eight elements a
// lane.  FAST: rd/2 is a multiple of 8, so a rotary partner is the same element of
// another lane; otherwise partners meet in shared memory.
template <bool F32, bool FAST>
__global__ void __launch_bounds__(kWarps * 32, F32 ? 2 : 3)
prompt_rows_kernel(const __grid_constant__ PromptRowsArgs a, int parts)
{
    __shared__ float2 table[kWarps][128];
    __shared__ float swap[FAST ? 1 : kWarps][256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(job / parts), part = (int)(job % parts);
    if (t >= a.sq.total)
        return;
    const int s = find_seq_warp(a.sq, t);
    if (s < 0)
        return;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    const long long p0 = a.pos[s], p = p0 + (t - r0);
    const bool ok = slot >= 0 && p0 >= 0 && p0 + len <= a.cap;
    if (!ok && lane == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    const int half = a.rd / 2;
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
    const int lpu = a.d == 64 ? 8 : (a.d == 128 ? 16 : 32);   // lanes per head row
    const int sub = lane & (lpu - 1), at = lane / lpu, upw = 32 / lpu;
    const int j0 = sub * 8;
    const bool act = j0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    float cosv[8], sinv[8];
    Raw<false> wq, wk;
    wq.clear();
    wk.clear();
    if (act) {
        wq.load(a.q_norm, j0);
        wk.load(a.k_norm, j0);
    }
    // y cos + partner (-sin or sin); 1 and 0 past the rotary elements
    int mate = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = j0 + i;
        if (j < half) {
            cosv[i] = cs[j].x;
            sinv[i] = -cs[j].y;
        } else if (j < a.rd) {
            cosv[i] = cs[j - half].x;
            sinv[i] = cs[j - half].y;
        } else {
            cosv[i] = 1.f;
            sinv[i] = 0.f;
        }
    }
    if (FAST && j0 < a.rd)
        mate = j0 < half ? lane + half / 8 : lane - half / 8;
    float *const buf = FAST ? nullptr : swap[warp] + at * lpu * 8;
    const int units = a.H + 2 * a.Hk, step = parts * upw;
    for (int u0 = part * upw + at; u0 - at < units; u0 += kFly * step) {
        Raw<F32> raw[kFly];
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int u = u0 + f * step;
            raw[f].clear();
            if (act && ok && u < units) {
                const int kind = u < a.H ? 0 : (u < a.H + a.Hk ? 1 : 2);
                const RowStride st = kind == 0 ? a.qs : (kind == 1 ? a.ks : a.vs);
                const int head = kind == 0 ? u : (kind == 1 ? u - a.H : u - a.H - a.Hk);
                raw[f].load(kind == 0 ? a.q : (kind == 1 ? a.k : a.v), t * st.tok + head * st.head + j0);
            }
        }
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int u = u0 + f * step;
            if (u - at >= units)               // the whole warp is past the last unit
                break;
            const int kind = u < a.H ? 0 : (u < a.H + a.Hk ? 1 : 2);
            float x[8];
            raw[f].get(x);
            // (values come along so that every lane meets the shuffles)
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss = fmaf(x[i], x[i], ss);
            for (int o = lpu / 2; o; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (kind < 2 || upw > 1) {
                const float inv = rsqrtf(ss * inv_d + a.eps);
                float y[8], z[8], w[8];
                if (kind == 0)
                    wq.get(w);
                else
                    wk.get(w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    y[i] = x[i] * (inv * w[i]);
                if (FAST) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        z[i] = __shfl_sync(0xffffffffu, y[i], mate);
                } else {
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        buf[j0 + i] = y[i];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = j0 + i;
                        z[i] = j < a.rd ? buf[j < half ? j + half : j - half] : 0.f;
                    }
                }
                if (kind < 2)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = j0 + i < a.rd ? y[i] * cosv[i] + z[i] * sinv[i] : y[i];
            }
            if (!act || u >= units)
                continue;
            if (kind == 0)
                store8(a.q_out + t * a.os.tok + u * a.os.head + j0, x);
            else if (ok && kind == 1)
                store8(a.kc + slot * a.kcb + (u - a.H) * a.kch + p * a.kct + j0, x);
            else if (ok)
                store8(a.vc + slot * a.vcb + (u - a.H - a.Hk) * a.vch + p * a.vct + j0, x);
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
    // warps per row: two keep the row's own work (angles, sequence) small against
    // its bytes; eight while there are too few rows to fill the GPU
    const int parts = (long long)a.sq.total * 2 >= (long long)sms * 32 ? 2 : 8;
    const long long jobs = (long long)a.sq.total * parts;
    const dim3 grid((unsigned)((jobs + kWarps - 1) / kWarps)), block(kWarps * 32);
    const bool fast = (a.rd / 2) % 8 == 0;
    auto *fn = x_f32 ? (fast ? prompt_rows_kernel<true, true> : prompt_rows_kernel<true, false>)
                     : (fast ? prompt_rows_kernel<false, true> : prompt_rows_kernel<false, false>);
    return launch_seq(fn, grid, block, s, a, parts);
}

}  // namespace gattn
