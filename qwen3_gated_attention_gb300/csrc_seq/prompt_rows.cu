// prompt_rows.cu -- QK RMSNorm, partial RoPE and KV append of packed prompt rows.
//
// Per head row x of d elements at position p:
//   y = x / sqrt(mean(x^2) + eps) * w,  then for i < rd/2
//   (y_i, y_{i+rd/2}) <- (y_i cos - y_{i+rd/2} sin, y_{i+rd/2} cos + y_i sin),
// angle p * theta^(-2i/rd); values are copied.  Every element is read once and
// written once.
#include "seq.cuh"

namespace gattn {

namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ void load8(const void *base, long long off, float (&f)[8])
{
    if (F32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
        const float4 u = p[0], w = p[1];
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
        f[4] = w.x; f[5] = w.y; f[6] = w.z; f[7] = w.w;
    } else {
        ld_bf16x8(static_cast<const __nv_bfloat16 *>(base) + off, f);
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8])
{
    uint4 u;
    u.x = pack_bf16x2(f[0], f[1]);
    u.y = pack_bf16x2(f[2], f[3]);
    u.z = pack_bf16x2(f[4], f[5]);
    u.w = pack_bf16x2(f[6], f[7]);
    *reinterpret_cast<uint4 *>(p) = u;
}

// One CTA per packed row; a group of d/8 lanes (padded to a power of two) per
// head, eight elements a lane.
template <bool F32>
__global__ void __launch_bounds__(kThreads) prompt_rows_kernel(const __grid_constant__ PromptRowsArgs a)
{
    __shared__ float2 cs[128];
    __shared__ float rowbuf[kThreads * 8];
    const int t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = find_seq_warp(a.sq, t);
    if (s < 0)
        return;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    const long long p0 = a.pos[s];
    const long long p = p0 + (t - r0);
    const bool ok = slot >= 0 && p0 >= 0 && p0 + len <= a.cap;
    if (!ok && threadIdx.x == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    const int half = a.rd / 2;
    if (threadIdx.x < half) {
        // The angle p * inv_freq as an unevaluated float pair, reduced modulo
        // 2 pi in two steps: good to a few 1e-7 rad at far positions without
        // double arithmetic
        const float pos = (float)p;
        const float2 fq = a.inv_freq[threadIdx.x];
        const float ph = pos * fq.x;
        const float pl = fmaf(pos, fq.x, -ph) + pos * fq.y;
        const float turns = rintf(ph * 0.15915494f);
        float red = fmaf(-turns, 6.2831855f, ph);
        red = fmaf(-turns, -1.7484555e-07f, red);
        red += pl;
        float sn, c;
        __sincosf(red, &sn, &c);
        cs[threadIdx.x] = make_float2(c, sn);
    }
    __syncthreads();
    const int lpu = a.d == 64 ? 8 : (a.d == 128 ? 16 : 32);   // lanes per head
    const int sub = lane & (lpu - 1);
    const int upw = 32 / lpu;
    const int j0 = sub * 8;
    const bool act = j0 < a.d;
    float *buf = rowbuf + warp * 256 + (lane - sub) * 8;
    const int units = a.H + 2 * a.Hk;
    const float inv_d = 1.f / (float)a.d;
    for (int u0 = warp * upw; u0 < units; u0 += (kThreads / 32) * upw) {
        const int u = u0 + lane / lpu;
        const bool on = act && u < units;
        const int kind = u < a.H ? 0 : (u < a.H + a.Hk ? 1 : 2);
        const int head = kind == 0 ? u : (kind == 1 ? u - a.H : u - a.H - a.Hk);
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on && ok) {
            const RowStride st = kind == 0 ? a.qs : (kind == 1 ? a.ks : a.vs);
            load8<F32>(kind == 0 ? a.q : (kind == 1 ? a.k : a.v), t * st.tok + head * st.head + j0, x);
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(x[i], x[i], ss);
        for (int o = lpu / 2; o; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (on && kind < 2) {
            const float inv = rsqrtf(ss * inv_d + a.eps);
            float w[8];
            ld_bf16x8(reinterpret_cast<const __nv_bfloat16 *>(kind == 0 ? a.q_norm : a.k_norm) + j0, w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] *= inv * w[i];
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            buf[j0 + i] = x[i];
        __syncwarp();
        if (on && kind < 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = j0 + i;
                if (j < half) {
                    const float2 c = cs[j];
                    x[i] = x[i] * c.x - buf[j + half] * c.y;
                } else if (j < a.rd) {
                    const float2 c = cs[j - half];
                    x[i] = x[i] * c.x + buf[j - half] * c.y;
                }
            }
        }
        if (!on)
            continue;
        if (kind == 0)
            store8(a.q_out + t * a.os.tok + head * a.os.head + j0, x);
        else if (ok && kind == 1)
            store8(a.kc + slot * a.kcb + head * a.kch + p * a.kct + j0, x);
        else if (ok)
            store8(a.vc + slot * a.vcb + head * a.vch + p * a.vct + j0, x);
    }
}

}  // namespace

cudaError_t launch_prompt_rows(const PromptRowsArgs &a, int x_f32, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.sq.total);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, x_f32 ? prompt_rows_kernel<true> : prompt_rows_kernel<false>, a);
}

}  // namespace gattn
