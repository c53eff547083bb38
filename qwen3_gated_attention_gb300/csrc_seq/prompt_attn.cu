// prompt_attn.cu -- causal attention of packed prompt rows with grouped heads and
// the sigmoid output gate.
//
// A warp per (row, query head): one pass over the keys with the running maximum
// m and sum l of the softmax (base 2),
//   m' = max(m, s_j),  l <- l 2^(m-m') + 2^(s_j-m'),  o <- o 2^(m-m') + 2^(s_j-m') v_j,
// lanes split over the head's elements.
#include "seq.cuh"

namespace gattn {

namespace {

constexpr int kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32) prompt_attn_simple(const __grid_constant__ PromptAttnArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + warp;
    const int t = (int)(unit / a.H), h = (int)(unit % a.H);
    if (t >= a.sq.total)
        return;
    const int s = find_seq_warp(a.sq, t);
    if (s < 0)
        return;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int i = t - r0;
    // keys: row `kv0` of batch row `slot`, the first `seen` visible
    long long kv0 = 0, keys;
    int slot = 0;
    bool ok;
    if (a.pos) {
        slot = seq_slot_warp(a.sq, s, false);
        const long long p0 = a.pos[s];
        keys = p0 + len;
        ok = slot >= 0 && p0 >= 0 && keys <= a.kv_rows;
    } else {
        kv0 = a.cu_kv[s];
        const long long kv1 = a.cu_kv[s + 1];
        keys = kv1 - kv0;
        ok = kv0 >= 0 && kv1 >= kv0 && kv1 <= a.kv_rows;
    }
    if (!ok && lane == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    const long long seen = ok ? keys - len + i + 1 : 0;
    const int g = h / (a.H / a.Hk);
    const int j0 = lane * 8;
    const bool act = j0 < a.d;
    float q[8] = {}, o[8] = {};
    if (act && seen > 0)
        ld_bf16x8(a.q + t * a.qs.tok + h * a.qs.head + j0, q);
    float m = -INFINITY, l = 0.f;
    const __nv_bfloat16 *kp = a.k + slot * a.kb + g * a.kh + kv0 * a.kt + j0;
    const __nv_bfloat16 *vp = a.v + slot * a.vb + g * a.vh + kv0 * a.vt + j0;
    for (long long j = 0; j < seen; ++j) {
        float k[8], v[8];
        float sc = 0.f;
        if (act) {
            ld_bf16x8(kp + j * a.kt, k);
            ld_bf16x8(vp + j * a.vt, v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sc = fmaf(q[e], k[e], sc);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1)
            sc += __shfl_xor_sync(0xffffffffu, sc, x);
        sc *= a.scale_log2;
        const float mn = fmaxf(m, sc);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float al = exp2f(m - ref), p = exp2f(sc - ref);
        m = mn;
        l = l * al + p;
        if (act)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = o[e] * al + p * v[e];
    }
    if (!act)
        return;
    const float inv = seen > 0 ? 1.f / l : 0.f;
    float gt[8];
    if (a.gate) {
        const long long go = t * a.gs.tok + h * a.gs.head + j0;
        if (a.gate_f32) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                gt[e] = static_cast<const float *>(a.gate)[go + e];
        } else {
            ld_bf16x8(static_cast<const __nv_bfloat16 *>(a.gate) + go, gt);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        o[e] = seen > 0 ? o[e] * inv : 0.f;
        if (a.gate && seen > 0)
            o[e] *= 1.f / (1.f + expf(-gt[e]));
    }
    uint4 u;
    u.x = pack_bf16x2(o[0], o[1]);
    u.y = pack_bf16x2(o[2], o[3]);
    u.z = pack_bf16x2(o[4], o[5]);
    u.w = pack_bf16x2(o[6], o[7]);
    *reinterpret_cast<uint4 *>(a.out + t * a.os.tok + h * a.os.head + j0) = u;
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttnArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    const long long units = (long long)a.sq.total * a.H;
    cfg.gridDim = dim3((unsigned)((units + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, prompt_attn_simple, a);
}

}  // namespace gattn
