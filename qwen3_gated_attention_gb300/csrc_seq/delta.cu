// delta.cu -- the gated delta rule, row by row.
//
//   S <- e^g S,  w = beta (v - S^T k),  S <- S + k w^T,  out = scale S^T q
//
// The columns of S are independent of one another: a CTA owns 32 of them for one
// (sequence, head), four lanes to a column, each holding k_dim/4 of its
// elements in registers (element 4 i + lane%4), so the state is read and written
// once per call.  k and q of a row are staged in shared memory (divided by their
// norms there).
#include "seq.cuh"

namespace gattn {

namespace {

constexpr int kThreads = 128;
constexpr int kCols = 32;

template <int DK>
__global__ void __launch_bounds__(kThreads) delta_rows_kernel(const __grid_constant__ DeltaArgs a)
{
    __shared__ float kq[2][2][DK];     // [buffer][k, q]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, s = blockIdx.x, hk = h / (a.Hv / a.Hk);
    const int col = blockIdx.z * kCols + warp * 8 + (lane >> 2), sub = lane & 3;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    __nv_bfloat16 *out = a.out + (long long)h * a.os.head + col;
    if (slot < 0) {
        if (threadIdx.x == 0)
            seq_flag(a.sq, GATTN_STATUS_RANGE);
        if (sub == 0)
            for (int t = r0; t < r0 + len; ++t)
                out[t * a.os.tok] = __float2bfloat16_rn(0.f);
        return;
    }
    float S[DK / 4];
    const long long so = slot * a.state_stride + (long long)h * DK * a.dv + col;
#pragma unroll
    for (int i = 0; i < DK / 4; ++i)
        S[i] = a.state ? a.state[so + (long long)(4 * i + sub) * a.dv] : 0.f;
    for (int r = 0; r < len; ++r) {
        const int t = r0 + r, b = r & 1;
        // warp 0 stages k, warp 1 stages q
        if (warp < 2) {
            const __nv_bfloat16 *src = warp == 0 ? a.k + t * a.ks.tok + hk * a.ks.head
                                                 : a.q + t * a.qs.tok + hk * a.qs.head;
            float x[DK / 32], ss = 0.f;
#pragma unroll
            for (int i = 0; i < DK / 32; ++i) {
                x[i] = __bfloat162float(src[lane + 32 * i]);
                ss = fmaf(x[i], x[i], ss);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
            float f = a.l2norm ? 1.f / sqrtf(ss + a.l2_eps) : 1.f;
            if (warp == 1)
                f *= a.scale;
#pragma unroll
            for (int i = 0; i < DK / 32; ++i)
                kq[b][warp][lane + 32 * i] = x[i] * f;
        }
        const float decay = expf(a.g[t * a.gt + h]), beta = a.beta[t * a.bt + h];
        const float v = __bfloat162float(a.v[t * a.vs.tok + h * a.vs.head + col]);
        __syncthreads();     // one a row: the buffers alternate
        float d[4] = {};
#pragma unroll
        for (int i = 0; i < DK / 4; ++i) {
            S[i] *= decay;
            d[i & 3] = fmaf(S[i], kq[b][0][4 * i + sub], d[i & 3]);
        }
        float dot = (d[0] + d[1]) + (d[2] + d[3]);
        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
        dot += __shfl_xor_sync(0xffffffffu, dot, 2);
        const float w = beta * (v - dot);
        float o[4] = {};
#pragma unroll
        for (int i = 0; i < DK / 4; ++i) {
            S[i] = fmaf(kq[b][0][4 * i + sub], w, S[i]);
            o[i & 3] = fmaf(S[i], kq[b][1][4 * i + sub], o[i & 3]);
        }
        float y = (o[0] + o[1]) + (o[2] + o[3]);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        if (sub == 0)
            out[t * a.os.tok] = __float2bfloat16_rn(y);
    }
    if (a.state_out && (len > 0 || a.state_out != a.state))
#pragma unroll
        for (int i = 0; i < DK / 4; ++i)
            a.state_out[so + (long long)(4 * i + sub) * a.dv] = S[i];
}

cudaError_t launch_rows(const DeltaArgs &a, cudaStream_t s)
{
    // one CTA per (sequence, head, 32 columns); x is the dimension that may be long
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.sq.n, a.Hv, a.dv / kCols);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, a.dk == 64 ? delta_rows_kernel<64> : delta_rows_kernel<128>, a);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs &a, cudaStream_t s) { return launch_rows(a, s); }

}  // namespace gattn
