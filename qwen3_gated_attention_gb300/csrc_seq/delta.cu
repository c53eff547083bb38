// delta.cu -- the gated delta rule, row by row.
//
//   S <- e^g S,  w = beta (v - S^T k),  S <- S + k w^T,  out = scale S^T q
//
// Bound by the state: 8 bytes an element, read and written once per call.  The
// columns of S are independent of one another: a CTA owns CT of them for one
// (sequence, head), four to a thread (16-byte accesses, whole lines per warp), the
// k-elements split over the groups of CT/4 threads; the state stays in registers
// from the first row to the last.  One pass over it gives both sums of a row,
//   S^T k and S^T q  (out = scale (e^g S^T q + (q.k) w)),
// which the groups add up through shared memory at one barrier a row.
#include "seq.cuh"

namespace gattn {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;          // rows staged at a time, one per warp

template <int DK, int CT>
__global__ void __launch_bounds__(kThreads) delta_rows_kernel(const __grid_constant__ DeltaArgs a)
{
    constexpr int LANES = CT / 4;                 // threads across the columns
    constexpr int NR = kThreads / LANES;          // groups across the k-elements
    constexpr int RPT = DK / NR;                  // k-elements of a thread: RPT grp + i
    constexpr int WARPS = kThreads / 32;
    static_assert(RPT >= 1 && DK % NR == 0, "every group has k-elements");
    __shared__ __align__(16) float ks[kBatch][DK], qs[kBatch][DK];
    __shared__ float qk[kBatch], decay[kBatch], beta[kBatch];
    __shared__ __align__(16) float sums[2][2][WARPS][CT];   // row parity; S^T k, S^T q
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y, s = blockIdx.x, hk = h / (a.Hv / a.Hk);
    const int c4 = (threadIdx.x % LANES) * 4, grp = threadIdx.x / LANES;
    const int col = blockIdx.z * CT + c4;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    __nv_bfloat16 *out = a.out + (long long)h * a.os.head + col;
    if (slot < 0) {
        if (threadIdx.x == 0)
            seq_flag(a.sq, GATTN_STATUS_RANGE);
        for (int t = r0 + grp; t < r0 + len; t += NR)
            *reinterpret_cast<uint2 *>(out + (long long)t * a.os.tok) = make_uint2(0, 0);
        return;
    }
    const long long so = slot * a.state_stride + ((long long)h * DK + grp * RPT) * a.dv + col;
    float4 S[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        S[i] = a.state ? *reinterpret_cast<const float4 *>(a.state + so + (long long)i * a.dv)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b0 = 0; b0 < len; b0 += kBatch) {
        const int rows = min(kBatch, len - b0);
        if (warp < rows) {
            // a row's k and q, divided by their norms, and their product
            const int t = r0 + b0 + warp;
            const __nv_bfloat16 *kp = a.k + t * a.ks.tok + hk * a.ks.head;
            const __nv_bfloat16 *qp = a.q + t * a.qs.tok + hk * a.qs.head;
            float x[DK / 32], y[DK / 32], kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
            for (int i = 0; i < DK / 32; ++i) {
                x[i] = __bfloat162float(kp[lane + 32 * i]);
                y[i] = __bfloat162float(qp[lane + 32 * i]);
                kk = fmaf(x[i], x[i], kk);
                qq = fmaf(y[i], y[i], qq);
                kq = fmaf(x[i], y[i], kq);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                kk += __shfl_xor_sync(0xffffffffu, kk, o);
                qq += __shfl_xor_sync(0xffffffffu, qq, o);
                kq += __shfl_xor_sync(0xffffffffu, kq, o);
            }
            const float fk = a.l2norm ? 1.f / sqrtf(kk + a.l2_eps) : 1.f;
            const float fq = a.l2norm ? 1.f / sqrtf(qq + a.l2_eps) : 1.f;
#pragma unroll
            for (int i = 0; i < DK / 32; ++i) {
                ks[warp][lane + 32 * i] = x[i] * fk;
                qs[warp][lane + 32 * i] = y[i] * fq;
            }
            if (lane == 0) {
                qk[warp] = kq * fk * fq;
                decay[warp] = expf(a.g[t * a.gt + h]);
                beta[warp] = a.beta[t * a.bt + h];
            }
        }
        uint2 vn = *reinterpret_cast<const uint2 *>(a.v + (long long)(r0 + b0) * a.vs.tok + h * a.vs.head + col);
        __syncthreads();
        for (int r = 0; r < rows; ++r) {
            const int t = r0 + b0 + r, par = r & 1;
            const uint2 vw = vn;
            if (r + 1 < rows)
                vn = *reinterpret_cast<const uint2 *>(a.v + (long long)(t + 1) * a.vs.tok + h * a.vs.head + col);
            float dk[4] = {}, dq[4] = {};
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float k = ks[r][grp * RPT + i], q = qs[r][grp * RPT + i];
                dk[0] = fmaf(S[i].x, k, dk[0]);
                dk[1] = fmaf(S[i].y, k, dk[1]);
                dk[2] = fmaf(S[i].z, k, dk[2]);
                dk[3] = fmaf(S[i].w, k, dk[3]);
                dq[0] = fmaf(S[i].x, q, dq[0]);
                dq[1] = fmaf(S[i].y, q, dq[1]);
                dq[2] = fmaf(S[i].z, q, dq[2]);
                dq[3] = fmaf(S[i].w, q, dq[3]);
            }
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dk[e] += __shfl_xor_sync(0xffffffffu, dk[e], o);
                    dq[e] += __shfl_xor_sync(0xffffffffu, dq[e], o);
                }
            if (lane < LANES) {
                *reinterpret_cast<float4 *>(&sums[par][0][warp][c4]) = make_float4(dk[0], dk[1], dk[2], dk[3]);
                *reinterpret_cast<float4 *>(&sums[par][1][warp][c4]) = make_float4(dq[0], dq[1], dq[2], dq[3]);
            }
            __syncthreads();       // the buffers alternate: one barrier a row
            float4 sk = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(&sums[par][0][w][c4]);
                sk.x += x.x;
                sk.y += x.y;
                sk.z += x.z;
                sk.w += x.w;
            }
            const float de = decay[r], be = beta[r];
            const float w0 = be * (bf16_lo(vw.x) - de * sk.x), w1 = be * (bf16_hi(vw.x) - de * sk.y);
            const float w2 = be * (bf16_lo(vw.y) - de * sk.z), w3 = be * (bf16_hi(vw.y) - de * sk.w);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float k = ks[r][grp * RPT + i];
                S[i].x = fmaf(k, w0, S[i].x * de);
                S[i].y = fmaf(k, w1, S[i].y * de);
                S[i].z = fmaf(k, w2, S[i].z * de);
                S[i].w = fmaf(k, w3, S[i].w * de);
            }
            if (grp == r % NR) {
                float4 sq = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(&sums[par][1][w][c4]);
                    sq.x += x.x;
                    sq.y += x.y;
                    sq.z += x.z;
                    sq.w += x.w;
                }
                const float p = qk[r], sc = a.scale;
                *reinterpret_cast<uint2 *>(out + (long long)t * a.os.tok) =
                    make_uint2(pack_bf16x2(sc * fmaf(p, w0, de * sq.x), sc * fmaf(p, w1, de * sq.y)),
                               pack_bf16x2(sc * fmaf(p, w2, de * sq.z), sc * fmaf(p, w3, de * sq.w)));
            }
        }
        __syncthreads();           // the staged rows are replaced
    }
    if (a.state_out && (len > 0 || a.state_out != a.state))
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            *reinterpret_cast<float4 *>(a.state_out + so + (long long)i * a.dv) = S[i];
}

template <int DK, int CT>
cudaError_t launch(const DeltaArgs &a, cudaStream_t s)
{
    // one CTA per (sequence, head, CT columns); x is the dimension that may be long
    return launch_seq(delta_rows_kernel<DK, CT>, dim3((unsigned)a.sq.n, a.Hv, a.dv / CT), dim3(kThreads), s, a);
}

template <int DK>
cudaError_t launch_dk(const DeltaArgs &a, cudaStream_t s)
{
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    // wide column blocks read whole lines of the state and repeat the rows' work
    // least; narrow ones give a small batch enough CTAs
    const long long cols = (long long)a.sq.n * a.Hv * a.dv;
    if (a.dv % 128 == 0 && cols / 128 >= 2 * sms)
        return launch<DK, 128>(a, s);
    if (a.dv % 64 == 0 && cols / 64 >= 2 * sms)
        return launch<DK, 64>(a, s);
    return launch<DK, 32>(a, s);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs &a, cudaStream_t s)
{
    return a.dk == 64 ? launch_dk<64>(a, s) : launch_dk<128>(a, s);
}

}  // namespace gattn
