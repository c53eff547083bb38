// delta.cu -- the gated delta rule, row by row.
//
//   S <- e^g S,  w = beta (v - S^T k),  S <- S + k w^T,  out = scale S^T q
//
// Bound by the state: 8 bytes an element, read and written once per call.  The
// columns of S are independent of one another, so a warp works alone on 16 of them
// for one (sequence, head), the state in registers from the first row to the last:
// lane 4 g + c holds k-elements RPT g .. of columns 4 c .. 4 c + 3 (16-byte accesses,
// whole sectors).  One pass over it gives both sums of a row,
//   S^T k and S^T q  (out = scale (e^g S^T q + (q.k) w)),
// added up over the groups by shuffles: no shared memory, no barrier, and warps at
// different points cover each other's latencies.  (A CTA per head with the sums in
// shared memory spent a fifth of its time at barriers: 39 us for 32 sequences of 4
// rows and 32 heads of 128 x 128.)  32 sequences of one row take 25 us, 79 % of the copy
// rate over 134 MB of state; of four rows 38 us, 53 %: a row adds 4 us of arithmetic
// and shuffles to each warp's way.  One sequence of one row: 3.7 us.
#include "seq.cuh"
#include "tc5.cuh"

namespace gattn {

namespace {

constexpr int kWarps = 4;          // per CTA

// A row's operands as they come from memory.
template <int RPT>
struct RowIn {
    uint4 k[RPT / 8], q[RPT / 8];
    uint2 v;
    float g, beta;
};

template <int N>
__device__ __forceinline__ void unpack_row(const uint4 (&u)[N], float (&f)[8 * N])
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t w[4] = {u[n].x, u[n].y, u[n].z, u[n].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[8 * n + 2 * i] = bf16_lo(w[i]);
            f[8 * n + 2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <int DK>
__global__ void __launch_bounds__(kWarps * 32) delta_rows_kernel(const __grid_constant__ DeltaArgs a)
{
    constexpr int RPT = DK / 8;                   // k-elements of a lane
    const int lane = threadIdx.x & 31, grp = lane >> 2;
    const int parts = a.dv / 16;
    const long long job = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int h = (int)(job / parts % a.Hv), hk = h / (a.Hv / a.Hk);
    const long long sl = job / parts / a.Hv;
    if (sl >= a.sq.n)
        return;
    const int s = (int)sl, col = (int)(job % parts) * 16 + (lane & 3) * 4;
    int r0, len;
    seq_rows(a.sq, s, r0, len);
    const int slot = seq_slot_warp(a.sq, s, true);
    __nv_bfloat16 *out = a.out + (long long)h * a.os.head + col;
    if (slot < 0) {
        if (lane == 0)
            seq_flag(a.sq, GATTN_STATUS_RANGE);
        for (int t = r0 + grp; t < r0 + len; t += 8)
            *reinterpret_cast<uint2 *>(out + (long long)t * a.os.tok) = make_uint2(0, 0);
        return;
    }
    const long long so = slot * a.state_stride + ((long long)h * DK + grp * RPT) * a.dv + col;
    uint64_t S[RPT][2];                           // columns (0, 1) and (2, 3)
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const ulonglong2 x = a.state ? *reinterpret_cast<const ulonglong2 *>(a.state + so + (long long)i * a.dv)
                                     : make_ulonglong2(0, 0);
        S[i][0] = x.x;
        S[i][1] = x.y;
    }
    auto load = [&](int t) {
        RowIn<RPT> r;
        const uint4 *kp = reinterpret_cast<const uint4 *>(a.k + t * a.ks.tok + hk * a.ks.head + grp * RPT);
        const uint4 *qp = reinterpret_cast<const uint4 *>(a.q + t * a.qs.tok + hk * a.qs.head + grp * RPT);
#pragma unroll
        for (int n = 0; n < RPT / 8; ++n) {
            r.k[n] = kp[n];
            r.q[n] = qp[n];
        }
        r.v = *reinterpret_cast<const uint2 *>(a.v + t * a.vs.tok + h * a.vs.head + col);
        r.g = a.g[t * a.gt + h];
        r.beta = a.beta[t * a.bt + h];
        return r;
    };
    RowIn<RPT> in;
    if (len > 0)
        in = load(r0);
    for (int r = 0; r < len; ++r) {
        float k[RPT], q[RPT];
        unpack_row(in.k, k);
        unpack_row(in.q, q);
        const uint2 v = in.v;
        const float de = expf(in.g), be = in.beta;
        if (r + 1 < len)
            in = load(r0 + r + 1);
        float kk = 0.f, qq = 0.f, kq = 0.f;
        uint64_t dk[2] = {0, 0}, dq[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
            kq = fmaf(k[i], q[i], kq);
            const uint64_t k2 = pack2(k[i], k[i]), q2 = pack2(q[i], q[i]);
            dk[0] = fma2(S[i][0], k2, dk[0]);
            dk[1] = fma2(S[i][1], k2, dk[1]);
            dq[0] = fma2(S[i][0], q2, dq[0]);
            dq[1] = fma2(S[i][1], q2, dq[1]);
        }
        float x[11] = {kk, qq, kq};
        unpack2(dk[0], x[3], x[4]);
        unpack2(dk[1], x[5], x[6]);
        unpack2(dq[0], x[7], x[8]);
        unpack2(dq[1], x[9], x[10]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int e = 0; e < 11; ++e)
                x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
        // k and q count divided by their norms: fk, fq stand beside the sums
        const float fk = a.l2norm ? 1.f / sqrtf(x[0] + a.l2_eps) : 1.f;
        const float fq = a.l2norm ? 1.f / sqrtf(x[1] + a.l2_eps) : 1.f;
        const float dfk = de * fk;
        const float w0 = be * (bf16_lo(v.x) - dfk * x[3]), w1 = be * (bf16_hi(v.x) - dfk * x[4]);
        const float w2 = be * (bf16_lo(v.y) - dfk * x[5]), w3 = be * (bf16_hi(v.y) - dfk * x[6]);
        const uint64_t u0 = pack2(fk * w0, fk * w1), u1 = pack2(fk * w2, fk * w3), d2 = pack2(de, de);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const uint64_t k2 = pack2(k[i], k[i]);
            S[i][0] = fma2(k2, u0, mul2(S[i][0], d2));
            S[i][1] = fma2(k2, u1, mul2(S[i][1], d2));
        }
        if (grp == 0) {
            const float p = x[2] * fk, sc = a.scale * fq;
            *reinterpret_cast<uint2 *>(out + (long long)(r0 + r) * a.os.tok) =
                make_uint2(pack_bf16x2(sc * fmaf(p, w0, de * x[7]), sc * fmaf(p, w1, de * x[8])),
                           pack_bf16x2(sc * fmaf(p, w2, de * x[9]), sc * fmaf(p, w3, de * x[10])));
        }
    }
    if (a.state_out && (len > 0 || a.state_out != a.state))
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            *reinterpret_cast<ulonglong2 *>(a.state_out + so + (long long)i * a.dv) =
                make_ulonglong2(S[i][0], S[i][1]);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs &a, cudaStream_t s)
{
    const long long jobs = (long long)a.sq.n * a.Hv * (a.dv / 16);
    if (jobs / kWarps >= 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    return launch_seq(a.dk == 64 ? delta_rows_kernel<64> : delta_rows_kernel<128>,
                      dim3((unsigned)((jobs + kWarps - 1) / kWarps)), dim3(kWarps * 32), s, a);
}

}  // namespace gattn
