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
// different points cover each other's latencies.  A warp takes one such job after
// another; the next one's state and first row are on their way while it works.
//
// 32 sequences and 32 heads of 128 x 128: one row each 25 us, 80 % of the copy rate over
// 134 MB of state; four rows 37 us, 55 %: a row adds 4 us, its 560 instructions at three
// warps a scheduler.  One sequence of one row: 3.5 us.  (A CTA per head with the sums in
// shared memory spent a fifth of its time at barriers: 39 us for the four rows; each job
// a warp of its own 25.4 and 38.9 us; pairs along k instead of along the columns made
// no difference.)
#include <algorithm>

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
__global__ void __launch_bounds__(kWarps * 32, 3) delta_rows_kernel(const __grid_constant__ DeltaArgs a)
{
    constexpr int RPT = DK / 8;                   // k-elements of a lane
    __shared__ ulonglong2 ahead[kWarps][RPT][32]; // the next job's state: a lane's own elements
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane >> 2;
    // all of it below 2^31, see the launch
    const unsigned parts = a.dv / 16, heads = a.Hv, per_key = a.Hv / a.Hk;
    const unsigned jobs = a.sq.n * heads * parts, stride = gridDim.x * kWarps;
    ulonglong2 (*const buf)[32] = ahead[warp];
    struct Job {
        int h, col, r0, len, slot;
    };
    auto find = [&](unsigned job) {
        Job j;
        const unsigned sh = job / parts, s = sh / heads;
        j.h = sh - s * heads;
        j.col = (job - sh * parts) * 16 + (lane & 3) * 4;
        seq_rows(a.sq, s, j.r0, j.len);
        j.slot = seq_slot_warp(a.sq, s, true);
        return j;
    };
    auto place = [&](const Job &j) {
        return j.slot * a.state_stride + ((long long)j.h * DK + grp * RPT) * a.dv + j.col;
    };
    auto load = [&](const Job &j, int t) {
        RowIn<RPT> r;
        const int hk = (unsigned)j.h / per_key;
        const uint4 *kp = reinterpret_cast<const uint4 *>(a.k + t * a.ks.tok + hk * a.ks.head + grp * RPT);
        const uint4 *qp = reinterpret_cast<const uint4 *>(a.q + t * a.qs.tok + hk * a.qs.head + grp * RPT);
#pragma unroll
        for (int n = 0; n < RPT / 8; ++n) {
            r.k[n] = kp[n];
            r.q[n] = qp[n];
        }
        r.v = *reinterpret_cast<const uint2 *>(a.v + t * a.vs.tok + j.h * a.vs.head + j.col);
        r.g = a.g[t * a.gt + j.h];
        r.beta = a.beta[t * a.bt + j.h];
        return r;
    };
    unsigned job = blockIdx.x * kWarps + warp;
    if (job >= jobs)
        return;
    Job cur = find(job);
    uint64_t S[RPT][2];                           // columns (0, 1) and (2, 3)
    RowIn<RPT> in;
    {
        const long long so = place(cur);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const ulonglong2 x = a.state && cur.slot >= 0
                                     ? *reinterpret_cast<const ulonglong2 *>(a.state + so + (long long)i * a.dv)
                                     : make_ulonglong2(0, 0);
            S[i][0] = x.x;
            S[i][1] = x.y;
        }
        if (cur.slot >= 0 && cur.len > 0)
            in = load(cur, cur.r0);
    }
    for (;;) {
        job += stride;
        const bool more = job < jobs;
        Job nxt = cur;
        if (more) {
            nxt = find(job);
            __syncwarp();                         // the buffer has been read
            if (a.state && nxt.slot >= 0) {
                const float *from = a.state + place(nxt);
#pragma unroll
                for (int i = 0; i < RPT; ++i)
                    cp_async<16>(&buf[i][lane], from + (long long)i * a.dv);
            }
        }
        const bool rows_next = more && nxt.slot >= 0 && nxt.len > 0;
        const int len = cur.slot >= 0 ? cur.len : 0;
        __nv_bfloat16 *out = a.out + (long long)cur.h * a.os.head + cur.col;
        if (cur.slot < 0) {
            if (lane == 0)
                seq_flag(a.sq, GATTN_STATUS_RANGE);
            for (int t = cur.r0 + grp; t < cur.r0 + cur.len; t += 8)
                *reinterpret_cast<uint2 *>(out + (long long)t * a.os.tok) = make_uint2(0, 0);
        }
        if (len == 0 && rows_next)
            in = load(nxt, nxt.r0);
        for (int r = 0; r < len; ++r) {
            float k[RPT], q[RPT];
            unpack_row(in.k, k);
            unpack_row(in.q, q);
            const uint2 v = in.v;
            const float de = expf(in.g), be = in.beta;
            if (r + 1 < len)
                in = load(cur, cur.r0 + r + 1);
            else if (rows_next)
                in = load(nxt, nxt.r0);
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
                *reinterpret_cast<uint2 *>(out + (long long)(cur.r0 + r) * a.os.tok) =
                    make_uint2(pack_bf16x2(sc * fmaf(p, w0, de * x[7]), sc * fmaf(p, w1, de * x[8])),
                               pack_bf16x2(sc * fmaf(p, w2, de * x[9]), sc * fmaf(p, w3, de * x[10])));
            }
        }
        if (cur.slot >= 0 && a.state_out && (len > 0 || a.state_out != a.state)) {
            float *to = a.state_out + place(cur);
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                *reinterpret_cast<ulonglong2 *>(to + (long long)i * a.dv) = make_ulonglong2(S[i][0], S[i][1]);
        }
        if (!more)
            return;
        cp_async_wait_all();
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const ulonglong2 x = a.state && nxt.slot >= 0 ? buf[i][lane] : make_ulonglong2(0, 0);
            S[i][0] = x.x;
            S[i][1] = x.y;
        }
        cur = nxt;
    }
}

}  // namespace

cudaError_t launch_delta_step(const DeltaArgs &a, cudaStream_t s)
{
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    const long long jobs = (long long)a.sq.n * a.Hv * (a.dv / 16), ctas = (jobs + kWarps - 1) / kWarps;
    if (jobs > 0x7fffffff - 3 * kWarps * sms)
        return cudaErrorInvalidConfiguration;
    return launch_seq(a.dk == 64 ? delta_rows_kernel<64> : delta_rows_kernel<128>,
                      dim3((unsigned)std::min<long long>(ctas, 3 * sms)), dim3(kWarps * 32), s, a);
}

}  // namespace gattn
