// paged_weights.cu -- how much softmax weight the positions of a paged cache received:
//
//   w_out[p] = w[p] + sum over rows i that see p and heads h of the group of
//              exp(scale q_ih . k_p - lse_ih)
//
// with the logarithms of the softmax sums that the attention left.  Bound by memory: the
// keys are read once for all rows and heads of a group (64 of them; more take another
// pass over the CTA's own units, which L2 mostly still holds).  The work is cut as
// paged_ring.cuh says; a warp alone takes a unit, sums over the rows in its registers and
// writes each position once, so there are no atomics and the sums have one order.
// Measured: 16 sequences of 64 to 15001 positions, one to four rows of 32 heads of 256 over
// 8: 66 us, 6.3 TB/s, 94 % of the copy rate.  One token over 4001 positions: 5.4 us.  Many rows
// are slow: chunks of 30 to 500 rows of 16 heads over 4, behind 256 to 30000 positions, 1.6
// ms; one of 200 rows among seven single ones 1.2 ms, because the line counts a unit once
// however many passes it takes.
#include "paged_ring.cuh"

namespace gattn {

using namespace paged;

namespace {

template <int D>
struct Cfg {
    static constexpr int M = 64, CW = 8, NP = 4, THREADS = (CW + NP) * 32;
    static constexpr int U = kUnit<D>, UNIT = U * D * 2;
    static constexpr int FIT = (227 * 1024 - 2 * M * D * 2 - 4096) / UNIT;
    static constexpr int SLOTS = (FIT > 24 ? 24 : FIT) / CW * CW;
    static constexpr int SMEM = SLOTS * UNIT + 2 * M * D * 2 + 1024;
    using R = Ring<D, U, M, false, SLOTS, NP, CW, 1, CW>;
    static_assert(SMEM + sizeof(R) + 512 <= 227 * 1024 && SLOTS > 0, "");
};

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
    paged_weights_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap, int min_units)
{
    using C = Cfg<D>;
    using R = typename C::R;
    constexpr int CW = C::CW, U = C::U;
    extern __shared__ uint8_t raw[];
    __shared__ R ring;
    uint8_t *units = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = units + C::SLOTS * C::UNIT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.H / a.Hk;
    if (threadIdx.x == 0) {
        ring.init();
        prefetch_tensormap(&kmap);
    }
    pdl_wait();
    pdl_launch_dependents();
    const Run run = plan_run<C::THREADS, 0, U>(a, group, min_units);
    if (run.bad && blockIdx.x == 0 && threadIdx.x == 0)
        seq_flag(a.sq, GATTN_STATUS_RANGE);
    if (run.x0 >= run.x1)
        return;
    if (warp >= CW) {
        produce(a, ring, units, qbuf, &kmap, &kmap, run, group, warp - CW, [](const Part &, int) {});
        return;
    }
    const int g = lane >> 2, cq = lane & 3;
    const int btl = box_log2(a.pg.page, U), box = (1 << btl) * D * 2, dbs = (1 << btl) * 128;
    int it = 0;                        // units of the CTA before this part, modulo CW
    int slot = warp, phase = 0;        // of this warp's next unit
    for (int parts = 0;; ++parts) {
        const int b = parts & 1;
        if (!ring_wait(&ring.qfull[b], (uint32_t)((parts >> 1) & 1), &ring.abort, a.sq))
            return;
        const Part p = ring.part[b];
        if (!p.live)
            return;
        // a further pass over the same units adds to what the one before it wrote: every
        // warp has left that one
        if (p.pass && !ring_wait(&ring.qempty[b ^ 1], (uint32_t)(((parts - 1) >> 1) & 1), &ring.abort, a.sq))
            return;
        const int first_row = p.p0 + p.rowf, end = p.p0 + p.len;
        const int count = p.u1 - p.u0, tiles = (p.nrows + 7) / 8;
        const uint32_t qrow = smem_u32(qbuf) + b * R::QB + (lane & 7) * (D * 2);
        const long long at = p.s * a.w_seq + p.hk * a.w_head;
        const float *const from = p.pass ? a.w_out : a.w;
        const int known = p.pass ? end : p.p0;          // positions that have a weight
        for (int n = (warp - it) & (CW - 1); n < count; n += CW) {
            const int t0 = (p.u0 + n) * U;
            // what the positions have: g and 8 on of each 16
            float old[U / 16][2];
#pragma unroll
            for (int q = 0; q < U / 16; ++q)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int t = t0 + q * 16 + g + 8 * x;
                    old[q][x] = cq == 0 && from && t < known ? from[at + t] : 0.f;
                }
            if (!ring_wait(&ring.full[slot], phase, &ring.abort, a.sq))
                return;
            const uint32_t ks = smem_u32(units) + slot * C::UNIT;
            const unsigned there = ring.ok[slot];
            const bool mask = t0 + U - 1 > first_row || there != (1u << (U >> btl)) - 1u;
            // the unit, once for all rows
            uint32_t ak[D / 16][U / 16][4];
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int q = 0; q < U / 16; ++q) {
                    const int in = (q * 16) >> btl, off = (q * 16) & ((1 << btl) - 1);
                    ldsm_x4(ak[k][q], ks + in * box + (k >> 2) * dbs + (off + (lane & 15)) * 128 +
                                          ((((2 * k + (lane >> 4)) & 7) ^ (lane & 7)) << 4));
                }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&ring.empty[slot]);         // the slot is free
            slot += CW;
            if (slot >= R::SLOTS) {
                slot -= R::SLOTS;
                phase ^= 1;
            }
            float sum[U / 16][2];
#pragma unroll
            for (int q = 0; q < U / 16; ++q)
                sum[q][0] = sum[q][1] = 0.f;
            for (int rt = 0; rt < tiles; ++rt) {
                constexpr int CHAINS = 64 / U;
                float sc[CHAINS][U / 16][4];
#pragma unroll
                for (int c = 0; c < CHAINS; ++c)
#pragma unroll
                    for (int q = 0; q < U / 16; ++q)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[c][q][e] = 0.f;
#pragma unroll
                for (int k = 0; k < D / 16; k += 2) {
                    uint32_t qf[4];
                    ldsm_x4(qf, qrow + rt * 8 * (D * 2) + (((2 * k + (lane >> 3)) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int q = 0; q < U / 16; ++q)
                            mma(sc[(k + x) % CHAINS][q], ak[k + x][q], qf[2 * x], qf[2 * x + 1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = rt * 8 + 2 * cq + e;
                    const float lse = ring.lse[b][i];
                    // (a row that saw nothing gives nothing, whatever its keys hold)
                    const int lim = i < p.nrows && lse != INFINITY ? first_row + (p.hf + i) / group : -1;
#pragma unroll
                    for (int q = 0; q < U / 16; ++q)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int t = q * 16 + g + 8 * x;
                            float v = sc[0][q][2 * x + e];
                            if (CHAINS >= 2)
                                v += sc[1 % CHAINS][q][2 * x + e];
                            if (CHAINS == 4)
                                v += sc[2 % CHAINS][q][2 * x + e] + sc[3 % CHAINS][q][2 * x + e];
                            v = exp2_approx(fmaf(v, a.scale_log2, -lse));
                            if (lim < 0 || (mask && (t0 + t > lim || !((there >> (t >> btl)) & 1u))))
                                v = 0.f;
                            sum[q][x] += v;
                        }
                }
            }
#pragma unroll
            for (int q = 0; q < U / 16; ++q)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float v = sum[q][x];
                    v += __shfl_xor_sync(0xffffffffu, v, 1);
                    v += __shfl_xor_sync(0xffffffffu, v, 2);
                    const int t = t0 + q * 16 + g + 8 * x;
                    if (cq == 0 && t < end)
                        a.w_out[at + t] = old[q][x] + v;
                }
        }
        it = (it + count) & (CW - 1);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&ring.qempty[b]);
    }
}

template <int D>
cudaError_t launch(const PagedAttnArgs &a, cudaStream_t s)
{
    using C = Cfg<D>;
    auto *fn = paged_weights_kernel<D>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(fn, C::SMEM, done);
    if (e != cudaSuccess)
        return e;
    int sms = 0;
    e = sm_count(&sms);
    if (e != cudaSuccess)
        return e;
    CUtensorMap km;
    if (!encode_pages(&km, a.pg, false, a.Hk, D, 1 << box_log2(a.pg.page, C::U)))
        return cudaErrorInvalidValue;
    return launch_paged(fn, dim3(sms < kMaxCtas ? sms : kMaxCtas), dim3(C::THREADS), C::SMEM, s, a, km, 4);
}

}  // namespace

cudaError_t launch_paged_weights(const PagedAttnArgs &a, cudaStream_t s)
{
    switch (a.d) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    case 192: return launch<192>(a, s);
    default: return launch<256>(a, s);
    }
}

}  // namespace gattn
