// seq.cuh -- what the packed-sequence operators share: parameter blocks,
// launchers and the lookup of a row's sequence (internal; not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "gattn.h"

namespace gattn {

// element strides of a row tensor
struct RowStride {
    long long tok, head;
};

// Packed sequences as the kernels see them.
struct SeqArgs {
    const int *cu;        // [n + 1]; null: `uniform` rows each
    const int *slots;     // [n] or null
    int n, total, uniform;
    int num_slots;
    unsigned *status;
};

struct PromptRowsArgs {
    SeqArgs sq;
    const int *pos;
    const void *q, *k, *v;
    RowStride qs, ks, vs, os;
    const uint16_t *q_norm, *k_norm;
    __nv_bfloat16 *q_out, *kc, *vc;
    int cap;
    long long kct, kch, kcb, vct, vch, vcb;
    int H, Hk, d, rd;
    float eps;
    float2 inv_freq[128];     // [rd / 2] as float (hi, lo) pairs
};

struct PromptAttnArgs {
    SeqArgs sq;
    const int *cu_kv, *pos;
    const __nv_bfloat16 *q, *k, *v;
    RowStride qs, os, gs;
    const void *gate;
    int gate_f32;
    int kv_batch, kv_rows;
    long long kt, kh, kb, vt, vh, vb;
    __nv_bfloat16 *out;
    int H, Hk, d;
    float scale_log2;
    int max_kv;
};

struct DeltaArgs {
    SeqArgs sq;
    const __nv_bfloat16 *q, *k, *v;
    RowStride qs, ks, vs, os;
    const float *g, *beta;
    long long gt, bt;
    const float *state;
    float *state_out;
    long long state_stride;
    __nv_bfloat16 *out;
    int Hk, Hv, dk, dv;
    float scale, l2_eps;
    int l2norm;
};

// Lets a kernel take `bytes` of dynamic shared memory on the current device, once
// per device (`done`: a bit for each of the first 64).
template <class F>
inline cudaError_t allow_smem(F *fn, int bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit))
        return cudaSuccess;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

inline cudaError_t sm_count(int *n)
{
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return e == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : e;
}

// A plain launch that reports its own status only.
template <class... K, class... A>
inline cudaError_t launch_seq(void (*f)(K...), dim3 grid, dim3 block, cudaStream_t s, A &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, f, static_cast<A &&>(args)...);
}

cudaError_t launch_prompt_rows(const PromptRowsArgs &a, int x_f32, cudaStream_t s);
cudaError_t launch_prompt_attn(const PromptAttnArgs &a, cudaStream_t s);
cudaError_t launch_delta_step(const DeltaArgs &a, cudaStream_t s);
cudaError_t launch_delta_prompt(const DeltaArgs &a, cudaStream_t s);

#ifdef __CUDACC__

__device__ __forceinline__ int seq_begin(const SeqArgs &q, int s)
{
    return q.cu ? q.cu[s] : s * q.uniform;
}

// Rows of sequence s, clipped to the rows the tensors hold.
__device__ __forceinline__ void seq_rows(const SeqArgs &q, int s, int &r0, int &len)
{
    r0 = seq_begin(q, s);
    const int r1 = min(seq_begin(q, s + 1), q.total);
    r0 = max(r0, 0);
    len = max(r1 - r0, 0);
}

// The sequence that owns packed row t (the last s with cu[s] <= t), or -1 for a
// row outside [cu[0], cu[n]).  Called by a whole warp: 32-way search.
__device__ __forceinline__ int find_seq_warp(const SeqArgs &q, int t)
{
    const int lane = threadIdx.x & 31;
    if (!q.cu)
        return q.uniform > 0 && t / q.uniform < q.n ? t / q.uniform : -1;
    if (t < q.cu[0] || t >= q.cu[q.n])
        return -1;
    int lo = 0, hi = q.n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < hi && q.cu[i] <= t);
        // cu is non-decreasing, so the set lanes are the first ones
        const int c = 31 - __clz(m | 1u);
        lo += c * step;
        hi = min(lo + step, hi);
    }
    return lo;
}

// The slot of sequence s, or -1 when it lies outside the slots or an earlier
// sequence has it already.  Called by a whole warp.
__device__ __forceinline__ int seq_slot_warp(const SeqArgs &q, int s, bool unique)
{
    if (!q.slots)
        return s < q.num_slots ? s : -1;
    const int slot = q.slots[s];
    if (slot < 0 || slot >= q.num_slots)
        return -1;
    if (unique) {
        bool taken = false;
        for (int i = threadIdx.x & 31; i < s; i += 32)
            taken |= q.slots[i] == slot;
        if (__any_sync(0xffffffffu, taken))
            return -1;
    }
    return slot;
}

__device__ __forceinline__ void seq_flag(const SeqArgs &q, unsigned bit)
{
    if (q.status)
        atomicOr(q.status, bit);
}

// 8 bf16 at a 16-byte boundary as floats
__device__ __forceinline__ void ld_bf16x8(const __nv_bfloat16 *p, float (&f)[8])
{
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

#endif  // __CUDACC__

}  // namespace gattn

void gattn_set_error(const char *msg);
