// paged.cuh -- what the paged-cache operators share: parameter blocks and launchers
// (internal; not part of the ABI).
#pragma once

#include <type_traits>

#include "seq.cuh"

namespace gattn {

constexpr int kMaxPos = 1 << 24;       // positions are exact in fp32 up to here

// element strides of a pool of pages
struct PageStride {
    long long tok, head, page;
};

// Pools of pages and the table that says where a sequence's positions are.
struct Pages {
    void *kp, *vp;
    PageStride k, v;
    const int *table;
    long long table_stride;
    int pages, page, width;    // pages of the pools, positions of a page, pages of a table row
};

struct PagedRowsArgs {
    SeqArgs sq;
    Pages pg;
    const int *pos, *positions;
    const void *q, *k, *v;
    RowStride qs, ks, vs, os;
    const uint16_t *q_norm, *k_norm;
    __nv_bfloat16 *q_out;
    long long cap;
    int H, Hk, d, rd, pairs;
    float eps, turn_size;
    float2 inv_freq[128];      // [rd / 2] as float (hi, lo) pairs
};

// Attention of new rows over pages, and the weights that they give to positions.
struct PagedAttnArgs {
    SeqArgs sq;
    Pages pg;
    const int *pos;
    const __nv_bfloat16 *q;
    RowStride qs, os, gs;
    int H, Hk, d;
    long long cap;             // positions that a sequence may have
    float scale_log2;
    // attention
    const void *gate;
    int gate_f32;
    __nv_bfloat16 *out;
    float *lse;                // [total][H], null: not wanted; read by the weights
    void *ws;
    // weights: strides of both; w null: zeros
    const float *w;
    float *w_out;
    long long w_seq, w_head;
};

struct PagedEvictArgs {
    Pages pg;
    const int *out_table;      // null: in place
    long long out_stride;
    int n;
    const int *lengths;
    int *lengths_out;
    const float *w;
    float *w_out;
    long long w_seq, w_head, wo_seq, wo_head;
    int *kept;                 // [n][Hk][keep]
    int Hk, d, keep, recent;
    long long cap, out_cap;    // positions that a sequence may have before and after
    unsigned *status;
};

// Launches that may be set up while the work before them on the stream ends.  The rules of
// these kernels:
//   - Every block waits for that work (pdl_wait) before it ends, and before it touches
//     memory; but see paged_move_kernel.
//   - A kernel that lets the next one be set up early (pdl_launch_dependents; attention,
//     moves and the close in place do not) does so in every block behind its own wait.
// So a kernel that has started behind one of them knows, before its own wait, that all work
// in front of that one has ended: paged_move_kernel, always behind paged_select_kernel, reads
// and writes what the selection does not write or read.
template <class... K, class... A>
inline cudaError_t launch_paged(void (*f)(K...), dim3 grid, dim3 block, int smem, cudaStream_t s, A &&...args)
{
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, static_cast<A &&>(args)...);
}

cudaError_t launch_paged_rows(const PagedRowsArgs &a, int x_f32, cudaStream_t s);
cudaError_t launch_paged_attn(const PagedAttnArgs &a, cudaStream_t s);
cudaError_t launch_paged_weights(const PagedAttnArgs &a, cudaStream_t s);
cudaError_t launch_paged_evict(const PagedEvictArgs &a, cudaStream_t s);
// bytes of device memory that an attention of these shapes needs
long long paged_attn_workspace(int d, int group, int n, int total);

}  // namespace gattn
