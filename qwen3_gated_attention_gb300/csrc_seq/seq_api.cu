// seq_api.cu -- host side of the packed-sequence entry points of gattn.h:
// argument checks and parameter blocks.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "seq.cuh"

using namespace gattn;

namespace {

gattn_status bad(gattn_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
gattn_status bad(gattn_status st, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    gattn_set_error(buf);
    return st;
}

#define CHECK(expr)                        \
    do {                                   \
        const gattn_status st_ = (expr);   \
        if (st_ != GATTN_OK)               \
            return st_;                    \
    } while (0)

gattn_status cuda_status(const char *what, cudaError_t e)
{
    return e == cudaSuccess ? GATTN_OK
                            : bad(GATTN_E_CUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// A row tensor: 16-byte aligned base, positive strides in multiples of 8 elements.
gattn_status check_rows(const char *name, const void *p, int64_t tok, int64_t head)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "%s is NULL", name);
    if (misaligned(p))
        return bad(GATTN_E_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (tok <= 0 || head <= 0 || ((tok | head) & 7))
        return bad(GATTN_E_INVALID_ARG,
                   "%s strides must be positive multiples of 8 elements (got %lld, %lld)", name,
                   (long long)tok, (long long)head);
    // the tensor maps hold strides below 2^40 bytes
    if (tok >= (1ll << 38) || head >= (1ll << 38))
        return bad(GATTN_E_INVALID_ARG, "%s strides are too large", name);
    return GATTN_OK;
}

// One axis of a tensor that is written: its step in elements and its entries.
struct Axis {
    int64_t step, n;
};

// Rows of d elements that are written: no two of them may share memory.  From the
// nearest step on, each has to span all that the nearer ones reach.
gattn_status check_apart(const char *name, int64_t d, std::initializer_list<Axis> axes)
{
    Axis a[3];
    int n = 0;
    for (const Axis &x : axes)
        if (x.n > 1)
            a[n++] = x;
    std::sort(a, a + n, [](const Axis &x, const Axis &y) { return x.step < y.step; });
    // steps stay below 2^38 and entries below 2^31: with a span of at most 2^62 so far,
    // the next one is compared by division and cannot overflow before it is refused
    int64_t span = d;
    for (int i = 0; i < n; ++i) {
        if (a[i].step < span)
            return bad(GATTN_E_INVALID_ARG, "%s strides make its rows overlap (a step of %lld within %lld elements)",
                       name, (long long)a[i].step, (long long)span);
        if (a[i].n - 1 > ((1ll << 62) - span) / a[i].step)
            span = 1ll << 62;
        else
            span += (a[i].n - 1) * a[i].step;
    }
    return GATTN_OK;
}

gattn_status check_out(const char *name, const void *p, int64_t tok, int64_t head, int64_t d, int64_t rows,
                       int64_t heads)
{
    CHECK(check_rows(name, p, tok, head));
    return check_apart(name, d, {{tok, rows}, {head, heads}});
}

// Device arrays of 32-bit words; NULL passes.
gattn_status check_words(std::initializer_list<const void *> p)
{
    for (const void *x : p)
        if (reinterpret_cast<uintptr_t>(x) & 3)
            return bad(GATTN_E_INVALID_ARG, "offsets, positions, slots and status must be 4-byte aligned");
    return GATTN_OK;
}

gattn_status check_seqs(int32_t n, int32_t total)
{
    if (n < 0 || total < 0)
        return bad(GATTN_E_INVALID_ARG, "num_seqs and total_rows must be >= 0");
    if (total > (1 << 30) || n > (1 << 24))
        return bad(GATTN_E_INVALID_ARG, "num_seqs or total_rows is too large");
    return GATTN_OK;
}

gattn_status check_heads(int32_t H, int32_t Hk)
{
    if (H <= 0 || Hk <= 0 || H % Hk)
        return bad(GATTN_E_INVALID_ARG, "heads must be > 0 and a multiple of the key heads");
    return GATTN_OK;
}

}  // namespace

extern "C" {

gattn_status gattn_prompt_rows(const gattn_prompt_rows_desc *p, gattn_stream stream)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    CHECK(check_heads(p->num_heads, p->num_kv_heads));
    CHECK(check_seqs(p->num_seqs, p->total_rows));
    if (p->head_dim <= 0 || p->head_dim % 64 || p->head_dim > 256)
        return bad(GATTN_E_UNSUPPORTED, "head_dim %d: a multiple of 64 <= 256 is needed", p->head_dim);
    if (p->x_dtype != GATTN_DTYPE_F32 && p->x_dtype != GATTN_DTYPE_BF16)
        return bad(GATTN_E_INVALID_ARG, "x_dtype must be GATTN_DTYPE_F32 or GATTN_DTYPE_BF16");
    if (!(p->partial_rotary_factor > 0.f && p->partial_rotary_factor <= 1.f))
        return bad(GATTN_E_INVALID_ARG, "partial_rotary_factor must be in (0, 1]");
    const int rd = (int)((double)p->head_dim * (double)p->partial_rotary_factor);
    if (rd < 2 || (rd & 1))
        return bad(GATTN_E_INVALID_ARG, "rotary dims %d must be even and >= 2", rd);
    if (!(p->rope_theta > 0.f) || !std::isfinite(p->rope_theta) || !(p->rms_eps >= 0.f))
        return bad(GATTN_E_INVALID_ARG, "rope_theta must be > 0 and rms_eps >= 0");
    CHECK(check_rows("q", p->q, p->q_stride_token, p->q_stride_head));
    CHECK(check_rows("k", p->k, p->k_stride_token, p->k_stride_head));
    CHECK(check_rows("v", p->v, p->v_stride_token, p->v_stride_head));
    CHECK(check_out("q_out", p->q_out, p->o_stride_token, p->o_stride_head, p->head_dim, p->total_rows,
                    p->num_heads));
    CHECK(check_rows("k_cache", p->k_cache, p->kc_stride_token, p->kc_stride_head));
    CHECK(check_rows("k_cache", p->k_cache, p->kc_stride_batch, 8));
    CHECK(check_rows("v_cache", p->v_cache, p->vc_stride_token, p->vc_stride_head));
    CHECK(check_rows("v_cache", p->v_cache, p->vc_stride_batch, 8));
    CHECK(check_apart("k_cache", p->head_dim, {{p->kc_stride_token, p->cache_capacity},
                                               {p->kc_stride_head, p->num_kv_heads},
                                               {p->kc_stride_batch, p->cache_batch}}));
    CHECK(check_apart("v_cache", p->head_dim, {{p->vc_stride_token, p->cache_capacity},
                                               {p->vc_stride_head, p->num_kv_heads},
                                               {p->vc_stride_batch, p->cache_batch}}));
    CHECK(check_words({p->cu_rows, p->cache_pos, p->slots, p->status}));
    if (misaligned(p->q_norm) || misaligned(p->k_norm))
        return bad(GATTN_E_INVALID_ARG, "q_norm and k_norm must be 16-byte aligned");
    if (!p->cu_rows || !p->cache_pos || !p->q_norm || !p->k_norm)
        return bad(GATTN_E_INVALID_ARG, "cu_rows, cache_pos, q_norm or k_norm is NULL");
    if (p->cache_batch <= 0 || p->cache_capacity <= 0)
        return bad(GATTN_E_INVALID_ARG, "cache_batch and cache_capacity must be > 0");
    if (p->cache_capacity > (1 << 24))
        return bad(GATTN_E_UNSUPPORTED, "cache_capacity %d: positions are exact up to 2^24", p->cache_capacity);
    if (p->num_seqs == 0 || p->total_rows == 0)
        return GATTN_OK;
    PromptRowsArgs a{};
    a.sq = {p->cu_rows, p->slots, p->num_seqs, p->total_rows, 0, p->cache_batch, p->status};
    a.pos = p->cache_pos;
    a.q = p->q;
    a.k = p->k;
    a.v = p->v;
    a.qs = {p->q_stride_token, p->q_stride_head};
    a.ks = {p->k_stride_token, p->k_stride_head};
    a.vs = {p->v_stride_token, p->v_stride_head};
    a.os = {p->o_stride_token, p->o_stride_head};
    a.q_norm = p->q_norm;
    a.k_norm = p->k_norm;
    a.q_out = static_cast<__nv_bfloat16 *>(p->q_out);
    a.kc = static_cast<__nv_bfloat16 *>(p->k_cache);
    a.vc = static_cast<__nv_bfloat16 *>(p->v_cache);
    a.cap = p->cache_capacity;
    a.kct = p->kc_stride_token;
    a.kch = p->kc_stride_head;
    a.kcb = p->kc_stride_batch;
    a.vct = p->vc_stride_token;
    a.vch = p->vc_stride_head;
    a.vcb = p->vc_stride_batch;
    a.H = p->num_heads;
    a.Hk = p->num_kv_heads;
    a.d = p->head_dim;
    a.rd = rd;
    a.eps = p->rms_eps;
    // theta^(-2i/rd), by the power anew every 8th time: a few ulp of a double apart
    const double step = std::pow((double)p->rope_theta, -2.0 / rd);
    double f = 1.;
    for (int i = 0; i < rd / 2; ++i) {
        f = i % 8 ? f * step : std::pow((double)p->rope_theta, -2.0 * i / rd);
        a.inv_freq[i].x = (float)f;
        a.inv_freq[i].y = (float)(f - (double)a.inv_freq[i].x);
    }
    return cuda_status("gattn_prompt_rows",
                       launch_prompt_rows(a, p->x_dtype == GATTN_DTYPE_F32,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

gattn_status gattn_prompt_attention(const gattn_prompt_attention_desc *p, gattn_stream stream)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    CHECK(check_heads(p->num_heads, p->num_kv_heads));
    CHECK(check_seqs(p->num_seqs, p->total_rows));
    if (p->head_dim <= 0 || p->head_dim % 64 || p->head_dim > 256)
        return bad(GATTN_E_UNSUPPORTED, "head_dim %d: a multiple of 64 <= 256 is needed", p->head_dim);
    if (p->num_heads > 65536 / p->head_dim)
        return bad(GATTN_E_UNSUPPORTED, "num_heads * head_dim must be <= 65536");
    if (!(p->scale > 0.f) || !std::isfinite(p->scale))
        return bad(GATTN_E_INVALID_ARG, "scale must be finite and > 0");
    CHECK(check_rows("q", p->q, p->q_stride_token, p->q_stride_head));
    const bool keys = p->k || p->v || p->kv_rows != 0;
    if (keys) {
        CHECK(check_rows("k", p->k, p->k_stride_token, p->k_stride_head));
        CHECK(check_rows("v", p->v, p->v_stride_token, p->v_stride_head));
        CHECK(check_rows("k", p->k, p->k_stride_batch, 8));
        CHECK(check_rows("v", p->v, p->v_stride_batch, 8));
    }
    CHECK(check_out("out", p->out, p->o_stride_token, p->o_stride_head, p->head_dim, p->total_rows,
                    p->num_heads));
    CHECK(check_words({p->cu_rows, p->cu_kv, p->cache_pos, p->slots, p->status}));
    if (p->gate) {
        CHECK(check_rows("gate", p->gate, p->g_stride_token, p->g_stride_head));
        if (p->gate_dtype != GATTN_DTYPE_F32 && p->gate_dtype != GATTN_DTYPE_BF16)
            return bad(GATTN_E_INVALID_ARG, "gate_dtype must be GATTN_DTYPE_F32 or GATTN_DTYPE_BF16");
    }
    if (!p->cu_rows)
        return bad(GATTN_E_INVALID_ARG, "cu_rows is NULL");
    if (p->kv_batch <= 0 || (keys && p->kv_rows <= 0) || p->max_kv < 0)
        return bad(GATTN_E_INVALID_ARG, "kv_batch and kv_rows must be > 0 (kv_rows 0 without k and v), max_kv >= 0");
    if (p->kv_rows > (1 << 30))
        return bad(GATTN_E_INVALID_ARG, "kv_rows is too large");
    if (!p->cache_pos && (p->kv_batch != 1 || p->slots))
        return bad(GATTN_E_INVALID_ARG, "packed keys have kv_batch 1 and no slots");
    if (p->cache_pos && p->cu_kv)
        return bad(GATTN_E_INVALID_ARG, "cu_kv is for packed keys: cache_pos must be NULL");
    if (p->num_seqs == 0 || p->total_rows == 0)
        return GATTN_OK;
    PromptAttnArgs a{};
    a.sq = {p->cu_rows, p->slots, p->num_seqs, p->total_rows, 0, p->kv_batch, p->status};
    a.cu_kv = p->cu_kv ? p->cu_kv : p->cu_rows;
    a.pos = p->cache_pos;
    a.q = static_cast<const __nv_bfloat16 *>(p->q);
    a.k = static_cast<const __nv_bfloat16 *>(p->k);
    a.v = static_cast<const __nv_bfloat16 *>(p->v);
    a.qs = {p->q_stride_token, p->q_stride_head};
    a.os = {p->o_stride_token, p->o_stride_head};
    a.gs = {p->g_stride_token, p->g_stride_head};
    a.gate = p->gate;
    a.gate_f32 = p->gate_dtype == GATTN_DTYPE_F32;
    a.kv_batch = p->kv_batch;
    a.kv_rows = p->kv_rows;
    a.kt = p->k_stride_token;
    a.kh = p->k_stride_head;
    a.kb = p->k_stride_batch;
    a.vt = p->v_stride_token;
    a.vh = p->v_stride_head;
    a.vb = p->v_stride_batch;
    a.out = static_cast<__nv_bfloat16 *>(p->out);
    a.H = p->num_heads;
    a.Hk = p->num_kv_heads;
    a.d = p->head_dim;
    a.scale_log2 = (float)(1.4426950408889634 * (double)p->scale);
    a.max_kv = p->max_kv;
    return cuda_status("gattn_prompt_attention",
                       launch_prompt_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

static gattn_status delta_args(const gattn_delta_desc *p, DeltaArgs &a)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    CHECK(check_heads(p->num_v_heads, p->num_k_heads));
    CHECK(check_seqs(p->num_seqs, p->total_rows));
    if (p->k_dim != 64 && p->k_dim != 128)
        return bad(GATTN_E_UNSUPPORTED, "k_dim %d: 64 or 128 is needed", p->k_dim);
    if (p->v_dim <= 0 || p->v_dim % 32 || p->v_dim > 256)
        return bad(GATTN_E_UNSUPPORTED, "v_dim %d: a multiple of 32 <= 256 is needed", p->v_dim);
    if (p->num_v_heads > 65535)
        return bad(GATTN_E_UNSUPPORTED, "num_v_heads must be <= 65535");
    if (!std::isfinite(p->scale))
        return bad(GATTN_E_INVALID_ARG, "scale must be finite");
    if (p->qk_l2norm && !(p->l2_eps >= 0.f))
        return bad(GATTN_E_INVALID_ARG, "l2_eps must be >= 0");
    if (p->total_rows > 0) {
        CHECK(check_rows("q", p->q, p->q_stride_token, p->q_stride_head));
        CHECK(check_rows("k", p->k, p->k_stride_token, p->k_stride_head));
        CHECK(check_rows("v", p->v, p->v_stride_token, p->v_stride_head));
        CHECK(check_out("out", p->out, p->o_stride_token, p->o_stride_head, p->v_dim, p->total_rows,
                        p->num_v_heads));
        if (!p->g || !p->beta)
            return bad(GATTN_E_INVALID_ARG, "g or beta is NULL");
        if ((reinterpret_cast<uintptr_t>(p->g) | reinterpret_cast<uintptr_t>(p->beta)) & 3)
            return bad(GATTN_E_INVALID_ARG, "g and beta must be 4-byte aligned");
        if (p->g_stride_token < p->num_v_heads || p->beta_stride_token < p->num_v_heads)
            return bad(GATTN_E_INVALID_ARG, "g and beta row strides must be >= num_v_heads");
    }
    CHECK(check_words({p->cu_rows, p->slots, p->status}));
    if (!p->cu_rows && p->num_seqs > 0 && p->total_rows % p->num_seqs)
        return bad(GATTN_E_INVALID_ARG, "without cu_rows total_rows must be a multiple of num_seqs");
    if (p->state || p->state_out) {
        if (p->num_slots <= 0)
            return bad(GATTN_E_INVALID_ARG, "num_slots must be > 0");
        if (misaligned(p->state) || misaligned(p->state_out))
            return bad(GATTN_E_INVALID_ARG, "state and state_out must be 16-byte aligned");
        if (p->state_stride < (int64_t)p->num_v_heads * p->k_dim * p->v_dim || (p->state_stride & 3))
            return bad(GATTN_E_INVALID_ARG,
                       "state_stride must be a multiple of 4 and cover a slot's heads");
    } else if (p->slots) {
        return bad(GATTN_E_INVALID_ARG, "slots without a state");
    }
    a = DeltaArgs{};
    const bool stateless = !p->state && !p->state_out;
    a.sq = {p->cu_rows, p->slots, p->num_seqs, p->total_rows,
            !p->cu_rows && p->num_seqs > 0 ? p->total_rows / p->num_seqs : 0,
            stateless ? p->num_seqs : p->num_slots, p->status};
    a.q = static_cast<const __nv_bfloat16 *>(p->q);
    a.k = static_cast<const __nv_bfloat16 *>(p->k);
    a.v = static_cast<const __nv_bfloat16 *>(p->v);
    a.qs = {p->q_stride_token, p->q_stride_head};
    a.ks = {p->k_stride_token, p->k_stride_head};
    a.vs = {p->v_stride_token, p->v_stride_head};
    a.os = {p->o_stride_token, p->o_stride_head};
    a.g = p->g;
    a.beta = p->beta;
    a.gt = p->g_stride_token;
    a.bt = p->beta_stride_token;
    a.state = p->state;
    a.state_out = p->state_out;
    a.state_stride = p->state_stride;
    a.out = static_cast<__nv_bfloat16 *>(p->out);
    a.Hk = p->num_k_heads;
    a.Hv = p->num_v_heads;
    a.dk = p->k_dim;
    a.dv = p->v_dim;
    a.scale = p->scale;
    a.l2norm = p->qk_l2norm != 0;
    a.l2_eps = p->l2_eps;
    return GATTN_OK;
}

gattn_status gattn_delta_prompt(const gattn_delta_desc *p, gattn_stream stream)
{
    DeltaArgs a;
    CHECK(delta_args(p, a));
    if (a.sq.n == 0)
        return GATTN_OK;
    return cuda_status("gattn_delta_prompt",
                       launch_delta_prompt(a, reinterpret_cast<cudaStream_t>(stream)));
}

gattn_status gattn_delta_step(const gattn_delta_desc *p, gattn_stream stream)
{
    DeltaArgs a;
    CHECK(delta_args(p, a));
    if (a.sq.n == 0)
        return GATTN_OK;
    return cuda_status("gattn_delta_step",
                       launch_delta_step(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
