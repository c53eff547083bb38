// paged_api.cu -- host side of the paged-cache entry points of gattn.h: argument checks
// and parameter blocks.
#include <cmath>

#include "paged.cuh"
#include "seq_check.h"

using namespace gattn;
using namespace gattn::check;

namespace {

gattn_status check_dim(int32_t d)
{
    if (d <= 0 || d % 64 || d > 256)
        return bad(GATTN_E_UNSUPPORTED, "head_dim %d: a multiple of 64 <= 256 is needed", d);
    return GATTN_OK;
}

gattn_status check_pool(const char *name, const void *p, int64_t tok, int64_t head, int64_t page)
{
    CHECK(check_rows(name, p, tok, head));
    return check_rows(name, p, page, 8);
}

// The pools that a call writes must keep their rows apart.
gattn_status check_pages(const gattn_pages &g, int32_t Hk, int32_t d, bool values, bool written)
{
    if (g.page_size < 16 || g.page_size % 16)
        return bad(GATTN_E_UNSUPPORTED, "page_size %d: a multiple of 16 is needed", g.page_size);
    if (g.num_pages <= 0 || g.table_width <= 0)
        return bad(GATTN_E_INVALID_ARG, "num_pages and table_width must be > 0");
    if (g.table_width > (1 << 24) / g.page_size)
        return bad(GATTN_E_UNSUPPORTED, "table_width * page_size: positions are exact up to 2^24");
    if (!g.table)
        return bad(GATTN_E_INVALID_ARG, "table is NULL");
    if (g.table_stride < g.table_width)
        return bad(GATTN_E_INVALID_ARG, "table_stride must be >= table_width");
    CHECK(check_words({g.table}));
    CHECK(check_pool("k_pages", g.k_pages, g.k_stride_token, g.k_stride_head, g.k_stride_page));
    if (values)
        CHECK(check_pool("v_pages", g.v_pages, g.v_stride_token, g.v_stride_head, g.v_stride_page));
    if (written) {
        CHECK(check_apart("k_pages", d, {{g.k_stride_token, g.page_size}, {g.k_stride_head, Hk}, {g.k_stride_page, g.num_pages}}));
        CHECK(check_apart("v_pages", d, {{g.v_stride_token, g.page_size}, {g.v_stride_head, Hk}, {g.v_stride_page, g.num_pages}}));
    }
    return GATTN_OK;
}

Pages pages_of(const gattn_pages &g)
{
    return {g.k_pages, g.v_pages, {g.k_stride_token, g.k_stride_head, g.k_stride_page},
            {g.v_stride_token, g.v_stride_head, g.v_stride_page}, g.table, g.table_stride,
            g.num_pages, g.page_size, g.table_width};
}

// Received weights as they lie in memory: n sequences of Hk heads of `width` floats.
struct Received {
    const float *p;
    int64_t width, seq, head;
};

int64_t floor_div(int64_t x, int64_t y) { return x / y - (x % y < 0); }

struct Found {
    int64_t first, last;
};

// The i in [0, n) whose rows, `len` elements from i * step on, meet [x, x + width).
Found rows_met(int64_t x, int64_t width, int64_t step, int64_t n, int64_t len)
{
    return {std::max<int64_t>(floor_div(x - len, step) + 1, 0), std::min(floor_div(x + width - 1, step), n - 1)};
}

// Weights that are written share no memory with those that are read, unless they are the
// same ones.
gattn_status check_beside(const Received &in, const Received &out, int64_t n, int64_t Hk)
{
    // what there is one of has no stride
    const int64_t is = n == 1 ? 0 : in.seq, ih = Hk == 1 ? 0 : in.head, os = n == 1 ? 0 : out.seq, oh = Hk == 1 ? 0 : out.head;
    if (!in.p || (in.p == out.p && is == os && ih == oh))
        return GATTN_OK;
    if (in.p == out.p)
        return bad(GATTN_E_INVALID_ARG, "weights_out in place of weights must have its strides");
    if (n == 0)
        return GATTN_OK;
    for (const int64_t step : {is, os})
        if (step > (1ll << 60) / n)
            return bad(GATTN_E_INVALID_ARG, "weights strides are too large");
    for (const int64_t step : {ih, oh})
        if (step > (1ll << 60) / Hk)
            return bad(GATTN_E_INVALID_ARG, "weights strides are too large");
    const int64_t from = (reinterpret_cast<intptr_t>(in.p) - reinterpret_cast<intptr_t>(out.p)) / 4;
    const int64_t in_span = (n - 1) * is + (Hk - 1) * ih + in.width, out_span = (n - 1) * os + (Hk - 1) * oh + out.width;
    if (from >= out_span || from + in_span <= 0)
        return GATTN_OK;
    bool meet = false;
    if (is == os && ih == oh) {
        // rows between each other: only how far apart they are counts
        for (int64_t h = 1 - Hk; h < Hk && !meet; ++h) {
            const Found f = rows_met(from + (n - 1) * is + h * ih, in.width, std::max<int64_t>(is, 1), 2 * n - 1, out.width);
            meet = f.first <= f.last;
        }
    } else {
        // the axis of out whose steps are further apart, and the nearer one within it
        const bool by_seq = os >= oh;
        const int64_t S = std::max<int64_t>(by_seq ? os : oh, 1), N = by_seq ? n : Hk;
        const int64_t T = std::max<int64_t>(by_seq ? oh : os, 1), M = by_seq ? Hk : n;
        for (int64_t i = 0; i < n * Hk && !meet; ++i) {
            const int64_t x = from + i / Hk * is + i % Hk * ih;
            const Found f = rows_met(x, in.width, S, N, (M - 1) * T + out.width);
            meet = f.last - f.first >= 2;      // whatever lies between is covered
            for (int64_t j = f.first; j <= f.last && !meet; ++j) {
                const Found g = rows_met(x - j * S, in.width, T, M, out.width);
                meet = g.first <= g.last;
            }
        }
    }
    if (meet)
        return bad(GATTN_E_INVALID_ARG, "weights_out overlaps weights and is not the same: it is written while weights are read");
    return GATTN_OK;
}

// Frequencies as float pairs, theta^(-2i/rd) stretched as the descriptor asks.
gattn_status frequencies(const gattn_paged_rows_desc *p, int rd, float2 *to)
{
    const double theta = p->rope_theta, pi = 3.14159265358979323846;
    double lo = 0, hi = 0;
    if (p->rope_scaling != GATTN_ROPE_PLAIN && p->rope_scaling != GATTN_ROPE_LINEAR && p->rope_scaling != GATTN_ROPE_YARN)
        return bad(GATTN_E_INVALID_ARG, "rope_scaling must be one of GATTN_ROPE_*");
    if (p->rope_scaling != GATTN_ROPE_PLAIN && (!(p->rope_factor >= 1.f) || !std::isfinite(p->rope_factor)))
        return bad(GATTN_E_INVALID_ARG, "rope_factor must be finite and >= 1");
    if (p->rope_scaling == GATTN_ROPE_YARN) {
        if (p->rope_original <= 0 || !(p->rope_beta_fast > 0.f) || !(p->rope_beta_slow > 0.f) ||
            p->rope_beta_fast < p->rope_beta_slow || !std::isfinite(p->rope_beta_fast) || !(theta > 1.))
            return bad(GATTN_E_INVALID_ARG,
                       "YaRN needs rope_original > 0, rope_theta > 1 and rope_beta_fast >= rope_beta_slow > 0");
        // the pair that turns `beta` times within the original positions
        auto pair = [&](double beta) { return rd * std::log(p->rope_original / (beta * 2 * pi)) / (2 * std::log(theta)); };
        lo = std::max(std::floor(pair(p->rope_beta_fast)), 0.);
        hi = std::min(std::ceil(pair(p->rope_beta_slow)), rd - 1.);
    }
    // by the power anew every 8th time: a few ulp of a double apart
    const double step = std::pow(theta, -2. / rd);
    double plain = 1.;
    for (int i = 0; i < rd / 2; ++i) {
        plain = i % 8 ? plain * step : std::pow(theta, -2. * i / rd);
        double f = plain;
        if (p->rope_scaling == GATTN_ROPE_LINEAR) {
            f /= p->rope_factor;
        } else if (p->rope_scaling == GATTN_ROPE_YARN) {
            const double slow = std::min(std::max((i - lo) / std::max(hi - lo, 1e-3), 0.), 1.);
            f = f * (1 - slow) + f / p->rope_factor * slow;
        }
        to[i].x = (float)f;
        to[i].y = (float)(f - (double)to[i].x);
    }
    return GATTN_OK;
}

}  // namespace

extern "C" {

gattn_status gattn_paged_rows(const gattn_paged_rows_desc *p, gattn_stream stream)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    CHECK(check_heads(p->num_heads, p->num_kv_heads));
    CHECK(check_seqs(p->num_seqs, p->total_rows));
    CHECK(check_dim(p->head_dim));
    if (p->x_dtype != GATTN_DTYPE_F32 && p->x_dtype != GATTN_DTYPE_BF16)
        return bad(GATTN_E_INVALID_ARG, "x_dtype must be GATTN_DTYPE_F32 or GATTN_DTYPE_BF16");
    const int rd = p->rotary_dims;
    if (rd < 2 || (rd & 1) || rd > p->head_dim)
        return bad(GATTN_E_INVALID_ARG, "rotary_dims %d must be even, >= 2 and <= head_dim", rd);
    if (!(p->rope_theta > 0.f) || !std::isfinite(p->rope_theta) || !(p->rms_eps >= 0.f))
        return bad(GATTN_E_INVALID_ARG, "rope_theta must be > 0 and rms_eps >= 0");
    if (!(p->rope_size >= 0.f) || !std::isfinite(p->rope_size))
        return bad(GATTN_E_INVALID_ARG, "rope_size must be finite and >= 0");
    CHECK(check_rows("q", p->q, p->q_stride_token, p->q_stride_head));
    CHECK(check_rows("k", p->k, p->k_stride_token, p->k_stride_head));
    CHECK(check_rows("v", p->v, p->v_stride_token, p->v_stride_head));
    CHECK(check_out("q_out", p->q_out, p->o_stride_token, p->o_stride_head, p->head_dim, p->total_rows,
                    p->num_heads));
    CHECK(check_pages(p->pages, p->num_kv_heads, p->head_dim, true, true));
    CHECK(check_words({p->cu_rows, p->cache_pos, p->positions, p->status}));
    if (misaligned(p->q_norm) || misaligned(p->k_norm))
        return bad(GATTN_E_INVALID_ARG, "q_norm and k_norm must be 16-byte aligned");
    if (!p->cu_rows || !p->cache_pos)
        return bad(GATTN_E_INVALID_ARG, "cu_rows or cache_pos is NULL");
    PagedRowsArgs a{};
    CHECK(frequencies(p, rd, a.inv_freq));
    if (p->num_seqs == 0 || p->total_rows == 0)
        return GATTN_OK;
    a.sq = {p->cu_rows, nullptr, p->num_seqs, p->total_rows, 0, p->num_seqs, p->status};
    a.pg = pages_of(p->pages);
    a.pos = p->cache_pos;
    a.positions = p->positions;
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
    a.cap = (long long)p->pages.table_width * p->pages.page_size;
    a.H = p->num_heads;
    a.Hk = p->num_kv_heads;
    a.d = p->head_dim;
    a.rd = rd;
    a.pairs = p->rope_pairs != 0;
    a.eps = p->rms_eps;
    a.turn_size = p->rope_size > 0.f ? p->rope_size
                  : p->rope_scaling == GATTN_ROPE_YARN ? (float)(0.1 * std::log((double)p->rope_factor) + 1.)
                                                       : 1.f;
    return cuda_status("gattn_paged_rows", launch_paged_rows(a, p->x_dtype == GATTN_DTYPE_F32,
                                                             reinterpret_cast<cudaStream_t>(stream)));
}

// Shapes that the attention takes.
static gattn_status check_attended(int32_t H, int32_t Hk, int32_t d, int32_t n, int32_t total)
{
    CHECK(check_heads(H, Hk));
    CHECK(check_seqs(n, total));
    CHECK(check_dim(d));
    if (H > 65536 / d)
        return bad(GATTN_E_UNSUPPORTED, "num_heads * head_dim must be <= 65536");
    if ((long long)total * H > 0x7fffffffll)
        return bad(GATTN_E_UNSUPPORTED, "total_rows * num_heads must be below 2^31");
    return GATTN_OK;
}

// What attention and weights have in common.
static gattn_status paged_args(const gattn_paged_attention_desc *p, bool values, PagedAttnArgs &a)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    CHECK(check_attended(p->num_heads, p->num_kv_heads, p->head_dim, p->num_seqs, p->total_rows));
    if (!(p->scale > 0.f) || !std::isfinite(p->scale))
        return bad(GATTN_E_INVALID_ARG, "scale must be finite and > 0");
    CHECK(check_rows("q", p->q, p->q_stride_token, p->q_stride_head));
    CHECK(check_pages(p->pages, p->num_kv_heads, p->head_dim, values, false));
    CHECK(check_words({p->cu_rows, p->cache_pos, p->lse, p->status}));
    if (!p->cu_rows || !p->cache_pos)
        return bad(GATTN_E_INVALID_ARG, "cu_rows or cache_pos is NULL");
    a = PagedAttnArgs{};
    a.sq = {p->cu_rows, nullptr, p->num_seqs, p->total_rows, 0, p->num_seqs, p->status};
    a.pg = pages_of(p->pages);
    a.pos = p->cache_pos;
    a.q = static_cast<const __nv_bfloat16 *>(p->q);
    a.qs = {p->q_stride_token, p->q_stride_head};
    a.H = p->num_heads;
    a.Hk = p->num_kv_heads;
    a.d = p->head_dim;
    a.cap = (long long)p->pages.table_width * p->pages.page_size;
    a.scale_log2 = (float)(1.4426950408889634 * (double)p->scale);
    a.lse = p->lse;
    return GATTN_OK;
}

int64_t gattn_paged_attention_workspace(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_seqs,
                                        int32_t total_rows)
{
    if (check_attended(num_heads, num_kv_heads, head_dim, num_seqs, total_rows) != GATTN_OK)
        return -1;
    // what all rows in one sequence need: tiles go by the rows of an average sequence, so fewer
    // sequences may need more
    return paged_attn_workspace(head_dim, num_heads / num_kv_heads, 1, total_rows);
}

gattn_status gattn_paged_attention(const gattn_paged_attention_desc *p, gattn_stream stream)
{
    PagedAttnArgs a;
    CHECK(paged_args(p, true, a));
    if (p->gate) {
        CHECK(check_rows("gate", p->gate, p->g_stride_token, p->g_stride_head));
        if (p->gate_dtype != GATTN_DTYPE_F32 && p->gate_dtype != GATTN_DTYPE_BF16)
            return bad(GATTN_E_INVALID_ARG, "gate_dtype must be GATTN_DTYPE_F32 or GATTN_DTYPE_BF16");
    }
    CHECK(check_out("out", p->out, p->o_stride_token, p->o_stride_head, p->head_dim, p->total_rows, p->num_heads));
    if (!p->workspace || misaligned(p->workspace))
        return bad(GATTN_E_INVALID_ARG, "workspace must be 16-byte aligned and not NULL");
    const int64_t need =
        paged_attn_workspace(p->head_dim, p->num_heads / p->num_kv_heads, p->num_seqs, p->total_rows);
    if (p->workspace_bytes < need)
        return bad(GATTN_E_INVALID_ARG, "workspace of %lld bytes: %lld are needed", (long long)p->workspace_bytes,
                   (long long)need);
    if (p->num_seqs == 0 || p->total_rows == 0)
        return GATTN_OK;
    a.gate = p->gate;
    a.gate_f32 = p->gate_dtype == GATTN_DTYPE_F32;
    a.gs = {p->g_stride_token, p->g_stride_head};
    a.out = static_cast<__nv_bfloat16 *>(p->out);
    a.os = {p->o_stride_token, p->o_stride_head};
    a.ws = p->workspace;
    return cuda_status("gattn_paged_attention", launch_paged_attn(a, reinterpret_cast<cudaStream_t>(stream)));
}

gattn_status gattn_paged_weights(const gattn_paged_weights_desc *p, gattn_stream stream)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    PagedAttnArgs a;
    CHECK(paged_args(&p->attention, false, a));
    if (!a.lse)
        return bad(GATTN_E_INVALID_ARG, "lse is NULL");
    if (!p->weights_out)
        return bad(GATTN_E_INVALID_ARG, "weights_out is NULL");
    CHECK(check_words({p->weights, p->weights_out}));
    if (p->weights_width <= 0)
        return bad(GATTN_E_INVALID_ARG, "weights_width must be > 0");
    CHECK(check_apart("weights", p->weights_width, {{p->w_stride_head, a.Hk}, {p->w_stride_seq, a.sq.n}}));
    CHECK(check_beside({p->weights, p->weights_width, p->w_stride_seq, p->w_stride_head},
                       {p->weights_out, p->weights_width, p->w_stride_seq, p->w_stride_head}, a.sq.n, a.Hk));
    if (a.sq.n == 0 || a.sq.total == 0)
        return GATTN_OK;
    a.cap = std::min<long long>(a.cap, p->weights_width);
    a.w = p->weights;
    a.w_out = p->weights_out;
    a.w_seq = p->w_stride_seq;
    a.w_head = p->w_stride_head;
    return cuda_status("gattn_paged_weights", launch_paged_weights(a, reinterpret_cast<cudaStream_t>(stream)));
}

gattn_status gattn_paged_evict(const gattn_paged_evict_desc *p, gattn_stream stream)
{
    if (!p)
        return bad(GATTN_E_INVALID_ARG, "desc is NULL");
    if (p->num_kv_heads <= 0 || p->num_kv_heads > 65536)
        return bad(GATTN_E_INVALID_ARG, "num_kv_heads must be in 1..65536");
    CHECK(check_dim(p->head_dim));
    CHECK(check_seqs(p->num_seqs, 0));
    if (p->keep <= 0 || p->keep > (1 << 24) || p->recent < 0 || p->recent > p->keep)
        return bad(GATTN_E_INVALID_ARG, "keep must be in 1..2^24 and recent in 0..keep");
    CHECK(check_pages(p->pages, p->num_kv_heads, p->head_dim, true, true));
    CHECK(check_words({p->out_table, p->lengths, p->lengths_out, p->weights, p->weights_out, p->kept, p->status}));
    if (!p->lengths || !p->lengths_out || !p->weights || !p->kept)
        return bad(GATTN_E_INVALID_ARG, "lengths, lengths_out, weights or kept is NULL");
    const char *li = reinterpret_cast<const char *>(p->lengths), *lo = reinterpret_cast<const char *>(p->lengths_out);
    if (p->num_seqs > 0 && std::abs(lo - li) < 4ll * p->num_seqs)
        return bad(GATTN_E_INVALID_ARG, "lengths_out must not overlap lengths: every head reads them");
    if (p->weights_width <= 0 || p->w_stride_seq < 0 || p->w_stride_head < 0)
        return bad(GATTN_E_INVALID_ARG, "weights_width must be > 0 and the weights' strides >= 0");
    if (p->weights_out) {
        if (p->weights_out_width <= 0)
            return bad(GATTN_E_INVALID_ARG, "weights_out_width must be > 0");
        CHECK(check_apart("weights_out", p->weights_out_width,
                          {{p->wo_stride_head, p->num_kv_heads}, {p->wo_stride_seq, p->num_seqs}}));
        // (a stride over one sequence or head is none)
        if (p->weights_out == p->weights && ((p->num_seqs != 1 && p->wo_stride_seq != p->w_stride_seq) ||
                                             (p->num_kv_heads != 1 && p->wo_stride_head != p->w_stride_head)))
            return bad(GATTN_E_INVALID_ARG, "weights_out in place of weights must have its strides");
        CHECK(check_beside({p->weights, p->weights_width, p->w_stride_seq, p->w_stride_head},
                           {p->weights_out, p->weights_out_width, p->wo_stride_seq, p->wo_stride_head}, p->num_seqs,
                           p->num_kv_heads));
    }
    if (p->out_table && (p->out_table_width <= 0 || p->out_table_stride < p->out_table_width ||
                         p->out_table_width > (1 << 24) / p->pages.page_size))
        return bad(GATTN_E_INVALID_ARG, "out_table_width must be > 0, within 2^24 positions and out_table_stride");
    if ((long long)p->num_seqs * p->num_kv_heads > (1ll << 26) ||
        (long long)p->num_seqs * p->num_kv_heads * ((p->keep + 7) / 8) > (1ll << 33))
        return bad(GATTN_E_UNSUPPORTED, "num_seqs * num_kv_heads is too large");
    if (p->num_seqs == 0)
        return GATTN_OK;
    PagedEvictArgs a{};
    a.pg = pages_of(p->pages);
    const bool in_place = !p->out_table || p->out_table == p->pages.table;
    if (in_place && p->out_table && p->out_table_stride != p->pages.table_stride)
        return bad(GATTN_E_INVALID_ARG, "out_table in place of table must have its stride");
    a.out_table = in_place ? nullptr : p->out_table;
    a.out_stride = p->out_table_stride;
    a.n = p->num_seqs;
    a.lengths = p->lengths;
    a.lengths_out = p->lengths_out;
    a.w = p->weights;
    a.w_out = p->weights_out;
    a.w_seq = p->w_stride_seq;
    a.w_head = p->w_stride_head;
    a.wo_seq = p->wo_stride_seq;
    a.wo_head = p->wo_stride_head;
    a.kept = p->kept;
    a.Hk = p->num_kv_heads;
    a.d = p->head_dim;
    a.keep = p->keep;
    a.recent = p->recent;
    const long long room = (long long)a.pg.width * a.pg.page;
    a.cap = std::min<long long>(room, p->weights_width);
    a.out_cap = p->out_table ? (long long)p->out_table_width * a.pg.page : room;
    if (p->weights_out)
        a.out_cap = std::min<long long>(a.out_cap, p->weights_out_width);
    a.status = p->status;
    return cuda_status("gattn_paged_evict", launch_paged_evict(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
