// seq_check.h -- argument checks that the packed-sequence and paged-cache entry points
// share (host only).
#pragma once

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "seq.cuh"

namespace gattn {
namespace check {

inline gattn_status bad(gattn_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
inline gattn_status bad(gattn_status st, const char *fmt, ...)
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

inline gattn_status cuda_status(const char *what, cudaError_t e)
{
    return e == cudaSuccess ? GATTN_OK
                            : bad(GATTN_E_CUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

inline bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// A row tensor: 16-byte aligned base, positive strides in multiples of 8 elements.
inline gattn_status check_rows(const char *name, const void *p, int64_t tok, int64_t head)
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
inline gattn_status check_apart(const char *name, int64_t d, std::initializer_list<Axis> axes)
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

inline gattn_status check_out(const char *name, const void *p, int64_t tok, int64_t head, int64_t d, int64_t rows,
                       int64_t heads)
{
    CHECK(check_rows(name, p, tok, head));
    return check_apart(name, d, {{tok, rows}, {head, heads}});
}

// Device arrays of 32-bit words; NULL passes.
inline gattn_status check_words(std::initializer_list<const void *> p)
{
    for (const void *x : p)
        if (reinterpret_cast<uintptr_t>(x) & 3)
            return bad(GATTN_E_INVALID_ARG, "offsets, positions, slots and status must be 4-byte aligned");
    return GATTN_OK;
}

inline gattn_status check_seqs(int32_t n, int32_t total)
{
    if (n < 0 || total < 0)
        return bad(GATTN_E_INVALID_ARG, "num_seqs and total_rows must be >= 0");
    if (total > (1 << 30) || n > (1 << 24))
        return bad(GATTN_E_INVALID_ARG, "num_seqs or total_rows is too large");
    return GATTN_OK;
}

inline gattn_status check_heads(int32_t H, int32_t Hk)
{
    if (H <= 0 || Hk <= 0 || H % Hk)
        return bad(GATTN_E_INVALID_ARG, "heads must be > 0 and a multiple of the key heads");
    return GATTN_OK;
}

}  // namespace check
}  // namespace gattn
