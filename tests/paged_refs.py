"""float64 forms of the paged-cache operators, from their formulas, and pools of pages to
run them on (torch, on the CPU)."""
from __future__ import annotations

import math

import torch

from tests.seq_refs import U_BF16, U_F32

BF = torch.bfloat16


def pool(n_pages, Hk, P, d, g, token_major=False):
    """A pool [pages][Hk][P][d], or a view of [pages][P][Hk][d] with that shape."""
    if token_major:
        return torch.randn(n_pages, P, Hk, d, generator=g).to(BF).transpose(1, 2)
    return torch.randn(n_pages, Hk, P, d, generator=g).to(BF)


def tables(totals, P, g, spare=3, width=None):
    """Pages for sequences of these many positions, in no order: (table, pages)."""
    need = [-(-t // P) for t in totals]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    t = torch.zeros(len(totals), width or max(max(need), 1), dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = order[at:at + k]
        at += k
    return t, pages


def gather(pool_, row, P, m):
    """The first m positions of a table row: [m][Hk][d]; zeros where there is no page."""
    out = torch.zeros(m, pool_.shape[1], pool_.shape[3], dtype=torch.float64)
    there = torch.ones(m, dtype=torch.bool)
    for p in range(m):
        page = int(row[p // P])
        if 0 <= page < pool_.shape[0]:
            out[p] = pool_[page, :, p % P].double()
        else:
            there[p] = False
    return out, there


def attention64(q, k, v, there, gate, scale, past):
    """One sequence: q [n][H][d], k and v [m][Hk][d]; row i sees the positions <= past + i that
    are there.  Returns (out, weight, lse, size): weight = sigmoid(gate) * softmax @ |v|,
    what relative errors of the probabilities act on; size = the largest sum of a score's
    products, in size."""
    n, H, d = q.shape
    Hk = k.shape[1]
    own = torch.arange(H) // (H // Hk)
    out = torch.zeros(n, H, d, dtype=torch.float64)
    weight, lse = torch.zeros_like(out), torch.full((n, H), -math.inf, dtype=torch.float64)
    size = 0.0
    q, k, v = q.double(), k.double(), v.double()
    for i in range(n):
        e = past + i + 1
        on = there[:e].nonzero()[:, 0]
        if not len(on):
            continue
        kk, vv = k[on][:, own], v[on][:, own]
        s = torch.einsum("hd,mhd->hm", q[i], kk) * scale
        size = max(size, float(torch.einsum("hd,mhd->hm", q[i].abs(), kk.abs()).max()) * scale)
        p = torch.softmax(s, -1)
        lse[i] = torch.logsumexp(s, -1)
        out[i] = torch.einsum("hm,mhd->hd", p, vv)
        weight[i] = torch.einsum("hm,mhd->hd", p, vv.abs())
        if gate is not None:
            sg = torch.sigmoid(gate[i].double())
            out[i], weight[i] = out[i] * sg, weight[i] * sg
    return out, weight, lse, size


def score_error(d, size, scale, lse=0.0):
    """|fl(s) - s| of a d-term fp32 sum of exact products whose sizes add up to size, with
    its scaling; then the exponent's own rounding beside a reference of up to `lse`."""
    return (d + 4) * U_F32 * size + 4 * U_F32 * (size + abs(lse))


def attention_bound(out, weight, error):
    """One rounding to bf16 (half a step of |out|); numerators of 16 bits (2^-16 with the
    second part's own rounding); scores off by e scale a numerator and the sum by
    exp(e) each; sums of up to 2^17 terms in fp32, in blocks, exponentials, the
    gate's exponential and division: below 2^-14 together."""
    return U_BF16 * out.abs() + (math.expm1(2 * error) + 2.0 ** -16 + 2.0 ** -14) * weight * (1 + U_BF16) + 1e-30


def turn64(x, w, pos, rd, pairs, theta=1e6, eps=1e-6, rope_factor=None, rope_yarn=None, rope_size=0.0):
    """One row [heads][d]: RMSNorm by w (None: as it is), the first rd elements turned."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    size = rope_size
    freq = []
    for i in range(rd // 2):
        f = theta ** (-2.0 * i / rd)
        if rope_factor is not None:
            f /= rope_factor
        if rope_yarn is not None:
            y = dict(beta_fast=32.0, beta_slow=1.0, **{k: v for k, v in rope_yarn.items() if not k.startswith("beta")})
            y.update(rope_yarn)
            at = lambda turns: rd * math.log(y["original"] / (2 * math.pi * turns)) / (2 * math.log(theta))  # noqa: E731
            lo, hi = max(math.floor(at(y["beta_fast"])), 0), min(math.ceil(at(y["beta_slow"])), rd - 1)
            c = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = f * (1 - c) + f / y["factor"] * c
        freq.append(f)
    if not size:
        size = 0.1 * math.log(rope_yarn["factor"]) + 1 if rope_yarn is not None else 1.0
    ang = torch.tensor(freq, dtype=torch.float64) * pos
    cos, sin = ang.cos() * size, ang.sin() * size
    out = x.clone()
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if pairs else (x[..., :rd // 2], x[..., rd // 2:rd])
    if pairs:
        out[..., 0:rd:2], out[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
    else:
        out[..., :rd // 2], out[..., rd // 2:rd] = a * cos - b * sin, b * cos + a * sin
    return out


def evicted(w, length, keep, recent):
    """The kept positions of one head, in order; w [positions]."""
    m = min(length, keep)
    new = min(recent, m)
    value = lambda i: -math.inf if math.isnan(w[i]) else w[i]      # noqa: E731
    best = sorted(range(length - new), key=lambda i: (-value(i), i))[:m - new]
    return sorted(best) + list(range(length - new, length))
