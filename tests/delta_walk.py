"""The gated delta rule row by row on the CPU, in 64 and in 32 bits, with a bound of
the error that each row leaves in a state column and in its answers."""
from __future__ import annotations

import torch

from tests.seq_refs import U_BF16

# What one row may leave, relative to the norms it multiplies.  Row by row in fp32: a
# dot product of at most 256 terms in partial sums (20 roundings one after another), the
# decay, the update and the unit of a normalized row, each a few 2^-24.  In chunks: a
# product's operands are pairs of 11-bit parts, off by 2^-24 each and 2^-24 more for the
# product of the two lower parts that is left out; 24 fp32 accumulations of at most
# 2^-23 each.  Both stay below 64 * 2^-24.
U_ROW = 2.0 ** -18


def unit(x, eps):
    return x if eps is None else x / torch.sqrt((x * x).sum(-1, keepdim=True) + eps)


def walk(q, k, v, g, beta, S, scale, eps=None, dtype=torch.float64, chunk=0):
    """One sequence: q, k [n][Hk][dk], v [n][Hv][dv], S [Hv][dk][dv].  Returns (out, state,
    bound of out before its rounding, bound of the state's columns [Hv][1][dv]).  With
    `chunk` rows that are taken at once, a row leaves in a column 2^-24 more of the largest
    norm that the column, or a write to it, has in the chunk: a 16-bit operand's lower part
    ends at 2^-25 of a unit of at most a quarter of the largest element, in two products
    (W and, for answers, A W)."""
    n, Hk, dk = q.shape
    Hv = v.shape[1]
    own = torch.arange(Hv) // (Hv // Hk)
    q, k, v, g, beta, S = (x.to(dtype) for x in (q, k, v, g, beta, S))
    q, k = unit(q, eps)[:, own], unit(k, eps)[:, own]
    out = torch.zeros(n, Hv, v.shape[2], dtype=dtype)
    eo = torch.zeros_like(out)
    sizes, local = [], []
    for t in range(n):
        before = S.norm(dim=1)
        a = torch.exp(g[t])[:, None]
        S = a[..., None] * S
        size = S.norm(dim=1)
        b, kn = beta[t].abs()[:, None], k[t].norm(dim=-1)[:, None]
        w = beta[t][:, None] * (v[t] - torch.einsum("ha,hab->hb", k[t], S))
        S = S + k[t][:, :, None] * w[:, None, :]
        out[t] = scale * torch.einsum("ha,hab->hb", q[t], S)
        # the row's map I - beta k k^T stretches by 1 or by |1 - beta |k|^2|
        stretch = a * torch.clamp((1 - beta[t][:, None] * kn * kn).abs(), min=1)
        sizes.append(torch.maximum(torch.maximum(before, S.norm(dim=1)), kn * torch.maximum(w.abs(), b * v[t].abs())))
        local.append((stretch, U_ROW * (size + b * kn * (v[t].abs() + kn * size)),
                      abs(scale) * q[t].norm(dim=-1)[:, None], U_ROW * (size + kn * w.abs())))
    e = torch.zeros(Hv, v.shape[2], dtype=dtype)
    for t, (stretch, row, qn, answer) in enumerate(local):
        most = torch.stack(sizes[t // chunk * chunk:][:chunk]).amax(0) if chunk else 0
        e = stretch * e + row + 2.0 ** -24 * most
        eo[t] = qn * (e + answer + 2.0 ** -23 * most)
    return out, S, eo, e[:, None, :]


def hold_to_rule(case, out, state, scale, eps=None, bounded=True, chunk=32):
    """Holds out [n][Hv][dv] and state [Hv][dk][dv] (or None) of one sequence to the rule.
    Element by element: the last rounding and the bound above, where no row stretches the
    state (`bounded`).  Always, per head and per `chunk` rows: the 2-norm of the error
    within eight times that of the same recurrence in fp32 (parts of 22 bits and
    accumulations that truncate against 24 bits and rounding), one rounding of the
    answers and 2^-20 of the size."""
    want, last, eo, es = walk(*case, scale, eps)
    out32, last32, _, _ = walk(*case, scale, eps, dtype=torch.float32)
    assert out.isfinite().all()
    err = (out.double() - want).abs()
    if bounded:
        tol = U_BF16 * want.abs() + (1 + U_BF16) * eo + 1e-37
        assert (err <= tol).all(), ("out", float((err - tol).max()), float((err / tol).max()))
    for r in range(0, len(want), chunk):
        a = slice(r, r + chunk)
        e, w, e32 = (x[a].double().transpose(0, 1).flatten(1).norm(dim=1) for x in (err, want, out32.double() - want))
        assert (e <= (U_BF16 + 2.0 ** -20) * w + 8 * e32 + 1e-37).all(), ("out rows", r, (e / w).tolist())
    if state is None:
        return
    assert state.isfinite().all()
    err = (state.double() - last).abs()
    if bounded:
        assert (err <= es + 1e-37).all(), ("state", float((err - es).max()), float((err / es).max()))
    e, w, e32 = (x.double().flatten(1).norm(dim=1) for x in (err, last, last32.double() - last))
    assert (e <= 2.0 ** -20 * w + 8 * e32 + 1e-37).all(), ("state", (e / w).tolist(), (e32 / w).tolist())
