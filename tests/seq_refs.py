"""float64 forms of the packed-sequence operators, from their formulas, and the
bounds their kernels are held to (torch, on the CPU)."""
from __future__ import annotations

import math

import torch

U_BF16 = 2.0 ** -8         # half a step of bf16, relative
U_F32 = 2.0 ** -24


def cu_of(lens, device="cpu"):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32, device=device)


def rope64(x, pos, rd, theta):
    """x [rows][heads][d] float64, rotate-half on the first rd elements at pos [rows]."""
    half = rd // 2
    inv = torch.tensor([theta ** (-2.0 * i / rd) for i in range(half)], dtype=torch.float64)
    ang = pos.double()[:, None, None] * inv
    a, b = x[..., :half], x[..., half:rd]
    return torch.cat((a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin(), x[..., rd:]), -1)


def rows64(x, w, pos, rd, theta, eps):
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    return rope64(y, pos, rd, theta)


def attention64(q, k, v, gate, scale, past):
    """One sequence: q [n][H][d], k and v [m][Hk][d]; row i sees keys j <= past + i.
    Returns (out, weight): weight = sigmoid(gate) * softmax @ |v|, the size that
    relative errors of the probabilities act on."""
    n, H, d = q.shape
    m, Hk = k.shape[:2]
    out = torch.zeros(n, H, d, dtype=torch.float64)
    weight = torch.zeros_like(out)
    for i in range(n):
        e = min(m, past + i + 1)
        if e <= 0:
            continue
        for h in range(H):
            kk, vv = k[:e, h // (H // Hk)].double(), v[:e, h // (H // Hk)].double()
            s = (kk @ q[i, h].double()) * scale
            p = torch.softmax(s, 0)
            out[i, h] = p @ vv
            weight[i, h] = p @ vv.abs()
    if gate is not None:
        sg = torch.sigmoid(gate.double())
        out, weight = out * sg, weight * sg
        seen = torch.tensor([past + i + 1 > 0 for i in range(n)])
        out[~seen], weight[~seen] = 0, 0
    return out, weight


def attention_bound(out, weight, score_error):
    """The out row is rounded once (half a bf16 step of |out|); every probability
    is rounded once to bf16 before it meets its value (half a step of `weight`);
    a score off by e scales a probability and the sum by exp(e) each; the sums
    and the base-2 exponentials (a few units of 2^-22) stay below 2^-12."""
    return U_BF16 * out.abs() + (U_BF16 * (1 + U_BF16) + math.expm1(2 * score_error) + 2.0 ** -12) * weight + 1e-30


def score_error(q, k, scale):
    """|fl(s) - s| of a d-term fp32 dot product of exact bf16 products."""
    d = q.shape[-1]
    big = q.double().abs().amax(0).amax(0) @ k.double().abs().amax(0).amax(0)
    return float((d + 2) * U_F32 * big * scale)


def delta64(q, k, v, g, beta, S, scale, l2_eps=None):
    """One sequence: q, k [n][Hk][dk], v [n][Hv][dv], S [Hv][dk][dv].  Returns
    (out, state after the last row, largest column norm met)."""
    n, Hk, dk = q.shape
    Hv = v.shape[1]
    own = torch.arange(Hv) // (Hv // Hk)
    q, k, v, g, beta, S = (x.double() for x in (q, k, v, g, beta, S))
    if l2_eps is not None:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + l2_eps)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + l2_eps)
    q, k = q[:, own], k[:, own]
    out = torch.zeros(n, Hv, v.shape[2], dtype=torch.float64)
    top = float(S.norm(dim=1).max()) if S.numel() else 0.0
    for t in range(n):
        S = torch.exp(g[t])[:, None, None] * S
        w = beta[t][:, None] * (v[t] - torch.einsum("ha,hab->hb", k[t], S))
        S = S + k[t][:, :, None] * w[:, None, :]
        out[t] = scale * torch.einsum("ha,hab->hb", q[t], S)
        top = max(top, float(S.norm(dim=1).max()), float(v[t].abs().max()))
    return out, S, top


def delta_bound(rows, top, dk):
    """Absolute error of a state entry after `rows` rows, for |k| <= 1, beta <= 1 and
    g <= 0, where one row's map I - beta k k^T (times the decay) does not expand.
    Row by row a row adds the rounding of a dk-term dot product and of the update
    and decay, at most (dk + 6) 2^-24 of a column's norm.  In chunks the three
    products (k S, T Y, k W) take fp32 operands as pairs of 16-bit floats, each
    pair within 2^-16 of its value."""
    return rows * max((dk + 6) * U_F32, 3 * 2.0 ** -16) * top
