"""The packed-sequence operators as a hybrid stack uses them: a prompt pass that
fills the layer's cache (rows, attention) and the delta layers' states, then
decode steps on top, against the same tokens fed one at a time."""
import numpy as np
import pytest
import torch

from qwen3_gated_attention_gb300 import gattn, synth
from tests.cases import bf16_ulp_distance
from tests.seq_refs import (U_BF16, attention64, attention_bound, cu_of, delta64, delta_bound,
                            score_error)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _layer(spec, cap, layout):
    from qwen3_gated_attention_gb300.device import DeviceLayer
    packed = [gattn.pack_affine_host(w, spec.bits[i], spec.group[i])
              for i, w in enumerate(synth.weights_f32(spec))]
    qn, kn = synth.norm_weights_bf16(spec)
    return DeviceLayer(spec, packed, qn, kn, cap, layout=layout), qn, kn


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("layout", ["bhtd", "btd"])
@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (4, 1, 256)])
def test_prompt_then_decode_equals_decode_from_the_start(H, Hk, d, layout):
    from qwen3_gated_attention_gb300 import device
    lens, n = [37, 12, 25], 3
    cap, T = 64, sum(lens)
    spec = synth.WORKLOADS["tiny"].with_(name="stack", num_heads=H, num_kv_heads=Hk, head_dim=d,
                                         batch=n, q_len=1, x_dtype="bf16", cache_pos=(0,))
    a, qn, kn = _layer(spec, cap, layout)
    b, _, _ = _layer(spec, cap, layout)
    g = torch.Generator().manual_seed(d)
    x = torch.randn(n, max(lens) + 2, spec.hidden, generator=g).to(BF).cuda()
    y = torch.zeros(n, spec.n_q + 2 * spec.n_kv, device="cuda")
    at = torch.zeros(n, H * d, device="cuda")
    out = torch.zeros(n, 1, spec.hidden, dtype=BF, device="cuda")
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    a.set_taps(y, at)
    ys, ats = [], []
    for t in range(max(lens)):                     # token by token through the layer
        pos.fill_(t)
        a.step(x[:, t].contiguous(), pos, out)
        ys.append(y.clone())
        ats.append(at.clone())
    a.poll()
    ys, ats = torch.stack(ys, 1), torch.stack(ats, 1)
    rows = torch.cat([ys[s, :m] for s, m in enumerate(lens)])        # packed projection outputs
    want = torch.cat([ats[s, :m] for s, m in enumerate(lens)]).view(T, H, d)
    qg = rows[:, :2 * H * d].view(T, H, 2 * d)
    k = rows[:, 2 * H * d:2 * H * d + Hk * d].view(T, Hk, d)
    v = rows[:, 2 * H * d + Hk * d:].view(T, Hk, d)
    kc, vc = (t if layout == "bhtd" else t.transpose(1, 2) for t in (b.k, b.v))
    cu, zero = cu_of(lens, "cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    w = [torch.from_numpy(np.ascontiguousarray(z).view(np.int16)).view(BF).cuda() for z in (qn, kn)]
    q = device.prompt_rows(qg[..., :d], k, v, *w, kc, vc, cu, zero,
                           partial_rotary_factor=spec.partial_rotary_factor,
                           rope_theta=spec.rope_theta, rms_eps=spec.rms_eps)
    gate = qg[..., d:]
    o = device.prompt_attention(q, kc, vc, cu, cache_pos=zero, gate=gate)
    torch.cuda.synchronize()
    ka, va = (t if layout == "bhtd" else t.transpose(1, 2) for t in (a.k, a.v))
    r = 0
    for s, m in enumerate(lens):
        for mine, theirs in ((kc, ka), (vc, va)):
            # both round the same fp32 values to bf16: a unit apart at most
            assert bf16_ulp_distance(_bits(mine[s, :, :m]), _bits(theirs[s, :, :m])).max() <= 1
        kk, vv = (t[s, :, :m].transpose(0, 1).cpu() for t in (kc, vc))
        qq = q[r:r + m].cpu()
        ref, weight = attention64(qq, kk, vv, gate[r:r + m].cpu(), d ** -0.5, 0)
        tol = attention_bound(ref, weight, score_error(qq, kk, d ** -0.5))
        assert ((o[r:r + m].cpu().double() - ref).abs() <= tol).all()
        # the layer's own attention (before its gate), whose keys may be a unit off
        mine = o[r:r + m].float().cpu()
        theirs = (want[r:r + m] * torch.sigmoid(gate[r:r + m])).cpu()
        assert (mine - theirs).abs().max() <= 0.05 * theirs.abs().max()
        r += m
    # decode goes on from the filled cache
    last = []
    for L in (a, b):
        pos.copy_(torch.tensor(lens, dtype=torch.int32))
        nxt = torch.stack([x[s, m] for s, m in enumerate(lens)])
        L.set_taps(None, at)
        L.step(nxt, pos, out)
        L.poll()
        last.append(at.clone())
    assert (last[0] - last[1]).abs().max() <= 0.05 * last[0].abs().max()
    a.close()
    b.close()


def test_delta_prompt_then_steps_and_a_rejected_draft():
    from qwen3_gated_attention_gb300 import device
    Hk, Hv, dk, dv, lens, n = 2, 4, 128, 128, [45, 33], 2
    g = torch.Generator().manual_seed(3)
    full = [m + 6 for m in lens]
    parts = [dict(q=torch.randn(m, Hk, dk, generator=g).to(BF), k=torch.randn(m, Hk, dk, generator=g).to(BF),
                  v=torch.randn(m, Hv, dv, generator=g).to(BF), g=-torch.rand(m, Hv, generator=g),
                  beta=torch.sigmoid(torch.randn(m, Hv, generator=g))) for m in full]
    pool = torch.zeros(5, Hv, dk, dv, device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    args = lambda cut: [torch.cat([p[key][cut(m)] for p, m in zip(parts, lens)]).cuda()  # noqa: E731
                        for key in ("q", "k", "v", "g", "beta")]
    outs = [device.delta_prompt(*args(lambda m: slice(0, m)), cu_of(lens, "cuda"), state=pool,
                                state_out=pool, slots=slots, qk_l2norm=True).cpu()]
    before = pool.clone()
    draft = args(lambda m: slice(m, m + 4))
    four = device.delta_step(*draft, num_seqs=n, state=pool, slots=slots, qk_l2norm=True).cpu()
    torch.cuda.synchronize()
    assert torch.equal(pool, before)                       # a draft that is not kept
    took = [3, 1]                                          # accepted rows differ by sequence
    kept = [torch.cat([d[4 * s:4 * s + t] for s, t in enumerate(took)]) for d in draft]
    three = device.delta_step(*kept, cu_of(took, "cuda"), state=pool, state_out=pool, slots=slots,
                              qk_l2norm=True).cpu()
    assert torch.equal(three[:3], four[:3]) and torch.equal(three[3:], four[4:5])
    r = 0
    for s, m in enumerate(lens):
        rows = m + took[s]
        p = {key: x[:rows] for key, x in parts[s].items()}
        want, S, top = delta64(p["q"], p["k"], p["v"], p["g"], p["beta"], torch.zeros(Hv, dk, dv),
                               dk ** -0.5, 1e-6)
        e = delta_bound(rows, top, dk)
        mine = torch.cat((outs[0][r:r + m], four[4 * s:4 * s + took[s]])).double()
        assert ((mine - want).abs() <= U_BF16 * want.abs() + e + 2.0 ** -14 * top).all()
        assert float((pool[int(slots[s])].cpu().double() - S).abs().max()) <= e
        r += m
    assert (pool[[0, 2, 3]] == 0).all()
