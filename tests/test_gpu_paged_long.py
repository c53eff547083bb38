"""One new row behind a very long context: equal calls give equal bits whatever lies in the
workspace or ran in between, and each output is float64's within the derived bound."""
import pytest
import torch

from tests.paged_refs import BF, attention_bound, score_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _case(seed, past, H, Hk, d, P):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")      # noqa: E731
    n = -(-(past + 1) // P)
    kp, vp = (torch.cat([randn(min(512, n + 2 - i), Hk, P, d).to(BF) for i in range(0, n + 2, 512)]) for _ in range(2))
    table = torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32)[None]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    return dict(q=randn(1, H, d).to(BF), kp=kp, vp=vp, table=table, cu=i32([0, 1]), pos=i32([past]), gate=randn(1, H, d).to(BF))


def _run(s, ws):
    from qwen3_gated_attention_gb300 import device
    lse = torch.full(s["q"].shape[:2], float("nan"), device="cuda")
    out = device.paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["cu"], s["pos"], gate=s["gate"], lse=lse, workspace=ws)
    return out, lse


@pytest.mark.parametrize("H,Hk,d,P", [(24, 2, 256, 64), (8, 1, 64, 16), (40, 2, 128, 128)])
def test_a_long_context(H, Hk, d, P):
    from qwen3_gated_attention_gb300 import device
    past = 131071
    s, other = (_case(seed, past, H, Hk, d, P) for seed in (1, 2))
    ws = device.paged_attention_workspace(s["q"], s["kp"], s["cu"])
    out, lse = _run(s, ws)
    for i in range(12):
        ws.fill_((0, 0x7F, 0xFF)[i % 3])              # zeros, large numbers, NaN
        if i % 2:
            _run(other, ws)
        again, lse2 = _run(s, ws)
        assert torch.equal(again, out) and torch.equal(lse2, lse)
    G, scale = H // Hk, d ** -0.5
    sg = torch.sigmoid(s["gate"].double())[0]
    for hk in range(Hk):
        rows = slice(hk * G, hk * G + G)
        k, v = (p[s["table"][0].long(), hk].reshape(-1, d)[:past + 1].double() for p in (s["kp"], s["vp"]))
        q = s["q"][0, rows].double()
        score = (q @ k.t()) * scale
        size = float((q.abs() @ k.abs().t()).max()) * scale
        p = torch.softmax(score, -1)
        want, weight = (p @ v) * sg[rows], (p @ v.abs()) * sg[rows]
        total = torch.logsumexp(score, -1)
        e = score_error(d, size, 1.0, float(total.max()))
        assert ((out[0, rows].double() - want).abs() <= attention_bound(want, weight, e)).all()
        # the sum of 2^17 terms in fp32, in blocks, and its logarithm; the reference's rounding
        assert ((lse[0, rows].double() - total).abs() <= e + 2.0 ** -16 + 2.0 ** -22 * total.abs()).all()
