"""gattn_prompt_attention: a row's probabilities add up to one as they were multiplied,
and keys that are not there."""
import pytest
import torch

from tests.seq_refs import U_BF16, cu_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _attn(*a, **k):
    from qwen3_gated_attention_gb300 import device
    return device.prompt_attention(*a, **k)


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _holds_the_value(out, v, gate, keys):
    """The average of equal values is the value: numerator and sum add up the same
    numbers, in fp32 (2^-24 a key each), a division, a sigmoid of base-2 exponential and
    reciprocal (2^-20 together); one rounding."""
    want = v.double().repeat_interleave(out.shape[1] // v.shape[0], 0) * torch.sigmoid(gate.double())
    tol = (U_BF16 / 2 * 2 ** torch.ceil(torch.log2(want.abs())) +
           (2 * keys * 2.0 ** -24 + 2.0 ** -20) * want.abs())
    err = (out.double() - want).abs()
    assert (err <= tol).all(), (float((err / tol).max()), float((err > tol).double().mean()))


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (4, 1, 128), (6, 2, 192), (4, 2, 256)])
def test_equal_values_come_back(H, Hk, d):
    g = torch.Generator().manual_seed(d)
    T = 300
    q, k = (2 * torch.randn(T, h, d, generator=g) for h in (H, Hk))
    v = (1 + torch.rand(Hk, d, generator=g)).to(BF)
    gate = torch.randn(T, H, d, generator=g)
    out = _attn(q.to(BF).cuda(), k.to(BF).cuda(), v.cuda().expand(T, Hk, d).contiguous(), cu_of([T], "cuda"),
                gate=gate.cuda())
    _holds_the_value(out.cpu(), v, gate, T)


def test_equal_values_come_back_from_shares_of_a_cache():
    g = torch.Generator().manual_seed(1)
    H, Hk, d, past, n = 8, 2, 256, 3000, 8
    q, k = 2 * torch.randn(n, H, d, generator=g), torch.randn(1, Hk, past + n, d, generator=g)
    v = (1 + torch.rand(Hk, d, generator=g)).to(BF)
    gate = torch.randn(n, H, d, generator=g)
    vc = v.cuda()[None, :, None].expand(1, Hk, past + n, d).contiguous()
    out = _attn(q.to(BF).cuda(), k.to(BF).cuda(), vc, cu_of([n], "cuda"), cache_pos=_i32(past), gate=gate.cuda(),
                max_kv=past + n)
    _holds_the_value(out.cpu(), v, gate, past + n)
