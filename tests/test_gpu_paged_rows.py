"""gattn_paged_rows on the GPU against float64: both layouts of the turned elements, scaled
frequencies, positions apart from places, absent norms, pages, what is left alone."""
import math

import pytest
import torch

from tests.paged_refs import BF, pool, tables, turn64
from tests.seq_refs import U_BF16, cu_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _dev():
    from qwen3_gated_attention_gb300 import device
    return device


YARN = dict(factor=4.0, original=4096)


def _case(H, Hk, d, P, lens, past, dtype, seed, norm=True, token_major=False, lead=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + 2 * lead
    table, pages = tables([a + b for a, b in zip(lens, past)], P, g)
    c = dict(H=H, Hk=Hk, d=d, P=P, lens=lens, past=past, table=table, lead=lead, cu=cu_of(lens) + lead)
    c["kp"], c["vp"] = (pool(pages, Hk, P, d, g, token_major) for _ in range(2))
    c["y"] = torch.randn(T, 2 * H * d + 2 * Hk * d, generator=g).to(dtype)
    c["qn"], c["kn"] = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF) if norm else None for _ in range(2))
    return c


def _split(c, y):
    T, H, Hk, d = y.shape[0], c["H"], c["Hk"], c["d"]
    return (y[:, :2 * H * d].view(T, H, 2 * d)[..., :d], y[:, 2 * H * d:2 * H * d + Hk * d].view(T, Hk, d),
            y[:, 2 * H * d + Hk * d:].view(T, Hk, d))


def _strided(x):
    return torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)


def _run(c, rd, pairs, positions=None, **rope):
    kp, vp = _strided(c["kp"]), _strided(c["vp"])
    y = c["y"].cuda()
    out = torch.full((y.shape[0], c["H"], c["d"]), 7.0, dtype=BF, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    on = lambda x: None if x is None else x.cuda()      # noqa: E731
    _dev().paged_rows(*_split(c, y), kp, vp, c["table"].cuda(), c["cu"].cuda(),
                      torch.tensor(c["past"], dtype=torch.int32, device="cuda"), rotary_dims=rd, rope_theta=1e6,
                      rope_pairs=pairs, q_norm=on(c["qn"]), k_norm=on(c["kn"]), rms_eps=1e-6, positions=on(positions),
                      q_out=out, status=st, **rope)
    torch.cuda.synchronize()
    return out.cpu(), kp.cpu(), vp.cpu(), int(st)


def _check(c, rd, pairs, got, positions=None, skipped=(), **rope):
    out, kp, vp, st = got
    q, k, v = _split(c, c["y"])
    want_k, want_v = c["kp"].clone(), c["vp"].clone()
    seen = torch.zeros(out.shape[0], dtype=torch.bool)
    for b, n in enumerate(c["lens"]):
        for i in range(n):
            t, p = int(c["cu"][b]) + i, c["past"][b] + i
            seen[t] = True
            if b in skipped:
                assert (out[t] == 0).all()
                continue
            at = p if positions is None else int(positions[t])
            y = turn64(q[t], c["qn"], at, rd, pairs, **rope)
            # fp32 products beside a bf16 rounding, an angle good to 2^-20 of the pair's size
            size = y.abs().amax() * 2.0 ** -17
            assert ((out[t].double() - y).abs() <= U_BF16 * y.abs() + size).all(), (b, i)
            page, row = int(c["table"][b, p // c["P"]]), p % c["P"]
            if 0 <= page < kp.shape[0]:
                y = turn64(k[t], c["kn"], at, rd, pairs, **rope)
                size = y.abs().amax() * 2.0 ** -17
                assert ((kp[page, :, row].double() - y).abs() <= U_BF16 * y.abs() + size).all()
                want_k[page, :, row] = kp[page, :, row]
                want_v[page, :, row] = v[t].to(BF)
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)      # nothing else was written
    assert (out[~seen] == 7).all()
    return st


@pytest.mark.parametrize("H,Hk,d", [(16, 4, 256), (6, 2, 192), (16, 8, 128), (8, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("pairs", [False, True])
def test_layouts_and_types(H, Hk, d, dtype, pairs):
    for rd in (d, d // 4, 20):
        c = _case(H, Hk, d, 16, [1, 5, 0, 33], [0, 11, 3, 1000], dtype, seed=d + rd)
        assert _check(c, rd, pairs, _run(c, rd, pairs)) == 0


@pytest.mark.parametrize("rope", [dict(rope_factor=8.0), dict(rope_yarn=YARN), dict(rope_yarn=dict(YARN, beta_fast=16, beta_slow=2)),
                                  dict(rope_yarn=YARN, rope_size=1.0), dict(rope_size=0.5),
                                  dict(rope_yarn=dict(factor=1.0, original=4096))])
@pytest.mark.parametrize("pairs", [False, True])
def test_scaled_frequencies(rope, pairs):
    c = _case(4, 2, 128, 48, [3, 2], [0, 60000], BF, seed=1)
    assert _check(c, 128, pairs, _run(c, 128, pairs, **rope), **rope) == 0


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("token_major", [True, False])
def test_positions_of_their_own_norms_and_layouts(norm, token_major):
    c = _case(4, 2, 64, 32, [4, 1], [30, 0], BF, seed=2, norm=norm, token_major=token_major, lead=3)
    pos = torch.tensor([9, 9, 9, 100000, 0, 2 ** 24, 77, 5, 9, 9, 9], dtype=torch.int32)
    assert _check(c, 64, False, _run(c, 64, False, positions=pos), positions=pos) == 0


@pytest.mark.parametrize("rows", [1, 8, 100, 2000, 6000])
def test_row_counts(rows):
    c = _case(8, 2, 64, 16, [rows], [5], BF, seed=rows)
    out, kp, vp, st = _run(c, 16, False)
    assert st == 0
    pick = sorted({0, rows - 1, rows // 2, min(rows - 1, 517)})
    q, k, v = _split(c, c["y"])
    for t in pick:
        y = turn64(q[t], c["qn"], 5 + t, 16, False)
        assert ((out[t].double() - y).abs() <= U_BF16 * y.abs() + y.abs().amax() * 2.0 ** -17).all()
        page, row = int(c["table"][0, (5 + t) // 16]), (5 + t) % 16
        assert torch.equal(vp[page, :, row], v[t])


def test_what_does_not_fit_is_skipped():
    c = _case(4, 2, 64, 16, [2, 3, 1, 2], [30, 10, 5, 0], BF, seed=3)
    width = c["table"].shape[1]
    c["past"] = [16 * width - 1, 10, -1, 2 ** 31 - 1]
    assert _check(c, 32, False, _run(c, 32, False), skipped=(0, 2, 3)) == 1


def test_entries_that_are_no_page_and_positions_out_of_range():
    c = _case(4, 2, 64, 16, [3, 2], [14, 0], BF, seed=4)
    c["table"][0, 1] = c["kp"].shape[0]                 # positions 16 on
    c["table"][1, 0] = -5
    assert _check(c, 32, True, _run(c, 32, True)) == 1
    c = _case(4, 2, 64, 16, [3], [14], BF, seed=4)
    pos = torch.tensor([4, -1, 2 ** 24 + 1], dtype=torch.int32)
    out, kp, vp, st = _run(c, 32, True, positions=pos)
    assert st == 1 and (out[1:] == 0).all()
    y = turn64(_split(c, c["y"])[0][0], c["qn"], 4, 32, True)
    assert ((out[0].double() - y).abs() <= U_BF16 * y.abs() + y.abs().amax() * 2.0 ** -17).all()
    page = int(c["table"][0, 1])
    assert torch.equal(kp[page], c["kp"][page]) and torch.equal(vp[page], c["vp"][page])


def test_matches_the_contiguous_form():
    """Pages in order are the cache of prompt_rows: equal bits."""
    c = _case(16, 4, 256, 64, [5, 70], [0, 58], BF, seed=5)
    c["table"] = torch.arange(4, dtype=torch.int32).view(2, 2)
    got = _run(c, 64, False)
    kc, vc = (torch.zeros(2, 4, 128, 256, dtype=BF, device="cuda") for _ in range(2))
    q_out = _dev().prompt_rows(*_split(c, c["y"].cuda()), c["qn"].cuda(), c["kn"].cuda(), kc, vc, c["cu"].cuda(),
                               torch.tensor(c["past"], dtype=torch.int32, device="cuda"), partial_rotary_factor=0.25,
                               rope_theta=1e6, rms_eps=1e-6)
    assert torch.equal(q_out.cpu(), got[0])
    for x, y in ((kc, got[1]), (vc, got[2])):
        for b, (n, p) in enumerate(zip(c["lens"], c["past"])):
            flat = y[c["table"][b].long()].transpose(0, 1).reshape(4, -1, 256)
            assert torch.equal(x[b, :, p:p + n].cpu(), flat[:, p:p + n])
