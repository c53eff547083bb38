"""gattn_paged_attention on the GPU against float64: head layouts, pages, lengths from one
to long ones, odd sizes, strides, what a row does not see, bad tables."""
import math

import pytest
import torch

from tests.paged_refs import BF, attention64, attention_bound, gather, pool, score_error, tables
from tests.seq_refs import cu_of

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


def _case(H, Hk, d, P, lens, past, seed, gate=BF, token_major=False, width=None, lead=0):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens), len(lens)
    table, pages = tables([a + b for a, b in zip(lens, past)], P, g, width=width)
    c = dict(H=H, Hk=Hk, d=d, P=P, lens=lens, past=past, table=table, scale=d ** -0.5, lead=lead)
    c["kp"], c["vp"] = (pool(pages, Hk, P, d, g, token_major) for _ in range(2))
    y = torch.randn(T + 2 * lead, H, 2 * d, generator=g).to(BF)
    c["q"] = y[..., :d]
    c["gate"] = None if gate is None else torch.randn(T + 2 * lead, H, 2 * d, generator=g).to(gate)[..., d:]
    c["cu"] = cu_of(lens) + lead
    return c


def _to(x):
    """On the GPU with its strides."""
    if x is None:
        return None
    base = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
    return base.copy_(x)


def _run(c, **kw):
    dev = {k: _to(c[k]) for k in ("q", "kp", "vp", "table", "gate")}
    lse = torch.full((c["q"].shape[0], c["H"]), 7.0, device="cuda")
    out = torch.full((c["q"].shape[0], c["H"], c["d"]), 7.0, dtype=BF, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    _dev().paged_attention(dev["q"], dev["kp"], dev["vp"], dev["table"], c["cu"].cuda(),
                           torch.tensor(c["past"], dtype=torch.int32, device="cuda"), gate=dev["gate"],
                           scale=c["scale"], out=out, lse=lse, status=st, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(st)


def _check(c, out, lse, seqs=None):
    for b, n in enumerate(c["lens"]):
        if not n or (seqs is not None and b not in seqs):
            continue
        t0, p = int(c["cu"][b]), c["past"][b]
        rows = slice(t0, t0 + n)
        k, there = gather(c["kp"], c["table"][b], c["P"], n + p)
        v, _ = gather(c["vp"], c["table"][b], c["P"], n + p)
        gate = None if c["gate"] is None else c["gate"][rows]
        want, weight, ls, size = attention64(c["q"][rows], k, v, there, gate, c["scale"], p)
        top = float(ls[ls.isfinite()].abs().max()) if ls.isfinite().any() else 0.0
        e = score_error(c["d"], size, c["scale"], top)
        err = (out[rows].double() - want).abs()
        bound = attention_bound(want, weight, e)
        assert (err <= bound).all(), (b, float((err - bound).max()), float(err.max()))
        got = lse[rows].double()
        assert torch.equal(got.isfinite(), ls.isfinite())
        off = (got - ls)[ls.isfinite()].abs()
        # the score's error, then logarithm, product and the sum's 2^-20
        assert (off <= e + 2.0 ** -19 + 4 * 2.0 ** -24 * top).all(), (b, float(off.max()))
    lead, T = c["lead"], sum(c["lens"])
    for x in (out, lse):            # rows of no sequence
        assert (x[:lead] == 7).all() and (x[lead + T:] == 7).all()


HEADS = [(16, 4, 256), (24, 2, 256), (32, 8, 256), (8, 2, 64), (16, 8, 128), (6, 2, 192), (5, 1, 128), (3, 3, 64),
         (40, 1, 64), (66, 2, 64)]


@pytest.mark.parametrize("H,Hk,d", HEADS)
@pytest.mark.parametrize("lens,past,P", [
    ([1], [0], 16),
    ([1], [1003], 64),
    ([1, 1, 1], [15, 16, 17], 16),
    ([1, 3, 0, 2], [63, 0, 5, 700], 48),
    ([4, 4], [100, 61], 32),
])
def test_against_float64(H, Hk, d, lens, past, P):
    c = _case(H, Hk, d, P, lens, past, seed=H + d + P)
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse)


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("gate,token_major", [(None, False), (torch.float32, True), (BF, True)])
def test_gates_and_pool_layouts(d, gate, token_major):
    c = _case(8, 2, d, 16, [1, 2, 5], [300, 33, 12], seed=d, gate=gate, token_major=token_major, lead=3)
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse)


@pytest.mark.parametrize("P", [16, 48, 80, 128, 512])
def test_many_sequences_share_the_work(P):
    """Runs of the work that begin and end anywhere: hundreds of short and a few long
    sequences, parts of one segment in many CTAs."""
    g = torch.Generator().manual_seed(P)
    lens = [int(x) for x in torch.randint(0, 4, (300,), generator=g)]
    past = [int(x) for x in torch.randint(0, 200, (300,), generator=g)]
    past[7], past[150], lens[7], lens[150] = 9000, 4001, 1, 3
    c = _case(4, 1, 64, P, lens, past, seed=P)
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse, seqs=set(range(0, 300, 17)) | {7, 150})


@pytest.mark.parametrize("d", [64, 128, 192, 256])
@pytest.mark.parametrize("seed", [0, 1])
def test_rows_of_all_numbers_side_by_side(d, seed):
    """Parts of one to 72 rows in turn in every CTA: groups of one to eight warps, some of
    them whole, some joined."""
    g = torch.Generator().manual_seed(seed)
    lens = [int(x) for x in torch.randint(1, 7, (150,), generator=g)]
    past = [int(x) for x in torch.randint(0, 400, (150,), generator=g)]
    past[40] = 6000
    c = _case(24, 2, d, 16, lens, past, seed=d + seed)
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse, seqs=set(range(seed, 150, 7)) | {40})
    again, lse2, _ = _run(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("H,Hk,d,lens,past", [(24, 2, 256, [1], [20000]), (24, 2, 256, [3], [9999]),
                                              (16, 1, 64, [2, 1], [30000, 1]), (4, 4, 128, [1], [70000])])
def test_long_contexts(H, Hk, d, lens, past):
    c = _case(H, Hk, d, 64, lens, past, seed=1)
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse)


@pytest.mark.parametrize("d,P", [(256, 16), (64, 64), (128, 32), (192, 16)])
def test_a_prompt_of_many_rows(d, P):
    c = _case(4, 2, d, P, [70, 1, 33], [0, 40, 90], seed=d)
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse)


@pytest.mark.parametrize("d,P", [(256, 16), (64, 64), (128, 48)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_row_does_not_see(d, P, bad):
    """Keys and values behind a row's last position hold anything: in the rest of its page,
    in pages of nobody, and in the later rows of its own sequence."""
    c = _case(4, 2, d, P, [3, 1], [37, 5], seed=d)
    clean, clean_lse, _ = _run(c)
    for b, (n, p) in enumerate(zip(c["lens"], c["past"])):
        end = n + p
        page = int(c["table"][b, (end - 1) // P])
        for x in (c["kp"], c["vp"]):
            x[page, :, (end - 1) % P + 1:] = bad
    used = {int(c["table"][b, i]) for b in range(2) for i in range((c["lens"][b] + c["past"][b] - 1) // P + 1)}
    for i in range(c["kp"].shape[0]):
        if i not in used:
            c["kp"][i] = bad
            c["vp"][i] = bad
    out, lse, st = _run(c)
    assert st == 0 and torch.equal(out, clean) and torch.equal(lse, clean_lse)
    # the value of row 2 (position 39): rows 0 and 1 do not see it
    page, at = int(c["table"][0, 39 // P]), 39 % P
    c["vp"][page, :, at] = bad
    out, lse, st = _run(c)
    weight = (out[:2].double() - clean[:2].double()).abs()
    assert (weight <= 2 * 2.0 ** -8 * clean[:2].double().abs() + 2.0 ** -12).all()      # another order of sums
    assert torch.equal(lse, clean_lse) and not out[2].isfinite().any()
    assert torch.equal(out[3], clean[3])
    c["kp"][page, :, at] = bad
    out, lse, _ = _run(c)
    assert out[:2].isfinite().all() and torch.equal(lse[:2], clean_lse[:2])


def test_entries_that_are_no_page():
    c = _case(8, 2, 128, 32, [1, 2, 1], [200, 90, 64], seed=4)
    c["table"][0, 2] = -1
    c["table"][1, 0] = c["kp"].shape[0]
    c["table"][2, :] = 2 ** 31 - 1
    out, lse, st = _run(c)
    assert st == 1
    _check(c, out, lse)
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()


def test_sequences_that_do_not_fit_their_table():
    c = _case(8, 2, 64, 16, [1, 2, 1, 3], [20, 30, 31, 0], seed=5, width=2)
    c["past"] = [20, 31, -1, 2 ** 31 - 2]
    out, lse, st = _run(c)
    assert st == 1
    _check(c, out, lse, seqs={0})
    assert (out[1:] == 0).all() and (lse[1:] == -math.inf).all()


def test_a_long_prompt_that_does_not_fit():
    """Its rows are zeroed by the whole grid, beside sequences that do fit."""
    c = _case(4, 2, 64, 16, [1, 300, 1], [20, 0, 9], seed=12)
    big = 200000
    c["lens"], c["cu"] = [1, big, 1], cu_of([1, big, 1])
    c["q"] = torch.randn(big + 2, 4, 64).to(BF)
    c["gate"] = torch.randn(big + 2, 4, 64).to(BF)
    out, lse, st = _run(c)
    assert st == 1 and (out[1:-1] == 0).all() and (lse[1:-1] == -math.inf).all()
    _check(c, out, lse, seqs={0, 2})


def test_peaked_scores():
    """Scores of very different sizes: the reference moves often, and far."""
    c = _case(8, 2, 128, 16, [1, 3], [500, 77], seed=6)
    c["kp"] *= torch.linspace(0.01, 30, c["kp"].shape[0]).to(BF)[:, None, None, None]
    out, lse, st = _run(c)
    assert st == 0
    _check(c, out, lse)


def test_shared_prefix_and_equal_calls():
    c = _case(8, 2, 64, 16, [1, 1], [40, 40], seed=8)
    c["table"][1, :2] = c["table"][0, :2]
    out, lse, st = _run(c)
    _check(c, out, lse)
    again, lse2, _ = _run(c)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
