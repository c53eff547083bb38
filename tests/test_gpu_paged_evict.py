"""gattn_paged_weights and gattn_paged_evict on the GPU: the weights against float64, the kept
positions and moved rows exactly, in place and into other pages."""
import math

import pytest
import torch

from tests.paged_refs import BF, evicted, gather, pool, score_error, tables
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ weights

def _weights_case(H, Hk, d, P, lens, past, seed, extra=3):
    g = torch.Generator().manual_seed(seed)
    totals = [a + b for a, b in zip(lens, past)]
    table, pages = tables(totals, P, g)
    c = dict(H=H, Hk=Hk, d=d, P=P, lens=lens, past=past, table=table, cu=cu_of(lens))
    c["kp"] = pool(pages, Hk, P, d, g)
    c["q"] = torch.randn(max(sum(lens), 1), H, d, generator=g).to(BF)[:sum(lens)]
    c["w"] = torch.rand(len(lens), Hk, max(totals) + extra, generator=g)
    own = torch.arange(H) // (H // Hk)
    c["lse"] = torch.full((sum(lens), H), -math.inf)
    c["want"] = torch.full(c["w"].shape, 7.0, dtype=torch.float64)
    c["size"] = 0.0
    scale = d ** -0.5
    for b, (n, p) in enumerate(zip(lens, past)):
        k, there = gather(c["kp"], table[b], P, n + p)
        if n:
            c["want"][b, :, :p] = c["w"][b, :, :p].double()
            c["want"][b, :, p:n + p] = 0
        for i in range(n):
            t, e = int(c["cu"][b]) + i, p + i + 1
            s = torch.einsum("hd,mhd->hm", c["q"][t].double(), k[:e][:, own]) * scale
            c["size"] = max(c["size"], float(torch.einsum("hd,mhd->hm", c["q"][t].double().abs(), k[:e][:, own].abs()).max()) * scale)
            lse = torch.logsumexp(s, -1)
            c["lse"][t] = lse.float()
            c["want"][b, :, :e] += torch.exp(s - c["lse"][t].double()[:, None]).view(Hk, H // Hk, e).sum(1)
    return c


def _run_weights(c, w="w", out=None, **kw):
    o = torch.full(c["w"].shape, 7.0, device="cuda") if out is None else out
    _dev().paged_weights(c["q"].cuda(), c["kp"].cuda(), c["table"].cuda(), c["cu"].cuda(), _i32(c["past"]), c["lse"].cuda(),
                         weights=None if w is None else c["w"].cuda() if w == "w" else w, weights_out=o, **kw)
    torch.cuda.synchronize()
    return o.cpu()


def _weights_bound(c):
    """A term is off by its score's error and 2^-21 of the exponential, the sum of rows and
    heads by 2^-20; the old weight's addition by half a step."""
    rows = max(c["lens"]) * c["H"] // c["Hk"]
    e = score_error(c["d"], c["size"], 1.0, 12.0)
    return lambda want: (math.expm1(e) + 2.0 ** -20) * want.abs() + 2.0 ** -24 * want.abs() + rows * 1e-37


@pytest.mark.parametrize("H,Hk,d", [(16, 4, 256), (24, 2, 256), (8, 2, 64), (16, 8, 128), (6, 2, 192), (5, 1, 128), (40, 1, 64)])
@pytest.mark.parametrize("lens,past,P", [([1], [0], 16), ([1], [1003], 64), ([1, 3, 0, 2], [63, 0, 5, 700], 48), ([6, 1], [100, 17], 32)])
def test_weights_against_float64(H, Hk, d, lens, past, P):
    c = _weights_case(H, Hk, d, P, lens, past, seed=H + P)
    got = _run_weights(c).double()
    assert ((got - c["want"]).abs() <= _weights_bound(c)(c["want"])).all()


@pytest.mark.parametrize("d", [64, 256])
def test_more_rows_than_a_pass_takes(d):
    c = _weights_case(8, 1, d, 16, [30, 2, 9], [50, 600, 0], seed=d)          # 240 rows of one head
    got = _run_weights(c).double()
    assert ((got - c["want"]).abs() <= _weights_bound(c)(c["want"])).all()
    assert torch.equal(got, _run_weights(c).double())


def test_weights_in_place_and_from_nothing():
    c = _weights_case(8, 2, 64, 16, [2, 1], [40, 90], seed=3)
    want = _run_weights(c)
    w = c["w"].cuda()
    w[:, :, 90:] = math.nan                 # new positions and what is behind them
    _run_weights(c, w=w, out=w)
    assert torch.equal(w[0, :, :42].cpu(), want[0, :, :42]) and torch.equal(w[1, :, :91].cpu(), want[1, :, :91])
    assert w[1, :, 91:].isnan().all()
    none = _run_weights(c, w=None)
    assert torch.equal(none[0, :, 40:42], want[0, :, 40:42])
    assert ((none[0, :, :40] - (want[0, :, :40] - c["w"][0, :, :40])).abs() <= 2.0 ** -23 * want[0, :, :40]).all()


def test_weights_skips():
    c = _weights_case(8, 2, 64, 16, [1, 1, 1], [20, 47, 30], seed=4, extra=0)
    c["past"][1] = 48                        # one beyond the weights
    c["lse"][2] = -math.inf
    c["table"][0, 1] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _run_weights(c, status=st)
    assert int(st) == 1 and (got[1] == 7).all()
    assert torch.equal(got[2, :, :30], c["w"][2, :, :30]) and (got[2, :, 30] == 0).all()
    assert torch.equal(got[0, :, 16:20], c["w"][0, :, 16:20]) and (got[0, :, 20] == 0).all()
    assert (got[0, :, :16] > c["w"][0, :, :16]).all()


def test_weights_add_up_to_the_rows():
    """One token's weights are a distribution, with the log sums that attention leaves."""
    g = torch.Generator().manual_seed(5)
    table, pages = tables([900], 32, g)
    kp, vp = (pool(pages, 2, 32, 128, g).cuda() for _ in range(2))
    q = torch.randn(1, 8, 128, generator=g).to(BF).cuda()
    lse = torch.empty(1, 8, device="cuda")
    _dev().paged_attention(q, kp, vp, table.cuda(), _i32([0, 1]), _i32([899]), lse=lse)
    w = _dev().paged_weights(q, kp, table.cuda(), _i32([0, 1]), _i32([899]), lse,
                             weights_out=torch.zeros(1, 2, 900, device="cuda"))
    assert (w.sum(-1) - 4).abs().max() < 4 * 2.0 ** -18


# ----------------------------------------------------------------- eviction

def _evict_case(Hk, d, P, lengths, keep, seed, width=None, spare=None, draw=None):
    g = torch.Generator().manual_seed(seed)
    out = [min(x, keep) for x in lengths]
    table, pages = tables(lengths + out, P, g, width=width)
    n = len(lengths)
    c = dict(Hk=Hk, d=d, P=P, lengths=lengths, keep=keep, table=table[:n], out=table[n:])
    c["kp"], c["vp"] = (pool(pages, Hk, P, d, g) for _ in range(2))
    L = max(max(lengths), 1)
    c["w"] = torch.exp(2.5 * torch.randn(n, Hk, L, generator=g) - 6) if draw is None else draw(n, Hk, L, g)
    return c


def _run_evict(c, recent, into_pages, alias=False, **kw):
    x = {k: c[k].cuda() for k in ("kp", "vp", "table", "out", "w")}
    n, Hk, keep = len(c["lengths"]), c["Hk"], c["keep"]
    wo = x["w"] if alias else torch.full((n, Hk, keep), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, lens = _dev().paged_evict(x["kp"], x["vp"], x["table"], _i32(c["lengths"]), x["w"], keep=keep, recent=recent,
                                    out_table=x["out"] if into_pages else None, weights_out=wo, status=st, **kw)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in dict(kept=kept, lens=lens, kp=x["kp"], vp=x["vp"], w=wo, status=st).items()}


def _check_evict(c, recent, got, into_pages, skipped=()):
    P = c["P"]
    want_k, want_v = c["kp"].clone(), c["vp"].clone()
    for b, length in enumerate(c["lengths"]):
        if b in skipped:
            assert (got["kept"][b] == -1).all() and int(got["lens"][b]) == length
            continue
        m = min(length, c["keep"])
        assert int(got["lens"][b]) == m
        to = c["out"][b] if into_pages else c["table"][b]
        for h in range(c["Hk"]):
            at = evicted(c["w"][b, h].tolist(), length, c["keep"], recent)
            assert got["kept"][b, h, :m].tolist() == at and (got["kept"][b, h, m:] == -1).all(), (b, h)
            f, t = torch.tensor(at, dtype=torch.int64), torch.arange(m)
            a, o = got["w"][b, h, :m], c["w"][b, h, f]
            assert torch.equal(a.isnan(), o.isnan()) and torch.equal(a.nan_to_num(), o.nan_to_num())
            src, dst = c["table"][b].long()[f // P], to.long()[t // P]
            want_k[dst, h, t % P] = c["kp"][src, h, f % P]
            want_v[dst, h, t % P] = c["vp"][src, h, f % P]
    assert torch.equal(got["kp"], want_k) and torch.equal(got["vp"], want_v)


@pytest.mark.parametrize("into_pages", [True, False])
@pytest.mark.parametrize("Hk,d,P", [(4, 256, 16), (1, 64, 48), (3, 128, 32), (2, 192, 128)])
@pytest.mark.parametrize("keep,recent", [(100, 20), (1, 0), (1, 1), (64, 64), (5000, 100), (777, 0)])
def test_evict(Hk, d, P, keep, recent, into_pages):
    c = _evict_case(Hk, d, P, [1000, 0, 1, 100, 101, 3000], keep, seed=keep + d)
    got = _run_evict(c, recent, into_pages)
    assert int(got["status"]) == 0
    _check_evict(c, recent, got, into_pages)
    if keep <= c["w"].shape[2]:
        again = _run_evict(c, recent, into_pages, alias=True)
        _check_evict(c, recent, again, into_pages)
        assert torch.equal(again["kp"], got["kp"]) and torch.equal(again["w"][..., c["keep"]:], c["w"][..., c["keep"]:])


@pytest.mark.parametrize("draw", ["equal", "few", "signs", "odd", "tiny"])
@pytest.mark.parametrize("keep,recent", [(500, 0), (500, 100), (4100, 33)])
def test_order_of_weights(draw, keep, recent):
    """Ties go to the lowest position; zeros of both signs are one; NaN counts as -infinity."""
    def make(n, Hk, L, g):
        w = torch.randn(n, Hk, L, generator=g)
        if draw == "equal":
            return torch.full((n, Hk, L), 0.25)
        if draw == "few":
            return torch.randint(0, 3, (n, Hk, L), generator=g).float()
        if draw == "signs":
            return torch.where(w > 1, w, torch.where(w < 0, torch.tensor(-0.0), torch.tensor(0.0)))
        if draw == "odd":
            w[w > 2] = math.inf
            w[w < -1] = math.nan
            w[(w > -0.5) & (w < -0.4)] = -math.inf
            return w
        return w * 1e-42
    c = _evict_case(2, 64, 16, [5000, 4096, 12], keep, seed=7, draw=make)
    for into_pages in (True, False):
        _check_evict(c, recent, _run_evict(c, recent, into_pages), into_pages)


@pytest.mark.parametrize("into_pages", [True, False])
def test_long_sequences(into_pages):
    """More positions than stay in shared memory while they are selected."""
    c = _evict_case(1, 64, 64, [70000, 32769], 20000, seed=8)
    _check_evict(c, 4000, _run_evict(c, 4000, into_pages), into_pages)


@pytest.mark.parametrize("into_pages", [True, False])
def test_evict_skips(into_pages):
    c = _evict_case(2, 64, 16, [100, 120, 90, 80], 50, seed=9)
    c["lengths"] = [100, 121, -1, 80]
    got = _run_evict(c, 5, into_pages)
    assert int(got["status"]) == 1
    _check_evict(c, 5, got, into_pages, skipped=(1, 2))
    # a table row that is too short for what is kept
    c = _evict_case(2, 64, 16, [100, 20], 50, seed=9)
    c["out"] = c["out"][:, :2].contiguous()
    got = _run_evict(c, 5, True)
    assert int(got["status"]) == 1
    _check_evict(c, 5, got, True, skipped=(0,))


@pytest.mark.parametrize("into_pages", [True, False])
def test_evict_leaves_what_has_no_page(into_pages):
    c = _evict_case(1, 64, 16, [64], 40, seed=10)
    bad = int(c["table"][0, 3])
    c["table"][0, 3] = -1
    got = _run_evict(c, 16, into_pages)
    assert int(got["status"]) == 1 and got["kept"][0, 0, 24:].tolist() == list(range(48, 64))
    at = evicted(c["w"][0, 0].tolist(), 64, 40, 16)
    to = c["out"][0] if into_pages else c["table"][0]
    for j in range(24):
        assert torch.equal(got["kp"][int(to[j // 16]), 0, j % 16], c["kp"][int(c["table"][0, at[j] // 16]), 0, at[j] % 16])
    for j in range(24, 40):                 # as they were
        assert torch.equal(got["kp"][int(to[j // 16]), 0, j % 16], c["kp"][int(to[j // 16]), 0, j % 16])
    assert torch.equal(got["kp"][bad], c["kp"][bad])


def test_one_sequence_through_all_four():
    """Tokens appended, attended and weighed, the sequence cut, more tokens at their own
    positions: attention over what is left equals float64 over the kept keys."""
    from tests.paged_refs import attention64, attention_bound, turn64
    g = torch.Generator().manual_seed(11)
    H, Hk, d, P, W = 8, 2, 128, 16, 8
    kp, vp = (torch.zeros(W + 1, Hk, P, d, dtype=BF, device="cuda") for _ in range(2))
    table = torch.randperm(W + 1, generator=g)[:W].to(torch.int32)[None].cuda()
    w = torch.zeros(1, Hk, W * P, device="cuda")
    qn, kn = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF) for _ in range(2))
    keys = [[] for _ in range(Hk)]          # (position, value row) of each head
    dev, at = _dev(), 0
    length = 0
    for step, n in enumerate([30, 1, 1, 3, 1, 40, 1]):
        y = torch.randn(n, (H + 2 * Hk) * d, generator=g).to(BF)
        q, k, v = (y[:, :H * d].view(n, H, d), y[:, H * d:(H + Hk) * d].view(n, Hk, d), y[:, (H + Hk) * d:].view(n, Hk, d))
        pos = torch.arange(at, at + n, dtype=torch.int32)
        q_out = dev.paged_rows(q.cuda(), k.cuda(), v.cuda(), kp, vp, table, _i32([0, n]), _i32([length]), rope_theta=1e6,
                               rotary_dims=32, q_norm=qn.cuda(), k_norm=kn.cuda(), positions=pos.cuda())
        for i in range(n):
            kk = turn64(k[i], kn, at + i, 32, False).to(BF)
            for h in range(Hk):
                keys[h].append((kk[h], v[i, h]))
        lse = torch.empty(n, H, device="cuda")
        out = dev.paged_attention(q_out, kp, vp, table, _i32([0, n]), _i32([length]), lse=lse)
        dev.paged_weights(q_out, kp, table, _i32([0, n]), _i32([length]), lse, weights=w)
        kf = torch.stack([torch.stack([x[0] for x in keys[h]]) for h in range(Hk)], 1)
        vf = torch.stack([torch.stack([x[1] for x in keys[h]]) for h in range(Hk)], 1)
        there = torch.ones(len(kf), dtype=torch.bool)
        want, weight, ls, size = attention64(q_out.cpu(), kf, vf, there, None, d ** -0.5, length)
        # keys of the cache and of the reference may round apart: 2^-8 of a score's size
        bound = attention_bound(want, weight, score_error(d, size, 1.0, 10.0) + 2.0 ** -12 * size)
        assert ((out.cpu().double() - want).abs() <= bound).all(), step
        length += n
        at += n
        if length > 32:
            kept, lens = dev.paged_evict(kp, vp, table, _i32([length]), w, keep=24, recent=8, weights_out=w)
            for h in range(Hk):
                keys[h] = [keys[h][i] for i in kept[0, h].tolist()]
            length = int(lens)
            assert length == 24
