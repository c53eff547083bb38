"""The paged-cache operators at their edges: captured and replayed, on other streams, at
once, far offsets, many sequences, uneven batches, equal bits from equal calls."""
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


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _step(s, **kw):
    """A decode step of a layer: append, attend, weigh."""
    d = _dev()
    q = d.paged_rows(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["cu"], s["pos"], rope_theta=1e6,
                     rotary_dims=32, q_out=s.get("q_out"), **kw)
    out = d.paged_attention(q, s["kp"], s["vp"], s["table"], s["cu"], s["pos"], gate=s["gate"], lse=s["lse"],
                            out=s.get("out"), workspace=s.get("ws"), **kw)
    d.paged_weights(q, s["kp"], s["table"], s["cu"], s["pos"], s["lse"], weights=s["w"], **kw)
    return out


def _state(n, seed, H=8, Hk=2, d=128, P=16, width=40):
    g = torch.Generator().manual_seed(seed)
    s = dict(kp=pool(n * width, Hk, P, d, g).cuda(), vp=pool(n * width, Hk, P, d, g).cuda(),
             table=torch.randperm(n * width, generator=g).view(n, width).to(torch.int32).cuda(), cu=cu_of([1] * n).cuda(),
             pos=torch.randint(0, width * P - 40, (n,), generator=g).to(torch.int32).cuda(),
             w=torch.zeros(n, Hk, width * P, device="cuda"), lse=torch.zeros(n, H, device="cuda"))
    for k, h in (("q", H), ("k", Hk), ("v", Hk), ("gate", H)):
        s[k] = torch.randn(n, h, d, generator=g).to(BF).cuda()
    return s


def _clone(s):
    return {k: v.clone() for k, v in s.items()}


def _same(a, b):
    return all(torch.equal(a[k], b[k]) for k in ("kp", "vp", "w", "lse"))


def test_captured_and_replayed_with_other_lengths_and_tables():
    s = _state(5, 1)
    eager = _clone(s)
    s["out"], s["q_out"] = (torch.zeros_like(s["q"]) for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(_clone(s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = _clone(s)
    with torch.cuda.graph(graph):
        _step(s)                            # the workspace is the graph's own
    for k, v in keep.items():
        s[k].copy_(v)
    g = torch.Generator().manual_seed(2)
    for step in range(6):
        graph.replay()
        want = _step(eager)
        torch.cuda.synchronize()
        assert torch.equal(s["out"], want) and _same(s, eager), step
        for x in (s, eager):
            x["pos"].add_(1)
        if step == 2:
            pos = torch.tensor([0, 639 - 40, 1, 16, 300], dtype=torch.int32)
            table = torch.randperm(200, generator=g).view(5, 40).to(torch.int32)
            for x in (s, eager):
                x["pos"].copy_(pos)
                x["table"].copy_(table)


def test_two_at_once_on_streams_of_their_own():
    states = [_state(9, 3), _state(4, 4, H=24, Hk=2, d=256, width=100)]
    for s in states:
        s["ws"] = _dev().paged_attention_workspace(s["q"], s["kp"], s["cu"])
    alone = [_clone(s) for s in states]
    want = []
    for s in alone:
        for _ in range(20):
            o = _step(s)
            s["pos"].add_(1)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for i in range(20):
        for j, (s, st) in enumerate(zip(states, streams)):
            with torch.cuda.stream(st):
                got[j] = _step(s)
                s["pos"].add_(1)
    torch.cuda.synchronize()
    for s, a, o, w in zip(states, alone, got, want):
        assert _same(s, a) and torch.equal(o, w)


def test_stream_handles():
    s = _state(3, 5)
    want = _step(_clone(s))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = _step(s, stream=st.cuda_stream)
    kept, lens = _dev().paged_evict(s["kp"], s["vp"], s["table"], s["pos"], s["w"], keep=7, recent=2, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(got, want)
    assert lens.tolist() == [min(7, x) for x in s["pos"].tolist()]


def test_eviction_captured():
    s = _state(4, 6)
    _step(s)
    s["pos"].add_(1)
    eager = _clone(s)
    kept, lens = torch.empty(4, 2, 50, dtype=torch.int32, device="cuda"), torch.empty(4, dtype=torch.int32, device="cuda")
    call = lambda x: _dev().paged_evict(x["kp"], x["vp"], x["table"], x["pos"], x["w"], keep=50, recent=9,     # noqa: E731
                                        weights_out=x["w"], kept=kept, lengths_out=lens)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(_clone(s))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(s)
    graph.replay()
    torch.cuda.synchronize()
    a, b = kept.clone(), lens.clone()
    call(eager)
    assert torch.equal(a, kept) and torch.equal(b, lens) and _same(s, eager)


def test_offsets_past_32_bits():
    """Pools of more than 2^32 elements, rows of queries, gates and outputs 2^31 apart."""
    H, Hk, d, P = 4, 2, 256, 16
    g = torch.Generator().manual_seed(7)
    pages = (1 << 32) // (Hk * P * d) + 9
    kp, vp = (torch.empty(pages, Hk, P, d, dtype=BF, device="cuda") for _ in range(2))
    ids = [pages - 1, 3, pages - 5, pages - 2, pages // 2 + 1, pages - 7]
    table = torch.tensor(ids, dtype=torch.int32)[None]
    past, n = 70, 3
    small = [pool(len(ids), Hk, P, d, g) for _ in range(2)]
    for i, p in enumerate(ids):
        kp[p], vp[p] = small[0][i].cuda(), small[1][i].cuda()
    far = (1 << 31) + 8
    store = torch.zeros(2 * far + H * d, dtype=BF, device="cuda")
    q = torch.as_strided(store, (n, H, d), (far, d, 1))
    gate = torch.as_strided(torch.zeros(2 * far + H * d, dtype=BF, device="cuda"), (n, H, d), (far, d, 1))
    out = torch.as_strided(torch.zeros(2 * far + H * d, dtype=BF, device="cuda"), (n, H, d), (far, d, 1))
    q.copy_(torch.randn(n, H, d, generator=g).to(BF))
    gate.copy_(torch.randn(n, H, d, generator=g).to(BF))
    k, v = (torch.randn(n, Hk, d, generator=g).to(BF).cuda() for _ in range(2))
    d_ = _dev()
    qo = d_.paged_rows(q, k, v, kp, vp, table.cuda(), _i32([0, n]), _i32([past]), rope_theta=1e6, rotary_dims=64)
    d_.paged_attention(qo, kp, vp, table.cuda(), _i32([0, n]), _i32([past]), gate=gate, out=out)
    # the same with pages in order
    kc, vc = (torch.zeros(1, Hk, 96, d, dtype=BF, device="cuda") for _ in range(2))
    for x, y in ((kc, small[0]), (vc, small[1])):
        x[0] = y.transpose(0, 1).reshape(Hk, -1, d).cuda()
    kp2, vp2 = (x[0].view(Hk, 6, P, d).transpose(0, 1).contiguous() for x in (kc, vc))
    t2 = torch.arange(6, dtype=torch.int32, device="cuda")[None]
    qo2 = d_.paged_rows(q, k, v, kp2, vp2, t2, _i32([0, n]), _i32([past]), rope_theta=1e6, rotary_dims=64)
    want = d_.paged_attention(qo2, kp2, vp2, t2, _i32([0, n]), _i32([past]), gate=gate.contiguous())
    assert torch.equal(qo, qo2) and torch.equal(out, want)
    for i, p in enumerate(ids):
        assert torch.equal(kp[p], kp2[i]) and torch.equal(vp[p], vp2[i])
    w = torch.rand(1, Hk, 96, generator=g).cuda()
    for x in ((kp, vp, table.cuda()), (kp2, vp2, t2)):
        kept, lens = d_.paged_evict(*x, _i32([past + n]), w, keep=20, recent=4)
    torch.cuda.synchronize()
    for i, p in enumerate(ids):
        assert torch.equal(kp[p], kp2[i]) and torch.equal(vp[p], vp2[i])


@pytest.mark.parametrize("n", [1, 400, 5000])
def test_many_sequences(n):
    """More sequences than threads of a block; most of them empty or of one position."""
    H, Hk, d, P = 4, 1, 64, 16
    g = torch.Generator().manual_seed(n)
    lens = [int(x) for x in torch.randint(0, 2, (n,), generator=g)]
    past = [int(x) for x in torch.randint(0, 30, (n,), generator=g)]
    lens[0], lens[-1], past[0] = 1, 1, 100
    table, pages = tables([a + b for a, b in zip(lens, past)], P, g)
    kp, vp = (pool(pages, Hk, P, d, g) for _ in range(2))
    q = torch.randn(sum(lens), H, d, generator=g).to(BF)
    lse = torch.empty(sum(lens), H, device="cuda")
    cu = cu_of(lens)
    out = _dev().paged_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), cu.cuda(), _i32(past), lse=lse).cpu()
    w = _dev().paged_weights(q.cuda(), kp.cuda(), table.cuda(), cu.cuda(), _i32(past), lse,
                             weights_out=torch.zeros(n, Hk, 128, device="cuda")).cpu()
    has = torch.tensor(lens, dtype=torch.bool)
    assert (w.sum((1, 2))[has] - H).abs().max() < H * 2.0 ** -16 and (w[~has] == 0).all()
    for b in sorted({0, n - 1, n // 2, n // 3, min(n - 1, 383), min(n - 1, 384), min(n - 1, 288)}):
        if not lens[b]:
            continue
        k, there = gather(kp, table[b], P, 1 + past[b])
        v, _ = gather(vp, table[b], P, 1 + past[b])
        t = int(cu[b])
        want, weight, ls, size = attention64(q[t:t + 1], k, v, there, None, d ** -0.5, past[b])
        e = score_error(d, size, 1.0, 10.0)
        assert ((out[t:t + 1].double() - want).abs() <= attention_bound(want, weight, e)).all(), b
    kept, left = _dev().paged_evict(kp.cuda(), vp.cuda(), table.cuda(), _i32([a + b for a, b in zip(lens, past)]), w.cuda(),
                                    keep=8, recent=3)
    assert left.tolist() == [min(8, a + b) for a, b in zip(lens, past)]


@pytest.mark.parametrize("H,Hk,d,lens,past,P", [
    (4, 1, 256, [1] * 40 + [150], [10] * 40 + [300], 16),        # small tiles, one long sequence
    (8, 1, 64, [200] + [1] * 9, [0] * 10, 4096),                 # pages larger than everything
    (64, 1, 128, [2, 1], [50, 5], 16),                           # more heads of a group than a tile has rows
])
def test_uneven_batches(H, Hk, d, lens, past, P):
    g = torch.Generator().manual_seed(d)
    table, pages = tables([a + b for a, b in zip(lens, past)], P, g, spare=1)
    kp, vp = (pool(pages, Hk, P, d, g) for _ in range(2))
    q = torch.randn(sum(lens), H, d, generator=g).to(BF)
    cu = cu_of(lens)
    out = _dev().paged_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), cu.cuda(), _i32(past)).cpu()
    for b in (0, len(lens) // 2, len(lens) - 1):
        t, m = int(cu[b]), lens[b] + past[b]
        k, there = gather(kp, table[b], P, m)
        v, _ = gather(vp, table[b], P, m)
        want, weight, ls, size = attention64(q[t:t + lens[b]], k, v, there, None, d ** -0.5, past[b])
        e = score_error(d, size, 1.0, 10.0)
        assert ((out[t:t + lens[b]].double() - want).abs() <= attention_bound(want, weight, e)).all(), b


@pytest.mark.parametrize("H,lens", [(2, 1), (8, 1), (12, 2), (12, 4), (24, 3)])
def test_equal_bits_from_equal_calls(H, lens):
    """Whatever the copies' order: repeated with the caches cold and warm."""
    g = torch.Generator().manual_seed(H)
    past = [3001, 17, 9000, 600, 12001, 1, 256, 5000]
    n = [lens, 1, lens, 1, 1, lens, lens, 1]
    table, pages = tables([a + b for a, b in zip(n, past)], 32, g)
    kp, vp = (pool(pages, 2, 32, 256, g).cuda() for _ in range(2))
    q = torch.randn(sum(n), 2 * H, 256, generator=g).to(BF).cuda()
    cold = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    first = None
    for i in range(12):
        if i % 2:
            cold.fill_(i)
        lse = torch.empty(sum(n), 2 * H, device="cuda")
        out = _dev().paged_attention(q, kp, vp, table.cuda(), cu_of(n).cuda(), _i32(past), lse=lse)
        w = _dev().paged_weights(q, kp, table.cuda(), cu_of(n).cuda(), _i32(past), lse,
                                 weights_out=torch.zeros(8, 2, 12016, device="cuda"))
        got = (out, lse, w)
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got)), i


def test_captured_behind_copies_and_other_streams():
    """In a graph the calls follow copies, fills and work of another stream that joins, and
    precede such; each finds what came before it finished."""
    s = _state(6, 12)
    src = {k: torch.randn_like(s[k].float()).to(BF) for k in ("q", "k", "v", "gate")}
    eager = _clone(s)

    def go(x, side):
        for k in ("q", "k"):
            x[k].copy_(src[k])              # a copy node
        x["w"].zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for k in ("v", "gate"):
                x[k].copy_(src[k])
                x[k].mul_(0.5)
        torch.cuda.current_stream().wait_stream(side)
        first = _step(x)
        x["pos"].add_(1)
        x["q"].copy_(first)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):       # beside the next step's rows
            twice = first * 2
        second = _step(x)
        torch.cuda.current_stream().wait_stream(side)
        return first, twice, second

    side = torch.cuda.Stream()
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        go(_clone(s), side)
    torch.cuda.synchronize()
    want = go(eager, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    keep = _clone(s)
    with torch.cuda.graph(graph):
        got = go(s, side)
    for _ in range(3):
        for k, v in keep.items():
            s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and _same(s, eager)


def test_calls_in_a_row_without_waiting():
    """A chain of small calls, each set up while the one before it ends, against the same
    with a wait after every call."""
    a = _state(3, 13, width=30)
    b = _clone(a)
    d = _dev()
    outs = [[], []]
    for x, wait, out in ((a, False, outs[0]), (b, True, outs[1])):
        length = x["pos"].clamp(min=60)
        x["pos"].copy_(length)
        for i in range(40):
            out.append(_step(x))
            if wait:
                torch.cuda.synchronize()
            x["pos"].add_(1)
            if i % 8 == 7:
                kept, lens = d.paged_evict(x["kp"], x["vp"], x["table"], x["pos"], x["w"], keep=55, recent=11,
                                           weights_out=x["w"])
                if wait:
                    torch.cuda.synchronize()
                x["pos"].copy_(lens)
                out.append(kept)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*outs)) and _same(a, b)


def test_the_longest_table():
    """2^24 positions, in pages that repeat: as many keys as pages differ, each counted."""
    Hk, d, P = 1, 64, 16
    g = torch.Generator().manual_seed(14)
    kp, vp = (pool(4, Hk, P, d, g) for _ in range(2))
    width = (1 << 24) // P
    table = (torch.arange(width, dtype=torch.int32) % 4)[None].contiguous()
    q = torch.randn(1, 4, d, generator=g).to(BF)
    lse = torch.empty(1, 4, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    past = (1 << 24) - 1
    out = _dev().paged_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([0, 1]), _i32([past]), lse=lse, status=st)
    k, v = (x[:, 0].reshape(-1, d).double() for x in (kp, vp))
    s = (k @ q[0].double().t()).t() / 8
    p = torch.softmax(s, -1)
    want, weight = p @ v, p @ v.abs()
    e = score_error(d, float((k.abs() @ q[0].double().abs().t()).max()) / 8, 1.0, 25.0)
    # a CTA adds 2^24 / 152 terms, in runs of 64: 2^-14 more than the shorter ones
    assert ((out[0].cpu().double() - want).abs() <= attention_bound(want, weight, e) + 2.0 ** -14 * weight).all()
    assert (lse[0].cpu().double() - torch.logsumexp(s, -1) - torch.log(torch.tensor(2.0 ** 18))).abs().max() < 2.0 ** -13
    w = _dev().paged_weights(q.cuda(), kp.cuda(), table.cuda(), _i32([0, 1]), _i32([past]), lse,
                             weights_out=torch.zeros(1, 1, 1 << 24, device="cuda"), status=st)
    got = w.view(-1, 64).double().sum(0).cpu()
    assert (got - p.sum(0)).abs().max() < 4 * 2.0 ** -12 and int(st) == 0
    _dev().paged_attention(q.cuda(), kp.cuda(), vp.cuda(), table.cuda(), _i32([0, 1]), _i32([past + 1]), status=st)
    assert int(st) == 1
