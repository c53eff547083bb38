"""gattn_prompt_attention on the GPU against float64: head layouts, ragged and
empty sequences, packed keys and caches, gates, strides, and what hidden or
foreign rows must not do."""
import pytest
import torch

from tests.seq_refs import attention64, attention_bound, cu_of, score_error

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _attn(*a, **k):
    from qwen3_gated_attention_gb300 import device
    return device.prompt_attention(*a, **k)


def _randn(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g).to(dtype)


def _check_packed(out, q, k, v, gate, lens, klens=None, scale=None, rows=None):
    klens = klens or lens
    scale = scale or q.shape[-1] ** -0.5
    r = kr = 0
    for n, m in zip(lens, klens):
        a, b = slice(r, r + n), slice(kr, kr + m)
        if n:
            want, weight = attention64(q[a], k[b], v[b], None if gate is None else gate[a], scale, m - n)
            se = score_error(q[a], k[b], scale) if m else 0.0
            tol = attention_bound(want, weight, se)
            err = (out[a].double() - want).abs()
            assert (err <= tol).all(), (n, m, float((err - tol).max()), float(err.max()))
        r, kr = r + n, kr + m


SHAPES = [(4, 2, 64), (5, 1, 64), (6, 2, 192), (8, 8, 128), (12, 1, 256), (16, 4, 256), (24, 2, 256)]


@pytest.mark.parametrize("H,Hk,d", SHAPES)
@pytest.mark.parametrize("lens", [[1], [3, 0, 1, 20], [130, 64, 1]], ids=["one", "short", "tiles"])
def test_packed(H, Hk, d, lens):
    g = torch.Generator().manual_seed(H * d + len(lens))
    T = sum(lens)
    q, k, v, gate = (_randn(g, T, h, d) for h in (H, Hk, Hk, H))
    out = _attn(q.cuda(), k.cuda(), v.cuda(), cu_of(lens, "cuda"), gate=gate.cuda())
    _check_packed(out.cpu(), q, k, v, gate, lens)


@pytest.mark.parametrize("n", [63, 64, 65, 127, 128, 129, 257, 300])
@pytest.mark.parametrize("d", [64, 256])
def test_lengths_around_the_tiles(n, d):
    g = torch.Generator().manual_seed(n)
    q, k, v = (_randn(g, n, h, d) for h in (2, 1, 1))
    out = _attn(q.cuda(), k.cuda(), v.cuda(), cu_of([n], "cuda"))
    _check_packed(out.cpu(), q, k, v, None, [n])


@pytest.mark.parametrize("lens,klens", [([5, 3], [9, 3]), ([7, 4, 2], [3, 0, 300]), ([130], [20])])
@pytest.mark.parametrize("gate_dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_other_key_counts(lens, klens, gate_dtype):
    """More keys than rows (earlier rows), fewer (first rows see nothing), none."""
    g = torch.Generator().manual_seed(sum(klens))
    H, Hk, d = 4, 2, 128
    q, gate = _randn(g, sum(lens), H, d), _randn(g, sum(lens), H, d, dtype=gate_dtype)
    k, v = (_randn(g, sum(klens), Hk, d) for _ in range(2))
    out = _attn(q.cuda(), k.cuda(), v.cuda(), cu_of(lens, "cuda"), cu_kv=cu_of(klens, "cuda"),
                gate=gate.cuda())
    _check_packed(out.cpu(), q, k, v, gate, lens, klens)


def test_no_keys_at_all():
    q = torch.randn(3, 2, 64, device="cuda").to(BF)
    kv = torch.empty(0, 1, 64, device="cuda", dtype=BF)
    out = _attn(q, kv, kv, cu_of([3], "cuda"), cu_kv=cu_of([0], "cuda"))
    assert (out == 0).all()


@pytest.mark.parametrize("layout", ["bhtd", "btd"])
@pytest.mark.parametrize("H,Hk,d,past", [(4, 2, 64, [0, 77, 500]), (24, 2, 256, [46, 0, 900]), (16, 4, 256, [1, 127, 128])])
def test_cache(layout, H, Hk, d, past):
    """Rows appended behind earlier ones; stale slots hold NaN; slots permuted."""
    g = torch.Generator().manual_seed(H)
    lens, B, cap = [4, 33, 1], 5, max(past) + 40
    slots = [3, 0, 4]
    shape = (B, Hk, cap, d) if layout == "bhtd" else (B, cap, Hk, d)
    kc, vc = (torch.full(shape, NAN).to(BF) for _ in range(2))
    kv = [t if layout == "bhtd" else t.transpose(1, 2) for t in (kc, vc)]
    for s, (n, p) in enumerate(zip(lens, past)):
        for t in kv:
            t[slots[s], :, :p + n] = _randn(g, Hk, p + n, d)
    q, gate = _randn(g, sum(lens), H, d), _randn(g, sum(lens), H, d)
    dev = [t.cuda() if layout == "bhtd" else t.transpose(1, 2).contiguous().cuda().transpose(1, 2) for t in kv]
    for hint in (0, 32768):
        out = _attn(q.cuda(), *dev, cu_of(lens, "cuda"), gate=gate.cuda(), max_kv=hint,
                    cache_pos=torch.tensor(past, dtype=torch.int32, device="cuda"),
                    slots=torch.tensor(slots, dtype=torch.int32, device="cuda")).cpu()
        r = 0
        for s, (n, p) in enumerate(zip(lens, past)):
            kk, vv = (t[slots[s], :, :p + n].transpose(0, 1) for t in kv)
            _check_packed(out[r:r + n], q[r:r + n], kk, vv, gate[r:r + n], [n], [p + n])
            r += n


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("poison", [NAN, float("inf"), -float("inf")])
def test_hidden_values_do_not_reach_a_row(d, poison):
    """A value or key that is not finite spoils the rows that see it and no other."""
    g = torch.Generator().manual_seed(d)
    lens, H, Hk = [100, 60], 4, 2
    q, k, v = (_randn(g, 160, h, d) for h in (H, Hk, Hk))
    clean = _attn(q.cuda(), k.cuda(), v.cuda(), cu_of(lens, "cuda")).cpu()
    at = 70                                                 # a row in the middle of the first sequence
    v2 = v.clone()
    v2[at, 0, 5] = poison
    out = _attn(q.cuda(), k.cuda(), v2.cuda(), cu_of(lens, "cuda")).cpu()
    assert torch.equal(out[:at], clean[:at]) and torch.equal(out[100:], clean[100:])
    assert torch.equal(out[:, 2:], clean[:, 2:])            # the other KV head
    touched = out[at:100, :2, 5].float()
    assert (touched.isnan() if poison != poison else touched == poison).all()
    keep = [j for j in range(d) if j != 5]
    assert torch.equal(out[:, :, keep], clean[:, :, keep])
    k2 = k.clone()
    k2[at, 0] = NAN
    out = _attn(q.cuda(), k2.cuda(), v.cuda(), cu_of(lens, "cuda")).cpu()
    assert torch.equal(out[:at], clean[:at]) and torch.equal(out[100:], clean[100:])
    assert torch.equal(out[:, 2:], clean[:, 2:]) and out[at:100, :2].isnan().all()


def test_extreme_scores():
    """Scores far apart: the running maximum moves up by large steps, and a row of
    scores all at the type's lowest end is still a softmax."""
    g = torch.Generator().manual_seed(5)
    n, d = 300, 64
    q, k, v = (_randn(g, n, 1, d) for _ in range(3))
    k = (k.float() * torch.linspace(0.01, 30, n)[:, None, None]).to(BF)
    out = _attn(q.cuda(), k.cuda(), v.cuda(), cu_of([n], "cuda")).cpu()
    _check_packed(out, q, k, v, None, [n])
    q2 = torch.full_like(q, 1e15)
    k2 = torch.full_like(k, -1e15)
    out = _attn(q2.cuda(), k2.cuda(), v.cuda(), cu_of([n], "cuda")).cpu()
    _check_packed(out, torch.zeros_like(q), torch.zeros_like(k), v, None, [n])   # equal scores


def test_strided_slices_and_rows_behind_the_last_sequence():
    g = torch.Generator().manual_seed(6)
    H, Hk, d, T, lens = 6, 2, 128, 70, [31, 20]
    y = _randn(g, T, 2 * H * d + 2 * Hk * d).cuda()
    qg = y[:, :2 * H * d].view(T, H, 2 * d)
    q, gate = qg[..., :d], qg[..., d:]
    k = y[:, 2 * H * d:2 * H * d + Hk * d].view(T, Hk, d)
    v = y[:, 2 * H * d + Hk * d:].view(T, Hk, d)
    wide = torch.full((T, H, 2 * d), 3.0, dtype=BF, device="cuda")
    y[51:] = NAN
    out = _attn(q, k, v, cu_of(lens, "cuda"), gate=gate, out=wide[..., :d], scale=0.05)
    torch.cuda.synchronize()
    assert (wide[..., d:] == 3.0).all() and (wide[51:] == 3.0).all()
    _check_packed(out.cpu(), q.cpu(), k.cpu(), v.cpu(), gate.cpu(), lens, scale=0.05)


def test_skipped_sequences():
    g = torch.Generator().manual_seed(7)
    q, (kc, vc) = _randn(g, 9, 2, 64).cuda(), (_randn(g, 3, 1, 32, 64).cuda() for _ in range(2))
    lens = [3, 3, 3]
    for pos, slots, skipped in (([0, 30, 5], [0, 1, 2], 1), ([0, -1, 5], [0, 1, 2], 1),
                                ([0, 4, 5], [0, 3, 2], 1), ([0, 4, 5], [0, -1, 2], 1)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = _attn(q, kc, vc, cu_of(lens, "cuda"), status=status,
                    cache_pos=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                    slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
        assert int(status) == 1 and (out[3 * skipped:3 * skipped + 3] == 0).all()
        ok = [s for s in range(3) if s != skipped]
        for s in ok:
            a = slice(3 * s, 3 * s + 3)
            kk, vv = (t[slots[s], :, :pos[s] + 3].transpose(0, 1).cpu() for t in (kc, vc))
            _check_packed(out[a].cpu(), q[a].cpu(), kk, vv, None, [3], [pos[s] + 3])
    # packed keys past the tensor
    k = _randn(g, 8, 1, 64).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _attn(q, k, k, cu_of(lens, "cuda"), status=status)
    assert int(status) == 1 and (out[6:] == 0).all()
    _check_packed(out[:6].cpu(), q[:6].cpu(), k[:6].cpu(), k[:6].cpu(), None, [3, 3])


def test_many_sequences():
    g = torch.Generator().manual_seed(8)
    lens = [(5 * i) % 4 for i in range(1300)]
    T = sum(lens)
    q, k, v = (_randn(g, T, h, 64) for h in (2, 1, 1))
    out = _attn(q.cuda(), k.cuda(), v.cuda(), cu_of(lens, "cuda")).cpu()
    _check_packed(out, q, k, v, None, lens)


def test_long_split_is_deterministic_and_right():
    """Few rows over a long cache: the keys are split, the answer does not depend
    on the hint beyond its bound, and a run repeats bit for bit."""
    g = torch.Generator().manual_seed(9)
    H, Hk, d, p, n = 8, 2, 256, 5000, 3
    kc, vc = (_randn(g, 1, Hk, p + n, d) for _ in range(2))
    q = _randn(g, n, H, d)
    args = (q.cuda(), kc.cuda(), vc.cuda(), cu_of([n], "cuda"))
    pos = torch.tensor([p], dtype=torch.int32, device="cuda")
    for hint in (0, 1, p + n, 1 << 30):
        a = _attn(*args, cache_pos=pos, max_kv=hint)
        b = _attn(*args, cache_pos=pos, max_kv=hint)
        assert torch.equal(a, b)
        _check_packed(a.cpu(), q, kc[0].transpose(0, 1), vc[0].transpose(0, 1), None, [n], [p + n])


def test_other_stream_and_graph():
    g = torch.Generator().manual_seed(10)
    lens = [70, 9]
    q, k, v = (_randn(g, 79, h, 128).cuda() for h in (4, 2, 2))
    cu = cu_of(lens, "cuda")
    want = _attn(q, k, v, cu)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = torch.zeros_like(want)
    with torch.cuda.stream(st):
        _attn(q, k, v, cu, out=out)
    st.synchronize()
    assert torch.equal(out, want)
    graph, outs = [], []
    for _ in range(2):                       # two graphs of the same call, replayed at once
        o = torch.zeros_like(want)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            _attn(q, k, v, cu, out=o)
        graph.append(gr)
        outs.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for gr, s in zip(graph, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
