"""The packed-sequence operators where calls are unusual: every width of a CTA's
share of the state, columns of very different sizes, offsets past 32 bits, several
calls at once, graphs whose lengths change between replays, streams of their own."""
import pytest
import torch

from tests import seq_refs as R
from tests.test_gpu_delta import _case, _check, _fn, _parts, _run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _dev():
    from qwen3_gated_attention_gb300 import device
    return device


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(g, *shape, dtype=BF):
    return torch.randn(*shape, generator=g).to(dtype)


# 10 sequences of 8 heads: more column groups than SMs, so a CTA takes 64 or 128 columns
WIDE = [(64, 64), (64, 128), (128, 64), (128, 128), (128, 192), (64, 256)]
LENS = [1, 0, 33, 70, 32, 5, 64, 31, 2, 47]


@pytest.mark.parametrize("dk,dv", WIDE)
def test_wide_shares_of_the_state(dk, dv):
    c = _case(4, 8, dk, dv, LENS, dk + dv, extra=3)
    c["y"][-3:] = float("nan")
    out, so = _run("prompt", c)
    _check(c, out, so)
    again, so2 = _run("prompt", c, inplace=True)
    assert torch.equal(again, out) and torch.equal(so2, so)


@pytest.mark.parametrize("dv", [64, 128])
def test_wide_shares_with_spoilt_rows_and_slots(dv):
    c = _case(4, 8, 128, dv, LENS, 50 + dv, slots=[3, 1, 12, 0, 5, 5, 9, 11, -1, 2], nslots=12)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    base, so = _run("prompt", c, status=status)
    _check(c, base, so, skipped=(2, 5, 8))
    assert int(status) == 1
    d = dict(c, y=c["y"].clone(), g=c["g"].clone())
    r0 = sum(LENS[:3])
    d["y"][r0 + 41, 4 * 128 + 7] = float("inf")        # key head 0 of the 70-row sequence
    d["g"][r0 + 50, 4] = float("nan")                  # value head 4, key head 2
    out, s2 = _run("prompt", d)
    own = [i for i in range(out.shape[0]) if not r0 <= i < r0 + 70]
    assert torch.equal(out[own], base[own])
    assert torch.equal(out[r0:r0 + 41], base[r0:r0 + 41])
    assert not out[r0 + 41:r0 + 70, :2].isfinite().any()
    assert torch.equal(out[r0:r0 + 50, 2:], base[r0:r0 + 50, 2:])
    assert not out[r0 + 50:r0 + 70, 4].isfinite().any()
    heads = [2, 3, 5, 6, 7]
    assert torch.equal(out[r0:r0 + 70, heads], base[r0:r0 + 70, heads])
    assert torch.equal(s2[0, heads], so[0, heads])


@pytest.mark.parametrize("name", ["prompt", "step"])
@pytest.mark.parametrize("dv,n", [(32, 1), (64, 10), (128, 10)])
def test_columns_of_very_different_sizes(name, dv, n):
    """The columns of a state do not meet, and powers of two commute with every
    rounding: scaling column j of the state and of the values by 2^e_j scales its
    outputs by 2^e_j.  Each column is held to a bound of its own size."""
    c = _case(4 if n > 1 else 1, 8 if n > 1 else 2, 128, dv, [40] * n, 60 + dv)
    e = (torch.arange(dv) * 7 % 61 - 30).float()
    f = torch.exp2(e)
    Hv, a = c["Hv"], 2 * c["Hk"] * 128
    want, base_state = _run(name, c)
    d = dict(c, y=c["y"].clone(), S=c["S"] * f)
    d["y"][:, a:] = (c["y"][:, a:].view(-1, Hv, dv).float() * f).to(BF).view(-1, Hv * dv)
    out, so = _run(name, d)
    q, k, v = _parts(c, c["y"])
    for s in (0, n - 1):
        r = slice(40 * s, 40 * s + 40)
        w, last, top = R.delta64(q[r], k[r], v[r], c["g"][r], c["beta"][r], c["S"][s], 128 ** -0.5, 1e-6)
        err = R.delta_bound(40, top, 128)
        tol = R.U_BF16 * w.abs() + 128 ** -0.5 * (128 ** 0.5 * err + 3 * 2.0 ** -16 * top + 2.0 ** -17 * top)
        assert ((out[r].double() / f - w).abs() <= tol).all()
        assert float((so[s].double() / f - last).abs().max()) <= err
    assert want.isfinite().all() and base_state.isfinite().all()


@pytest.mark.parametrize("name", ["prompt", "step"])
def test_rows_of_very_different_sizes(name):
    """Normalized keys and queries do not depend on their rows' sizes (no epsilon)."""
    c = _case(1, 2, 64, 64, [45], 70)
    a = 2 * 64
    f = torch.exp2((torch.arange(45) * 11 % 81 - 40).float())[:, None]
    y = c["y"].clone()
    y[:, :a] = (y[:, :a].float() * f).to(BF)
    q, k, v = _parts(c, c["y"])
    want, last, top = R.delta64(q, k, v, c["g"], c["beta"], c["S"][0], 0.125, 0.0)
    so = torch.zeros_like(c["S"]).cuda()
    out = _fn(name)(*_parts(c, y.cuda()), c["g"].cuda(), c["beta"].cuda(), num_seqs=1, state=c["S"].cuda(),
                    state_out=so, qk_l2norm=True, l2_eps=0.0)
    e = R.delta_bound(45, top, 64)
    tol = R.U_BF16 * want.abs() + 0.125 * (8 * e + 3 * 2.0 ** -16 * top + 2.0 ** -18 * top)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert float((so.cpu()[0].double() - last).abs().max()) <= e


@pytest.mark.parametrize("H,Hk,d", [(128, 1, 64), (256, 1, 64), (7, 1, 128), (192, 3, 64)])
def test_large_and_odd_groups(H, Hk, d):
    from tests.test_gpu_prompt_attention import _check_packed
    g = torch.Generator().manual_seed(H)
    lens, klens = [3, 1, 18], [3, 200, 150]
    q = _randn(g, 22, H, d)
    k, v = (_randn(g, sum(klens), Hk, d) for _ in range(2))
    out = _dev().prompt_attention(q.cuda(), k.cuda(), v.cuda(), R.cu_of(lens, "cuda"),
                                  cu_kv=R.cu_of(klens, "cuda")).cpu()
    _check_packed(out, q, k, v, None, lens, klens)


def test_many_longer_sequences():
    """More sequences than lanes, with tiles of several blocks among them."""
    from tests.test_gpu_prompt_attention import _check_packed
    g = torch.Generator().manual_seed(80)
    lens = [(37 * i) % 300 if i % 4 else i % 3 for i in range(45)]
    T = sum(lens)
    q, k, v, gate = _randn(g, T, 4, 128), _randn(g, T, 2, 128), _randn(g, T, 2, 128), _randn(g, T, 4, 128)
    out = _dev().prompt_attention(*(x.cuda() for x in (q, k, v)), R.cu_of(lens, "cuda"), gate=gate.cuda()).cpu()
    _check_packed(out, q, k, v, gate, lens)


def test_offsets_past_32_bits():
    """Rows, cache slots and state slots more than 2^32 elements apart."""
    from tests.test_gpu_prompt_attention import _check_packed
    dv, g = _dev(), torch.Generator().manual_seed(81)
    far = (1 << 32) + 64
    big = torch.empty(far + (1 << 20), dtype=BF, device="cuda")

    def spread(x, step):
        """x [n][h][d] with its rows `step` elements apart"""
        n, h, d = x.shape
        out = big.as_strided((n, h, d), (step, d, 1))
        out.copy_(x.cuda())
        return out

    # three query rows, the last past 2^32
    T, H, Hk, d = 3, 4, 2, 64
    q, k, v = _randn(g, T, H, d), _randn(g, T, Hk, d), _randn(g, T, Hk, d)
    cu = R.cu_of([T], "cuda")
    out = dv.prompt_attention(spread(q, far // 2 + 8), k.cuda(), v.cuda(), cu)
    _check_packed(out.cpu(), q, k, v, None, [T])
    out = dv.prompt_attention(q.cuda(), spread(k, far // 2 + 8), v.cuda(), cu)
    _check_packed(out.cpu(), q, k, v, None, [T])
    far_out = big.as_strided((T, H, d), (far // 2 + 8, d, 1))
    dv.prompt_attention(q.cuda(), k.cuda(), v.cuda(), cu, out=far_out)
    _check_packed(far_out.cpu(), q, k, v, None, [T])
    # a cache slot past 2^32: written, then read
    small = torch.zeros(2, Hk, 16, d, dtype=BF, device="cuda")
    kc = big.as_strided((2, Hk, 16, d), (far, 16 * d, d, 1))
    kc.zero_()
    w = torch.ones(d, dtype=BF, device="cuda")
    kw = dict(partial_rotary_factor=0.5, rope_theta=1e4, rms_eps=1e-6, slots=_i32(1))
    rows = (q.cuda(), k.cuda(), v.cuda(), w, w)
    a = dv.prompt_rows(*rows, small, small.clone(), cu, _i32(5), **kw)
    b = dv.prompt_rows(*rows, kc, small.clone(), cu, _i32(5), **kw)
    assert torch.equal(a, b) and torch.equal(kc, small)
    near = dv.prompt_attention(a, small, small, cu, cache_pos=_i32(5), slots=_i32(1))
    assert torch.equal(dv.prompt_attention(a, kc, small, cu, cache_pos=_i32(5), slots=_i32(1)), near)
    # rows and states of the delta rule
    c = _case(1, 2, 64, 64, [T], 82)
    y, gl, be = c["y"].cuda(), c["g"].cuda(), c["beta"].cuda()
    qd, kd, vd = _parts(c, y)
    states = big.view(torch.float32).as_strided((2, 2, 64, 64), (far // 2, 4096, 64, 1))
    for name in ("prompt", "step"):
        want_state = c["S"].cuda()
        want = _fn(name)(qd, kd, vd, gl, be, cu, state=want_state, state_out=want_state)
        states[1].copy_(c["S"][0])
        assert torch.equal(_fn(name)(qd, kd, vd, gl, be, cu, state=states, state_out=states, slots=_i32(1)), want)
        assert torch.equal(states[1], want_state[0])
        s2 = c["S"].cuda()
        assert torch.equal(_fn(name)(qd, kd, spread(vd.cpu(), far // 2 + 8), gl, be, cu, state=s2), want)


def _stack(dv, x, cu, pos, kc, vc, st):
    """One pass of every operator; a list of what it writes."""
    w = torch.ones(64, dtype=BF, device="cuda")
    q = dv.prompt_rows(x["q"], x["k"], x["v"], w, w, kc, vc, cu, pos, partial_rotary_factor=0.25, rope_theta=1e6,
                       rms_eps=1e-6)
    a = dv.prompt_attention(q, kc, vc, cu, cache_pos=pos, gate=x["gate"])
    d = dv.delta_prompt(x["k"], x["v"], a, x["g"], x["beta"], cu, state=st, state_out=st, qk_l2norm=True)
    e = dv.delta_step(x["k"], x["v"], d, x["g"], x["beta"], cu, state=st, state_out=st, qk_l2norm=True)
    return [q, a, d, e, kc, vc, st]


def _stack_inputs(seed, T=90, n=4):
    g = torch.Generator().manual_seed(seed)
    x = {k: _randn(g, T, h, 64).cuda() for k, h in (("q", 4), ("k", 2), ("v", 2), ("gate", 4))}
    x["g"] = -torch.rand(T, 4, generator=g).cuda()
    x["beta"] = torch.rand(T, 4, generator=g).cuda()
    kc, vc = (_randn(g, n, 2, 128, 64).cuda() for _ in range(2))
    return x, kc, vc, torch.randn(n, 4, 64, 64, generator=g).cuda()


def test_calls_at_once_on_several_streams():
    """Calls share nothing: three streams, each with tensors of its own."""
    dv = _dev()
    cu, pos = R.cu_of([40, 0, 1, 49], "cuda"), _i32(3, 0, 100, 9)
    sets = [_stack_inputs(90 + i) for i in range(3)]
    want = [[t.clone() for t in _stack(dv, x, cu, pos, kc.clone(), vc.clone(), st.clone())]
            for x, kc, vc, st in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        copies = [(kc.clone(), vc.clone(), st.clone()) for _, kc, vc, st in sets]
        torch.cuda.synchronize()
        for (x, *_), own, s in zip(sets, copies, streams):
            with torch.cuda.stream(s):
                got.append(_stack(dv, x, cu, pos, *own))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_a_stream_handle_of_its_own():
    dv = _dev()
    x, kc, vc, st = _stack_inputs(95)
    cu, pos = R.cu_of([40, 0, 1, 49], "cuda"), _i32(3, 0, 100, 9)
    want = dv.prompt_attention(x["q"], kc, vc, cu, cache_pos=pos)
    wd = dv.delta_prompt(x["k"], x["v"], x["q"], x["g"], x["beta"], cu, state=st)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = dv.prompt_attention(x["q"], kc, vc, cu, cache_pos=pos, stream=s.cuda_stream)
    d = dv.delta_prompt(x["k"], x["v"], x["q"], x["g"], x["beta"], cu, state=st, stream=s.cuda_stream)
    s.synchronize()
    # bit by bit: with keys that are not normalized a row multiplies the state by
    # 1 - beta |k|^2, some -60, so 49 of them pass fp32's range and leave NaN in both
    assert torch.equal(a, want) and torch.equal(d.view(torch.int16), wd.view(torch.int16))


def test_one_graph_of_all_with_other_lengths_at_each_replay():
    """Lengths, positions and rows live on the device: a captured pass serves other
    batches of the same buffers."""
    dv = _dev()
    x, kc, vc, st = _stack_inputs(99)
    cu, pos = R.cu_of([40, 0, 1, 49], "cuda"), _i32(3, 0, 100, 9)
    own = [t.clone() for t in (kc, vc, st)]
    _stack(dv, x, cu, pos, *own)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = _stack(dv, x, cu, pos, *own)
    for lens, p in (([40, 0, 1, 49], (3, 0, 100, 9)), ([1, 1, 1, 1], (7, 127, 0, 63)), ([0, 90, 0, 0], (0, 38, 5, 5)),
                    ([17, 33, 16, 24], (0, 1, 2, 3))):
        cu.copy_(R.cu_of(lens, "cuda"))
        pos.copy_(_i32(*p))
        for t, u in zip(own, (kc, vc, st)):
            t.copy_(u)
        for t in got[:4]:
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        fresh = [t.clone() for t in (kc, vc, st)]
        want = _stack(dv, x, cu.clone(), pos.clone(), *fresh)
        T = sum(lens)
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a[:T], b[:T]) and not a[T:].any()
        assert all(torch.equal(a, b) for a, b in zip(own, fresh))


@pytest.mark.parametrize("own", [True, False], ids=["stream", "default"])
def test_an_output_belongs_to_the_stream_that_writes_it(own):
    """Memory freed on the stream that is current must not come back as the output of
    a call on another stream while the first still writes it."""
    dv = _dev()
    x, kc, vc, _ = _stack_inputs(96)
    cu, pos = R.cu_of([40, 0, 1, 49], "cuda"), _i32(3, 0, 100, 9)
    want = dv.prompt_attention(x["q"], kc, vc, cu, cache_pos=pos)
    side, s = torch.cuda.Stream(), torch.cuda.Stream() if own else torch.cuda.default_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy = torch.empty(1 << 28, device="cuda")
        for _ in range(20):
            busy.fill_(1.0)
        late = torch.empty_like(want)
        late.fill_(7.0)                    # behind the busy work
        at = late.data_ptr()
        del late
        out = dv.prompt_attention(x["q"], kc, vc, cu, cache_pos=pos, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert out.data_ptr() != at and torch.equal(out, want)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 96)])
@pytest.mark.parametrize("how", ["apart", "inplace", "no_state", "not_kept"])
def test_more_states_than_warps(dk, dv, how):
    """A warp takes several (sequence, head, columns) in turn, with empty and skipped
    sequences among them."""
    n = 44
    lens = [(3 * i) % 4 for i in range(n)]
    slots = [(7 * i) % 50 for i in range(n)]
    slots[5], slots[9], slots[20], slots[43] = -1, slots[8], 50, slots[0]
    skipped = (5, 9, 20, 43)
    if how == "no_state":
        slots, skipped = None, ()
    c = _case(4, 8, dk, dv, lens, dk + dv + 7, slots=slots, nslots=50 if slots else None, extra=2)
    out, so = _run("step", c, state=how != "no_state", inplace=how == "inplace",
                   keep=how not in ("not_kept", "no_state"))
    if how != "inplace":
        _check(c, out, so, state=how != "no_state", skipped=skipped)
        return
    # in place: the same, and what no sequence owns as it was
    want, apart = _run("step", c)
    assert torch.equal(out, want)
    own = [slots[i] for i in range(n) if i not in skipped]
    assert torch.equal(so[own], apart[own])
    rest = [i for i in range(50) if i not in own]
    assert torch.equal(so[rest], c["S"][rest])


@pytest.mark.parametrize("T", [700, 1450])
@pytest.mark.parametrize("H,Hk,d,x_dtype", [(9, 3, 192, BF), (4, 1, 64, torch.float32)])
def test_rows_by_two_and_four_warps(T, H, Hk, d, x_dtype):
    from tests import test_gpu_prompt_rows as P
    c = P._case(H, Hk, d, [T - 301, 0, 300, 1], [5, 2, 0, 9], T, x_dtype, 0.25, T)
    P._check(c, P._run(c))
