"""gattn_delta_prompt and gattn_delta_step on the GPU against the float64
recurrence: lengths around the chunks, head layouts, states in and out, slots."""
import pytest
import torch

from tests.seq_refs import U_BF16, cu_of, delta64, delta_bound

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _fn(name):
    from qwen3_gated_attention_gb300 import device
    return {"prompt": device.delta_prompt, "step": device.delta_step}[name]


def _case(Hk, Hv, dk, dv, lens, seed, slots=None, nslots=None, extra=0, fast=1.0):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens) + extra, len(lens)
    y = torch.randn(T, 2 * Hk * dk + Hv * dv, generator=g).to(BF)
    gl = -fast * torch.rand(T, Hv, generator=g) * (1 + 15 * torch.rand(Hv, generator=g)) * 0.1
    beta = torch.sigmoid(torch.randn(T, Hv, generator=g))
    S = 0.3 * torch.randn(nslots or n, Hv, dk, dv, generator=g)
    return dict(Hk=Hk, Hv=Hv, dk=dk, dv=dv, lens=lens, y=y, g=gl, beta=beta, S=S, slots=slots)


def _parts(c, y):
    T, a = y.shape[0], c["Hk"] * c["dk"]
    return (y[:, :a].view(T, c["Hk"], -1), y[:, a:2 * a].view(T, c["Hk"], -1),
            y[:, 2 * a:].view(T, c["Hv"], -1))


def _run(name, c, state=True, inplace=False, keep=True, status=None, out=None):
    y = c["y"].cuda()
    st = c["S"].cuda() if state else None
    so = None if not keep else st if inplace else torch.full(c["S"].shape, 9.0, device="cuda")
    slots = None if c["slots"] is None else torch.tensor(c["slots"], dtype=torch.int32, device="cuda")
    if out is None:
        out = torch.full((y.shape[0], c["Hv"], c["dv"]), 7.0, dtype=BF, device="cuda")
    _fn(name)(*_parts(c, y), c["g"].cuda(), c["beta"].cuda(), cu_of(c["lens"], "cuda"), state=st,
              state_out=so, slots=slots if st is not None or so is not None else None,
              qk_l2norm=True, out=out, status=status)
    torch.cuda.synchronize()
    return out.cpu(), None if so is None else so.cpu()


def _check(c, out, so, state=True, skipped=(), scale=None):
    q, k, v = _parts(c, c["y"])
    scale = scale or c["dk"] ** -0.5
    r, touched = 0, set()
    for s, n in enumerate(c["lens"]):
        a = slice(r, r + n)
        r += n
        if s in skipped:
            assert (out[a] == 0).all()
            continue
        slot = s if c["slots"] is None else c["slots"][s]
        S0 = c["S"][slot] if state else torch.zeros_like(c["S"][0])
        want, last, top = delta64(q[a], k[a], v[a], c["g"][a], c["beta"][a], S0, scale, 1e-6)
        e = delta_bound(n, top, c["dk"])
        if n:
            # out = q . S: |q| <= 1 turns a state error of e per entry into
            # sqrt(dk) e at most, the chunk's own products once more; one rounding
            tol = U_BF16 * want.abs() + scale * (c["dk"] ** 0.5 * e + 3 * 2.0 ** -16 * top + c["dk"] * 2.0 ** -24 * top)
            err = (out[a].double() - want).abs()
            assert (err <= tol).all(), (s, n, float((err - tol).max()))
        if so is not None:
            err = (so[slot].double() - last).abs()
            assert float(err.max()) <= e + 1e-30 if n else torch.equal(so[slot], S0), (s, n, float(err.max()), e)
            touched.add(slot)
    assert (out[r:] == 7.0).all()
    if so is not None:
        for slot in range(c["S"].shape[0]):
            if slot not in touched:
                assert (so[slot] == 9.0).all() or torch.equal(so[slot], c["S"][slot])


@pytest.mark.parametrize("name", ["prompt", "step"])
@pytest.mark.parametrize("Hk,Hv,dk,dv", [(2, 4, 128, 128), (1, 3, 64, 32), (2, 2, 128, 64), (1, 1, 64, 256), (1, 2, 128, 96)])
@pytest.mark.parametrize("lens", [[1], [0, 3, 70], [33, 16, 64, 5]], ids=["one", "ragged", "chunks"])
def test_rule(name, Hk, Hv, dk, dv, lens):
    c = _case(Hk, Hv, dk, dv, lens, Hv * dk + dv)
    _check(c, *_run(name, c))


@pytest.mark.parametrize("n", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200])
def test_lengths_around_the_chunks(n):
    c = _case(1, 2, 128, 128, [n], n)
    _check(c, *_run("prompt", c))


@pytest.mark.parametrize("name", ["prompt", "step"])
def test_states(name):
    """No state in, in place, not kept, permuted slots, a pass cut in two."""
    c = _case(1, 2, 64, 64, [20, 37], 1, slots=[3, 1], nslots=5)
    base, so = _run(name, c)
    _check(c, base, so)
    out, so2 = _run(name, c, inplace=True)
    assert torch.equal(out, base) and torch.equal(so2[[3, 1]], so[[3, 1]])
    assert torch.equal(so2[[0, 2, 4]], c["S"][[0, 2, 4]])
    out, _ = _run(name, c, keep=False)
    assert torch.equal(out, base)
    _check(c, *_run(name, c, state=False), state=False)
    out, _ = _run(name, dict(c, slots=None), state=False, keep=False)
    _check(dict(c, slots=None), out, None, state=False)
    # the second half from the state after the first
    y, gl, b = c["y"], c["g"], c["beta"]
    one = dict(c, lens=[20], y=y[:20], g=gl[:20], beta=b[:20], slots=[3])
    _, mid = _run(name, dict(one, lens=[13], y=y[:13], g=gl[:13], beta=b[:13]), inplace=True)
    tail, last = _run(name, dict(one, lens=[7], y=y[13:20], g=gl[13:20], beta=b[13:20], S=mid), inplace=True)
    _check(one, torch.cat((base[:13], tail)), torch.where(torch.ones(5, 1, 1, 1).bool(), last, last))


@pytest.mark.parametrize("name", ["prompt", "step"])
@pytest.mark.parametrize("slots,skipped", [([0, 3, 1], (1,)), ([0, -1, 1], (1,)), ([2, 2, 0], (1,))])
def test_bad_slots_are_skipped(name, slots, skipped):
    c = _case(1, 2, 64, 32, [4, 3, 35], 2, slots=slots, nslots=3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, so = _run(name, c, status=status)
    _check(c, out, so, skipped=skipped)
    assert int(status) == 1


@pytest.mark.parametrize("name", ["prompt", "step"])
def test_decays(name):
    """No decay, strong decay, a full reset (-inf) in the middle, weak after strong."""
    c = _case(1, 4, 64, 32, [80], 3)
    c["g"][:, 0] = 0
    c["g"][:, 1] = -20
    c["g"][40, 2] = -float("inf")
    c["g"][::7, 3] = -5000
    c["g"][1::7, 3] = -0.001
    _check(c, *_run(name, c))


@pytest.mark.parametrize("name", ["prompt", "step"])
def test_repeated_keys_and_full_writes(name):
    """One key over and over with beta = 1: each row replaces what the last wrote."""
    c = _case(1, 2, 128, 64, [70], 4, fast=0.0)
    a = c["Hk"] * c["dk"]
    c["y"][:, a:2 * a] = c["y"][:1, a:2 * a]
    c["beta"][:] = 1.0
    _check(c, *_run(name, c))


def test_without_l2norm_and_scale():
    c = _case(1, 2, 64, 64, [50], 5)
    q, k, v = _parts(c, c["y"].clone())
    k = (k.float() / k.float().norm(dim=-1, keepdim=True)).to(BF)
    k = (k.float() * 0.99).to(BF)
    want, last, top = delta64(q, k, v, c["g"], c["beta"], c["S"][0], 0.03)
    e = delta_bound(50, top, 64)
    for name in ("prompt", "step"):
        so = torch.zeros_like(c["S"]).cuda()
        out = _fn(name)(q.cuda(), k.cuda(), v.cuda(), c["g"].cuda(), c["beta"].cuda(), num_seqs=1,
                        state=c["S"].cuda(), state_out=so, scale=0.03)
        qn = float(q.float().norm(dim=-1).max())
        tol = U_BF16 * want.abs() + 0.03 * qn * (64 ** 0.5 * e + 4 * 2.0 ** -16 * top)
        assert ((out.cpu().double() - want).abs() <= tol).all()
        assert float((so.cpu()[0].double() - last).abs().max()) <= e


@pytest.mark.parametrize("name", ["prompt", "step"])
def test_rows_behind_the_last_sequence_stay(name):
    c = _case(1, 2, 64, 32, [5, 40], 6, extra=9)
    c["y"][45:] = float("nan")
    _check(c, *_run(name, c))


@pytest.mark.parametrize("name", ["prompt", "step"])
def test_foreign_rows_do_not_reach_a_sequence(name):
    """A sequence whose rows are not finite leaves its neighbours as they were."""
    c = _case(1, 2, 64, 32, [17, 6, 20], 7)
    base, so = _run(name, c)
    d = dict(c, y=c["y"].clone(), g=c["g"].clone(), beta=c["beta"].clone())
    d["y"][17:23] = float("nan")
    d["g"][17:23] = float("nan")
    d["beta"][17:23] = float("inf")
    out, s2 = _run(name, d)
    assert torch.equal(out[:17], base[:17]) and torch.equal(out[23:], base[23:])
    assert torch.equal(s2[[0, 2]], so[[0, 2]]) and out[17:23].isnan().all()


@pytest.mark.parametrize("name", ["prompt", "step"])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_before_a_spoilt_one_stay_as_they_were(name, what, bad):
    """A row that is not finite reaches the rows after it, in the columns it
    touches, and none before it."""
    c = _case(1, 2, 64, 32, [70], 10)
    base, _ = _run(name, c)
    d = dict(c, y=c["y"].clone(), g=c["g"].clone(), beta=c["beta"].clone())
    for row, col in ((41, 5), (45, 7)):
        if what in ("g", "beta"):
            d[what][row] = bad
        else:
            d["y"][row, {"q": 0, "k": 64, "v": 128}[what] + col] = bad
    out, _ = _run(name, d)
    assert torch.equal(out[:41], base[:41])
    if what == "q":                                  # its own row's answer only
        keep = [i for i in range(70) if i not in (41, 45)]
        assert torch.equal(out[keep], base[keep]) and not out[[41, 45]].isfinite().any()
    elif what == "v":
        cols = [j for j in range(32) if j not in (5, 7)]
        assert torch.allclose(out[:, :, cols].float(), base[:, :, cols].float(), rtol=2.0 ** -7, atol=2.0 ** -13)
        assert torch.equal(out[:, 1], base[:, 1])    # the other head has its own values
        assert not out[41:, 0, 5].isfinite().any() and not out[45:, 0, 7].isfinite().any()
        assert torch.allclose(out[:45, 0, 7].float(), base[:45, 0, 7].float(), rtol=2.0 ** -7, atol=2.0 ** -13)
    else:
        assert not out[45:].isfinite().any()


def test_uniform_lengths_and_graph():
    c = _case(2, 4, 128, 128, [4] * 6, 8)
    y = c["y"].cuda()
    args = (*_parts(c, y), c["g"].cuda(), c["beta"].cuda())
    st = c["S"].cuda()
    want, so = _run("step", c)
    for name in ("step", "prompt"):
        so2, out = torch.zeros_like(st), torch.zeros(24, 4, 128, dtype=BF, device="cuda")
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            _fn(name)(*args, num_seqs=6, state=st, state_out=so2, qk_l2norm=True, out=out)
        gr.replay()
        gr.replay()
        torch.cuda.synchronize()
        _check(c, out.cpu(), so2.cpu())
        if name == "step":
            assert torch.equal(out.cpu(), want) and torch.equal(so2.cpu(), so)


def test_many_sequences():
    c = _case(1, 1, 64, 32, [(3 * i) % 4 for i in range(700)], 9)
    for name in ("prompt", "step"):
        _check(c, *_run(name, c))
