"""gattn_delta_prompt and gattn_delta_step over the whole range of the rule: keys of any
size, rows that stretch the state, states and values of very different sizes, answers
that are small differences.  Both forms are held to the same bounds."""
import pytest
import torch

from tests.delta_walk import hold_to_rule, walk
from tests.seq_refs import U_BF16, cu_of
from tests.test_gpu_delta import _fn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BOTH = pytest.mark.parametrize("name", ["prompt", "step"])
# 32, 64 and 128 state columns of a CTA: one sequence, and ten of eight heads
SHAPES = [(1, 2, 64, 32, 1), (4, 8, 64, 64, 10), (4, 8, 128, 128, 10), (1, 2, 128, 96, 1)]
SHAPE = pytest.mark.parametrize("Hk,Hv,dk,dv,n", SHAPES)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _inputs(Hk, Hv, dk, dv, n, rows, seed, decay=0.1):
    """n sequences of `rows` rows; keys and queries of unit length but for their rounding."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    T = n * rows
    norm = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    return dict(q=norm(r(T, Hk, dk)).to(BF), k=norm(r(T, Hk, dk)).to(BF), v=r(T, Hv, dv).to(BF),
                g=-decay * torch.rand(T, Hv, generator=g), beta=torch.sigmoid(r(T, Hv)),
                S=0.3 * r(n, Hv, dk, dv), rows=rows, n=n)


def _hold(name, x, scale=1.0, eps=None, state=True, bounded=True, only=None):
    """Runs a form on the inputs and holds every sequence (or the ones in `only`)."""
    dev = {key: t.cuda() for key, t in x.items() if isinstance(t, torch.Tensor)}
    so = torch.full_like(dev["S"], 9.0)
    out = _fn(name)(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], cu_of([x["rows"]] * x["n"], "cuda"),
                    state=dev["S"] if state else None, state_out=so, scale=scale, qk_l2norm=eps is not None,
                    l2_eps=eps or 0.0)
    torch.cuda.synchronize()
    out, so = out.cpu(), so.cpu()
    for s in range(x["n"]) if only is None else only:
        a = slice(s * x["rows"], (s + 1) * x["rows"])
        S0 = x["S"][s] if state else torch.zeros_like(x["S"][s])
        hold_to_rule([x[key][a] for key in ("q", "k", "v", "g", "beta")] + [S0], out[a], so[s], scale, eps, bounded)


# ------------------------------------------------------------------ key scales

@BOTH
@SHAPE
@pytest.mark.parametrize("e", [-27, -13, 10, 30])
def test_keys_of_any_size(name, Hk, Hv, dk, dv, n, e):
    """Keys of length 2^e with strengths of 4^-e: the state is 2^-e times the one of unit
    keys, and nothing else changes."""
    x = _inputs(Hk, Hv, dk, dv, n, 70, 1 + e + dv)
    x["k"] = (x["k"].float() * 2.0 ** e).to(BF)
    x["beta"], x["S"] = x["beta"] * 4.0 ** -e, x["S"] * 2.0 ** -e
    _hold(name, x, 2.0 ** e, only=(0, n - 1))


@BOTH
def test_rows_of_different_key_sizes(name):
    x = _inputs(1, 2, 128, 64, 1, 70, 2)
    f = torch.exp2((torch.arange(70) * 5 % 13 - 6).float())[:, None]
    x["k"] = (x["k"].float() * f[..., None]).to(BF)
    x["beta"] = x["beta"] / f ** 2
    _hold(name, x)


@BOTH
def test_large_keys_and_queries(name):
    """One row from a zero state: q.k of 4.6e7 times a write of 2^-20."""
    x = _inputs(1, 2, 128, 32, 1, 1, 3)
    for key in ("q", "k"):
        x[key] = torch.full_like(x[key], 600.0)
    x["beta"] = torch.full_like(x["beta"], 2.0 ** -26)
    _hold(name, x, state=False)


@BOTH
@pytest.mark.parametrize("state", [True, False], ids=["state", "zeros"])
def test_normalized_keys_far_below_epsilon(name, state):
    """Keys and queries of 2^-90, divided by the root of an epsilon of 1e-6."""
    x = _inputs(1, 2, 64, 32, 1, 40, 14)
    for key in ("q", "k"):
        x[key] = (x[key].float() * 2.0 ** -90).to(BF)
    _hold(name, x, eps=1e-6, state=state)


# ------------------------------ rows that stretch the state

@BOTH
@SHAPE
@pytest.mark.parametrize("size,beta,rows", [(128.0, 0.5, 10), (128.0, 0.5, 20), (32.0, 0.5, 33), (4.0, 0.9, 70)])
def test_rows_that_stretch_the_state(name, Hk, Hv, dk, dv, n, size, beta, rows):
    """Keys that nobody normalized: a row multiplies the state along its key by
    1 - beta |k|^2.  It grows by orders of magnitude and stays a number of fp32."""
    x = _inputs(Hk, Hv, dk, dv, n, rows, int(size) + rows)
    x["k"] = (x["k"].float() * size ** 0.5).to(BF)
    x["beta"][:] = beta
    _hold(name, x, bounded=False, only=(0, n - 1))


@BOTH
def test_one_key_again_and_again_that_stretches_the_state(name):
    x = _inputs(1, 2, 128, 64, 1, 40, 4, decay=0.0)
    x["k"] = (2 * x["k"][:1].float()).to(BF).expand(40, 1, 128).contiguous()
    x["beta"][:] = 0.9
    _hold(name, x, bounded=False)


@BOTH
def test_one_row_that_stretches_the_state_by_a_million(name):
    x = _inputs(1, 2, 64, 32, 1, 50, 5)
    x["k"][21] = (x["k"][21].float() * 1000).to(BF)
    _hold(name, x, bounded=False)


@BOTH
@SHAPE
def test_states_that_grow_by_their_decay(name, Hk, Hv, dk, dv, n):
    """A positive g is a growth: the state passes 2^40 and is a state like any other."""
    x = _inputs(Hk, Hv, dk, dv, n, 40, 6)
    x["g"] = x["g"] + 0.75
    x["g"][7, 0] = 5.0
    _hold(name, x, bounded=False, only=(0, n - 1))


# ------------------------------------------- states and values of different sizes

@BOTH
@SHAPE
@pytest.mark.parametrize("size", [1e4, 1e6, 1e8])
@pytest.mark.parametrize("how", ["reset", "strong", "steady", "last"])
def test_small_values_after_a_large_state(name, Hk, Hv, dk, dv, n, size, how):
    """What is written after the state has decayed is as exact as if it had been small."""
    x = _inputs(Hk, Hv, dk, dv, n, 75, 7)
    x["S"] = x["S"] * size
    for s in range(n):
        r = s * 75
        if how == "reset":
            x["g"][r + 13] = -float("inf")
        elif how == "strong":
            x["g"][r + 5] = -25.0
            x["g"][r + 40] = -8.0
        elif how == "steady":
            x["g"][r:r + 75] = -1.0
        else:
            x["g"][r + 31] = -1e9
    _hold(name, x, only=(0, n - 1))


@BOTH
@SHAPE
@pytest.mark.parametrize("state", [True, False], ids=["state", "zeros"])
@pytest.mark.parametrize("up", [True, False], ids=["up", "down"])
def test_values_whose_size_jumps(name, Hk, Hv, dk, dv, n, state, up):
    """Rows of 1e-6 and rows of 1e6 in one chunk, with a state that forgets."""
    x = _inputs(Hk, Hv, dk, dv, n, 75, 8)
    for s in range(n):
        r = s * 75
        for a, b in ((0, 9), (20, 45), (50, 75)):
            x["v"][r + a:r + b] = (x["v"][r + a:r + b].float() * (1e-6 if up else 1e6)).to(BF)
        x["g"][r:r + 75:10] = -40.0
    _hold(name, x, state=state, only=(0, n - 1))


@BOTH
@SHAPE
@pytest.mark.parametrize("size", [1e-30, 1e20, 1e30, 1e36])
def test_states_of_any_size(name, Hk, Hv, dk, dv, n, size):
    x = _inputs(Hk, Hv, dk, dv, n, 40, 9)
    x["S"] = x["S"] * size
    x["g"][:] = -0.5
    _hold(name, x, only=(0, n - 1))


@BOTH
def test_states_that_nothing_is_written_to(name):
    """Values of zero under a decay: the state fades out row by row."""
    x = _inputs(1, 2, 64, 32, 1, 100, 10)
    x["v"].zero_()
    x["g"][:] = -0.7
    _hold(name, x)
    x["beta"].zero_()
    _hold(name, x)


@BOTH
def test_a_state_that_was_wiped_out_takes_small_values(name):
    """After a reset to exactly zero the next chunks' values are far below the old state."""
    x = _inputs(1, 2, 64, 32, 1, 140, 11)
    x["S"] = x["S"] * 1e12
    x["g"][31] = -float("inf")
    x["v"][:64] = 0
    _hold(name, x)


@BOTH
@SHAPE
@pytest.mark.parametrize("cols", [1, 16])
@pytest.mark.parametrize("size", [1e-8, 0.0])
def test_columns_that_wake_up(name, Hk, Hv, dk, dv, n, cols, size):
    """Columns without a state or values for 32 rows, then with values, then with hardly
    any: what they hold by then is theirs."""
    x = _inputs(Hk, Hv, dk, dv, n, 100, 15)
    x["g"][:] = -0.5
    for s in range(n):
        r = s * 100
        x["v"][r:r + 32, :, :cols] = 0
        x["v"][r + 64:r + 100] = (x["v"][r + 64:r + 100].float() * size).to(BF)
    _hold(name, x, state=False, only=(0, n - 1))


@pytest.mark.parametrize("seed", range(36))
def test_sizes_of_every_kind_at_once(seed):
    """Rows, columns, states and keys of sizes far apart, resets, rows without a value or a
    strength, in any mixture: the prompt form is as exact as the step is, up to 2^-24 of
    the largest that a column held or was written within the same 32 rows."""
    pick = torch.Generator().manual_seed(seed)
    draw = lambda *x: x[int(torch.randint(len(x), (1,), generator=pick))]  # noqa: E731
    yes = lambda: draw(0, 0, 1)                                            # noqa: E731
    Hk, Hv, dk, dv, n = draw(*SHAPES, (4, 8, 64, 128, 10))
    rows = int(torch.randint(1, 110, (1,), generator=pick))
    x = _inputs(Hk, Hv, dk, dv, n, rows, 100 + seed, decay=draw(0.0, 0.01, 0.1, 0.5, 2.0, 8.0))
    T = n * rows
    two = lambda e, *s: torch.exp2(torch.randint(-e, e + 1, s, generator=pick).float())  # noqa: E731
    some = lambda p, *s: torch.rand(*s, generator=pick) < p                # noqa: E731
    eps = draw(None, 1e-6)
    if yes():
        x["v"] = (x["v"].float() * two(draw(2, 6, 14), T, 1, 1)).to(BF)
    if yes():
        f = two(draw(2, 10, 20), dv)
        x["v"], x["S"] = (x["v"].float() * f).to(BF), x["S"] * f
    if yes():
        x["v"] = (x["v"].float() * two(12, dv)).to(BF)
    if yes():
        x["S"] = x["S"] * two(30, 1)
    if yes():
        x["g"][some(draw(0.02, 0.2), T, Hv)] = -draw(3.0, 10.0, 30.0, 1e5)
    if yes():
        x["beta"][some(0.5, T, Hv)] = 0
    if yes():
        x["v"][some(0.5, T)] = 0
    if yes():
        x["v"][:, :, -8:], x["S"][..., -8:] = 0, draw(0.0, 1.0)
    if yes():
        f = two(4, T, 1, 1)
        x["k"], x["beta"], eps = (x["k"].float() * f).to(BF), x["beta"] / f[:, :, 0] ** 2, None
    if yes():
        x["q"] = x["k"].clone()
    state = draw(True, True, False)
    for name in ("prompt", "step"):
        dev = {key: t.cuda() for key, t in x.items() if isinstance(t, torch.Tensor)}
        so = torch.full_like(dev["S"], 9.0)
        out = _fn(name)(dev["q"], dev["k"], dev["v"], dev["g"], dev["beta"], cu_of([rows] * n, "cuda"),
                        state=dev["S"] if state else None, state_out=so, scale=1.0, qk_l2norm=eps is not None,
                        l2_eps=eps or 0.0).cpu()
        for s in {0, n - 1}:
            a = slice(s * rows, (s + 1) * rows)
            S0 = x["S"][s] if state else torch.zeros_like(x["S"][s])
            want, last, eo, es = walk(*(x[key][a] for key in ("q", "k", "v", "g", "beta")), S0, 1.0, eps,
                                      chunk=32 if name == "prompt" else 0)
            tol = U_BF16 * want.abs() + (1 + U_BF16) * eo + 1e-37
            assert ((out[a].double() - want).abs() <= tol).all(), (name, s)
            assert ((so[s].cpu().double() - last).abs() <= es + 1e-37).all(), (name, s)


# --------------------------------------------- answers that are small differences

@BOTH
@SHAPE
@pytest.mark.parametrize("size", [10.0, 1e3, 1e5])
def test_answers_that_are_small_differences(name, Hk, Hv, dk, dv, n, size):
    """The query is the key of a row that overwrites: its answer is the value, and what
    the state held along that key cancels."""
    x = _inputs(Hk, Hv, dk, dv, n, 70, 12, decay=0.0)
    x["q"] = x["k"].clone()
    x["beta"][:] = 1.0
    x["S"] = x["S"] * size
    _hold(name, x, eps=0.0, only=(0, n - 1))


@BOTH
@SHAPE
@pytest.mark.parametrize("rows", [1, 31, 32, 33, 70, 129, 200])
def test_every_length_to_fp32(name, Hk, Hv, dk, dv, n, rows):
    x = _inputs(Hk, Hv, dk, dv, n, rows, 13 + rows)
    _hold(name, x, dk ** -0.5, 1e-6, only=(0, n - 1))
    _hold(name, x, dk ** -0.5, 1e-6, state=False, only=(0,))
