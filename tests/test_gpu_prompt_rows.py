"""gattn_prompt_rows on the GPU: norm, rotary embedding and append of packed rows
against float64, over head layouts, types, strides, positions and slots."""
import pytest
import torch

from tests.seq_refs import U_BF16, cu_of, rows64

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


def _case(H, Hk, d, lens, past, cap, x_dtype, prf, seed, layout="bhtd", slots=None, B=None):
    g = torch.Generator().manual_seed(seed)
    T, n = sum(lens), len(lens)
    B = B or n
    y = torch.randn(T, 2 * H * d + 2 * Hk * d, generator=g).to(x_dtype)
    shape = (B, Hk, cap, d) if layout == "bhtd" else (B, cap, Hk, d)
    kc, vc = (torch.randn(shape, generator=g).to(BF) for _ in range(2))
    qn, kn = ((1 + 0.1 * torch.randn(d, generator=g)).to(BF) for _ in range(2))
    return dict(H=H, Hk=Hk, d=d, lens=lens, past=past, y=y, kc=kc, vc=vc, qn=qn, kn=kn, prf=prf,
                layout=layout, slots=slots)


def _split(c, y):
    T, H, Hk, d = y.shape[0], c["H"], c["Hk"], c["d"]
    q = y[:, :2 * H * d].view(T, H, 2 * d)[..., :d]
    k = y[:, 2 * H * d:2 * H * d + Hk * d].view(T, Hk, d)
    v = y[:, 2 * H * d + Hk * d:].view(T, Hk, d)
    return q, k, v


THETA, EPS = 1e7, 1e-6


def _run(c, extra_rows=0, status=None):
    y, kc, vc = c["y"].cuda(), c["kc"].cuda(), c["vc"].cuda()
    q, k, v = _split(c, y)
    kv = (kc, vc) if c["layout"] == "bhtd" else (kc.transpose(1, 2), vc.transpose(1, 2))
    out = torch.full((y.shape[0], c["H"], c["d"]), 7.0, dtype=BF, device="cuda")
    slots = None if c["slots"] is None else torch.tensor(c["slots"], dtype=torch.int32, device="cuda")
    _dev().prompt_rows(q, k, v, c["qn"].cuda(), c["kn"].cuda(), *kv, cu_of(c["lens"], "cuda"),
                       torch.tensor(c["past"], dtype=torch.int32, device="cuda"),
                       partial_rotary_factor=c["prf"], rope_theta=THETA, rms_eps=EPS, q_out=out,
                       slots=slots, status=status)
    torch.cuda.synchronize()
    return out.cpu(), kv[0].cpu(), kv[1].cpu()


def _check(c, got, skipped=()):
    out, kc, vc = got
    q, k, v = _split(c, c["y"])
    rd = int(c["d"] * c["prf"])
    kv0 = (c["kc"], c["vc"]) if c["layout"] == "bhtd" else (c["kc"].transpose(1, 2), c["vc"].transpose(1, 2))
    want_k, want_v = kv0[0].clone(), kv0[1].clone()
    touched = torch.zeros(want_k.shape[:3], dtype=torch.bool)
    r = 0
    for s, (n, p) in enumerate(zip(c["lens"], c["past"])):
        a = slice(r, r + n)
        r += n
        if s in skipped:
            assert (out[a] == 0).all()
            continue
        pos = torch.arange(p, p + n)
        b = s if c["slots"] is None else c["slots"][s]
        for got_rows, x, w in ((out[a], q[a], c["qn"]), (kc[b, :, p:p + n].transpose(0, 1), k[a], c["kn"])):
            want = rows64(x, w, pos, rd, THETA, EPS)
            # one rounding to bf16; before it the reduced angle (1e-6 rad), the
            # hardware sine and cosine (2^-21) and the fp32 norm act on the pair
            mag = rows64(x, w, pos * 0, rd, THETA, EPS).abs()
            pair = mag.clone()
            h = rd // 2
            pair[..., :h] = pair[..., h:rd] = mag[..., :h] + mag[..., h:rd]
            tol = U_BF16 * want.abs() + 4e-6 * pair + 1e-30
            assert ((got_rows.double() - want).abs() <= tol).all(), s
        assert torch.equal(vc[b, :, p:p + n].transpose(0, 1), v[a].to(BF))
        touched[b, :, p:p + n] = True
    assert (out[r:] == 7.0).all()
    # everything that was not written is as it was, bit for bit
    assert torch.equal(kc[~touched].view(torch.int16), kv0[0][~touched].view(torch.int16))
    assert torch.equal(vc[~touched].view(torch.int16), kv0[1][~touched].view(torch.int16))


@pytest.mark.parametrize("H,Hk,d", [(16, 4, 256), (24, 2, 256), (5, 1, 64), (6, 2, 192), (16, 8, 128), (3, 3, 64)])
@pytest.mark.parametrize("x_dtype", [torch.float32, BF], ids=["f32", "bf16"])
def test_rows(H, Hk, d, x_dtype):
    c = _case(H, Hk, d, [1, 17, 0, 40], [0, 100003, 5, 63], 100100 if d == 64 else 100020, x_dtype, 0.25, H * d) \
        if d <= 64 else _case(H, Hk, d, [1, 17, 0, 40], [0, 233, 5, 63], 250, x_dtype, 0.25, H * d)
    _check(c, _run(c))


@pytest.mark.parametrize("d,prf", [(64, 1.0), (64, 0.1), (128, 0.55), (192, 1.0), (256, 0.0079)])
def test_rotary_widths(d, prf):
    """Every pairing distance: rotary halves that are no multiple of a lane's share."""
    c = _case(4, 2, d, [9, 3], [1000, 0], 1100, BF, prf, d)
    assert int(d * prf) % 2 == 0
    _check(c, _run(c))


def test_token_major_cache_and_slots():
    c = _case(4, 2, 128, [5, 1, 8], [3, 0, 11], 40, BF, 0.25, 1, layout="btd", slots=[4, 0, 2], B=5)
    _check(c, _run(c))


def test_rows_behind_the_last_sequence_stay():
    c = _case(4, 2, 64, [5, 3, 6], [0, 1, 2], 16, BF, 0.25, 2)
    c["lens"], c["past"] = [5, 3], [0, 1]
    c["kc"], c["vc"] = c["kc"][:2], c["vc"][:2]
    _check(c, _run(c))


@pytest.mark.parametrize("past,slots,skipped", [
    ([0, -1, 3], None, (1,)),                 # negative position
    ([9, 0, 3], None, (0,)),                  # runs past the capacity
    ([0, 0, 0], [1, 3, 0], (1,)),             # slot past the cache
    ([0, 0, 0], [1, -1, 0], (1,)),
    ([0, 5, 0], [2, 2, 1], (1,)),             # a slot named twice
    ([2 ** 31 - 4, 0, 0], None, (0,)),
])
def test_sequences_outside_the_cache_are_skipped(past, slots, skipped):
    c = _case(4, 2, 64, [8, 2, 4], past, 16, BF, 0.5, 3, slots=slots)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check(c, _run(c, status=status), skipped)
    assert int(status) == 1


def test_skipped_rows_are_zero_without_epsilon():
    c = _case(4, 2, 64, [8, 2], [0, -3], 16, BF, 0.5, 5)
    y, kc, vc = c["y"].cuda(), c["kc"].cuda(), c["vc"].cuda()
    q, k, v = _split(c, y)
    out = _dev().prompt_rows(q, k, v, c["qn"].cuda(), c["kn"].cuda(), kc, vc, cu_of(c["lens"], "cuda"),
                             torch.tensor(c["past"], dtype=torch.int32, device="cuda"),
                             partial_rotary_factor=0.5, rope_theta=THETA, rms_eps=0.0)
    assert (out[8:] == 0).all() and out[:8].isfinite().all() and (out[:8] != 0).any()


def test_many_sequences():
    lens = [(7 * i) % 5 for i in range(1500)]
    c = _case(2, 1, 64, lens, [i % 3 for i in range(1500)], 16, BF, 0.25, 4)
    _check(c, _run(c))
