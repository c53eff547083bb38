"""Infinities and NaN in places that the paged-cache operators say do not count."""
import math

import pytest
import torch

from tests.paged_refs import BF, score_error
from tests.test_gpu_paged_evict import _run_weights, _weights_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("H,Hk,d", [(8, 2, 64), (16, 4, 256), (40, 1, 128)])
def test_a_row_without_a_log_sum_gives_nothing(H, Hk, d, value):
    """lse -infinity: its keys may hold anything."""
    c = _weights_case(H, Hk, d, 16, [2, 3], [70, 33], seed=H)
    want = _run_weights(c)
    c["lse"][0:2] = -math.inf
    page, row = int(c["table"][0, 1]), 5              # position 21 of the first sequence
    c["kp"][page, :, row] = torch.full((d,), value, dtype=BF)
    got = _run_weights(c)
    assert torch.equal(got[1], want[1])
    assert torch.equal(got[0, :, :70], c["w"][0, :, :70]) and bool((got[0, :, 70:72] == 0).all())


@pytest.mark.parametrize("rd", [64, 20])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_skipped_rows_are_zero_whatever_the_norms_hold(rd, value):
    """Of gattn_paged_rows and of gattn_prompt_rows, without an epsilon."""
    from qwen3_gated_attention_gb300 import device
    g = torch.Generator().manual_seed(rd)
    q, k = (torch.randn(5, h, 64, generator=g).to(BF).cuda() for h in (4, 2))
    w = torch.full((64,), value, dtype=BF, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    cu = i32([0, 3, 5])
    pages, caches = torch.zeros(4, 2, 16, 64, dtype=BF, device="cuda"), torch.zeros(2, 2, 32, 64, dtype=BF, device="cuda")
    st = i32([0])
    out = device.paged_rows(q, k, k, pages, pages.clone(), i32([[0, 1], [2, 3]]), cu, i32([0, 31]), rope_theta=1e6, rotary_dims=rd,
                            q_norm=w, k_norm=w, rms_eps=0.0, status=st)
    assert bool((out[3:] == 0).all()) and not bool(out[:3].isfinite().any()) and int(st) == 1
    out = device.paged_rows(q, k, k, pages, pages.clone(), i32([[0, 1], [2, 3]]), cu, i32([0, 0]), rope_theta=1e6, rotary_dims=rd,
                            q_norm=w, k_norm=w, rms_eps=0.0, positions=i32([0, -1, 2, (1 << 24) + 1, 1 << 24]), status=st)
    assert bool((out[[1, 3]] == 0).all()) and not bool(out[[0, 2, 4]].isfinite().any())
    out = device.prompt_rows(q, k, k, w, w, caches, caches.clone(), cu, i32([0, 31]), partial_rotary_factor=rd / 64, rope_theta=1e6,
                             rms_eps=0.0, status=st)
    assert bool((out[3:] == 0).all()) and not bool(out[:3].isfinite().any())


@pytest.mark.parametrize("past", [0, 37, 9000])
def test_a_row_with_scores_of_minus_infinity_only(past):
    """Zeros and a log sum of -infinity, as for a row that sees nothing, whether one CTA or many
    have its positions; with one finite score beside them it is that position's value."""
    from qwen3_gated_attention_gb300 import device
    g = torch.Generator().manual_seed(past)
    H, Hk, d, P = 8, 2, 128, 16
    n = past // P + 1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")      # noqa: E731
    q = torch.randn(1, H, d, generator=g).abs().to(BF).cuda()
    kp = torch.randn(n, Hk, P, d, generator=g).to(BF).cuda()
    kp[..., 3] = -math.inf
    vp = torch.randn(n, Hk, P, d, generator=g).to(BF).cuda()
    table, lse = torch.arange(n, dtype=torch.int32, device="cuda")[None], torch.zeros(1, H, device="cuda")
    w = torch.zeros(1, Hk, past + 1, device="cuda")
    call = (table, i32([0, 1]), i32([past]))
    out = device.paged_attention(q, kp, vp, *call, lse=lse)
    device.paged_weights(q, kp, *call, lse, weights=w)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and bool((w == 0).all())
    at = past // 2
    kp[at // P, :, at % P, 3] = 1.0
    out = device.paged_attention(q, kp, vp, *call, lse=lse)
    device.paged_weights(q, kp, *call, lse, weights=w)
    assert torch.equal(out[0], vp[at // P, :, at % P].repeat_interleave(H // Hk, 0)) and bool(lse.isfinite().all())
    # each of a group's four rows gives one, up to its score's rounding here and in the log sum
    size = float((q[0].double().abs() * kp[at // P, :, at % P].double().abs().repeat_interleave(H // Hk, 0)).sum(-1).max()) * d ** -0.5
    e = 2 * score_error(d, size, 1.0, size) + 2.0 ** -20
    assert bool(((w[0, :, at] - 4).abs() <= 4 * math.expm1(e)).all()) and bool((w.sum(-1) == w[0, :, at]).all())
