"""Infinities and NaN in places that the paged-cache operators say do not count."""
import math

import pytest
import torch

from tests.paged_refs import BF
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
