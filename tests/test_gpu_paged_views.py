"""Eviction through views: weights and pages in place, narrower than what they are views of."""
import pytest
import torch

from tests.test_gpu_paged_evict import _check_evict, _dev, _evict_case, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _evict(c, recent, weights_out, out_table=None):
    """weights_out and out_table are made from the weights and the table on the GPU."""
    x = {k: c[k].cuda() for k in ("kp", "vp", "table", "out", "w")}
    wo = weights_out(x["w"])
    to = x["out"] if out_table == "others" else None if out_table is None else out_table(x["table"])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, lens = _dev().paged_evict(x["kp"], x["vp"], x["table"], _i32(c["lengths"]), x["w"], keep=c["keep"], recent=recent,
                                    out_table=to, weights_out=wo, status=st)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in dict(kept=kept, lens=lens, kp=x["kp"], vp=x["vp"], w=wo, status=st, all=x["w"]).items()}


@pytest.mark.parametrize("into_pages", [True, False])
@pytest.mark.parametrize("n,Hk", [(1, 1), (1, 3), (3, 1), (2, 2)])
def test_weights_in_place_through_a_narrower_view(n, Hk, into_pages):
    c = _evict_case(Hk, 64, 16, [300, 77, 130][:n], 100, seed=10 * n + Hk)
    got = _evict(c, 20, lambda w: w[:, :, :100], "others" if into_pages else None)
    assert int(got["status"]) == 0
    _check_evict(c, 20, got, into_pages)
    assert torch.equal(got["all"][:, :, 100:], c["w"][:, :, 100:])


@pytest.mark.parametrize("n", [1, 2])
def test_pages_in_place_through_a_narrower_table(n):
    """out_table as a view of the table: in place, and as wide as the view is."""
    c = _evict_case(2, 64, 16, [300, 77][:n], 100, seed=20 + n)
    weights = lambda w: torch.zeros(n, 2, 100, device="cuda")      # noqa: E731
    for width in (c["table"].shape[1], 7):
        got = _evict(c, 20, weights, lambda t: t[:, :width])
        assert int(got["status"]) == 0
        _check_evict(c, 20, got, False)
    # 6 pages hold 96 positions: the first sequence would keep 100, the other one has fewer
    got = _evict(c, 20, weights, lambda t: t[:, :6])
    assert int(got["status"]) == 1
    _check_evict(c, 20, got, False, skipped=(0,))


def test_pages_in_place_through_a_wider_table():
    c = _evict_case(2, 64, 16, [100], 40, seed=23)
    x = {k: c[k].cuda() for k in ("kp", "vp", "w")}
    wide = torch.cat((c["table"], torch.full((1, 5), 1 << 30, dtype=torch.int32)), 1).cuda()
    wo = torch.zeros(1, 2, 40, device="cuda")
    kept, lens = _dev().paged_evict(x["kp"], x["vp"], wide[:, :c["table"].shape[1]], _i32([100]), x["w"], keep=40, recent=8,
                                    out_table=wide, weights_out=wo)
    got = {k: v.cpu() for k, v in dict(kept=kept, lens=lens, kp=x["kp"], vp=x["vp"], w=wo).items()}
    _check_evict(c, 8, got, False)


@pytest.mark.parametrize("into_pages", [True, False])
def test_weights_between_those_that_are_read(into_pages):
    """Read from one half of each row of a buffer, written to the other."""
    c = _evict_case(3, 64, 16, [300, 77], 100, seed=31)
    x = {k: c[k].cuda() for k in ("kp", "vp", "table", "out")}
    both = torch.full((2, 3, 2, 300), 7.0, device="cuda")
    both[:, :, 0] = c["w"].cuda()
    kept, lens = _dev().paged_evict(x["kp"], x["vp"], x["table"], _i32(c["lengths"]), both[:, :, 0], keep=100, recent=20,
                                    out_table=x["out"] if into_pages else None, weights_out=both[:, :, 1, :100])
    got = {k: v.cpu() for k, v in dict(kept=kept, lens=lens, kp=x["kp"], vp=x["vp"], w=both[:, :, 1]).items()}
    _check_evict(c, 20, got, into_pages)
    assert torch.equal(both[:, :, 0].cpu(), c["w"]) and bool((both[:, :, 1, 100:] == 7).all())


def test_received_weights_between_those_that_are_read():
    from tests.test_gpu_paged_evict import _run_weights, _weights_case
    c = _weights_case(8, 2, 64, 16, [2, 1], [40, 90], seed=32)
    want = _run_weights(c)
    both = torch.full((2, 2, 2, c["w"].shape[2]), 7.0, device="cuda")
    both[:, :, 1] = c["w"].cuda()
    assert torch.equal(_run_weights(c, w=both[:, :, 1], out=both[:, :, 0]), want)
    assert torch.equal(both[:, :, 1].cpu(), c["w"])
