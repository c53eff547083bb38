"""gattn_paged_attention_workspace: what it refuses, and how long an answer holds."""
import pytest

from qwen3_gated_attention_gb300 import gattn
from tests.test_paged_args import _attn


@pytest.fixture(scope="module", autouse=True)
def built():
    from qwen3_gated_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("H,Hk,d,n,T", [(2048, 2, 64, 1, 8), (1026, 2, 64, 1, 8), (512, 2, 192, 1, 8), (4, 2, 64, 1, 1 << 29),
                                        (1024, 2, 64, 1, 1 << 21)])
def test_shapes_that_the_attention_refuses(H, Hk, d, n, T):
    with pytest.raises(gattn.GattnError):
        gattn.paged_attention_workspace(H, Hk, d, n, T)
    assert gattn.lib().gattn_paged_attention_workspace(H, Hk, d, n, T) == -1
    # the call refuses them too: all else is right, and there are no sequences
    with pytest.raises(gattn.GattnError) as e:
        gattn.paged_attention(_attn(num_heads=H, num_kv_heads=Hk, head_dim=d, total_rows=T, kp_stride_token=256, kp_stride_head=4096,
                                    vp_stride_token=256, vp_stride_head=4096, q_stride_head=256, q_stride_token=1 << 20,
                                    o_stride_head=256, o_stride_token=1 << 20))
    assert e.value.status == 2


def test_shapes_at_the_limits():
    for H, Hk, d, n, T in [(1024, 2, 64, 1, 8), (256, 4, 256, 1, 8), (1024, 1, 64, 1, (1 << 21) - 1), (1, 1, 64, 1, 1 << 30)]:
        assert gattn.paged_attention_workspace(H, Hk, d, n, T) > 0


@pytest.mark.parametrize("H,Hk,d", [(16, 2, 256), (16, 4, 256), (8, 8, 64), (24, 2, 256), (5, 1, 128), (64, 1, 192)])
def test_a_size_holds_for_smaller_calls(H, Hk, d):
    """Sequences leave, rows are fewer: what was enough stays enough."""
    size = lambda n, t: gattn.paged_attention_workspace(H, Hk, d, n, t)      # noqa: E731
    for n, t in [(64, 64), (64, 256), (7, 9), (3, 3), (1, 1), (2, 2), (1, 4), (100, 0)]:
        most = size(n, t)
        for m in range(1, n + 1):
            for r in {1, t // 3, t - 1, t, min(m, t)}:
                if 0 <= r <= t:
                    assert size(m, r) <= most, (n, t, m, r)
                    # and the call itself asks for no more (none is refused, with its need)
                    if r:
                        with pytest.raises(gattn.GattnError) as e:
                            gattn.paged_attention(_attn(num_heads=H, num_kv_heads=Hk, head_dim=d, num_seqs=m, total_rows=r,
                                                        q_stride_head=256, q_stride_token=1 << 15, o_stride_head=256,
                                                        o_stride_token=1 << 15, workspace_bytes=0))
                        assert int(str(e.value).split("bytes: ")[1].split()[0]) <= most
