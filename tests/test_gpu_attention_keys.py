"""gattn_prompt_attention over keys that are not there."""
import pytest
import torch

from tests.seq_refs import cu_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from qwen3_gated_attention_gb300 import build
    build.build()


def _attn(*a, **k):
    from qwen3_gated_attention_gb300 import device
    return device.prompt_attention(*a, **k)


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("kw,bit", [(dict(), 1), (dict(cu_kv=(0, 0, 0)), 0), (dict(cu_kv=(0, 1, 1)), 1),
                                    (dict(cache_pos=(0, 0)), 1), (dict(cache_pos=(0, 0), slots=(1, 0)), 1)])
def test_a_tensor_without_keys_holds_none(kw, bit):
    """Rows that ask for keys of an empty tensor are skipped and reported, rows that ask
    for none are zero; rows of no sequence stay."""
    q = torch.ones(4, 2, 64, device="cuda", dtype=BF)
    shape = (2, 1, 0, 64) if "cache_pos" in kw else (0, 1, 64)
    kv = torch.empty(*shape, device="cuda", dtype=BF)
    kw = {key: _i32(*x) for key, x in kw.items()}
    status = _i32(0)
    out = torch.full_like(q, 7.0)
    _attn(q, kv, kv, cu_of([1, 2], "cuda"), out=out, status=status, **kw)
    assert (out[:3] == 0).all() and (out[3:] == 7).all() and int(status) == bit
