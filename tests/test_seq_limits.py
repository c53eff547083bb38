"""Limits of the packed-sequence entry points, without a GPU: what the descriptors must
not say about memory and sizes."""
import pytest

from qwen3_gated_attention_gb300 import gattn
from tests.test_seq_args import P, _attn, _rows


@pytest.fixture(scope="module", autouse=True)
def built():
    from qwen3_gated_attention_gb300 import build
    build.build()


def _refuses(fn, desc, status, word):
    with pytest.raises(gattn.GattnError) as e:
        fn(desc)
    assert e.value.status == status and word in gattn.last_error(), gattn.last_error()


@pytest.mark.parametrize("which", ["kc", "vc"])
@pytest.mark.parametrize("strides,fine", [
    # token, head, batch of a cache [3][2][16][64]
    ((64, 1024, 2048), True), ((64, 1024, 2040), False), ((64, 1024, 8), False), ((64, 1024, 512), False),
    ((128, 64, 2048), True), ((128, 64, 1024), False),
    # the slots inside a token: [16][3][2][64], then the heads outside: [2][16][3][64]
    ((384, 64, 128), True), ((384, 64, 64), False), ((376, 64, 128), False), ((192, 3136, 64), True),
    ((192, 2048, 64), False), ((192, 3136, 56), False),
])
def test_cache_slots_that_share_memory(which, strides, fine):
    """Two sequences that append to one place would be a race."""
    kw = dict(cache_batch=3)
    for c in ("kc", "vc"):
        use = strides if c == which else (64, 1024, 2048)
        kw.update({f"{c}_stride_{n}": s for n, s in zip(("token", "head", "batch"), use)})
    if fine:
        gattn.prompt_rows(_rows(**kw))
    else:
        _refuses(gattn.prompt_rows, _rows(**kw), 1, "overlap")


def test_one_slot_needs_no_batch_stride():
    gattn.prompt_rows(_rows(kc_stride_batch=8, vc_stride_batch=8))


def test_more_key_rows_than_there_can_be():
    gattn.prompt_attention(_attn(kv_rows=1 << 30))
    _refuses(gattn.prompt_attention, _attn(kv_rows=(1 << 30) + 1), 1, "too large")


def test_no_keys():
    """Null keys and values with kv_rows 0: a tensor without keys."""
    none = dict(k=None, v=None, kv_rows=0)
    gattn.prompt_attention(_attn(**none))
    gattn.prompt_attention(_attn(cache_pos=P, kv_batch=2, **none))
    for change in (dict(k=P), dict(v=P), dict(kv_rows=8), dict(kv_rows=-1)):
        _refuses(gattn.prompt_attention, _attn(**{**none, **change}), 1, "")
