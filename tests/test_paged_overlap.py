"""Received weights that are written beside those that are read: refused where they share
memory, against a look at every element.  No call here reaches a GPU: what is not refused for
the weights is refused for the table of pages after them."""
import random

import pytest
import torch

from qwen3_gated_attention_gb300 import device, gattn
from tests.test_paged_args import P, _evict, _weights


@pytest.fixture(scope="module", autouse=True)
def built():
    from qwen3_gated_attention_gb300 import build
    build.build()


FAR = 1 << 40


def _evict_says(base, n, Hk, width, seq, head, out, out_width, out_seq, out_head):
    """What refuses the eviction, base and out in elements."""
    with pytest.raises(gattn.GattnError) as e:
        gattn.paged_evict(_evict(num_seqs=n, num_kv_heads=Hk, kp_stride_head=64, kp_stride_token=64 * Hk, kp_stride_page=1024 * Hk,
                                 vp_stride_head=64, vp_stride_token=64 * Hk, vp_stride_page=1024 * Hk, keep=1, recent=0,
                                 lengths_out=FAR, kept=2 * FAR, weights=P + 4 * base, weights_width=width, w_stride_seq=seq,
                                 w_stride_head=head, weights_out=P + 4 * out, weights_out_width=out_width,
                                 wo_stride_seq=out_seq, wo_stride_head=out_head, out_table=3 * FAR, out_table_width=0,
                                 out_table_stride=2))
    assert e.value.status == 1
    return str(e.value)


def _elements(at, n, Hk, width, seq, head):
    return {at + s * seq + h * head + i for s in range(n) for h in range(Hk) for i in range(width)}


def _apart(n, Hk, width, seq, head):
    return len(_elements(0, n, Hk, width, seq, head)) == n * Hk * width


@pytest.mark.parametrize("seed", range(8))
def test_eviction_refuses_what_shares_memory(seed):
    r = random.Random(seed)
    seen = {True: 0, False: 0}
    while min(seen.values()) < 40:
        n, Hk, width, out_width = r.randint(1, 4), r.randint(1, 4), r.randint(1, 6), r.randint(1, 6)
        steps = lambda w: (w + r.randint(0, 9), (w + 9) * Hk + r.randint(0, 20))      # noqa: E731
        head, seq = steps(width)
        if r.random() < 0.3:
            seq, head = width + r.randint(0, 5), (width + 6) * n + r.randint(0, 9)      # heads outside
        if r.random() < 0.5:
            out_seq, out_head = seq, head
        else:
            out_head, out_seq = steps(out_width)
        if r.random() < 0.1:
            head = 0                                # read twice
        out, base = r.randint(0, 120), r.randint(0, 120)
        # the nested order that written rows have to have
        a = sorted((s, k) for s, k in ((out_seq, n), (out_head, Hk)) if k > 1)
        span, nested = out_width, True
        for s, k in a:
            nested, span = nested and s >= span, span + (k - 1) * s
        if not nested:
            continue
        assert _apart(n, Hk, out_width, out_seq, out_head)
        same = out == base and (n == 1 or seq == out_seq) and (Hk == 1 or head == out_head)
        meet = not same and bool(_elements(base, n, Hk, width, seq, head) & _elements(out, n, Hk, out_width, out_seq, out_head))
        said = _evict_says(base, n, Hk, width, seq, head, out, out_width, out_seq, out_head)
        assert ("weights" in said) == meet, (said, n, Hk, width, seq, head, out, out_width, out_seq, out_head, base)
        assert meet or "out_table_width" in said
        seen[meet] += 1


def test_halves_of_one_buffer_are_taken_and_many_rows_are_quick():
    # [seqs][2][heads][positions] and [seqs][heads][2][positions], read from one half
    for seq, head, out in ((2 * 8 * 512, 512, 8 * 512), (8 * 1024, 1024, 512)):
        assert "out_table_width" in _evict_says(0, 4096, 8, 512, seq, head, out, 512, seq, head)
        assert "overlaps" in _evict_says(0, 4096, 8, 512, seq, head, out - 1, 512, seq, head)
        assert "overlaps" in _evict_says(0, 4096, 8, 513, seq, head, out, 512, seq, head)
    assert "too large" in _evict_says(0, 2, 2, 16, 1 << 61, 16, 64, 16, 64, 32)


def test_weights_refuse_what_shares_memory():
    for kw in (dict(weights=P + 4, weights_out=P), dict(weights=P, weights_out=P + 4), dict(weights=P, weights_out=P + 4 * 31),
               dict(weights=P, weights_out=P + 4 * 32), dict(weights=P, weights_out=P + 4 * 100)):
        with pytest.raises(gattn.GattnError, match="overlaps") as e:
            gattn.paged_weights(_weights(total_rows=0, num_seqs=3, **kw))
        assert e.value.status == 1
    gattn.paged_weights(_weights(total_rows=0, num_seqs=3, weights=P, weights_out=P + 4 * 192))
    gattn.paged_weights(_weights(total_rows=0, num_seqs=3, weights=P, weights_out=P + 4 * 64, w_stride_seq=128))
    gattn.paged_weights(_weights(total_rows=0, num_seqs=3, weights=P, weights_out=P))
    gattn.paged_weights(_weights(total_rows=0, num_seqs=3, weights=0, weights_out=P))
