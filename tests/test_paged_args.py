"""The paged-cache entry points without a GPU: every refusal the header documents, taken
before any CUDA call."""
import math

import pytest
import torch

from qwen3_gated_attention_gb300 import device, gattn


@pytest.fixture(scope="module", autouse=True)
def built():
    from qwen3_gated_attention_gb300 import build
    build.build()


P = 4096                  # a 16-byte aligned address that no refused call touches

POOL = dict(k_pages=P, v_pages=P, num_pages=4, page_size=16, kp_stride_token=64, kp_stride_head=1024,
            kp_stride_page=2048, vp_stride_token=64, vp_stride_head=1024, vp_stride_page=2048, table=P,
            table_width=2, table_stride=2)


def _fill(d, base, kw):
    for k, v in {**base, **kw}.items():
        assert hasattr(d, k), k
        setattr(d, k, v)
    return d


def _rows(**kw):
    return _fill(gattn.gattn_paged_rows_desc(), dict(
        POOL, num_heads=4, num_kv_heads=2, head_dim=64, rotary_dims=16, rope_theta=1e7, rope_factor=1.0, rms_eps=1e-6,
        x_dtype=1, num_seqs=0, total_rows=8, cu_rows=P, cache_pos=P, q=P, k=P, v=P, q_stride_token=512,
        q_stride_head=128, k_stride_token=128, k_stride_head=64, v_stride_token=128, v_stride_head=64, q_norm=P,
        k_norm=P, q_out=P, o_stride_token=256, o_stride_head=64), kw)


ATTN = dict(POOL, num_heads=4, num_kv_heads=2, head_dim=64, scale=0.125, num_seqs=0, total_rows=8, cu_rows=P, cache_pos=P,
            q=P, q_stride_token=256, q_stride_head=64, gate_dtype=1, g_stride_token=8, g_stride_head=8, out=P,
            o_stride_token=256, o_stride_head=64, workspace=P, workspace_bytes=1 << 40)


def _attn(**kw):
    return _fill(gattn.gattn_paged_attention_desc(), ATTN, kw)


def _weights(**kw):
    return _fill(gattn.gattn_paged_weights_desc(),
                 dict(ATTN, lse=P, weights=P, weights_out=P, weights_width=32, w_stride_seq=64, w_stride_head=32), kw)


def _evict(**kw):
    return _fill(gattn.gattn_paged_evict_desc(), dict(
        POOL, num_kv_heads=2, head_dim=64, num_seqs=0, keep=16, recent=4, lengths=P, lengths_out=2 * P, weights=P,
        weights_width=32, w_stride_seq=64, w_stride_head=32, weights_out=P, weights_out_width=32, wo_stride_seq=64,
        wo_stride_head=32, kept=P), kw)


CALLS = {"rows": (gattn.paged_rows, _rows), "attention": (gattn.paged_attention, _attn),
         "weights": (gattn.paged_weights, _weights), "evict": (gattn.paged_evict, _evict)}

INV, UNS = 1, 2
POOLS = [
    (dict(k_pages=0), INV), (dict(k_pages=P + 2), INV), (dict(num_pages=0), INV), (dict(num_pages=-1), INV),
    (dict(page_size=0), UNS), (dict(page_size=8), UNS), (dict(page_size=24), UNS), (dict(page_size=-16), UNS),
    (dict(table=0), INV), (dict(table=P + 2), INV), (dict(table_width=0), INV), (dict(table_stride=1), INV),
    (dict(table_width=(1 << 20) + 1, table_stride=1 << 21), UNS), (dict(kp_stride_token=0), INV),
    (dict(kp_stride_token=68), INV), (dict(kp_stride_head=-8), INV), (dict(kp_stride_page=4), INV),
    (dict(kp_stride_page=1 << 38), INV), (dict(head_dim=0), UNS), (dict(head_dim=96), UNS), (dict(head_dim=320), UNS),
    (dict(status=P + 1), INV), (dict(num_seqs=-1), INV), (dict(num_seqs=(1 << 24) + 1), INV),
]
VALUES = [(dict(v_pages=0), INV), (dict(v_pages=P + 8), INV), (dict(vp_stride_token=4), INV)]
WRITTEN = [(dict(kp_stride_token=8), INV), (dict(vp_stride_head=64), INV), (dict(kp_stride_page=1024), INV),
           (dict(vp_stride_token=1024, vp_stride_head=1024), INV)]
HEADS = [(dict(num_heads=0), INV), (dict(num_heads=5), INV), (dict(num_kv_heads=0), INV), (dict(total_rows=-1), INV),
         (dict(total_rows=(1 << 30) + 1), INV), (dict(cu_rows=0), INV), (dict(cu_rows=P + 2), INV),
         (dict(cache_pos=0), INV), (dict(cache_pos=P + 1), INV), (dict(q=0), INV), (dict(q=P + 2), INV),
         (dict(q_stride_head=4), INV), (dict(q_stride_token=0), INV)]
OWN = {
    "rows": [(dict(x_dtype=2), INV), (dict(rotary_dims=0), INV), (dict(rotary_dims=15), INV), (dict(rotary_dims=66), INV),
             (dict(rope_theta=0.0), INV), (dict(rope_theta=math.nan), INV), (dict(rope_theta=math.inf), INV),
             (dict(rms_eps=-1.0), INV), (dict(rms_eps=math.nan), INV), (dict(rope_size=-1.0), INV),
             (dict(rope_size=math.inf), INV), (dict(rope_scaling=3), INV), (dict(rope_scaling=-1), INV),
             (dict(rope_scaling=1, rope_factor=0.5), INV), (dict(rope_scaling=1, rope_factor=math.nan), INV),
             (dict(rope_scaling=2, rope_factor=2.0, rope_original=0, rope_beta_fast=32.0, rope_beta_slow=1.0), INV),
             (dict(rope_scaling=2, rope_factor=2.0, rope_original=64, rope_beta_fast=1.0, rope_beta_slow=2.0), INV),
             (dict(rope_scaling=2, rope_factor=2.0, rope_original=64, rope_beta_fast=1.0, rope_beta_slow=0.0), INV),
             (dict(rope_scaling=2, rope_factor=2.0, rope_original=64, rope_beta_fast=math.inf, rope_beta_slow=1.0), INV),
             (dict(rope_scaling=2, rope_factor=2.0, rope_original=64, rope_beta_fast=2.0, rope_beta_slow=1.0,
                   rope_theta=1.0), INV),
             (dict(k=0), INV), (dict(v=P + 4), INV), (dict(k_stride_head=12), INV), (dict(v_stride_token=0), INV),
             (dict(q_norm=P + 8), INV), (dict(k_norm=P + 2), INV), (dict(positions=P + 2), INV), (dict(q_out=0), INV),
             (dict(o_stride_token=64), INV), (dict(o_stride_head=32), INV)],
    "attention": [(dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
                  (dict(num_heads=2048, num_kv_heads=2), UNS), (dict(total_rows=1 << 29), UNS), (dict(lse=P + 2), INV),
                  (dict(gate=P, gate_dtype=5), INV), (dict(gate=P + 4), INV), (dict(gate=P, g_stride_head=4), INV),
                  (dict(out=0), INV), (dict(o_stride_token=64), INV), (dict(workspace=0), INV),
                  (dict(workspace=P + 8), INV), (dict(workspace_bytes=1000), INV)],
    "weights": [(dict(scale=0.0), INV), (dict(lse=0), INV), (dict(weights_out=0), INV), (dict(weights=P + 2), INV),
                (dict(weights_out=P + 1), INV), (dict(weights_width=0), INV), (dict(w_stride_head=16), INV),
                (dict(num_seqs=2, w_stride_seq=32), INV), (dict(total_rows=1 << 29), UNS)],
    "evict": [(dict(num_kv_heads=0), INV), (dict(keep=0), INV), (dict(keep=-3), INV), (dict(recent=-1), INV),
              (dict(recent=17), INV), (dict(lengths=0), INV), (dict(lengths_out=0), INV), (dict(weights=0), INV),
              (dict(kept=0), INV), (dict(kept=P + 2), INV), (dict(lengths=P + 2), INV), (dict(weights_width=0), INV),
              (dict(num_seqs=1, lengths_out=P), INV), (dict(num_seqs=3, lengths_out=P + 8), INV), (dict(w_stride_head=-8), INV),
              (dict(weights_out_width=0), INV), (dict(wo_stride_head=16), INV), (dict(num_seqs=2, wo_stride_seq=32), INV),
              (dict(wo_stride_seq=128), INV), (dict(out_table=P + 2, out_table_width=2, out_table_stride=2), INV),
              (dict(out_table=2 * P, out_table_width=0, out_table_stride=2), INV),
              (dict(out_table=2 * P, out_table_width=3, out_table_stride=2), INV),
              (dict(num_seqs=1, out_table=P, out_table_width=2, out_table_stride=3), INV),
              (dict(num_seqs=1 << 24, num_kv_heads=16, kp_stride_page=1 << 15, vp_stride_page=1 << 15, weights_out=0,
                    lengths_out=1 << 40), UNS)],
}
CASES = [(c, kw, st) for c in CALLS for kw, st in
         POOLS + (VALUES if c != "weights" else []) + (WRITTEN if c in ("rows", "evict") else []) +
         (HEADS if c != "evict" else []) + OWN[c]]


@pytest.mark.parametrize("call,kw,status", CASES)
def test_refusals(call, kw, status):
    fn, make = CALLS[call]
    with pytest.raises(gattn.GattnError) as e:
        fn(make(**kw))
    assert e.value.status == status and str(e.value).split(": ", 1)[1]


@pytest.mark.parametrize("call", CALLS)
def test_calls_without_work_and_without_a_descriptor(call):
    fn, make = CALLS[call]
    fn(make())                              # no sequences
    if call != "evict":
        fn(make(num_seqs=3, total_rows=0))
    assert getattr(gattn.lib(), "gattn_paged_" + call)(None, None) == 1
    # reading calls take pools whose rows overlap
    if call in ("attention", "weights"):
        fn(make(kp_stride_token=8, kp_stride_head=8))


def test_workspace_sizes():
    w = gattn.paged_attention_workspace
    assert w(16, 4, 256, 1, 1) > 0 and w(16, 4, 256, 0, 0) > 0
    # more rows a sequence, larger tiles; never more than those of 64 rows
    sizes = [w(16, 4, 256, 4, 4 * r) for r in (1, 2, 3, 4, 8, 16, 100)]
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2]
    for bad in ((0, 4, 64, 1, 1), (16, 5, 64, 1, 1), (16, 4, 65, 1, 1), (16, 4, 64, -1, 1)):
        with pytest.raises(gattn.GattnError):
            w(*bad)


def _t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_tensor_forms_refuse():
    i32, f32 = torch.int32, torch.float32
    q, kv, pool, table = _t((3, 4, 64)), _t((3, 2, 64)), _t((5, 2, 16, 64)), _t((1, 3), i32)
    cu, pos = _t((2,), i32), _t((1,), i32)
    ok = dict(rope_theta=1e4)
    for args, kw in [
            ((q, kv, kv, pool, pool, table, cu, pos), ok),                            # on the CPU
            ((q, kv, kv, pool, pool[:4], table, cu, pos), ok),
            ((q, kv, kv, pool.float(), pool, table, cu, pos), ok),
            ((q, kv[:2], kv, pool, pool, table, cu, pos), ok),
            ((q, kv, kv, pool, pool, table.long(), cu, pos), ok),
            ((q, kv, kv, pool, pool, table[0], cu, pos), ok),
            ((q, kv, kv, pool, pool, _t((2, 3), i32), cu, pos), ok),
            ((q, kv, kv, pool, pool, _t((3, 1), i32).t(), cu, _t((2,), i32)), ok),
            ((q, kv, kv, pool, pool, table, cu, pos), dict(ok, rope_factor=2.0, rope_yarn=dict(factor=2.0, original=8))),
            ((q, kv, kv, pool, pool, table, cu, pos), dict(ok, rope_yarn=dict(factor=2.0))),
            ((q, kv, kv, pool, pool, table, cu, pos), dict(ok, rope_yarn=dict(factor=2.0, original=8, mscale=1))),
            ((q, kv, kv, pool, pool, table, cu, pos), dict(ok, positions=_t((2,), i32)))]:
        with pytest.raises((ValueError, RuntimeError)):
            device.paged_rows(*args, **kw)
    lse, w = _t((3, 4), f32), _t((1, 2, 48), f32)
    for args, kw in [
            ((q, pool, pool, table, cu, pos), {}),
            ((q.float(), pool, pool, table, cu, pos), {}),
            ((q, pool, pool, table, cu, pos), dict(lse=lse.t())),
            ((q, pool, pool, table, cu, pos), dict(lse=lse[:2])),
            ((q, pool, pool, table, cu, pos), dict(gate=q[..., :32])),
            ((q, pool, pool, table, cu, pos), dict(workspace=lse)),
            ((_t((3, 4, 128)), pool, pool, table, cu, pos), {})]:
        with pytest.raises((ValueError, RuntimeError)):
            device.paged_attention(*args, **kw)
    for kw in [dict(weights=w), dict(), dict(weights=w[..., :40], weights_out=w), dict(weights=w.double()),
               dict(weights=w[0])]:
        with pytest.raises((ValueError, RuntimeError)):
            device.paged_weights(q, pool, table, cu, pos, lse, **kw)
    with pytest.raises((ValueError, RuntimeError)):
        device.paged_weights(q, pool, table, cu, pos, None, weights=w)
    for args, kw in [
            ((pool, pool, table, pos, w), dict(keep=8)),
            ((pool, pool, table, pos, w), dict(keep=8, kept=_t((1, 2, 7), i32))),
            ((pool, pool, table, pos, w), dict(keep=8, lengths_out=_t((2,), i32))),
            ((pool, pool, table, pos, w[:, :1]), dict(keep=8)),
            ((pool, pool, table, 3, w), dict(keep=8)),
            ((pool, pool, table, pos, w), dict(keep=8, out_table=table.long()))]:
        with pytest.raises((ValueError, RuntimeError)):
            device.paged_evict(*args, **kw)
