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
    """What the tensors get wrong names the argument; all right otherwise, they lie on the CPU."""
    i32, f32 = torch.int32, torch.float32
    q, kv, pool, table = _t((3, 4, 64)), _t((3, 2, 64)), _t((5, 2, 16, 64)), _t((1, 3), i32)
    cu, pos = _t((2,), i32), _t((1,), i32)

    def bad(fn, ok, text, *change, **kw):
        args = list(ok)
        for i, x in change:
            args[i] = x
        with pytest.raises(ValueError, match=text):
            fn(*args, **kw)

    rows = (q, kv, kv, pool, pool, table, cu, pos)
    th = dict(rope_theta=1e4)
    bad(device.paged_rows, rows, "CUDA device", **th)
    out = _t((3, 4, 64))
    for i, x, text in [(0, q.double(), "q has type"), (0, q[0], "q must have shape"), (0, q.transpose(1, 2), "q needs contiguous|k_pages must have"),
                       (0, q.to_sparse(), "dense"), (1, kv[:2], "k must have shape"), (1, kv.float(), "k has type"),
                       (1, 3, "k must be a tensor"), (2, _t((3, 3, 64)), "v must have shape"), (3, pool.float(), "k_pages has type"),
                       (3, pool[0], "k_pages must have shape"), (3, _t((5, 2, 16, 128)), "v_pages must have k_pages"),
                       (4, pool[:4], "v_pages must have k_pages"), (4, None, "v_pages must be a tensor"),
                       (5, table.long(), "table has type"), (5, table[0], "table must have shape"),
                       (5, _t((2, 3), i32), "table must have shape"), (5, _t((1, 6), i32)[:, ::2], "table must have shape"),
                       (6, cu.long(), "cu_rows has type"), (6, cu[:0], "cu_rows must have shape"), (7, _t((2,), i32), "cache_pos must have shape"),
                       (7, pos.float(), "cache_pos has type")]:
        bad(device.paged_rows, rows, text, (i, x), q_out=out, rotary_dims=64, **th)
    for kw, text in [(dict(rope_factor=2.0, rope_yarn=dict(factor=2.0, original=8)), "part of rope_yarn"),
                     (dict(rope_yarn=dict(factor=2.0)), "rope_yarn takes"),
                     (dict(rope_yarn=dict(factor=2.0, original=8, mscale=1)), "rope_yarn takes"),
                     (dict(positions=_t((2,), i32)), "positions must have shape"), (dict(q_norm=_t((32,))), "q_norm must have shape"),
                     (dict(k_norm=_t((64,), f32)), "k_norm has type"), (dict(q_out=_t((3, 4, 32))), "q_out must have shape"),
                     (dict(q_out=out.float()), "q_out has type"), (dict(status=_t((2,), i32)), "status must have shape"),
                     (dict(rotary_dims=1 << 40), "rotary_dims is out of range")]:
        bad(device.paged_rows, rows, text, **dict(th, **kw))
    with pytest.raises(TypeError):
        device.paged_rows(*rows, rope_theta="1e4")
    attn = (q, pool, pool, table, cu, pos)
    lse, w = _t((3, 4), f32), _t((1, 2, 48), f32)
    bad(device.paged_attention, attn, "CUDA device")
    bad(device.paged_attention, attn, "q has type", (0, q.float()), out=out)
    bad(device.paged_attention, attn, "q's head_dim", (0, _t((3, 4, 128))))
    for kw, text in [(dict(lse=_t((4, 3), f32).t()), "lse must have shape"), (dict(lse=lse[:2]), "lse must have shape"),
                     (dict(lse=lse.double()), "lse has type"), (dict(gate=q[..., :32]), "gate must have shape"),
                     (dict(gate=q.half()), "gate has type"), (dict(workspace=lse), "workspace has type"),
                     (dict(workspace=_t((4, 4), torch.uint8).t()), "workspace must be contiguous"),
                     (dict(out=out[:2]), "out must have shape")]:
        bad(device.paged_attention, attn, text, **kw)
    weigh = (q, pool, table, cu, pos, lse)
    bad(device.paged_weights, weigh, "CUDA device", weights=w)
    for kw, text in [(dict(), "weights_out must be a tensor"), (dict(weights=w[..., :40], weights_out=w), "weights_out's shape"),
                     (dict(weights=w.double()), "weights_out has type"), (dict(weights=w[0]), "weights_out must have shape"),
                     (dict(weights=_t((1, 3, 48), f32)), "weights_out must have shape"),
                     (dict(weights_out=_t((1, 2, 96), f32)[..., ::2]), "weights_out must have shape")]:
        bad(device.paged_weights, weigh, text, **kw)
    bad(device.paged_weights, weigh, "lse must be a tensor", (5, None), weights=w)
    evict = (pool, pool, table, pos, w)
    bad(device.paged_evict, evict, "CUDA device", keep=8)
    for kw, text in [(dict(keep=8, kept=_t((1, 2, 7), i32)), "kept must be"), (dict(keep=8, lengths_out=_t((2,), i32)), "lengths_out must"),
                     (dict(keep=0), "keep must be"), (dict(keep=8, out_table=table.long()), "out_table has type"),
                     (dict(keep=8, weights_out=w[:, :1]), "weights_out must have shape")]:
        bad(device.paged_evict, evict, text, **kw)
    bad(device.paged_evict, evict, "lengths must be a tensor", (3, 3), keep=8)
    bad(device.paged_evict, evict, "weights must have shape", (4, w[:, :1]), keep=8)
    bad(device.paged_evict, evict, "table must have shape", (2, _t((2, 3), i32)), keep=8)
