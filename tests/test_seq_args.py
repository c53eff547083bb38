"""The packed-sequence entry points without a GPU: every refusal the header
documents, taken before any CUDA call."""
import pytest
import torch

from qwen3_gated_attention_gb300 import device, gattn


@pytest.fixture(scope="module", autouse=True)
def built():
    from qwen3_gated_attention_gb300 import build
    build.build()


P = 4096                  # a 16-byte aligned address that no refused call touches


def _rows(**kw):
    d = gattn.gattn_prompt_rows_desc()
    base = dict(num_heads=4, num_kv_heads=2, head_dim=64, partial_rotary_factor=0.25, rope_theta=1e7,
                rms_eps=1e-6, x_dtype=1, num_seqs=0, total_rows=8, cu_rows=P, cache_pos=P, q=P, k=P, v=P,
                q_stride_token=512, q_stride_head=128, k_stride_token=128, k_stride_head=64,
                v_stride_token=128, v_stride_head=64, q_norm=P, k_norm=P, q_out=P, o_stride_token=256,
                o_stride_head=64, k_cache=P, v_cache=P, cache_batch=1, cache_capacity=16,
                kc_stride_token=64, kc_stride_head=1024, kc_stride_batch=2048, vc_stride_token=64,
                vc_stride_head=1024, vc_stride_batch=2048)
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def _attn(**kw):
    d = gattn.gattn_prompt_attention_desc()
    base = dict(num_heads=4, num_kv_heads=2, head_dim=64, scale=0.125, num_seqs=0, total_rows=8, cu_rows=P,
                q=P, q_stride_token=256, q_stride_head=64, k=P, v=P, kv_batch=1, kv_rows=8,
                k_stride_token=128, k_stride_head=64, k_stride_batch=8, v_stride_token=128, v_stride_head=64,
                v_stride_batch=8, gate_dtype=1, g_stride_token=8, g_stride_head=8, out=P,
                o_stride_token=256, o_stride_head=64)
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


def _delta(**kw):
    d = gattn.gattn_delta_desc()
    base = dict(num_k_heads=2, num_v_heads=4, k_dim=64, v_dim=64, scale=0.125, qk_l2norm=1, l2_eps=1e-6,
                num_seqs=0, total_rows=8, num_slots=1, cu_rows=P, q=P, k=P, v=P, q_stride_token=128,
                q_stride_head=64, k_stride_token=128, k_stride_head=64, v_stride_token=256, v_stride_head=64,
                g=P, beta=P, g_stride_token=4, beta_stride_token=4, state=P, state_out=P,
                state_stride=4 * 64 * 64, out=P, o_stride_token=256, o_stride_head=64)
    for k, v in {**base, **kw}.items():
        setattr(d, k, v)
    return d


BAD_ROWS = [
    (dict(num_kv_heads=3), 1), (dict(num_heads=0), 1), (dict(num_seqs=-1), 1), (dict(total_rows=-1), 1),
    (dict(total_rows=2 ** 31 - 1), 1), (dict(head_dim=96), 2), (dict(head_dim=320), 2), (dict(x_dtype=2), 1),
    (dict(partial_rotary_factor=0.0), 1), (dict(partial_rotary_factor=1.5), 1),
    (dict(partial_rotary_factor=3 / 64), 1), (dict(rope_theta=0.0), 1), (dict(rms_eps=-1.0), 1),
    (dict(rms_eps=float("nan")), 1), (dict(q=None), 1), (dict(q=P + 8), 1), (dict(q_stride_token=4), 1),
    (dict(q_stride_head=0), 1), (dict(k_stride_token=-64), 1), (dict(v=None), 1), (dict(q_out=None), 1),
    (dict(k_cache=None), 1), (dict(vc_stride_batch=12), 1), (dict(cu_rows=None), 1),
    (dict(cache_pos=None), 1), (dict(q_norm=None), 1), (dict(cache_batch=0), 1), (dict(cache_capacity=0), 1),
    (dict(q_norm=P + 2), 1),
]
BAD_ATTN = [
    (dict(num_kv_heads=3), 1), (dict(head_dim=80), 2), (dict(num_heads=2048, num_kv_heads=2048), 2),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(q=None), 1), (dict(k=P + 4), 1), (dict(out=None), 1), (dict(k_stride_batch=0), 1),
    (dict(gate=P, gate_dtype=7), 1), (dict(gate=P + 2), 1), (dict(gate=P, g_stride_head=3), 1),
    (dict(cu_rows=None), 1), (dict(kv_rows=0), 1), (dict(kv_batch=0), 1), (dict(kv_batch=2), 1),
    (dict(slots=P), 1), (dict(cache_pos=P, cu_kv=P), 1), (dict(max_kv=-1), 1), (dict(num_seqs=-3), 1),
    (dict(q_stride_token=2 ** 40), 1),
]
BAD_DELTA = [
    (dict(num_k_heads=3), 1), (dict(k_dim=96), 2), (dict(k_dim=256), 2), (dict(v_dim=48), 2), (dict(v_dim=288), 2),
    (dict(v_dim=0), 2), (dict(scale=float("nan")), 1), (dict(l2_eps=-1.0), 1), (dict(q=None), 1), (dict(v=P + 2), 1),
    (dict(g=None), 1), (dict(beta=P + 1), 1), (dict(g_stride_token=3), 1), (dict(out=None), 1),
    (dict(cu_rows=None, num_seqs=3), 1), (dict(num_slots=0), 1), (dict(state=P + 4), 1),
    (dict(state_stride=4 * 64 * 64 - 4), 1), (dict(state_stride=4 * 64 * 64 + 2), 1),
    (dict(state=None, state_out=None, slots=P), 1), (dict(o_stride_head=4), 1), (dict(num_seqs=-1), 1),
]


@pytest.mark.parametrize("make,call,bad", [(_rows, "prompt_rows", BAD_ROWS), (_attn, "prompt_attention", BAD_ATTN),
                                           (_delta, "delta_prompt", BAD_DELTA), (_delta, "delta_step", BAD_DELTA)],
                         ids=["rows", "attention", "delta_prompt", "delta_step"])
def test_refusals(make, call, bad):
    fn = getattr(gattn, call)
    fn(make())                                   # no sequences: accepted, nothing launched
    for change, status in bad:
        with pytest.raises(gattn.GattnError) as e:
            fn(make(**change))
        assert e.value.status == status, change
        assert gattn.last_error()
    raw = getattr(gattn.lib(), "gattn_" + call)
    assert raw(None, None) == 1


def _refused(fn, args):
    """Refused for what was changed, not for lying on the CPU (checked last)."""
    with pytest.raises(ValueError) as e:
        fn(**args)
    assert "CUDA device" not in str(e.value)


def test_tensor_checks():
    bf, z = torch.bfloat16, torch.zeros
    q, k = z(4, 2, 64, dtype=bf), z(4, 1, 64, dtype=bf)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    ok = dict(q=q, k=k, v=k, cu_rows=cu)
    for change in (dict(q=q.float()), dict(q=q[0]), dict(k=z(4, 1, 32, dtype=bf)), dict(v=z(3, 1, 64, dtype=bf)),
                   dict(cu_rows=cu.long()), dict(cu_rows=cu[:0]), dict(gate=z(4, 2, 32)), dict(out=q.float()),
                   dict(q=z(4, 64, 2, dtype=bf).transpose(1, 2)), dict(cu_kv=cu[:1]), dict(status=z(1)),
                   dict(cache_pos=cu[:1])):
        _refused(device.prompt_attention, {**ok, **change})
    v, g = z(4, 2, 64, dtype=bf), z(4, 2)
    ok = dict(q=k, k=k, v=v, g=g, beta=g, cu_rows=cu)
    for change in (dict(g=g.to(bf)), dict(beta=z(4, 3)), dict(cu_rows=None), dict(num_seqs=2), dict(k=v),
                   dict(state=z(1, 2, 64, 32)), dict(state=z(1, 2, 64, 64), state_out=z(2, 2, 64, 64)),
                   dict(state=z(1, 2, 64, 64).transpose(2, 3)), dict(out=k), dict(slots=cu)):
        _refused(device.delta_step, {**ok, **change})
    kc = z(1, 1, 16, 64, dtype=bf)
    w = z(64, dtype=bf)
    ok = dict(q=q, k=k, v=k, q_norm=w, k_norm=w, k_cache=kc, v_cache=kc, cu_rows=cu, cache_pos=cu[:1],
              partial_rotary_factor=0.25, rope_theta=1e7, rms_eps=1e-6)
    for change in (dict(k=k.float()), dict(q_norm=w.float()), dict(q_norm=w[:32]), dict(k_cache=kc[0]),
                   dict(v_cache=kc[:, :, :8]), dict(cache_pos=cu), dict(q_out=k), dict(slots=cu)):
        _refused(device.prompt_rows, {**ok, **change})
    with pytest.raises(ValueError, match="CUDA device"):
        device.prompt_rows(**ok)


def test_outputs_whose_rows_share_memory():
    """Two rows of an output in one place would be a race."""
    for make, call, bad, good in (
            (_attn, "prompt_attention",
             [dict(o_stride_head=32), dict(o_stride_token=64), dict(o_stride_token=192), dict(o_stride_head=504),
              dict(o_stride_token=2 ** 37, o_stride_head=2 ** 37)],
             [dict(o_stride_head=512, o_stride_token=64), dict(o_stride_head=8, num_heads=1, num_kv_heads=1),
              dict(o_stride_token=8, total_rows=1), dict(o_stride_head=2 ** 37), dict(o_stride_token=2 ** 37)]),
            (_rows, "prompt_rows",
             [dict(o_stride_head=32), dict(kc_stride_token=32), dict(vc_stride_head=1016), dict(vc_stride_token=128)],
             [dict(kc_stride_token=128, kc_stride_head=64), dict(cache_capacity=17, vc_stride_head=1088,
                                                                kc_stride_head=1088)]),
            (_delta, "delta_step", [dict(o_stride_head=32), dict(o_stride_token=192)], [dict(o_stride_token=264)])):
        fn = getattr(gattn, call)
        for change in bad:
            with pytest.raises(gattn.GattnError) as e:
                fn(make(**change))
            assert e.value.status == 1 and "overlap" in gattn.last_error(), change
        for change in good:
            fn(make(**change))


def test_words_off_their_boundary_and_far_positions():
    for make, call, names in ((_rows, "prompt_rows", ("cu_rows", "cache_pos", "slots", "status")),
                              (_attn, "prompt_attention", ("cu_rows", "cu_kv", "status")),
                              (_delta, "delta_prompt", ("cu_rows", "slots", "status"))):
        for name in names:
            with pytest.raises(gattn.GattnError) as e:
                getattr(gattn, call)(make(**{name: P + 2}))
            assert e.value.status == 1 and "4-byte" in gattn.last_error(), name
    big = dict(kc_stride_head=2 ** 31, vc_stride_head=2 ** 31)
    gattn.prompt_rows(_rows(cache_capacity=1 << 24, **big))
    with pytest.raises(gattn.GattnError) as e:
        gattn.prompt_rows(_rows(cache_capacity=(1 << 24) + 1, **big))
    assert e.value.status == 2
