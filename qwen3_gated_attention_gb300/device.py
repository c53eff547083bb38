"""Device-memory plumbing around the C ABI: torch owns the buffers (weights in the
interchange layout, bf16 caches, inputs, outputs); every computation goes
through ``gattn.layer_step`` and friends.  ``DeviceLayer`` holds one layer;
``prompt_rows``, ``prompt_attention``, ``delta_prompt`` and ``delta_step`` call
the packed-sequence operators on tensors."""
from __future__ import annotations

import numpy as np
import torch

from . import gattn


def _dev_u16(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, np.uint16).view(np.int16)).to(device)


def _dev_u32(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, np.uint32).view(np.int32)).to(device)


def cache_strides(layout: str, batch: int, Hk: int, cap: int, d: int):
    """(shape, stride_token, stride_head, stride_batch) in elements."""
    if layout == "bhtd":          # [B][Hk][cap][d]
        return (batch, Hk, cap, d), d, cap * d, Hk * cap * d
    if layout == "btd":           # token-major [B][cap][Hk*d]
        return (batch, cap, Hk, d), Hk * d, d, cap * Hk * d
    raise ValueError(layout)


class DeviceLayer:
    """One layer handle with its weights set and one registered cache: bf16 K/V,
    or (kv_format="turbo4v") bf16 K with Turbo4 V code and E4M3 scale planes
    [B][Hk][cap][d/2] and [B][Hk][cap][d/16] uint8, or (kv_format="turbo4")
    such planes for K and V both."""

    def __init__(self, spec, packed, q_norm, k_norm, capacity, *, batch=None, max_batch=None,
                 max_q_len=None, head_chunk=True, layout="bhtd", device="cuda:0",
                 kv_format="bf16"):
        self.spec = spec
        self.device = torch.device(device)
        self.batch = batch or spec.batch
        self.layout = layout
        self.capacity = capacity
        self.kv_format = kv_format
        self.cfg = gattn.make_cfg(spec.hidden, spec.num_heads, spec.num_kv_heads, spec.head_dim,
                                  spec.partial_rotary_factor, spec.rope_theta, spec.rms_eps,
                                  tuple(spec.bits), tuple(spec.group), x_dtype=spec.x_dtype,
                                  max_batch=max_batch or self.batch,
                                  max_q_len=max_q_len or spec.q_len, head_chunk=head_chunk)
        self.h = gattn.layer_create(self.cfg)
        self.kv = 0
        try:
            self._w = [(_dev_u32(p, self.device), _dev_u16(s, self.device), _dev_u16(b, self.device))
                       for p, s, b in packed]
            self._qn = _dev_u16(q_norm, self.device)
            self._kn = _dev_u16(k_norm, self.device)
            stream = torch.cuda.current_stream(self.device).cuda_stream
            gattn.layer_set_weights(self.h, [(p.data_ptr(), s.data_ptr(), b.data_ptr())
                                             for p, s, b in self._w],
                                    self._qn.data_ptr(), self._kn.data_ptr(), stream)
            Hk, d = spec.num_kv_heads, spec.head_dim
            shape, st, sh, sb = cache_strides(layout, self.batch, Hk, capacity, d)
            self.k = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
            if kv_format == "turbo4":
                assert layout == "bhtd"
                B = self.batch
                pl = lambda w: torch.zeros((B, Hk, capacity, w), dtype=torch.uint8, device=self.device)
                self.kc, self.ks = pl(d // 2), pl(d // 16)
                self.vc, self.vs = pl(d // 2), pl(d // 16)
                self.kv = gattn.kv_register_turbo4(
                    self.h, self.kc.data_ptr(), self.ks.data_ptr(), self.vc.data_ptr(),
                    self.vs.data_ptr(), B, capacity, (capacity * d // 2, Hk * capacity * d // 2),
                    (capacity * d // 16, Hk * capacity * d // 16))
            elif kv_format == "turbo4v":
                assert layout == "bhtd"
                B = self.batch
                self.vc = torch.zeros((B, Hk, capacity, d // 2), dtype=torch.uint8, device=self.device)
                self.vs = torch.zeros((B, Hk, capacity, d // 16), dtype=torch.uint8,
                                      device=self.device)
                self.kv = gattn.kv_register_turbo4v(
                    self.h, self.k.data_ptr(), self.vc.data_ptr(), self.vs.data_ptr(), B, capacity,
                    (st, sh, sb), (capacity * d // 2, Hk * capacity * d // 2),
                    (capacity * d // 16, Hk * capacity * d // 16))
            else:
                self.v = torch.zeros(shape, dtype=torch.bfloat16, device=self.device)
                self.kv = gattn.kv_register(self.h, self.k.data_ptr(), self.v.data_ptr(),
                                            self.batch, capacity, st, sh, sb)
        except Exception:
            self.close()
            raise

    # caches are exchanged with the host as [B][Hk][cap][d] bf16 bit patterns
    def load_cache(self, k_bits: np.ndarray, v_bits, batches=None):
        """v_bits: bf16 bits [B][Hk][cap][d], or (codes, scales) for a turbo4v cache."""
        idx = list(range(self.batch)) if batches is None else list(batches)
        if self.kv_format == "turbo4":
            (kc, ks), (vc, vs) = k_bits, v_bits
            for j, b in enumerate(idx):
                for dst, src in ((self.kc, kc), (self.ks, ks), (self.vc, vc), (self.vs, vs)):
                    dst[b].copy_(torch.from_numpy(np.ascontiguousarray(src[j], np.uint8)))
            return
        if self.kv_format == "turbo4v":
            codes, scales = v_bits
            for j, b in enumerate(idx):
                self.vc[b].copy_(torch.from_numpy(np.ascontiguousarray(codes[j], np.uint8)))
                self.vs[b].copy_(torch.from_numpy(np.ascontiguousarray(scales[j], np.uint8)))
            pairs = ((self.k, k_bits),)
        else:
            pairs = ((self.k, k_bits), (self.v, v_bits))
        for dst, src in pairs:
            for j, b in enumerate(idx):
                t = _dev_u16(src[j], self.device).view(torch.bfloat16)      # [Hk][cap][d]
                if self.layout == "bhtd":
                    dst[b].copy_(t)
                else:
                    dst[b].copy_(t.transpose(0, 1))

    def read_cache(self, batches=None):
        """(K bits, V bits), or (K bits, (codes, scales)) for a turbo4v cache."""
        idx = list(range(self.batch)) if batches is None else list(batches)
        if self.kv_format == "turbo4":
            g = lambda t: np.stack([t[b].cpu().numpy() for b in idx])
            return (g(self.kc), g(self.ks)), (g(self.vc), g(self.vs))
        if self.kv_format == "turbo4v":
            k = np.stack([self.k[b].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
                          for b in idx])
            return k, (np.stack([self.vc[b].cpu().numpy() for b in idx]),
                       np.stack([self.vs[b].cpu().numpy() for b in idx]))
        outs = []
        for src in (self.k, self.v):
            parts = []
            for b in idx:
                t = src[b] if self.layout == "bhtd" else src[b].transpose(0, 1)
                parts.append(t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
            outs.append(np.stack(parts))
        return outs[0], outs[1]

    def step(self, x: torch.Tensor, cache_pos: torch.Tensor, out: torch.Tensor, batch=None,
             q_len=None, stream=None):
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        gattn.layer_step(self.h, x.data_ptr(), self.kv, cache_pos.data_ptr(), batch or self.batch,
                         q_len or self.spec.q_len, out.data_ptr(), s)

    def step_block(self, x: torch.Tensor, cache_pos: torch.Tensor, input_ln: torch.Tensor,
                   post_ln: torch.Tensor | None, out: torch.Tensor,
                   out_normed: torch.Tensor | None = None, batch=None, q_len=None, stream=None):
        s = stream if stream is not None else torch.cuda.current_stream(self.device).cuda_stream
        gattn.layer_step_block(self.h, x.data_ptr(), self.kv, cache_pos.data_ptr(),
                               batch or self.batch, q_len or self.spec.q_len, input_ln.data_ptr(),
                               post_ln.data_ptr() if post_ln is not None else None, out.data_ptr(),
                               out_normed.data_ptr() if out_normed is not None else None, s)

    def set_taps(self, y: torch.Tensor | None, attn: torch.Tensor | None):
        gattn.layer_set_taps(self.h, y.data_ptr() if y is not None else None,
                             attn.data_ptr() if attn is not None else None)

    def set_mask(self, mask: torch.Tensor | None):
        """mask: uint8 [B][1 or H][R][T] on the device (None clears it)."""
        if mask is None:
            gattn.layer_set_mask(self.h, None)
            return
        assert mask.dtype == torch.uint8 and mask.dim() == 4 and mask.is_contiguous()
        self._mask = mask
        gattn.layer_set_mask(self.h, mask.data_ptr(), mask.shape[1], mask.shape[3],
                             (mask.stride(2), mask.stride(1), mask.stride(0)))

    def poll(self):
        gattn.layer_poll_status(self.h, torch.cuda.current_stream(self.device).cuda_stream)

    def close(self):
        if getattr(self, "kv", 0):
            gattn.kv_destroy(self.kv)
            self.kv = 0
        if getattr(self, "h", 0):
            gattn.layer_destroy(self.h)
            self.h = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def x_to_device(spec, x: np.ndarray, device="cuda:0") -> torch.Tensor:
    if spec.x_dtype == "f32":
        return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(device)
    return _dev_u16(x, device).view(torch.bfloat16)


def bf16_tensor_to_f64(t: torch.Tensor) -> np.ndarray:
    return t.float().cpu().numpy().astype(np.float64)


# -------------------------------------------------------- packed sequences
#
# Torch forms of the packed-sequence entry points: shapes and strides are read
# off the tensors, the launch goes to the current stream of their device (or to
# `stream`, a cudaStream_t handle of that device).  Slices of a wider projection
# output are passed as they are, nothing is copied.  `status`, an int32 tensor of one
# entry that the caller zeroes and reads, collects gattn.STATUS_* bits; without it a
# sequence that was skipped shows in its zero rows only, and a time-out not at all.

_DTYPES = {torch.float32: gattn.DTYPE_F32, torch.bfloat16: gattn.DTYPE_BF16}
_BF16, _F32, _I32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _refuse(t, name, dev, dtypes, shape, what="must have shape"):
    """The message for a tensor that _rows, _planes or _flat does not take."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} lies on {t.device}, not beside the first tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has type {t.dtype}, not one of {dtypes}")
    raise ValueError(f"{name} {what} {shape} (got {tuple(t.shape)}, strides {t.stride()})")


# A dimension of one or no entries may have any stride: a valid one stands in.

def _rows(t, name, dev, dtypes, shape=None):
    """(address, token stride, head stride) of a [rows][heads][elements] tensor."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype not in dtypes:
        _refuse(t, name, dev, dtypes, shape)
    sh, st = t.shape, t.stride()
    if len(sh) != 3 or (shape is not None and sh != shape):
        _refuse(t, name, dev, dtypes, shape or "[rows][heads][elements]")
    if st[2] != 1 and sh[2] > 1:
        _refuse(t, name, dev, dtypes, shape, "needs contiguous elements:")
    return (t.data_ptr(), st[0] if sh[0] > 1 else max(8, sh[1] * sh[2]),
            st[1] if sh[1] > 1 else max(8, sh[2]))


def _planes(t, name, dev, dtypes, shape=None):
    """(address, token, head, batch stride) of a [batch][heads][tokens][elements] tensor."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype not in dtypes:
        _refuse(t, name, dev, dtypes, shape)
    sh, st = t.shape, t.stride()
    if len(sh) != 4 or (shape is not None and sh != shape):
        _refuse(t, name, dev, dtypes, shape or "[batch][heads][tokens][elements]")
    if st[3] != 1 and sh[3] > 1:
        _refuse(t, name, dev, dtypes, shape, "needs contiguous elements:")
    return (t.data_ptr(), st[2] if sh[2] > 1 else max(8, sh[3]),
            st[1] if sh[1] > 1 else max(8, sh[2] * sh[3]),
            st[0] if sh[0] > 1 else max(8, sh[1] * sh[2] * sh[3]))


def _flat(t, name, dev, dtypes, n):
    """Address of a contiguous vector of n entries; 0 for None."""
    if t is None:
        return 0
    if (not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype not in dtypes or
            t.shape != (n,) or not t.is_contiguous()):
        _refuse(t, name, dev, dtypes, f"[{n}], contiguous")
    return t.data_ptr()


def _cu(t, name, dev):
    """(address, sequences) of the row offsets."""
    if (not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not torch.int32 or
            t.dim() != 1 or t.shape[0] < 1 or not t.is_contiguous()):
        _refuse(t, name, dev, _I32, "[num_seqs + 1], contiguous")
    return t.data_ptr(), t.shape[0] - 1


def _output(shape, like, stream):
    """A bf16 tensor whose memory belongs to the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    own = (torch.cuda.ExternalStream(stream, device=like.device) if stream
           else torch.cuda.default_stream(like.device))        # handle 0
    with torch.cuda.stream(own):
        return torch.empty(shape, dtype=torch.bfloat16, device=like.device)


def _call(fn, desc, dev, stream):
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if stream is None:
        stream = _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    if _current_device() == dev:
        fn(desc, stream)
    else:
        with torch.cuda.device(dev):
            fn(desc, stream)


def prompt_rows(q, k, v, q_norm, k_norm, k_cache, v_cache, cu_rows, cache_pos, *,
                partial_rotary_factor, rope_theta, rms_eps, q_out=None, slots=None, status=None,
                stream=None):
    """QK RMSNorm, partial RoPE and KV append of packed rows (gattn_prompt_rows).

    q [T][H][d], k and v [T][Hk][d] (fp32 or bf16); q_norm, k_norm bf16 [d];
    k_cache, v_cache bf16 [B][Hk][capacity][d] views, written at cache_pos[s] + i;
    cu_rows int32 [n + 1], cache_pos and slots int32 [n]; status int32 [1].
    Returns q_out, bf16 [T][H][d] (allocated when not given)."""
    dev = q.get_device()
    qa = _rows(q, "q", dev, _DTYPES)
    T, H, d = q.shape
    dtype = q.dtype
    Hk = k.shape[1] if k.dim() == 3 else 0
    ka = _rows(k, "k", dev, (dtype,), (T, Hk, d))
    va = _rows(v, "v", dev, (dtype,), (T, Hk, d))
    kc = _planes(k_cache, "k_cache", dev, _BF16)
    B, _, cap, _ = shape = k_cache.shape
    if shape != (B, Hk, cap, d):
        _refuse(k_cache, "k_cache", dev, _BF16, (B, Hk, cap, d))
    vc = _planes(v_cache, "v_cache", dev, _BF16, shape)
    if q_out is None:
        q_out = _output((T, H, d), q, stream)
    oa = _rows(q_out, "q_out", dev, _BF16, (T, H, d))
    cu, n = _cu(cu_rows, "cu_rows", dev)
    desc = gattn.gattn_prompt_rows_desc.pack(
        H, Hk, d, partial_rotary_factor, rope_theta, rms_eps, _DTYPES[dtype], n, T, cu,
        _flat(cache_pos, "cache_pos", dev, _I32, n), _flat(slots, "slots", dev, _I32, n),
        qa[0], ka[0], va[0], qa[1], qa[2], ka[1], ka[2], va[1], va[2],
        _flat(q_norm, "q_norm", dev, _BF16, d), _flat(k_norm, "k_norm", dev, _BF16, d), oa[0],
        oa[1], oa[2], kc[0], vc[0], B, cap, kc[1], kc[2], kc[3], vc[1], vc[2], vc[3],
        _flat(status, "status", dev, _I32, 1))
    if n and T:
        _call(gattn.prompt_rows, desc, dev, stream)
    return q_out


def prompt_attention(q, k, v, cu_rows, *, cu_kv=None, cache_pos=None, slots=None, gate=None,
                     scale=None, max_kv=0, out=None, status=None, stream=None):
    """Causal attention of packed rows with the output gate (gattn_prompt_attention).

    q [T][H][d] bf16.  Without cache_pos: k, v [Tk][Hk][d] bf16 packed by cu_kv
    (default cu_rows).  With cache_pos int32 [n]: k, v are caches [B][Hk][rows][d]
    bf16 that already hold the new rows, slots int32 [n] their cache rows.  gate
    [T][H][d] fp32 or bf16 before its sigmoid, or None.  scale defaults to
    d ** -0.5; max_kv is a hint; status int32 [1].  Returns out, bf16 [T][H][d]."""
    dev = q.get_device()
    qa = _rows(q, "q", dev, _BF16)
    T, H, d = shape = q.shape
    if cache_pos is not None:
        ka = _planes(k, "k", dev, _BF16)
        B, Hk, rows, _ = k.shape
        va = _planes(v, "v", dev, _BF16, (B, Hk, rows, d))
    else:
        ka = _rows(k, "k", dev, _BF16) + (8,)
        B, (rows, Hk, _) = 1, k.shape
        va = _rows(v, "v", dev, _BF16, (rows, Hk, d)) + (8,)
    if k.shape[-1] != d:
        _refuse(k, "k", dev, _BF16, d, "must have q's head_dim")
    if gate is not None:
        ga, gdt = _rows(gate, "gate", dev, _DTYPES, shape), _DTYPES[gate.dtype]
    else:
        ga, gdt = (0, 8, 8), gattn.DTYPE_BF16
    if out is None:
        out = _output(shape, q, stream)
    oa = _rows(out, "out", dev, _BF16, shape)
    cu, n = _cu(cu_rows, "cu_rows", dev)
    ckv = 0
    if cu_kv is not None:
        ckv, nk = _cu(cu_kv, "cu_kv", dev)
        if nk != n:
            _refuse(cu_kv, "cu_kv", dev, _I32, n + 1, "must have cu_rows's length")
    if rows == 0:
        # a tensor without keys: no address, and rows that ask for some are skipped
        ka = va = (0, 8, 8, 8)
        B = max(B, 1)
    desc = gattn.gattn_prompt_attention_desc.pack(
        H, Hk, d, d ** -0.5 if scale is None else scale, n, T, cu, ckv,
        _flat(cache_pos, "cache_pos", dev, _I32, n), _flat(slots, "slots", dev, _I32, n), qa[0],
        qa[1], qa[2], ka[0], va[0], B, rows, ka[1], ka[2], ka[3], va[1], va[2], va[3], ga[0], gdt,
        max_kv, ga[1], ga[2], oa[0], oa[1], oa[2], _flat(status, "status", dev, _I32, 1))
    if n and T:
        _call(gattn.prompt_attention, desc, dev, stream)
    return out


def _per_head(t, name, dev, T, Hv):
    """(address, row stride) of g or beta."""
    if (not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not torch.float32 or
            t.shape != (T, Hv)):
        _refuse(t, name, dev, _F32, (T, Hv))
    st = t.stride()
    if st[1] != 1 and Hv > 1:
        _refuse(t, name, dev, _F32, (T, Hv))
    return t.data_ptr(), st[0] if T > 1 else Hv


def _states(t, name, dev, Hv, dk, dv):
    """(address, slots, slot stride) of a state tensor."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not torch.float32:
        _refuse(t, name, dev, _F32, ("slots", Hv, dk, dv))
    n = t.shape[0] if t.dim() == 4 else 0
    if n < 1 or t.shape != (n, Hv, dk, dv) or not (t.is_contiguous() or t[0].is_contiguous()):
        _refuse(t, name, dev, _F32, ("slots", Hv, dk, dv))
    return t.data_ptr(), n, t.stride(0) if n > 1 else Hv * dk * dv


def _delta(fn, q, k, v, g, beta, cu_rows, num_seqs, state, state_out, slots, scale, qk_l2norm,
           l2_eps, out, status, stream):
    dev = q.get_device()
    qp, qt, qh = _rows(q, "q", dev, _BF16)
    T, Hk, dk = shape = q.shape
    kp, kt, kh = _rows(k, "k", dev, _BF16, shape)
    vp, vt, vh = _rows(v, "v", dev, _BF16)
    Tv, Hv, dv = v.shape
    if Tv != T:
        _refuse(v, "v", dev, _BF16, T, "must have q's rows:")
    gp, gt = _per_head(g, "g", dev, T, Hv)
    bp, bt = _per_head(beta, "beta", dev, T, Hv)
    if cu_rows is not None:
        cu, n = _cu(cu_rows, "cu_rows", dev)
        if num_seqs is not None and num_seqs != n:
            raise ValueError("num_seqs and cu_rows disagree")
    elif num_seqs is None:
        raise ValueError("num_seqs is needed without cu_rows")
    else:
        cu, n = 0, num_seqs
    sp = so = nslots = stride = 0
    if state is not None:
        sp, nslots, stride = _states(state, "state", dev, Hv, dk, dv)
    if state_out is not None:
        so, n_out, stride_out = _states(state_out, "state_out", dev, Hv, dk, dv)
        if sp and (n_out != nslots or stride_out != stride):
            raise ValueError("state and state_out must have one shape and stride")
        nslots, stride = n_out, stride_out
    if out is None:
        out = _output((T, Hv, dv), q, stream)
    op, ot, oh = _rows(out, "out", dev, _BF16, (T, Hv, dv))
    desc = gattn.gattn_delta_desc.pack(
        Hk, Hv, dk, dv, dk ** -0.5 if scale is None else scale, 1 if qk_l2norm else 0, l2_eps, n, T,
        nslots, cu, _flat(slots, "slots", dev, _I32, n), qp, kp, vp, qt, qh, kt, kh, vt, vh, gp, bp,
        gt, bt, sp, so, stride, op, ot, oh, _flat(status, "status", dev, _I32, 1))
    if n:
        _call(fn, desc, dev, stream)
    return out


def delta_prompt(q, k, v, g, beta, cu_rows=None, *, num_seqs=None, state=None, state_out=None,
                 slots=None, scale=None, qk_l2norm=False, l2_eps=1e-6, out=None, status=None,
                 stream=None):
    """The gated delta rule over packed prompts (gattn_delta_prompt).

    q, k [T][Hk][dk] and v [T][Hv][dv] bf16; g (log decay) and beta fp32 [T][Hv];
    cu_rows int32 [n + 1], or num_seqs sequences of T / num_seqs rows; state and
    state_out fp32 [slots][Hv][dk][dv] (one tensor for both: in place); slots
    int32 [n].  scale defaults to dk ** -0.5.  Returns out, bf16 [T][Hv][dv]."""
    return _delta(gattn.delta_prompt, q, k, v, g, beta, cu_rows, num_seqs, state, state_out, slots,
                  scale, qk_l2norm, l2_eps, out, status, stream)


def delta_step(q, k, v, g, beta, cu_rows=None, *, num_seqs=None, state=None, state_out=None,
               slots=None, scale=None, qk_l2norm=False, l2_eps=1e-6, out=None, status=None,
               stream=None):
    """The gated delta rule for one to a few new rows of many sequences
    (gattn_delta_step); arguments as delta_prompt."""
    return _delta(gattn.delta_step, q, k, v, g, beta, cu_rows, num_seqs, state, state_out, slots,
                  scale, qk_l2norm, l2_eps, out, status, stream)
