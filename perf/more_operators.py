"""The paged-cache operators: cases, inputs, a plain form of each and a float64
form written apart from it.

Four operators of decoding over a key-value cache kept in pages: position p of
sequence s is row p % page_size of page table[s][p // page_size].

rows       per-head RMSNorm and rotary embedding (halves or pairs, part of the head,
           frequencies scaled for long contexts) of the projected queries and keys, and
           the append of keys and values at each sequence's next positions
attention  causal attention of one to a few new rows of each sequence over its pages,
           grouped heads, sigmoid output gate; with the log of each softmax's sum
weights    the softmax weight that each cached position received from those rows,
           added to what it had received before
evict      of a sequence's positions the newest and the most attended, per key head,
           moved to the front of other pages in their order

With ``own`` false, ``run`` computes the plain form (elementary torch operations
in 32 bits, 64 for rotary angles); with it true, the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BF = torch.bfloat16

ROPE_THETA, EPS = 1e7, 1e-6
# frequencies stretched for four times the positions that were trained on
YARN = dict(factor=4.0, original=32768, beta_fast=32.0, beta_slow=1.0)


# ------------------------------------------------------------------- cases

def listed():
    g16 = dict(H=16, Hk=4, d=256)
    g24 = dict(H=24, Hk=2, d=256)
    g32 = dict(H=32, Hk=8, d=256)
    d64 = dict(H=16, Hk=8, d=64)
    return [
        # one new token of eight conversations: launch latency
        dict(name="rows_step", op="rows", lens="1,1,1,1,1,1,1,1", past="1003,17,4095,64,2500,333,0,900",
             page=64, rd=64, pairs=False, scaled=False, f32=False, **g16),
        # a full prompt batch appended behind earlier turns, frequencies scaled: streaming
        dict(name="rows_prompt", op="rows", lens="2048,1,1777,3001,513,900", past="0,40950,17,1024,0,333",
             page=16, rd=64, pairs=False, scaled=True, f32=False, **g32),
        # whole heads turned in neighbouring pairs, fp32 projections
        dict(name="rows_pairs", op="rows", lens="700,129,1024,64,333,1,515", past="3,0,700,15,2047,31,1",
             page=48, rd=128, pairs=True, scaled=False, f32=True, H=16, Hk=8, d=128),
        # one new token of one short conversation: launch latency and the join
        dict(name="attn_token", op="attention", lens="1", past="1003", page=64, **g16),
        # one new token behind a very long context: the split over the cache
        dict(name="attn_long", op="attention", lens="1", past="131071", page=64, **g24),
        # a decode batch of uneven lengths: streaming
        dict(name="attn_batch", op="attention", lens="1x32", past="7001,129,2048,15000,64,3333,1,9000,511,4096,"
             "12001,800,6000,250,1777,10240,37,5000,2500,8191,300,14000,950,7777,16,4500,11000,1200,640,3001,9999,0",
             page=16, **g32),
        # drafted rows to verify, and a sequence that only gets one
        dict(name="attn_verify", op="attention", lens="4,4,4,4,4,1,4,4", past="8000,1001,4099,12345,256,30000,2047,6000",
             page=32, **g24),
        # small heads, many sequences
        dict(name="attn_d64", op="attention", lens="1x64", past="x37+211", page=16, **d64),
        # what one new token attended to
        dict(name="weights_token", op="weights", lens="1", past="4000", page=64, **g16),
        # what the rows of a decode batch attended to
        dict(name="weights_batch", op="weights", lens="1,4,1,1,2,4,1,1,1,3,1,1,1,4,1,1",
             past="7001,15000,64,3333,9000,511,4096,12001,800,6000,1777,10240,5000,2500,8191,14000", page=16, **g32),
        # one conversation over its budget
        dict(name="evict_one", op="evict", past="2500", keep=1024, recent=128, page=64, **g16),
        # a batch cut to a quarter, some of it within the budget already
        dict(name="evict_batch", op="evict", past="16000,16384,9001,4000,15000,12345,4097,16001", keep=4096, recent=1024,
             page=16, **g16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rows", "attention", "attention", "attention", "weights", "evict"))
    heads = rng.choice((dict(H=16, Hk=4, d=256), dict(H=24, Hk=2, d=256), dict(H=32, Hk=8, d=256),
                        dict(H=8, Hk=2, d=64), dict(H=16, Hk=8, d=128), dict(H=6, Hk=2, d=192),
                        dict(H=5, Hk=1, d=128)))
    page = rng.choice((16, 16, 32, 48, 64, 128, 256))
    txt = lambda v: ",".join(str(x) for x in v)  # noqa: E731
    if op == "rows":
        total, n = _log(rng, 1, 7000), rng.randint(1, 12)
        share = [rng.expovariate(1.0) + 0.02 for _ in range(n)]
        lens = [max(1, int(total * x / sum(share))) for x in share]
        return dict(op=op, lens=txt(lens), past=txt(rng.choice((0, rng.randint(0, 40000))) for _ in lens), page=page,
                    rd=rng.choice((heads["d"] // 4, heads["d"] // 2, heads["d"], 20)), pairs=rng.random() < 0.5,
                    scaled=rng.random() < 0.5, f32=rng.random() < 0.4, **heads)
    if op == "evict":
        n = rng.randint(1, 6)
        past = [_log(rng, 1, 12000) for _ in range(n)]
        keep = _log(rng, 1, max(past))
        return dict(op=op, past=txt(past), keep=keep, recent=rng.randint(0, keep), page=page, **heads)
    n = _log(rng, 1, 40)
    lens = [1 if rng.random() < 0.6 else rng.randint(1, 6) for _ in range(n)]
    total = _log(rng, 1, 120000)
    share = [rng.expovariate(1.0) for _ in range(n)]
    past = [min(100000, int(total * x / sum(share))) for x in share]
    return dict(op=op, lens=txt(lens), past=txt(past), page=page, **heads)


def _lens(text):
    if text.startswith("1x"):
        return [1] * int(text[2:])
    return [int(x) for x in text.split(",")]


def _past(text):
    """Numbers, or xA+B for 64 uneven ones: A * i * i % 4001 + B."""
    if text.startswith("x"):
        a, b = (int(x) for x in text[1:].split("+"))
        return [a * i * i % 4001 + b for i in range(64)]
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------- inputs

def _cu(lens):
    c = [0]
    for x in lens:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device=DEV)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device=DEV)      # noqa: E731
    op, H, Hk, d, P = case["op"], case["H"], case["Hk"], case["d"], case["page"]
    past = _past(case["past"])
    lens = _lens(case["lens"]) if "lens" in case else [0] * len(past)
    n, T = len(lens), sum(lens)
    s = dict(op=op, case=case, lens=lens, past=past, cu=_cu(lens), pos=_ints(past))
    # a pool of pages with some to spare, handed out in no order
    need = [-(-(a + b) // P) for a, b in zip(lens, past)]
    out = [-(-min(p, case["keep"]) // P) for p in past] if op == "evict" else [0] * n
    pages = sum(need) + sum(out) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    s["table"] = torch.zeros(n, max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b in range(n):
        s["table"][b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    s["kp"] = torch.empty(pages, Hk, P, d, dtype=BF, device=DEV)
    s["vp"] = torch.empty(pages, Hk, P, d, dtype=BF, device=DEV)
    for i in range(0, pages, 1024):
        s["kp"][i:i + 1024] = randn(min(1024, pages - i), Hk, P, d).to(BF)
        s["vp"][i:i + 1024] = randn(min(1024, pages - i), Hk, P, d).to(BF)
    if op == "evict":
        s["out_table"] = torch.zeros(n, max(max(out), 1), dtype=torch.int32, device=DEV)
        for b in range(n):
            s["out_table"][b, :out[b]] = order[at:at + out[b]]
            at += out[b]
        L = max(past)
        # received weight falls off steeply, as it does: a few positions have most of it
        s["w"] = torch.exp(2.5 * randn(n, Hk, L) - 6)
        s["w_out"] = torch.zeros(n, Hk, case["keep"], device=DEV)
        s["kept"] = torch.zeros(n, Hk, case["keep"], dtype=torch.int32, device=DEV)
        s["len_out"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        return s
    if op == "rows":
        # one projection output per row: per head query | gate, then the keys and values
        y = randn(T, 2 * H * d + 2 * Hk * d)
        y = y if case["f32"] else y.to(BF)
        s["q"] = y[:, :2 * H * d].view(T, H, 2 * d)[..., :d]
        s["k"] = y[:, 2 * H * d:2 * H * d + Hk * d].view(T, Hk, d)
        s["v"] = y[:, 2 * H * d + Hk * d:].view(T, Hk, d)
        s["qn"] = (1 + 0.1 * randn(d)).to(BF)
        s["kn"] = (1 + 0.1 * randn(d)).to(BF)
        s["q_out"] = torch.zeros(T, H, d, dtype=BF, device=DEV)
        return s
    s["q"] = randn(T, H, d).to(BF)
    s["scale"] = d ** -0.5
    if op == "attention":
        s["gate"] = randn(T, H, 2 * d).to(BF)[..., d:]      # beside the raw queries
        s["out"] = torch.zeros(T, H, d, dtype=BF, device=DEV)
        s["lse"] = torch.zeros(T, H, device=DEV)
        if own:
            from qwen3_gated_attention_gb300 import device
            s["ws"] = device.paged_attention_workspace(s["q"], s["kp"], s["cu"])
        return s
    # the log sums that the attention gave
    L = max(a + b for a, b in zip(lens, past))
    s["lse"] = torch.full((T, H), -math.inf, device=DEV)
    for b, t0 in enumerate(s["cu"].tolist()[:-1]):
        for i in range(lens[b]):
            k = _seen(s["kp"], s["table"], b, past[b] + i + 1).repeat_interleave(H // Hk, 0)
            s["lse"][t0 + i] = torch.logsumexp((k @ s["q"][t0 + i].float()[:, :, None])[..., 0] * s["scale"], -1)
    s["w"] = torch.exp(2.5 * randn(n, Hk, L) - 6)
    s["w_out"] = torch.zeros(n, Hk, L, device=DEV)
    return s


def _seen(pool, table, b, m):
    """The first m positions of sequence b in fp32: [Hk][m][d]."""
    P = pool.shape[2]
    x = pool[table[b, :-(-m // P)].long()].transpose(0, 1)
    return x.reshape(x.shape[0], -1, x.shape[-1])[:, :m].float()


# ---------------------------------------------------------------- plain form

def _where(cu, T):
    """Sequence and place within it of each packed row."""
    t = torch.arange(T, device=cu.device)
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    return seq, t - cu[seq]


def _plain_rows(s):
    c = s["case"]
    rd, P = c["rd"], c["page"]
    half = rd // 2
    seq, at = _where(s["cu"], s["q"].shape[0])
    pos = s["pos"][seq] + at
    i = torch.arange(half, device=DEV, dtype=torch.float64)
    inv, size = ROPE_THETA ** (-2.0 * i / rd), 1.0
    if c["scaled"]:
        # as many turns within the trained positions: kept where fast, stretched where slow
        edge = lambda turns: rd * math.log(YARN["original"] / (turns * 2 * math.pi)) / (2 * math.log(ROPE_THETA))  # noqa: E731
        lo = max(math.floor(edge(YARN["beta_fast"])), 0)
        hi = min(math.ceil(edge(YARN["beta_slow"])), rd - 1)
        slow = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        inv = inv * (1 - slow) + inv / YARN["factor"] * slow
        size = 0.1 * math.log(YARN["factor"]) + 1
    ang = pos.double()[:, None] * inv
    cos, sin = (torch.cos(ang) * size).float()[:, None], (torch.sin(ang) * size).float()[:, None]

    def turned(x, w):
        x = x.float()
        x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()
        y = x.clone()
        if c["pairs"]:
            a, b = x[..., 0:rd:2], x[..., 1:rd:2]
            y[..., 0:rd:2], y[..., 1:rd:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :half], x[..., half:rd]
            y[..., :half], y[..., half:rd] = a * cos - b * sin, b * cos + a * sin
        return y

    q, k = turned(s["q"], s["qn"]), turned(s["k"], s["kn"])
    s["q_out"].copy_(q)
    page, row = s["table"][seq, pos // P].long(), pos % P
    s["kp"][page, :, row] = k.to(BF)
    s["vp"][page, :, row] = s["v"].to(BF)
    return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]}


def _padded(s):
    """Queries [n][Hk][rows * group][d], scores' visibility and the row places, per longest row count."""
    c = s["case"]
    H, Hk, d = c["H"], c["Hk"], c["d"]
    n, T, R = len(s["lens"]), sum(s["lens"]), max(s["lens"])
    seq, at = _where(s["cu"], T)
    q = torch.zeros(n, R, H, d, device=DEV).index_put((seq, at), s["q"].float())
    q = q.view(n, R, Hk, H // Hk, d).permute(0, 2, 1, 3, 4).reshape(n, Hk, -1, d)
    m = max(a + b for a, b in zip(s["lens"], s["past"]))
    j, i = torch.arange(m, device=DEV), torch.arange(R, device=DEV)
    seen = j[None, None, :] <= (s["pos"][:, None] + i)[:, :, None]
    return q, seen, seq, at, m, R


def _gathered(s, pool, m):
    x = pool[s["table"][:, :-(-m // pool.shape[2])].long()].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])[:, :, :m].float()


def _plain_attention(s):
    c = s["case"]
    H, Hk, d = c["H"], c["Hk"], c["d"]
    n = len(s["lens"])
    q, seen, seq, at, m, R = _padded(s)
    x = (q @ _gathered(s, s["kp"], m).transpose(-1, -2)).mul_(s["scale"]).view(n, Hk, R, H // Hk, m)
    x.masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    sums = x.sum(-1, keepdim=True)
    lse = (top + sums.log())[..., 0].permute(0, 2, 1, 3).reshape(n, R, H)
    x.div_(sums)
    o = (x.view(n, Hk, -1, m) @ _gathered(s, s["vp"], m)).view(n, Hk, R, H // Hk, d)
    o = o.permute(0, 2, 1, 3, 4).reshape(n, R, H, d)[seq, at]
    s["out"].copy_(o / (1 + torch.exp(-s["gate"].float())))
    s["lse"].copy_(lse[seq, at])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_weights(s):
    c = s["case"]
    H, Hk = c["H"], c["Hk"]
    n = len(s["lens"])
    q, seen, seq, at, m, R = _padded(s)
    lse = torch.full((n, R, H), float("inf"), device=DEV).index_put((seq, at), s["lse"])
    lse = lse.view(n, R, Hk, H // Hk).permute(0, 2, 1, 3)
    x = (q @ _gathered(s, s["kp"], m).transpose(-1, -2)).mul_(s["scale"]).view(n, Hk, R, H // Hk, m)
    x.sub_(lse[..., None]).exp_().masked_fill_(~seen[:, None, :, None], 0)
    x = x.sum((2, 3))
    j = torch.arange(m, device=DEV)
    old = torch.where(j < s["pos"][:, None, None], s["w"], torch.zeros((), device=DEV))
    new = j < (s["pos"] + _ints(s["lens"]))[:, None, None]
    s["w_out"].copy_(torch.where(new, old + x, s["w_out"]))
    return {"weights": s["w_out"]}


def _plain_evict(s):
    c = s["case"]
    n, keep, P = len(s["past"]), c["keep"], c["page"]
    L = s["w"].shape[2]
    j = torch.arange(L, device=DEV)
    length = s["pos"][:, None, None]
    w = torch.where(j >= length - c["recent"], torch.full((), float("inf"), device=DEV), s["w"])
    w = torch.where(j < length, w, torch.full((), float("-inf"), device=DEV))
    m = min(keep, L)
    src = torch.sort(torch.sort(w, dim=-1, descending=True, stable=True)[1][..., :m], dim=-1)[0]
    ok = torch.arange(m, device=DEV) < length                      # as many as the sequence has
    ok = ok.expand(src.shape)
    s["kept"].fill_(-1)
    s["kept"][..., :m] = torch.where(ok, src, torch.full((), -1, device=DEV)).int()
    s["w_out"][..., :m] = torch.where(ok, torch.gather(s["w"], 2, src), s["w_out"][..., :m])
    b, h, i = torch.nonzero(ok, as_tuple=True)
    f = src[b, h, i]
    page, to = s["table"][b, f // P].long(), s["out_table"][b, i // P].long()
    for pool in (s["kp"], s["vp"]):
        pool[to, h, i % P] = pool[page, h, f % P]
    s["len_out"].copy_(s["pos"].clamp(max=keep))
    return {"k_pages": s["kp"], "v_pages": s["vp"], "kept": s["kept"], "weights": s["w_out"], "lengths": s["len_out"]}


def run(s):
    op = s["op"]
    if own:
        from qwen3_gated_attention_gb300 import device
        if op == "rows":
            c = s["case"]
            device.paged_rows(s["q"], s["k"], s["v"], s["kp"], s["vp"], s["table"], s["cu"], s["pos"], q_norm=s["qn"],
                              k_norm=s["kn"], rotary_dims=c["rd"], rope_theta=ROPE_THETA, rope_pairs=c["pairs"],
                              rope_yarn=YARN if c["scaled"] else None, rms_eps=EPS, q_out=s["q_out"])
            return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]}
        if op == "attention":
            device.paged_attention(s["q"], s["kp"], s["vp"], s["table"], s["cu"], s["pos"], gate=s["gate"],
                                   scale=s["scale"], out=s["out"], lse=s["lse"], workspace=s["ws"])
            return {"out": s["out"], "lse": s["lse"]}
        if op == "weights":
            device.paged_weights(s["q"], s["kp"], s["table"], s["cu"], s["pos"], s["lse"], scale=s["scale"],
                                 weights=s["w"], weights_out=s["w_out"])
            return {"weights": s["w_out"]}
        c = s["case"]
        device.paged_evict(s["kp"], s["vp"], s["table"], s["pos"], s["w"], keep=c["keep"], recent=c["recent"],
                           out_table=s["out_table"], weights_out=s["w_out"], kept=s["kept"], lengths_out=s["len_out"])
        return {"k_pages": s["kp"], "v_pages": s["vp"], "kept": s["kept"], "weights": s["w_out"], "lengths": s["len_out"]}
    return {"rows": _plain_rows, "attention": _plain_attention, "weights": _plain_weights, "evict": _plain_evict}[op](s)


# ---------------------------------------------------------------------- work

def work(case):
    op, H, Hk, d = case["op"], case["H"], case["Hk"], case["d"]
    past = _past(case["past"])
    if op == "evict":
        kept = sum(min(p, case["keep"]) for p in past)
        # weights read; what is kept moved and named
        return {"bytes": 4 * Hk * sum(past) + Hk * kept * (8 * d + 8), "flops": 0}
    lens = _lens(case["lens"])
    T = sum(lens)
    if op == "rows":
        x = 4 if case["f32"] else 2
        return {"bytes": (x + 2) * T * (H + 2 * Hk) * d + 4 * d, "flops": 8 * T * (H + Hk) * d}
    pairs = sum(x * p + x * (x + 1) // 2 for x, p in zip(lens, past))
    kv = sum(x + p for x, p in zip(lens, past))
    if op == "attention":
        return {"bytes": 2 * d * (3 * T * H + 2 * kv * Hk) + 4 * T * H, "flops": 4 * d * H * pairs}
    return {"bytes": 2 * d * (T * H + kv * Hk) + 4 * T * H + 8 * kv * Hk, "flops": 2 * d * H * pairs}


# ------------------------------------------------------------- float64 form

def _frequencies(rd, scaled):
    """(angle per position of each turned pair, size of the turned part), pair by pair."""
    out = []
    for i in range(rd // 2):
        f = math.exp(-2.0 * i / rd * math.log(ROPE_THETA))
        if scaled:
            border = []
            for turns, whole in ((YARN["beta_fast"], math.floor), (YARN["beta_slow"], math.ceil)):
                border.append(whole(rd / 2 * math.log(YARN["original"] / (2 * math.pi * turns)) / math.log(ROPE_THETA)))
            lo, hi = max(border[0], 0), min(border[1], rd - 1)
            mix = min(max((i - lo) / ((hi - lo) or 1e-3), 0.0), 1.0)
            f = f * ((1 - mix) + mix / YARN["factor"])
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device=DEV), 1 + 0.1 * math.log(YARN["factor"]) if scaled else 1.0


def _exact_rows(s):
    c = s["case"]
    rd, P = c["rd"], c["page"]
    freq, size = _frequencies(rd, c["scaled"])
    kc, vc = s["kp"].double(), s["vp"].double()
    cu = s["cu"].tolist()
    qs = []
    for b, (n, p) in enumerate(zip(s["lens"], s["past"])):
        a = slice(cu[b], cu[b] + n)
        where = torch.arange(p, p + n, device=DEV)
        turn = torch.polar(torch.full((), size, dtype=torch.float64, device=DEV), where.double()[:, None, None] * freq)
        both = []
        for x, w in ((s["q"][a].double(), s["qn"].double()), (s["k"][a].double(), s["kn"].double())):
            x = w * x / torch.sqrt(torch.einsum("thd,thd->th", x, x)[..., None] / c["d"] + EPS)
            if c["pairs"]:
                z = torch.view_as_complex(x[..., :rd].unflatten(-1, (rd // 2, 2)).contiguous()) * turn
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) * turn
                y = torch.cat((z.real, z.imag), -1)
            both.append(torch.cat((y, x[..., rd:]), -1))
        qs.append(both[0])
        page = s["table"][b].long()[where // P]
        kc[page, :, where % P] = both[1]
        vc[page, :, where % P] = s["v"][a].double()
    return {"q": torch.cat(qs), "k_pages": kc, "v_pages": vc}


def _exact_scores(s, b, m):
    """Scaled scores [Hk][group][rows][m] of sequence b, hidden ones -inf."""
    c = s["case"]
    H, Hk, d = c["H"], c["Hk"], c["d"]
    t0, n = int(s["cu"][b]), s["lens"][b]
    k = _seen(s["kp"], s["table"], b, m).double()
    q = s["q"][t0:t0 + n].double().view(n, Hk, H // Hk, d)
    x = torch.einsum("ikgd,kjd->kgij", q, k) / math.sqrt(d)
    hidden = torch.ones(n, m, dtype=torch.bool, device=DEV).triu(m - n + 1)
    return x.masked_fill(hidden, -math.inf), slice(t0, t0 + n)


def _exact_attention(s):
    c = s["case"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"]):
        m = n + s["past"][b]
        x, rows = _exact_scores(s, b, m)
        v = _seen(s["vp"], s["table"], b, m).double()
        lse[rows] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(n, c["H"])
        out[rows] = torch.einsum("kgij,kjd->ikgd", torch.softmax(x, -1), v).reshape(n, c["H"], c["d"])
    return {"out": out * torch.sigmoid(s["gate"].double()), "lse": lse}


def _exact_weights(s):
    c = s["case"]
    Hk, g = c["Hk"], c["H"] // c["Hk"]
    out = s["w_out"].double()
    for b, n in enumerate(s["lens"]):
        p = s["past"][b]
        x, rows = _exact_scores(s, b, n + p)
        lse = s["lse"][rows].double().view(n, Hk, g).permute(1, 2, 0)[..., None]
        out[b, :, :n + p] = torch.exp(x - lse).sum((1, 2))
        out[b, :, :p] += s["w"][b, :, :p].double()
    return {"weights": out}


def _exact_evict(s):
    c = s["case"]
    keep, P = c["keep"], c["page"]
    kc, vc, w = s["kp"].double(), s["vp"].double(), s["w_out"].double()
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int32)
    got = s["w"].double().cpu().tolist()
    for b, length in enumerate(s["past"]):
        m = min(length, keep)
        for h in range(c["Hk"]):
            old = range(max(length - c["recent"], 0))
            best = sorted(old, key=lambda i: (-got[b][h][i], i))[:m - min(c["recent"], m)]
            at = sorted(best) + list(range(length - (m - len(best)), length))
            kept[b, h, :m] = torch.tensor(at, dtype=torch.int32)
            f, t = torch.tensor(at, dtype=torch.int64, device=DEV), torch.arange(m, device=DEV)
            w[b, h, :m] = s["w"][b, h, f].double()
            src, dst = s["table"][b].long()[f // P], s["out_table"][b].long()[t // P]
            kc[dst, h, t % P] = s["kp"][src, h, f % P].double()
            vc[dst, h, t % P] = s["vp"][src, h, f % P].double()
    return {"k_pages": kc, "v_pages": vc, "kept": kept.to(DEV), "weights": w,
            "lengths": _ints([min(x, keep) for x in s["past"]])}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rows": _exact_rows, "attention": _exact_attention, "weights": _exact_weights, "evict": _exact_evict}[s["op"]](s)
