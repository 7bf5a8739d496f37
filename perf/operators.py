"""Cases of the query/key preparation and sink-window attention operators, with their plain forms.

  rope   rotary positions on the heads of one activation (forward, or the
         inverse rotation that is its gradient)
  qk     per-head norm of queries and keys with the rotation in the same
         pass; ``train`` adds its gradients
  sink   attention with a sliding window and a few first tokens that stay
         visible, over packed sequences; ``train`` adds its gradients
  step   one new token per sequence over a rolling cache of sinks and window,
         the new key and value written into their slot

Activations are row-major [rows, heads * d], head h at columns [h d, (h+1) d).
"""

import math

import torch

own = False

EPS = 1e-6
BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _rope(name, rows, heads, d, rot, layout, dtype, start, scaling, inverse):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "d": d, "rot": rot,
            "layout": layout, "dtype": dtype, "start": start, "scaling": scaling, "factor": 8.0,
            "inverse": inverse}


def _qk(name, train, frames, tokens, heads, kv_heads, d, rot, axes, layout, q_norm, k_norm, dtype):
    return {"name": name, "op": "qk", "train": train, "frames": frames, "tokens": tokens,
            "heads": heads, "kv_heads": kv_heads, "d": d, "rot": rot, "axes": axes,
            "layout": layout, "q_norm": q_norm, "k_norm": k_norm, "dtype": dtype}


def _sink(name, train, lens_q, lens_k, heads, kv_heads, d, window, sinks, ahead):
    return {"name": name, "op": "sink", "train": train, "lens_q": lens_q, "lens_k": lens_k,
            "heads": heads, "kv_heads": kv_heads, "d": d, "window": window, "sinks": sinks,
            "ahead": ahead}


def _step(name, batch, heads, kv_heads, d, window, sinks, pos_lo, pos_hi):
    return {"name": name, "op": "step", "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "d": d, "window": window, "sinks": sinks, "pos_lo": pos_lo, "pos_hi": pos_hi}


def listed():
    return [
        # the queries of one token of 8 streams, far into a long stream: latency
        _rope("rope_token", 8, 16, 128, 128, "half", "bf16", 1000000, "none", False),
        # the layer's heads over a long stream, half of each head rotated, context stretched
        _rope("rope_long", 32768, 24, 128, 64, "interleaved", "bf16", 0, "yarn", False),
        # an odd row count in single precision, the gradient's direction
        _rope("rope_grad_odd", 5003, 6, 64, 64, "half", "fp32", 77, "ntk", True),
        # 42 latent frames at the sweep's 1008 tokens: q RMS-normed, keys of unit length, as the
        # delta rule takes them, rotated by frame, row and column
        _qk("qk_video", False, 42, 1008, 24, 24, 128, 128, 3, "interleaved", "rms", "l2", "bf16"),
        # a ragged training step of shared key heads
        _qk("qk_train_shared", True, 1, 9001, 16, 4, 64, 32, 1, "half", "rms", "rms", "fp16"),
        # the training step of the layer's own heads
        _qk("qk_train_video", True, 10, 1008, 24, 24, 128, 128, 3, "half", "rms", "l2", "bf16"),
        # a training step of three short packed sequences looking both ways
        _sink("sink_packed", True, "700,1,323", "700,1,323", 6, 6, 64, 129, 5, 128),
        # one chunk of 64 new tokens behind a long context, nothing forgotten
        _sink("sink_chunk", False, "64", "24000", 16, 4, 128, 1 << 30, 0, 0),
        # a long stream with shared key heads
        _sink("sink_long", False, "16384", "16384", 16, 4, 128, 4096, 4, 0),
        # a training step over packed sequences of odd lengths
        _sink("sink_train", True, "4097,2500,1500", "4097,2500,1500", 16, 4, 128, 1024, 4, 0),
        # one token of one stream: latency
        _step("step_one", 1, 24, 24, 128, 1020, 4, 5000, 5001),
        # a batch of streams of different ages
        _step("step_batch", 32, 32, 8, 128, 4088, 8, 100, 12000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "qk", "sink", "step"])
    if op == "rope":
        d = rng.choice([32, 64, 96, 128, 256])
        rot = rng.choice([d, d // 2, 8 * rng.randint(1, d // 8)])
        heads = rng.randint(1, 32)
        rows = _log(rng, 1, min(40000, 90000000 // (heads * d)))
        c = _rope("", rows, heads, d, rot, rng.choice(["half", "interleaved"]),
                  rng.choice(["bf16", "bf16", "fp16", "fp32"]), rng.choice([0, _log(rng, 1, 2000000)]),
                  rng.choice(["none", "linear", "ntk", "yarn"]), rng.random() < 0.4)
    elif op == "qk":
        d = rng.choice([32, 64, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        axes = rng.choice([1, 3])
        rot = d if axes == 3 else rng.choice([d, d // 2])
        frames = rng.randint(1, 40)
        tokens = _log(rng, 1, max(2, 60000000 // (2 * heads * d * frames)))
        c = _qk("", rng.random() < 0.5, frames, tokens, heads, kv, d, rot, axes,
                rng.choice(["half", "interleaved"]), rng.choice(["rms", "l2"]),
                rng.choice(["rms", "l2"]), rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    elif op == "sink":
        train = rng.random() < 0.5
        n = rng.choice([1, 1, 2, 3, 5])
        most = 7000 if train else 12000
        lens_k = [_log(rng, 1, most // n) for _ in range(n)]
        lens_q = list(lens_k)
        if rng.random() < 0.3:  # chunks behind a context
            lens_q = [rng.randint(1, x) for x in lens_k]
        kv = rng.choice([1, 2, 4])
        c = _sink("", train, ",".join(map(str, lens_q)), ",".join(map(str, lens_k)),
                  kv * rng.choice([1, 2, 4]), kv, rng.choice([64, 128]), _log(rng, 1, 9000),
                  rng.choice([0, 1, 4, rng.randint(0, 300)]), rng.choice([0, 0, rng.randint(1, 2000)]))
    else:
        kv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 48)
        window = _log(rng, 1, 4000)
        lo = _log(rng, 1, 6000) - 1
        c = _step("", batch, kv * rng.choice([1, 2, 4, 8]), kv, rng.choice([64, 128]), window,
                  rng.choice([0, 1, 4, rng.randint(0, 64)]), lo, lo + _log(rng, 1, 8000))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _frequencies(case):
    """(radians per position of each rotated pair, in 64 bits; its axis; the scale of cos and sin)."""
    rot = case["rot"]
    if case.get("axes", 1) == 3:  # frame, row, column: the frame takes what thirds leave over
        third = rot // 2 // 3
        sections = [rot // 2 - 2 * third, third, third]
    else:
        sections = [rot // 2]
    freq, axis = [], []
    scaling, factor = case.get("scaling", "none"), case.get("factor", 1.0)
    scale = 1.0
    for a, n in enumerate(sections):
        dim = 2 * n
        base = BASE * factor ** (dim / (dim - 2)) if scaling == "ntk" and dim > 2 else BASE
        f = [base ** (-2.0 * i / dim) for i in range(n)]
        if scaling == "linear":
            f = [x / factor for x in f]
        if scaling == "yarn":
            def turn(b):  # the pair that turns b times over the original 4096 positions
                return dim * math.log(4096 / (b * 2 * math.pi)) / (2 * math.log(BASE))
            low, high = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), dim - 1)
            ramp = [min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0) for i in range(n)]
            f = [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)]
            scale = 0.1 * math.log(factor) + 1.0
        freq += f
        axis += [a] * n
    return (torch.tensor(freq, dtype=torch.float64, device="cuda"),
            torch.tensor(axis, dtype=torch.int64, device="cuda"), scale, sections)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _positions(case):
    if case["op"] == "rope":
        return torch.arange(case["start"], case["start"] + case["rows"], dtype=torch.int32,
                            device="cuda")[None]
    t, n = case["frames"], case["tokens"]
    if case["axes"] == 1:
        return torch.arange(t * n, dtype=torch.int32, device="cuda")[None]
    width = max(1, math.isqrt(n))
    i = torch.arange(t * n, dtype=torch.int32, device="cuda")
    return torch.stack([i // n, i % n // width, i % n % width])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    op, h, d = case["op"], case["heads"], case["d"]
    st = {"case": case}
    if op in ("rope", "qk"):
        st["positions"] = _positions(case)
        st["freq"], st["axis"], st["scale"], st["sections"] = _frequencies(case)
        dtype = DTYPES[case["dtype"]]
    if op == "rope":
        st["x"] = normal(case["rows"], h * d, dtype=dtype)
    elif op == "qk":
        rows, g = case["frames"] * case["tokens"], case["kv_heads"]
        st["q"], st["k"] = normal(rows, h * d, dtype=dtype), normal(rows, g * d, dtype=dtype)
        st["wq"] = 1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")
        st["wk"] = 1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda")
        if case["train"]:
            st["dq"], st["dk"] = normal(rows, h * d, dtype=dtype), normal(rows, g * d, dtype=dtype)
    elif op == "sink":
        lens_q, lens_k, g = _ints(case["lens_q"]), _ints(case["lens_k"]), case["kv_heads"]
        st["cu_q"], st["cu_k"] = _cu(lens_q), _cu(lens_k)
        nq, nk = sum(lens_q), sum(lens_k)
        st["q"] = normal(nq, h * d)
        st["k"], st["v"] = normal(nk, g * d), normal(nk, g * d)
        if case["train"]:
            st["d_o"] = normal(nq, h * d, scale=0.1)
    else:
        b, g, slots = case["batch"], case["kv_heads"], case["sinks"] + case["window"]
        st["q"] = normal(b, h * d)
        st["k_new"], st["v_new"] = normal(b, g * d), normal(b, g * d)
        st["k_cache"], st["v_cache"] = normal(b, slots, g * d), normal(b, slots, g * d)
        st["positions"] = torch.tensor(_step_positions(case), dtype=torch.int32, device="cuda")
    return st


def _step_positions(case):
    b, lo, hi = case["batch"], case["pos_lo"], case["pos_hi"]
    return [lo + i * (hi - lo) // b for i in range(b)]


# ---------------------------------------------------------------- plain forms

def _cos_sin(st, inverse=False):
    """[rows, 1, rot / 2] each; the angles in 64 bits, since positions run into the millions."""
    angle = st["positions"][st["axis"]].double().T * st["freq"]
    sin = torch.sin(angle) * st["scale"]
    return ((torch.cos(angle) * st["scale"]).float()[:, None],
            (-sin if inverse else sin).float()[:, None])


def _rotate(x, cos, sin, rot, layout):
    """x [rows, heads, d] in 32 bits."""
    y = x.clone()
    if layout == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(st):
    c = st["case"]
    cos, sin = _cos_sin(st, c["inverse"])
    x = st["x"].float().view(c["rows"], c["heads"], c["d"])
    return _rotate(x, cos, sin, c["rot"], c["layout"]).to(st["x"].dtype).view_as(st["x"])


def _plain_norm(x, w, heads, kind, cos, sin, c):
    x = x.float().view(x.shape[0], heads, c["d"])
    r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) * (1.0 / c["d"] if kind == "rms" else 1.0)
                         + EPS)
    return _rotate(x * r * w, cos, sin, c["rot"], c["layout"])


def _plain_norm_grad(x, w, g, heads, kind, cos, sin, c):
    x = x.float().view(x.shape[0], heads, c["d"])
    m = 1.0 / c["d"] if kind == "rms" else 1.0
    r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) * m + EPS)
    g = _rotate(g.float().view_as(x), cos, -sin, c["rot"], c["layout"])
    dw = (g * x * r).sum(0).sum(0)
    gw = g * w
    dx = r * gw - x * (r * r * r * m * (gw * x).sum(-1, keepdim=True))
    return dx, dw


def _plain_qk(st):
    c = st["case"]
    cos, sin = _cos_sin(st)
    sides = ((st["q"], st["wq"], c["heads"], c["q_norm"], "dq"),
             (st["k"], st["wk"], c["kv_heads"], c["k_norm"], "dk"))
    out = [_plain_norm(x, w, h, kind, cos, sin, c).to(x.dtype).view_as(x)
           for x, w, h, kind, _ in sides]
    if c["train"]:
        grads = [_plain_norm_grad(x, w, st[g], h, kind, cos, sin, c)
                 for x, w, h, kind, g in sides]
        out += [dx.to(x.dtype).view_as(x) for (dx, _), (x, *_) in zip(grads, sides)]
        out += [dw for _, dw in grads]
    return out


def _hidden(st):
    """[Lq, Lk] true where a query must not see a key: another sequence's, ahead, or left behind."""
    c = st["case"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    i = torch.arange(st["q"].shape[0], device="cuda")
    j = torch.arange(st["k"].shape[0], device="cuda")
    bq = torch.searchsorted(cu_q[1:], i, right=True)
    bk = torch.searchsorted(cu_k[1:], j, right=True)
    # a query's position counts from its sequence's first key; the last query has the last position
    p = (i - cu_q[bq + 1] + cu_k[bq + 1] - cu_k[bq])[:, None]
    j = (j - cu_k[bk])[None]
    seen = (j <= p + c["ahead"]) & ((p - j < c["window"]) | (j < c["sinks"]))
    return ~(seen & (bq[:, None] == bk[None]))


def _plain_sink(st):
    c = st["case"]
    h, g, d = c["heads"], c["kv_heads"], c["d"]
    nq, nk = st["q"].shape[0], st["k"].shape[0]
    scale = d ** -0.5
    hidden = _hidden(st)

    def heads_first(x, n):  # [n heads, rows, d], key heads beside their group of query heads
        return x.float().view(x.shape[0], n, d).transpose(0, 1)

    q = heads_first(st["q"], h).reshape(g, h // g * nq, d)
    k, v = heads_first(st["k"], g), heads_first(st["v"], g)
    s = torch.matmul(q, k.transpose(1, 2)).mul_(scale).view(h, nq, nk)
    s.masked_fill_(hidden, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    p /= torch.where(total == 0, 1.0, total)
    p = p.view(g, -1, nk)

    def rows_first(x, n):
        return x.view(n, -1, d).transpose(0, 1).reshape(-1, n * d)

    o = torch.matmul(p, v)
    out = [rows_first(o, h).bfloat16(), lse]
    if c["train"]:
        d_o = heads_first(st["d_o"], h).reshape(g, -1, d)
        dv = torch.matmul(p.transpose(1, 2), d_o)
        dp = torch.matmul(d_o, v.transpose(1, 2))
        ds = dp.sub_((d_o * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(1, 2), q)
        out += [rows_first(dq, h).bfloat16(), rows_first(dk, g).bfloat16(),
                rows_first(dv, g).bfloat16()]
    return out


def _plain_step(st):
    c = st["case"]
    b, h, g, d = c["batch"], c["heads"], c["kv_heads"], c["d"]
    slots = c["sinks"] + c["window"]
    pos = st["positions"].long()
    slot = torch.where(pos < slots, pos, c["sinks"] + (pos - c["sinks"]) % c["window"])
    row = torch.arange(b, device="cuda")
    st["k_cache"][row, slot] = st["k_new"]
    st["v_cache"][row, slot] = st["v_new"]
    live = torch.arange(slots, device="cuda") <= pos[:, None]  # [b, slots]
    q = st["q"].float().view(b, g, h // g, d)
    k = st["k_cache"].float().view(b, slots, g, d).permute(0, 2, 3, 1)
    v = st["v_cache"].float().view(b, slots, g, d).transpose(1, 2)
    s = torch.matmul(q, k).mul_(d ** -0.5)
    s.masked_fill_(~live[:, None, None], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p / p.sum(-1, keepdim=True), v)
    return [o.reshape(b, h * d).bfloat16(), st["k_cache"], st["v_cache"]]


# ---------------------------------------------------------------- the framework's calls

def _plan(st):
    """The rotation's plan, built once and kept, as a program does."""
    from video_diffusion_hybrid_vda_b200 import vdn
    c = st["case"]
    if "plan" not in st:
        scaling = c.get("scaling", "none")
        st["plan"] = vdn.RopePlan(c["d"], rot=c["rot"], base=BASE, layout=c["layout"],
                                  sections=st["sections"] if len(st["sections"]) > 1 else None,
                                  scaling=None if scaling == "none" else scaling,
                                  factor=c.get("factor", 1.0), original=4096)
    return st["plan"]


def _own_rope(st):
    from video_diffusion_hybrid_vda_b200 import vdn
    c = st["case"]
    return vdn.rope(st["x"], c["heads"], _plan(st), positions=st["positions"],
                    inverse=c["inverse"])


def _own_qk(st):
    from video_diffusion_hybrid_vda_b200 import vdn
    c = st["case"]
    kw = dict(wq=st["wq"], wk=st["wk"], q_norm=c["q_norm"], k_norm=c["k_norm"], eps=EPS,
              positions=st["positions"])
    out = list(vdn.qk_norm_rope(st["q"], st["k"], c["heads"], c["kv_heads"], _plan(st), **kw))
    if c["train"]:
        dq, dk, dwq, dwk, st["ws"] = vdn.qk_norm_rope_backward(
            st["q"], st["k"], st["dq"], st["dk"], c["heads"], c["kv_heads"], _plan(st),
            ws=st.get("ws"), **kw)
        out += [dq, dk, dwq, dwk]
    return out


def _own_sink(st):
    from video_diffusion_hybrid_vda_b200 import vdn
    c = st["case"]
    h, g, d = c["heads"], c["kv_heads"], c["d"]
    kw = dict(window=c["window"], sinks=c["sinks"], ahead=c["ahead"], cu_q=st["cu_q"],
              cu_k=st["cu_k"])
    lse = torch.empty((h, st["q"].shape[0]), dtype=torch.float32, device="cuda")
    o, st["ws"] = vdn.sink_attn(st["q"], st["k"], st["v"], h, g, d, lse=lse, ws=st.get("ws"), **kw)
    out = [o, lse]
    if c["train"]:
        dq, dk, dv, st["ws_grad"] = vdn.sink_attn_backward(
            st["q"], st["k"], st["v"], o, lse, st["d_o"], h, g, d, ws=st.get("ws_grad"), **kw)
        out += [dq, dk, dv]
    return out


def _own_step(st):
    from video_diffusion_hybrid_vda_b200 import vdn
    c = st["case"]
    o = vdn.sink_attn_step(st["q"], st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                           st["positions"], c["heads"], c["kv_heads"], c["d"], c["window"],
                           sinks=c["sinks"])
    return [o, st["k_cache"], st["v_cache"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "qk": _own_qk, "sink": _own_sink, "step": _own_step}[op](state)
    return {"rope": _plain_rope, "qk": _plain_qk, "sink": _plain_sink,
            "step": _plain_step}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(case):
    """Visible (query, key) pairs of one head."""
    n = 0
    for nq, nk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        p = torch.arange(nk - nq, nk, dtype=torch.int64)
        end = (p + case["ahead"] + 1).clamp(0, nk)
        begin = (p - case["window"] + 1).clamp(min=0)
        begin = torch.minimum(begin, end)
        sinks = torch.minimum(begin, torch.tensor(case["sinks"]))
        n += int((end - begin + sinks).sum())
    return n


def work(case):
    op, h, d = case["op"], case["heads"], case["d"]
    if op == "rope":
        n, e = case["rows"] * h * d, 4 if case["dtype"] == "fp32" else 2
        return {"bytes": 2 * n * e + 4 * case["rows"], "flops": 3 * n}
    g = case["kv_heads"]
    if op == "qk":
        rows = case["frames"] * case["tokens"]
        n, e = rows * (h + g) * d, 4 if case["dtype"] == "fp32" else 2
        streams, flops = (5, 18) if case["train"] else (2, 7)  # train: x, dy read, y, dx written;
        return {"bytes": streams * n * e + 4 * rows * case["axes"], "flops": flops * n}  # x again
    if op == "sink":
        nq, nk = sum(_ints(case["lens_q"])), sum(_ints(case["lens_k"]))
        q, kv = nq * h * d * 2, nk * g * d * 2
        pairs = _pairs(case) * h
        if case["train"]:  # q, k, v, o, d_o in; o, dq, dk, dv out; two and five products
            return {"bytes": 5 * q + 4 * kv + 8 * nq * h, "flops": 14 * pairs * d}
        return {"bytes": 2 * q + 2 * kv + 4 * nq * h, "flops": 4 * pairs * d}
    slots = case["sinks"] + case["window"]
    live = sum(min(p + 1, slots) for p in _step_positions(case))
    return {"bytes": live * g * d * 4 + case["batch"] * (2 * h + 4 * g) * d * 2,
            "flops": 4 * live * h * d}


# ---------------------------------------------------------------- the definition in 64 bits

def _turned(x, c, st, conj=False):
    """x [rows, heads, d] in 64 bits, its pairs taken as complex numbers and turned."""
    rot, half = c["rot"], c["rot"] // 2
    angle = st["positions"].double()[st["axis"]].T * st["freq"]
    turn = torch.polar(torch.full_like(angle, st["scale"]), -angle if conj else angle)[:, None]
    if c["layout"] == "half":
        z = torch.complex(x[..., :half], x[..., half:rot]) * turn
        return torch.cat([z.real, z.imag, x[..., rot:]], -1)
    z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)


def _exact_qk(c, st):
    out, grads = [], []
    for x, w, n, kind, g in ((st["q"], st["wq"], c["heads"], c["q_norm"], "dq"),
                             (st["k"], st["wk"], c["kv_heads"], c["k_norm"], "dk")):
        x = x.double().view(-1, n, c["d"]).requires_grad_(c["train"])
        w = w.double().requires_grad_(c["train"])
        sq = x.square().mean(-1, keepdim=True) if kind == "rms" else \
            x.square().sum(-1, keepdim=True)
        y = _turned(x * (sq + EPS).rsqrt() * w, c, st)
        out.append(y.detach().flatten(1))
        if c["train"]:
            dx, dw = torch.autograd.grad(y, [x, w], st[g].double().view_as(y))
            grads.append((dx.flatten(1), dw))
    return out + [dx for dx, _ in grads] + [dw for _, dw in grads]


def _exact_sink(c, st):
    h, g, d = c["heads"], c["kv_heads"], c["d"]
    q, k, v = (st[n].double().view(-1, m, d) for n, m in (("q", h), ("k", g), ("v", g)))
    o, lse = torch.zeros_like(q), torch.full((h, q.shape[0]), -math.inf, dtype=torch.float64,
                                             device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    a = b = 0
    for nq, nk in zip(_ints(c["lens_q"]), _ints(c["lens_k"])):
        p = torch.arange(nk - nq, nk, device="cuda")[:, None]
        j = torch.arange(nk, device="cuda")[None]
        see = (j <= p + c["ahead"]) & ((p - j < c["window"]) | (j < c["sinks"]))
        row = see.any(1)
        for i in range(h):
            e = i // (h // g)
            with torch.set_grad_enabled(c["train"]):
                qi = q[a:a + nq, i].clone().requires_grad_(c["train"])
                ki = k[b:b + nk, e].clone().requires_grad_(c["train"])
                vi = v[b:b + nk, e].clone().requires_grad_(c["train"])
                s = (qi @ ki.T / math.sqrt(d))[row].masked_fill(~see[row], -math.inf)
                oi = torch.softmax(s, -1) @ vi
            if c["train"]:
                got = torch.autograd.grad(
                    oi, [qi, ki, vi], st["d_o"].double().view(-1, h, d)[a:a + nq, i][row])
                dq[a:a + nq, i] += got[0]
                dk[b:b + nk, e] += got[1]
                dv[b:b + nk, e] += got[2]
            at = torch.arange(a, a + nq, device="cuda")[row]
            o[at, i] = oi.detach()
            lse[i, at] = torch.logsumexp(s.detach(), -1)
        a, b = a + nq, b + nk
    out = [o.flatten(1), lse]
    return out + [x.flatten(1) for x in (dq, dk, dv)] if c["train"] else out


def _exact_step(c, st):
    h, g, d, s0, w = c["heads"], c["kv_heads"], c["d"], c["sinks"], c["window"]
    kc, vc = st["k_cache"].double(), st["v_cache"].double()
    rows = []
    for i, p in enumerate(_step_positions(c)):
        at = p if p < s0 + w else s0 + (p - s0) % w
        kc[i, at], vc[i, at] = st["k_new"][i].double(), st["v_new"][i].double()
        n = min(p + 1, s0 + w)
        k = kc[i, :n].view(n, g, d).repeat_interleave(h // g, 1)
        v = vc[i, :n].view(n, g, d).repeat_interleave(h // g, 1)
        s = torch.einsum("hd,nhd->hn", st["q"][i].double().view(h, d), k) / math.sqrt(d)
        rows.append(torch.einsum("hn,nhd->hd", torch.softmax(s, -1), v).flatten())
    return [torch.stack(rows), kc, vc]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        x = st["x"].double().view(case["rows"], case["heads"], case["d"])
        return _turned(x, case, st, case["inverse"]).flatten(1)
    return {"qk": _exact_qk, "sink": _exact_sink, "step": _exact_step}[case["op"]](case, st)
