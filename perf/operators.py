"""The operators around the attention of a video transformer block, and how they are measured.

Three operators, each in its plain form (elementary torch operations in 32 bits) and as the
library's call:

* ``norm_rope``: the norm of every head's query and key (RMS or layer norm over the head's d
  elements) and the rotation by the token's position, in one pass, from the packed projection
  [batch, token, heads, d] to the attention's layout [batch, heads, token, d]; with ``back`` its
  gradients.  ``norm`` = "none" is the rotation alone.
* ``append``: the same on the way into a paged cache of keys and values, for ragged sequences.
* ``attn``: attention of each sequence's newest tokens over its paged cache.

Positions have one axis (a text's or a token stream's) or three (frame, row, column of the latent
grid); tokens behind the grid (text) are not rotated.
"""
import math

import torch

own = False

EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    rope3 = dict(layout="interleaved", theta=10000.0, scaling="none", factor=1.0, orig=0, far=0)
    wan = dict(heads=40, kv_heads=40, d=128, dtype="bf16", norm="rms", bias=False, dims="44,42,42",
               grid="21,45,80", **rope3)
    cog = dict(heads=30, kv_heads=30, d=64, dtype="bf16", norm="layer", bias=True, dims="16,24,24",
               grid="13,30,45", **rope3)
    text = dict(heads=32, kv_heads=8, d=128, dtype="bf16", norm="none", bias=False, dims="64", grid="131072",
                layout="half", theta=500000.0, scaling="yarn", factor=16.0, orig=8192, far=65536)
    gqa = dict(heads=32, kv_heads=8, d=128, dtype="bf16", page=16)
    return [
        # one new token between two attention calls: latency alone counts
        dict(name="norm_rope_one_token", op="norm_rope", back=False, batch=1, n=1, **wan),
        # every token of the headline attention call, all 40 heads
        dict(name="norm_rope_75600", op="norm_rope", back=False, batch=1, n=75600, **wan),
        # layer norm with a bias, 226 text tokens behind the grid that are not rotated
        dict(name="norm_rope_text_17776", op="norm_rope", back=False, batch=1, n=17776, **cog),
        # rotation alone: half layout, half of the head, shared heads, far positions scaled for a long context
        dict(name="rope_long_half", op="norm_rope", back=False, batch=2, n=9001, **text),
        # the gradients of a training step, two samples, with those of weights and biases
        dict(name="norm_rope_back_17776", op="norm_rope", back=True, batch=2, n=17776, **cog),
        # gradients in 32 bits, an odd number of tokens and of heads
        dict(name="norm_rope_back_f32", op="norm_rope", back=True, batch=1, n=2049,
             **{**wan, "heads": 5, "kv_heads": 5, "dtype": "f32"}),
        # one token of each of 16 sequences goes into the cache
        dict(name="append_16_tokens", op="append", seqs=16, new=1, kv=4099, ragged=True, page=16,
             **{**text, "norm": "rms", "scaling": "none", "dims": "128", "far": 0}),
        # three latent frames of every head go into the cache behind three earlier ones
        dict(name="append_3_frames", op="append", seqs=1, new=10800, kv=21600, ragged=False, page=64, **wan),
        # one new token over a short cache: latency alone counts
        dict(name="attn_one_token", op="attn", seqs=1, new=1, kv=777, ragged=False, block=1, window=0, **gqa),
        # one new token of each of 16 sequences of different lengths: the cache is read once
        dict(name="attn_16_tokens", op="attn", seqs=16, new=1, kv=8191, ragged=True, block=1, window=0, **gqa),
        # one or two frames of two sequences, causal by whole frames of 30 x 45 tokens
        dict(name="attn_frames_d64", op="attn", seqs=2, new=2700, kv=17550, ragged=True, block=1350, window=0,
             heads=30, kv_heads=30, d=64, dtype="bf16", page=32),
        # the last frame (45 x 80 tokens) of a clip over the whole clip, 40 heads
        dict(name="attn_frame_75600", op="attn", seqs=1, new=3600, kv=75600, ragged=False, block=3600, window=0,
             heads=40, kv_heads=40, d=128, dtype="bf16", page=128),
    ]


def draw(rng):
    def size(lo, hi):  # spread over the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm_rope", "norm_rope", "append", "attn", "attn"])
    d = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 3, 5, 8, 12, 16, 30, 40])
    group = rng.choice([1, 1, 1, 2, 4, 5, 8]) if kv_heads <= 8 else 1
    c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, d=d,
             dtype="bf16" if op == "attn" else rng.choice(["bf16", "bf16", "f32"]))
    if op == "attn":
        c.update(seqs=size(1, 32), ragged=rng.random() < 0.7, page=rng.choice([16, 32, 64, 128]))
        c["kv"] = size(1, 70000)
        c["new"] = min(c["kv"], rng.choice([1, 1, 2, size(1, 100), size(16, 4000)]))
        cost = 2.0e11  # pairs times heads times sequences times d of a call, at most
        while c["seqs"] > 1 and 1.0 * c["seqs"] * c["heads"] * c["new"] * c["kv"] * d > cost:
            c["seqs"] = (c["seqs"] + 1) // 2
        while c["new"] > 1 and 1.0 * c["seqs"] * c["heads"] * c["new"] * c["kv"] * d > cost:
            c["new"] = (c["new"] + 1) // 2
        while c["seqs"] > 1 and 1.0 * c["seqs"] * c["kv_heads"] * c["kv"] * d > 4.0e8:
            c["seqs"] = (c["seqs"] + 1) // 2
        c["block"] = rng.choice([0, 1, 1, size(2, 4000)])
        c["window"] = rng.choice([0, 0, 0, size(1, c["kv"] + 1)])
        return c
    axes = rng.choice([1, 3])
    c.update(norm=rng.choice(["none", "rms", "layer"]), layout=rng.choice(["interleaved", "half"]),
             theta=rng.choice([10000.0, 500000.0]), far=0)
    c["bias"] = c["norm"] == "layer"
    if axes == 3:
        frames, rows, cols = rng.randint(1, 30), rng.randint(3, 48), rng.randint(3, 80)
        c.update(dims="16,24,24" if d == 64 else "44,42,42", grid="%d,%d,%d" % (frames, rows, cols),
                 scaling="none", factor=1.0, orig=0)
        tokens = frames * rows * cols + rng.choice([0, 0, 1, 226])
    else:
        c.update(dims=str(rng.choice([32, 48, d])), grid="131072",
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]), orig=8192)
        c["factor"] = 1.0 if c["scaling"] == "none" else float(rng.choice([2, 8, 16]))
        tokens = size(1, 70000)
        c["far"] = 0 if op == "append" else rng.choice([0, 0, 131072 - tokens])
    if op == "append":
        c.update(seqs=size(1, 32), ragged=rng.random() < 0.7, page=rng.choice([16, 32, 64, 128]))
        c["new"] = rng.choice([1, 2, min(tokens, size(1, 8000))])
        c["kv"] = max(c["new"], min(tokens, 16384, 400000 // (c["seqs"] * c["kv_heads"])))
        while c["seqs"] > 1 and 1.0 * c["seqs"] * c["heads"] * c["new"] * d > 5.0e7:
            c["seqs"] = (c["seqs"] + 1) // 2
        return c
    c.update(back=rng.random() < 0.5, batch=rng.choice([1, 1, 2, 3]))
    c["n"] = max(1, min(tokens, int(3.0e8 / (c["batch"] * (c["heads"] + c["kv_heads"]) * d))))
    return c


def lengths(c):
    """New tokens and whole length of each sequence; ragged ones fall to about half of the first's."""
    fall = [i / (2.0 * c["seqs"]) if c["ragged"] else 0.0 for i in range(c["seqs"])]
    new = [max(1, int(c["new"] * (1 - f))) for f in fall]
    return new, [max(a, int(c["kv"] * (1 - f))) for a, f in zip(new, fall)]


def numbers(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------ inputs
def frequencies(c):
    """Angle per position of each pair, by axis, and the factor on cosine and sine (64 bits)."""
    out, mag = [], 1.0
    for dim in numbers(c["dims"]):
        j = torch.arange(0, dim, 2, dtype=torch.float64)
        theta = c["theta"]
        if c["scaling"] == "ntk":
            theta = theta * c["factor"] ** (dim / (dim - 2.0))
        f = theta ** (-j / dim)
        if c["scaling"] == "linear":
            f = f / c["factor"]
        if c["scaling"] == "yarn":
            turns = c["orig"] * f / (2 * math.pi)
            keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
            f = f * keep + f / c["factor"] * (1 - keep)
            mag = 0.1 * math.log(c["factor"]) + 1.0
        out.append(f)
    return out, mag


def coordinates(index, grid):
    """Row-major coordinates of token indices in the grid; -1 behind it."""
    inside = index < math.prod(grid)
    cols = []
    for g in reversed(grid):
        cols.insert(0, torch.where(inside, index % g, -1))
        index = torch.div(index, g, rounding_mode="floor")
    return torch.stack(cols, -1)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, hq, hk = DT[c["dtype"]], c["d"], c["heads"], c["kv_heads"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def projection(*lead):  # activations: every channel with its own scale, a few large ones
        scale = 0.3 + normal(hq + 2 * hk, d).abs() ** 2
        return (normal(*lead, hq + 2 * hk, d) * scale).to(dt)

    s = {"case": c}
    if c["op"] != "attn":
        freqs, mag = frequencies(c)
        grid = numbers(c["grid"])
        angles = [torch.arange(m, dtype=torch.float64, device="cuda")[:, None] * f.cuda() for m, f in zip(grid, freqs)]
        s["cos"] = [(a.cos() * mag).float() for a in angles]
        s["sin"] = [(a.sin() * mag).float() for a in angles]
        if c["norm"] != "none":
            s["wq"], s["wk"] = (1 + 0.2 * normal(d)).to(dt), (1 + 0.2 * normal(d)).to(dt)
        if c["bias"]:
            s["bq"], s["bk"] = (0.2 * normal(d)).to(dt), (0.2 * normal(d)).to(dt)
    if c["op"] == "norm_rope":
        x = projection(c["batch"], c["n"])
        s["q"], s["k"] = x[:, :, :hq], x[:, :, hq:hq + hk]
        s["pos"] = coordinates(torch.arange(c["n"], device="cuda"), grid)
        if len(grid) == 1:  # a stretch that begins at a far position, given with the call
            s["pos"] = s["pos"] + c["far"]
        if c["back"]:
            s["gq"], s["gk"] = (normal(c["batch"], h, c["n"], d).to(dt) for h in (hq, hk))
    else:
        new, kv = lengths(c)
        pages = [-(-n // c["page"]) for n in kv]
        table = torch.full((c["seqs"], max(pages)), -1, dtype=torch.int32)
        order = torch.randperm(sum(pages) + 3, generator=torch.Generator().manual_seed(seed)).int()
        first = 0
        for i, n in enumerate(pages):
            table[i, :n] = order[first:first + n]
            first += n
        s["block_table"] = table.cuda()
        s["q_start"] = torch.tensor([0] + new).cumsum(0).int().cuda()
        s["kv_len"] = torch.tensor(kv).int().cuda()
        s["max_q"], s["max_kv"] = max(new), max(kv)
        pool = (len(order), hk, c["page"], d)
        s["k_pages"], s["v_pages"] = normal(*pool).to(dt), normal(*pool).to(dt)
        if c["op"] == "append":
            x = projection(sum(new))
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        else:
            # scores of a trained layer: a few keys take most of a query's weight
            s["q"] = (1.5 * normal(sum(new), hq, d)).to(dt)
    if own:
        from clustered_sparse_attention_head_b200.layer import AttnLayer, LayerConfig
        cfg = dict(heads=hq, kv_heads=hk, d=d, dtype=c["dtype"])
        if c["op"] != "attn":
            cfg.update(norm=c["norm"], eps=EPS, rope_dims=tuple(numbers(c["dims"])), rope_max=tuple(grid),
                       rope_layout=c["layout"], rope_theta=c["theta"], rope_scaling=c["scaling"],
                       rope_factor=c["factor"], rope_orig=c["orig"])
        if c["op"] != "norm_rope":
            cfg.update(page_size=c["page"])
        if c["op"] == "attn":
            cfg.update(causal_block=c["block"], window=c["window"])
        s["layer"] = AttnLayer(LayerConfig(**cfg))
        if c["op"] != "attn":
            s["table"] = s["layer"].ac_rope_table()
        if c["op"] == "norm_rope":
            s["pos32"] = s["pos"].int() if c["far"] else None
    return s


# ------------------------------------------------------------------ plain forms
def pair_angles(s, pos):
    """cosine and sine of every token's pairs [tokens, pairs]; 1 and 0 where it is not rotated."""
    cos = torch.cat([t[p.clamp(min=0)] for t, p in zip(s["cos"], pos.unbind(-1))], -1)
    sin = torch.cat([t[p.clamp(min=0)] for t, p in zip(s["sin"], pos.unbind(-1))], -1)
    still = (pos < 0).any(-1, keepdim=True)
    return cos.masked_fill(still, 1.0), sin.masked_fill(still, 0.0)


def rotate(x, cos, sin, layout):
    """x [..., token, head, d] in 32 bits; cos, sin [token, pairs]."""
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if layout == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def normed(x, norm):
    """The norm before weight and bias, and its factor."""
    if norm == "none":
        return x, None
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def norm_rope(s, x, which, cos, sin):
    y, _ = normed(x.float(), s["case"]["norm"])
    if "w" + which in s:
        y = y * s["w" + which].float()
    if "b" + which in s:
        y = y + s["b" + which].float()
    return rotate(y, cos, sin, s["case"]["layout"])


def norm_rope_back(s, g, x, which, cos, sin):
    """g [batch, head, token, d] -> gradients of x [batch, token, head, d], of weight and bias."""
    c = s["case"]
    g = rotate(g.transpose(1, 2).float(), cos, -sin, c["layout"])
    if c["norm"] == "none":
        return [g.to(x.dtype)]
    y, r = normed(x.float(), c["norm"])
    dw, db = (g * y).sum((0, 1, 2)), g.sum((0, 1, 2))
    gy = g * s["w" + which].float()
    dx = gy - y * (gy * y).mean(-1, keepdim=True)
    if c["norm"] == "layer":
        dx = dx - gy.mean(-1, keepdim=True)
    grads = [(dx * r).to(x.dtype), dw.to(x.dtype)]
    return grads + [db.to(x.dtype)] if c["bias"] else grads


def new_tokens(s):
    """Sequence and place in the cache of every new token."""
    count = s["q_start"].diff().long()
    seq = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count, output_size=len(s["q"]))
    at = torch.arange(len(s["q"]), device="cuda") - s["q_start"][seq]
    return seq, at, at + s["kv_len"][seq] - count[seq]


def append(s):
    c = s["case"]
    seq, _, place = new_tokens(s)
    cos, sin = pair_angles(s, coordinates(place, numbers(c["grid"])))
    page = s["block_table"][seq, place // c["page"]].long()
    s["k_pages"][page, :, place % c["page"]] = norm_rope(s, s["k"], "k", cos, sin).to(s["k"].dtype)
    s["v_pages"][page, :, place % c["page"]] = s["v"]
    return norm_rope(s, s["q"], "q", cos, sin).to(s["q"].dtype), s["k_pages"], s["v_pages"]


def attend(s):
    c = s["case"]
    hk, group, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"]
    seq, at, _ = new_tokens(s)
    q = torch.zeros(c["seqs"], s["max_q"], hk, group, d, device="cuda")
    q[seq, at] = s["q"].float().unflatten(1, (hk, group))
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3) / math.sqrt(d)  # [seq, head, group x token, d]
    rows = s["block_table"].clamp(min=0).long()
    k, v = (p[rows].transpose(1, 2).flatten(2, 3)[:, :, :s["max_kv"]].float() for p in (s["k_pages"], s["v_pages"]))
    # what each new token sees of its sequence
    total, count = s["kv_len"].long(), s["q_start"].diff().long()
    place = (total - count)[:, None] + torch.arange(s["max_q"], device="cuda")
    end = total[:, None].expand_as(place)
    if c["block"]:
        end = torch.minimum(end, (torch.div(place, c["block"], rounding_mode="floor") + 1) * c["block"])
    begin = place - c["window"] + 1 if c["window"] else torch.zeros_like(place)
    key = torch.arange(s["max_kv"], device="cuda")
    hidden = ((key >= end[..., None]) | (key < begin[..., None])).repeat(1, group, 1)[:, None]
    out = torch.empty_like(q)
    step = max(1, 2 ** 30 // (c["seqs"] * q.shape[2] * s["max_kv"]))  # heads at a time, for the memory
    for h in range(0, hk, step):
        w = (q[:, h:h + step] @ k[:, h:h + step].transpose(2, 3)).masked_fill_(hidden, -math.inf)
        w = w.sub_(w.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
        out[:, h:h + step] = w @ v[:, h:h + step] / w.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.unflatten(2, (group, s["max_q"])).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return out[seq, at].to(s["q"].dtype)


def run(state):
    s = state
    c = s["case"]
    if own:
        layer = s["layer"]
        if c["op"] == "attn":
            return layer.ac_cache_attn(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["q_start"],
                                       s["kv_len"], max_q=s["max_q"], max_kv=s["max_kv"])
        weights = dict(w_q=s.get("wq"), w_k=s.get("wk"), b_q=s.get("bq"), b_k=s.get("bk"))
        if c["op"] == "append":
            q = layer.ac_cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["q_start"],
                                      s["kv_len"], q=s["q"], table=s["table"], **weights)
            return q, s["k_pages"], s["v_pages"]
        if not c["back"]:
            return layer.ac_qk_norm_rope(s["q"], s["k"], table=s["table"], pos=s["pos32"], **weights)
        grads = layer.ac_qk_norm_rope_backward(s["gq"], s["gk"], s["q"], s["k"], table=s["table"], pos=s["pos32"],
                                               **weights)
        return [grads[name] for name in ("q", "w_q", "b_q", "k", "w_k", "b_k") if grads[name] is not None]
    if c["op"] == "attn":
        return attend(s)
    if c["op"] == "append":
        return append(s)
    cos, sin = pair_angles(s, s["pos"])
    if c["back"]:
        return norm_rope_back(s, s["gq"], s["q"], "q", cos, sin) + norm_rope_back(s, s["gk"], s["k"], "k", cos, sin)
    return tuple(norm_rope(s, s[x], x, cos, sin).transpose(1, 2).contiguous().to(s[x].dtype) for x in "qk")


# ------------------------------------------------------------------ what a pass cannot do without
def seen(c):
    """(query, key) pairs of one head, and keys that any query sees, over all sequences."""
    pairs = keys = 0
    for new, kv in zip(*lengths(c)):
        place = torch.arange(kv - new, kv)
        end = ((place // c["block"] + 1) * c["block"]).clamp(max=kv) if c["block"] else torch.full_like(place, kv)
        begin = (place - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(place)
        pairs += int((end - begin).clamp(min=0).sum())
        keys += max(0, int(end.max()) - int(begin.min()))
    return pairs, keys


def work(case):
    c = case
    size = 2 if c["dtype"] == "bf16" else 4
    rows = c["heads"] + c["kv_heads"]
    if c["op"] == "attn":
        pairs, keys = seen(c)
        new = sum(lengths(c)[0])
        return {"bytes": size * c["d"] * (2 * new * c["heads"] + 2 * keys * c["kv_heads"]),
                "flops": 4 * c["d"] * pairs * c["heads"]}
    if c["op"] == "append":
        new = sum(lengths(c)[0])
        return {"bytes": 2 * size * c["d"] * new * (rows + c["kv_heads"]), "flops": 10 * c["d"] * new * rows}
    tokens = c["batch"] * c["n"]
    passes = 2 if not c["back"] or c["norm"] == "none" else 3
    return {"bytes": passes * size * c["d"] * tokens * rows,
            "flops": (20 if c["back"] else 10) * c["d"] * tokens * rows}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    double = {name: t.double() for name, t in s.items() if torch.is_tensor(t) and t.is_floating_point()}
    if c["op"] == "attn":
        if 4.0 * c["d"] * seen(c)[0] * c["heads"] > 2.0e13:
            return None
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        group, first = c["heads"] // c["kv_heads"], 0
        for i, (new, kv) in enumerate(zip(*lengths(c))):
            slots = s["block_table"][i].long()
            key = torch.arange(kv, device="cuda")
            place = torch.arange(kv - new, kv, device="cuda")[:, None]
            sees = torch.ones(new, kv, dtype=torch.bool, device="cuda")
            if c["block"]:
                sees &= key // c["block"] <= place // c["block"]
            if c["window"]:
                sees &= place - key < c["window"]
            for h in range(c["heads"]):
                k, v = (double[p][:, h // group][slots[key // c["page"]], key % c["page"]]
                        for p in ("k_pages", "v_pages"))
                w = double["q"][first:first + new, h] @ k.T * c["d"] ** -0.5
                w = torch.softmax(w.masked_fill(~sees, -math.inf), -1)
                out[first:first + new, h] = w @ v
            first += new
        return out

    # the rotation as a product of complex numbers
    freqs, mag = frequencies(c)
    grid = numbers(c["grid"])

    def turn(x, pos, back=False):  # x [..., d], pos [..., axes] of the same leading shape
        angle = torch.cat([pos[..., a:a + 1].double() * f.cuda() for a, f in enumerate(freqs)], -1)
        unit = torch.polar(torch.full_like(angle, mag), -angle if back else angle)
        unit = torch.where((pos < 0).any(-1, keepdim=True), torch.ones_like(unit), unit)
        half = angle.shape[-1]
        x = x.clone()
        if c["layout"] == "half":
            z = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * unit
            x[..., :half], x[..., half:2 * half] = z.real, z.imag
        else:
            z = torch.complex(x[..., 0:2 * half:2].contiguous(), x[..., 1:2 * half:2].contiguous()) * unit
            x[..., 0:2 * half:2], x[..., 1:2 * half:2] = z.real, z.imag
        return x

    def unit_rows(x):
        if c["norm"] == "layer":
            return (x - x.mean(-1, keepdim=True)) / (x.var(-1, keepdim=True, unbiased=False) + EPS).sqrt()
        return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() if c["norm"] == "rms" else x

    def forward(x, w, b, pos):
        y = unit_rows(x)
        y = y if w is None else y * w
        return turn(y if b is None else y + b, pos)

    if c["op"] == "append":
        first = 0
        q_out = torch.empty_like(double["q"])
        for i, (new, kv) in enumerate(zip(*lengths(c))):
            place = torch.arange(kv - new, kv, device="cuda")
            here = slice(first, first + new)
            page, at = s["block_table"][i].long()[place // c["page"]], place % c["page"]
            for out, name, heads in ((q_out, "q", c["heads"]), (None, "k", c["kv_heads"])):
                pos = coordinates(place, grid)[:, None].expand(new, heads, len(grid))
                y = forward(double[name][here], double.get("w" + name), double.get("b" + name), pos)
                if out is None:
                    double["k_pages"][page, :, at] = y
                else:
                    out[here] = y
            double["v_pages"][page, :, at] = double["v"][here]
            first += new
        return q_out, double["k_pages"], double["v_pages"]

    pos = s["pos"][None, :, None]
    outs = []
    for name in "qk":
        x, w, b = double[name], double.get("w" + name), double.get("b" + name)
        pos_x = pos.expand(*x.shape[:3], len(grid))
        if not c["back"]:
            outs.append(forward(x, w, b, pos_x).transpose(1, 2).contiguous())
            continue
        g = turn(double["g" + name].transpose(1, 2), pos_x, back=True)
        if c["norm"] == "none":
            outs.append(g)
            continue
        mean = x.mean(-1, keepdim=True) if c["norm"] == "layer" else torch.zeros_like(x[..., :1])
        scale = ((x - mean).square().mean(-1, keepdim=True) + EPS).sqrt()
        y, gy = (x - mean) / scale, g * w
        dx = gy / scale - (x - mean) * (gy * (x - mean)).sum(-1, keepdim=True) / (c["d"] * scale ** 3)
        if c["norm"] == "layer":
            dx = dx - (gy / scale).mean(-1, keepdim=True)
        outs += [dx, (g * y).sum((0, 1, 2))] + ([g.sum((0, 1, 2))] if c["bias"] else [])
    return tuple(outs) if not c["back"] else outs
