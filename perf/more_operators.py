"""Timed cases of the attention block's own operators, on the exchange's layouts.

Four operators on rank-stacked tensors (P layout ``[w, B, S, H, D]``, A layout
``[w, B, S*w, H/w, D]``):

* ``rope``   rotary positions with several axes (time, height, width), joined with
             the exchange or in place of a layout; the inverse rotation is its gradient;
* ``attn``   attention of gathered heads with a sliding window and a few first tokens
             that stay visible (sinks), the window in tokens or in chunks (frames);
* ``grad``   its backward pass, from the result and the log-sum-exp of each row;
* ``cache``  the same attention of new tokens (one for each sequence, or a chunk)
             over an 8-bit key/value cache.

What a query at position p sees, c(x) = x // chunk: positions j with
c(p) - left <= c(j) <= c(p) + right, and j < sinks; with right = 0 nothing past
p's own chunk, sinks or not.

``own`` selects between the plain form (elementary torch operations) and the
package's calls.
"""
import math

import torch

own = False

BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}            # largest value: 1.75 * 2**TOP


# --------------------------------------------------------------------- cases

def listed():
    return [
        # queries (or keys) of a 75,600-token video (21 frames of 45 x 80) on their way to attention
        dict(name="rope_video", op="rope", mode=0, w=8, B=1, S=9450, H=40, D=128, type="bf16", dims="44,42,42",
             halves=False, inverse=False),
        # the gradient of two images' queries, each with positions of its own, on its way back; halves of a head as pairs
        dict(name="rope_grad_halves", op="rope", mode=1, w=4, B=2, S=1531, H=16, D=64, type="fp16", dims="16,24,24",
             halves=True, inverse=True),
        # a new token for each of 32 sequences before they go to the cache: latency
        dict(name="rope_token", op="rope", mode=-1, w=8, B=1, S=4, H=8, D=128, type="bf16", dims="128",
             halves=True, inverse=False),
        # the same video generated frame by frame: each frame sees itself, two before it and the first
        dict(name="attn_video", op="attn", w=8, B=1, S=9450, H=40, kv=40, D=128, type="bf16", chunk=3600, left=2,
             right=0, sinks=3600, counts=False, lse=True),
        # two prompts of different lengths, shared key heads, a window of 1024 tokens and four sinks
        dict(name="attn_prompts", op="attn", w=4, B=2, S=1531, H=32, kv=8, D=64, type="fp16", chunk=1, left=1024,
             right=0, sinks=4, counts=True, lse=False),
        # a few tokens of an image, all of them visible: latency
        dict(name="attn_small", op="attn", w=2, B=1, S=33, H=4, kv=4, D=80, type="bf16", chunk=1, left=-1, right=-1,
             sinks=0, counts=False, lse=False),
        # training on a smaller video (21 frames of 30 x 52): the backward pass
        dict(name="grad_video", op="grad", w=4, B=1, S=8190, H=12, kv=12, D=128, type="bf16", chunk=1560, left=2,
             right=0, sinks=1560, counts=False),
        # training on packed prompts: padded rows, shared key heads, a window to both sides
        dict(name="grad_prompts", op="grad", w=4, B=2, S=1531, H=16, kv=4, D=64, type="fp16", chunk=1, left=512,
             right=512, sinks=8, counts=True),
        # one new token for each of 32 sequences, shared key heads, window and sinks
        dict(name="cache_tokens", op="cache", w=8, H=32, kv=8, D=128, type="bf16", fmt="e4m3", seqs=32, n=1, cap=8192,
             chunk=1, left=4095, right=0, sinks=4),
        # one new token of a single long sequence, everything visible
        dict(name="cache_long", op="cache", w=4, H=16, kv=8, D=128, type="bf16", fmt="e4m3", seqs=1, n=1, cap=131072,
             chunk=1, left=-1, right=0, sinks=0),
        # the next frame of a video: its tokens see the frame, three before it and the first
        dict(name="cache_frame", op="cache", w=4, H=12, kv=12, D=128, type="bf16", fmt="e4m3", seqs=1, n=1560,
             cap=18720, chunk=1560, left=3, right=0, sinks=1560),
        # a few sequences that have just begun, half precision: latency
        dict(name="cache_short", op="cache", w=2, H=8, kv=8, D=72, type="fp16", fmt="e5m2", seqs=3, n=1, cap=515,
             chunk=1, left=127, right=0, sinks=2),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "grad", "cache"])
    w = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([16, 32, 40, 64, 64, 72, 80, 96, 128, 128])
    c = dict(op=op, w=w, D=D)
    if op == "rope":
        D = c["D"] = rng.choice([16, 40, 64, 72, 80, 96, 128, 192, 256])
        H = c["H"] = w * _spread(rng, 1, max(1, 6144 // (w * D)))
        B = c["B"] = rng.choice([1, 1, 2, 3])
        c["type"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        values = 110_000_000 if c["type"] == "fp32" else 200_000_000
        c["S"] = max(1, _spread(rng, 16, max(16, min(75600, values // (H * D)))) // (w * B))
        axes = rng.choice([1, 2, 3, 3])
        part = 2 * (D // (2 * axes) - rng.choice([0, 1]))        # a few values of a head may stay as they are
        c["dims"] = ",".join([str(part)] * axes)
        c.update(mode=rng.choice([0, 0, 1, 1, -1, -2]), halves=rng.random() < 0.5, inverse=rng.random() < 0.5)
        return c
    c["type"] = rng.choice(["bf16", "bf16", "fp16"])
    kv = c["kv"] = w * _spread(rng, 1, max(1, 16 // w))
    H = c["H"] = kv * rng.choice([1, 1, 2, 4, 7])
    c["chunk"] = rng.choice([1, 1, rng.randint(2, 700)])
    c["right"] = rng.choice([0, 0, 0, -1, rng.randint(0, 600) // c["chunk"]])
    c["sinks"] = rng.choice([0, 1, 4, rng.randint(5, 900)])
    if op == "cache":
        c["fmt"] = rng.choice(["e4m3", "e5m2"])
        n = c["n"] = rng.choice([1, 1, 1, 2, _spread(rng, 3, 1024)])
        c["seqs"] = _spread(rng, 1, 64)
        room = 120_000_000 // (c["seqs"] * kv * D)               # positions of all sequences
        if n > 2:
            room = min(room, 600_000_000 // (c["seqs"] * H * n))
        c["cap"] = n + _spread(rng, 1, max(1, min(131072, room)))
        c["left"] = rng.choice([-1, _spread(rng, 1, c["cap"]) // c["chunk"]])
        return c
    c["B"] = rng.choice([1, 1, 2, 3])
    c["counts"] = rng.random() < 0.4
    c["lse"] = not c["counts"] and rng.random() < 0.5
    c["S"] = max(1, _spread(rng, 16, 24576) // (w * c["B"]))
    seen = 2_000_000_000 // (w * c["B"] * c["S"] * H // w)       # keys of a row, from the plain form's time
    c["left"] = rng.choice([-1, _spread(rng, 1, w * c["S"]) // c["chunk"]])
    if w * c["S"] > seen:
        c["right"] = max(0, c["right"]) if c["right"] * c["chunk"] <= seen // 2 else 0
        c["left"] = min(c["left"], seen // (2 * c["chunk"])) if c["left"] >= 0 else seen // (2 * c["chunk"])
    return c


def _pairs_seen(case, rows, first):
    """Pairs of a query and a key that it sees, of one head of one sequence."""
    total = 0
    end = first + rows
    for p in range(first, end):
        lo, hi = _range(case, p, end)
        s = min(case["sinks"], hi if case["right"] == 0 else end)
        total += hi - lo + min(s, lo)
    return total


def _range(case, p, end):
    """[lo, hi): the window of position p among [0, end)."""
    c = p // case["chunk"]
    lo = 0 if case["left"] < 0 else max(0, (c - case["left"]) * case["chunk"])
    hi = end if case["right"] < 0 else min(end, (c + case["right"] + 1) * case["chunk"])
    return min(lo, hi), hi


def work(case):
    w, H, D = case["w"], case["H"], case["D"]
    e = 4 if case["type"] == "fp32" else 2
    if case["op"] == "rope":
        n = w * case["B"] * case["S"] * H * D
        axes = len(case["dims"].split(","))
        return {"bytes": 2 * n * e + 4 * axes * case["B"] * case["S"] * w, "flops": 3 * n}
    if case["op"] == "cache":
        n, seqs = case["n"], case["seqs"]
        first = (case["cap"] - n) * 3 // 4 if seqs > 1 else case["cap"] - n      # the sequences' mean place
        lo, _ = _range(case, first, first + n)
        keys = first + n - lo + min(case["sinks"], lo)
        q = D + -(-D // BLOCK)
        return {"bytes": 2 * seqs * n * H * D * e + 2 * seqs * keys * case["kv"] * q,
                "flops": 4 * seqs * H * D * _pairs_seen(case, n, first)}
    SG = w * case["S"]
    share = 0.75 if case["counts"] else 1                        # the sequences' mean length
    tokens = int(case["B"] * SG * share)
    pairs = case["B"] * _pairs_seen(case, int(SG * share), 0)
    if case["op"] == "attn":
        b = tokens * D * e * (2 * H + 2 * case["kv"]) + (4 * tokens * H if case["lse"] else 0)
        return {"bytes": b, "flops": 4 * D * H * pairs}
    return {"bytes": tokens * D * e * (4 * H + 4 * case["kv"]) + 4 * tokens * H, "flops": 10 * D * H * pairs}


# -------------------------------------------------------------------- layouts

def _to_a(x, w):
    """P layout -> A layout."""
    j, B, S, H, d = x.shape
    return x.view(w, B, S, w, H // w, d).permute(3, 1, 0, 2, 4, 5).reshape(w, B, S * w, H // w, d)


def _to_p(x, w):
    """A layout -> P layout."""
    r, B, SG, hl, d = x.shape
    return x.view(w, B, w, SG // w, hl, d).permute(2, 1, 3, 0, 4, 5).reshape(w, B, SG // w, hl * w, d)


def _dims(case):
    return tuple(int(d) for d in case["dims"].split(","))


# ----------------------------------------------------------------- plain form

def _plain_rope(s):
    c = s["case"]
    w, dims = c["w"], _dims(c)
    pos = s["positions"].double()                                # [axes, B or 1, S*w]
    angles = []
    for a, d in enumerate(dims):
        f = 10000.0 ** (-torch.arange(0, d, 2, device=pos.device, dtype=torch.float64) / d)
        angles.append(pos[a].unsqueeze(-1) * f)
    angle = torch.cat(angles, -1)                                # [B or 1, S*w, pairs]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if c["inverse"]:
        sin = -sin
    x = s["x"]
    B, SG = c["B"], c["S"] * w
    if c["mode"] in (0, -1):                                     # x in P: rank, plane, token
        cos, sin = (t.expand(B, SG, -1).reshape(B, w, SG // w, -1).transpose(0, 1) for t in (cos, sin))
    else:
        cos, sin = (t.expand(B, SG, -1).unsqueeze(0) for t in (cos, sin))
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    v = x.float()
    R = sum(dims)
    if c["halves"]:
        a, b = v[..., :R // 2], v[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin, v[..., R:]], -1)
    else:
        a, b = v[..., 0:R:2], v[..., 1:R:2]
        y = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), v[..., R:]], -1)
    y = y.to(x.dtype)
    return {"out": _to_a(y, w) if c["mode"] == 0 else _to_p(y, w) if c["mode"] == 1 else y}


def _heads(x, group=1):
    """[w, B, tokens, heads, D] -> 32-bit [w*B, heads*group, tokens, D], contiguous."""
    x = x.float().transpose(2, 3).flatten(0, 1)
    if group > 1:
        x = x.repeat_interleave(group, 1)
    return x.contiguous()


def _visible(c, p, j):
    """Whether position p sees position j (integer tensors that broadcast)."""
    cp, cj = p // c["chunk"], j // c["chunk"]
    seen = torch.ones(torch.broadcast_shapes(p.shape, j.shape), dtype=torch.bool, device=p.device)
    if c["left"] >= 0:
        seen = seen & (cj >= cp - c["left"])
    if c["sinks"] > 0:
        seen = seen | (j < c["sinks"])
    if c["right"] >= 0:
        behind = cj > cp + c["right"]
        if c["right"] > 0 and c["sinks"] > 0:
            behind = behind & (j >= c["sinks"])
        seen = seen & ~behind
    return seen


def _row_blocks(c, SG):
    """(first row, rows, key places) of blocks of rows and the keys that one of them may see."""
    step = c["chunk"] * max(1, 2048 // c["chunk"])
    for r0 in range(0, SG, step):
        r1 = min(SG, r0 + step)
        lo, hi = _range(c, r0, SG)[0], _range(c, r1 - 1, SG)[1]
        s = min(c["sinks"], hi if c["right"] == 0 else SG, lo)
        yield r0, r1, list(range(0, s)) + list(range(lo, hi))


def _index(places, device):
    """An index tensor of two ranges, made on the device."""
    n = len(places)
    cut = next((i for i in range(n) if places[i] != i), n)
    parts = [torch.arange(cut, device=device)]
    if cut < n:
        parts.append(torch.arange(places[cut], places[-1] + 1, device=device))
    return torch.cat(parts)


def _softmax(sc, seen):
    """(weights, log-sum-exp) of rows, zeros and -inf where a row sees nothing."""
    sc = torch.where(seen, sc, float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = torch.exp(sc - top)
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), (torch.log(total) + top).squeeze(-1)


def _plain_forward(c, q, k, v, counts, dtype):
    """(out in A layout, lse [w, B, heads, tokens]) in 32 bits, rounded once."""
    w, B, SG, hl, D = q.shape
    group = hl // k.shape[3]
    Q, K, V = _heads(q), _heads(k, group), _heads(v, group)
    out = torch.empty(w, B, SG, hl, D, dtype=dtype, device=q.device)
    lse = torch.empty(w * B, hl, SG, device=q.device)
    end = None if counts is None else counts.view(1, B, 1, 1, 1).expand(w, -1, -1, -1, -1).reshape(w * B, 1, 1, 1)
    for r0, r1, places in _row_blocks(c, SG):
        j = _index(places, q.device)
        p = torch.arange(r0, r1, device=q.device)
        seen = _visible(c, p.view(-1, 1), j)
        if end is not None:
            seen = seen & (j < end) & (p.view(-1, 1) < end)
        sc = torch.matmul(Q[:, :, r0:r1], K[:, :, j].transpose(-1, -2).contiguous()) * D ** -0.5
        prob, lse[:, :, r0:r1] = _softmax(sc, seen)
        o = torch.matmul(prob, V[:, :, j])
        out[:, :, r0:r1] = o.view(w, B, hl, r1 - r0, D).transpose(2, 3).to(dtype)
    return out, lse.view(w, B, hl, SG)


def _plain_attn(s):
    c = s["case"]
    out, lse = _plain_forward(c, s["q"], s["k"], s["v"], s.get("counts"), s["q"].dtype)
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}


def _plain_grad(s):
    c = s["case"]
    q, k, counts = s["q"], s["k"], s.get("counts")
    w, B, SG, hl, D = q.shape
    kvl = k.shape[3]
    group = hl // kvl
    Q, K, V, DO = _heads(q), _heads(k, group), _heads(s["v"], group), _heads(s["dout"])
    delta = (DO * _heads(s["out"])).sum(-1, keepdim=True)
    lse = s["lse"].view(w * B, hl, SG, 1)
    dq, dk, dv = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    end = None if counts is None else counts.view(1, B, 1, 1, 1).expand(w, -1, -1, -1, -1).reshape(w * B, 1, 1, 1)
    for r0, r1, places in _row_blocks(c, SG):
        j = _index(places, q.device)
        p = torch.arange(r0, r1, device=q.device)
        seen = _visible(c, p.view(-1, 1), j)
        if end is not None:
            seen = seen & (j < end) & (p.view(-1, 1) < end)
        Qb, DOb, Kb = Q[:, :, r0:r1], DO[:, :, r0:r1], K[:, :, j]
        sc = torch.matmul(Qb, Kb.transpose(-1, -2).contiguous()) * D ** -0.5
        prob = torch.exp(torch.where(seen, sc - lse[:, :, r0:r1], float("-inf")))
        dv[:, :, j] += torch.matmul(prob.transpose(-1, -2), DOb)
        dp = torch.matmul(DOb, V[:, :, j].transpose(-1, -2).contiguous())
        ds = prob * (dp - delta[:, :, r0:r1]) * D ** -0.5
        dq[:, :, r0:r1] = torch.matmul(ds, Kb)
        dk[:, :, j] += torch.matmul(ds.transpose(-1, -2), Qb)

    def back(x, heads):
        x = x.view(w, B, heads, -1, SG, D).sum(3) if heads != hl else x.view(w, B, hl, SG, D)
        return x.transpose(2, 3).to(q.dtype).contiguous()

    return {"dq": back(dq, hl), "dk": back(dk, kvl), "dv": back(dv, kvl)}


def _pow2(k):
    """2.0**k in 32 bits, k an int32 tensor in [-127, 127], from its bits."""
    return torch.where(k > -127, (k + 127) << 23, torch.full_like(k, 1 << 22)).view(torch.float32)


def _quantise(v, fmt):
    """Codes and scales of 32-bit values [..., D]."""
    D = v.shape[-1]
    nb = -(-D // BLOCK)
    if nb * BLOCK != D:
        v = torch.cat([v, v.new_zeros(v.shape[:-1] + (nb * BLOCK - D,))], -1)
    v = v.unflatten(-1, (nb, BLOCK))
    m, ex = torch.frexp(v.abs().amax(-1))
    k = ex - 1 - TOP[fmt] + (m > 0.875).to(torch.int32)
    k = torch.where(m == 0, torch.full_like(k, -127), k.clamp_min(-127))
    codes = (v * _pow2(-k).unsqueeze(-1)).to(FORMATS[fmt]).flatten(-2)[..., :D].contiguous()
    return codes, (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_cache(s):
    c = s["case"]
    q = s["q"]
    w, seqs, n, hl, D = q.shape
    scale = _pow2(s["scales"].view(torch.uint8).to(torch.int32) - 127)
    kv = s["codes"].float() * scale.repeat_interleave(BLOCK, -1)[..., :D]
    kv = kv.to(q.dtype)                                          # what a read of the cache gives
    group = hl // kv.shape[4]
    K, V = (_heads(t, group) for t in kv)
    t = torch.arange(n, device=q.device)
    p = (s["starts"].view(-1, 1) + t).view(1, seqs, 1, n, 1)
    j = torch.arange(c["cap"], device=q.device)
    seen = _visible(c, p, j) & (j < s["starts"].view(1, seqs, 1, 1, 1) + s["counts"].view(1, seqs, 1, 1, 1))
    seen = seen.expand(w, -1, -1, -1, -1).flatten(0, 1)
    sc = torch.matmul(_heads(q), K.transpose(-1, -2).contiguous()) * D ** -0.5
    prob, _ = _softmax(sc, seen)
    o = torch.matmul(prob, V).view(w, seqs, hl, n, D).transpose(2, 3).to(q.dtype)
    live = (t < s["counts"].view(-1, 1)).view(1, seqs, n, 1, 1)
    s["out"].copy_(torch.where(live, o, s["out"]))
    return {"out": s["out"]}


# ------------------------------------------------------------ the package's calls

def _plan(s, B, S):
    if "plan" not in s:
        import ulysses_all_re_amd as ua
        c = s["case"]
        s["plan"] = ua.Plan(c["w"], B, S, c["H"], c["D"], TYPES[c["type"]])
    return s["plan"]


def _window(c):
    return dict(left=None if c["left"] < 0 else c["left"], right=None if c["right"] < 0 else c["right"],
                sinks=c["sinks"], chunk=c["chunk"])


def _own_rope(s):
    c = s["case"]
    plan = _plan(s, c["B"], c["S"])
    if "rotary" not in s:
        import ulysses_all_re_amd as ua
        s["rotary"] = ua.Rotary(c["D"], _dims(c), halves=c["halves"], device="cuda")
    if c["mode"] < 0:
        s["own_out"] = plan.rope(s["x"], s["rotary"], s["positions"], gathered=c["mode"] == -2, inverse=c["inverse"],
                                 out=s.get("own_out"))
    else:
        s["own_out"] = plan.rope_exchange(s["x"], s["rotary"], s["positions"], c["mode"], inverse=c["inverse"],
                                          out=s.get("own_out"))
    return {"out": s["own_out"]}


def _own_attn(s):
    c = s["case"]
    r = _plan(s, c["B"], c["S"]).window_attention(s["q"], s["k"], s["v"], counts=s.get("counts"), lse=c["lse"],
                                                  out=s.get("own_out"), **_window(c))
    s["own_out"] = r
    return {"out": r.out, "lse": r.lse} if c["lse"] else {"out": r.out}


def _own_grad(s):
    c = s["case"]
    r = _plan(s, c["B"], c["S"]).window_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"],
                                                           counts=s.get("counts"), grads=s.get("own_out"),
                                                           **_window(c))
    s["own_out"] = r
    return {"dq": r.dq, "dk": r.dk, "dv": r.dv}


def _own_cache(s):
    c = s["case"]
    plan = _plan(s, 1, 1)
    if "cache" not in s:
        import ulysses_all_re_amd as ua
        s["cache"] = ua.Cache.of(s["codes"], s["scales"])
    return {"out": plan.cache_attention(s["cache"], s["q"], s["starts"], s["counts"], out=s["out"], **_window(c))}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "grad": _own_grad, "cache": _own_cache}[op](s)
    return {"rope": _plain_rope, "attn": _plain_attn, "grad": _plain_grad, "cache": _plain_cache}[op](s)


# --------------------------------------------------------------------- inputs

def _activations(shape, gen, size=1.0):
    """Values as a norm or a projection gives them: normal, some channels of a head larger than others."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= size * torch.exp(0.4 * torch.randn(shape[-1], generator=gen, device="cuda"))
    return x


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    c, t = dict(case), TYPES[case["type"]]
    w, H, D, op = c["w"], c["H"], c["D"], c["op"]
    s = {"case": c}
    if op == "rope":
        p = (w, c["B"], c["S"], H, D)
        a = (w, c["B"], c["S"] * w, H // w, D)
        s["x"] = _activations(p if c["mode"] in (0, -1) else a, gen).to(t)
        axes, SG = len(_dims(c)), c["S"] * w
        if axes == 1:                                            # sequences at different places
            at = torch.randint(0, 100_000, (c["B"], 1), generator=gen, device="cuda", dtype=torch.int32)
            if c["S"] <= 4:
                at = torch.randint(0, 100_000, (c["B"], SG), generator=gen, device="cuda", dtype=torch.int32)
            s["positions"] = (at + torch.arange(SG, device="cuda", dtype=torch.int32) * (c["S"] > 4)).view(1, c["B"], SG)
        else:                                                    # a grid of frames, rows and columns, from some frame on
            wide = max(1, math.isqrt(max(1, SG // 12)))
            g = torch.arange(SG, device="cuda", dtype=torch.int32)
            first = torch.randint(0, 500, (c["B"], 1), generator=gen, device="cuda", dtype=torch.int32)
            frame = first + g // (wide * wide)
            rows = [frame, (g // wide % wide).expand(c["B"], -1), (g % wide).expand(c["B"], -1)]
            s["positions"] = torch.stack(rows[:axes] if axes == 3 else rows[1:])
        return s
    if op in ("attn", "grad"):
        SG, B = c["S"] * w, c["B"]
        s["q"] = _activations((w, B, SG, H // w, D), gen).to(t)
        s["k"] = _activations((w, B, SG, c["kv"] // w, D), gen).to(t)
        s["v"] = _activations((w, B, SG, c["kv"] // w, D), gen).to(t)
        if c["counts"]:
            s["counts"] = torch.randint(SG // 2, SG + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        if op == "grad":
            s["dout"] = (torch.randn(s["q"].shape, generator=gen, device="cuda") * 0.02).to(t)
            s["out"], s["lse"] = _plain_forward(c, s["q"], s["k"], s["v"], s.get("counts"), t)
        return s
    n, seqs, cap = c["n"], c["seqs"], c["cap"]
    s["q"] = _activations((w, seqs, n, H // w, D), gen).to(t)
    both = [_quantise(_activations((w, seqs, cap, c["kv"] // w, D), gen), c["fmt"]) for _ in range(2)]
    s["codes"] = torch.stack([q.view(torch.uint8) for q, _ in both]).view(FORMATS[c["fmt"]])
    s["scales"] = torch.stack([q.view(torch.uint8) for _, q in both]).view(torch.float8_e8m0fnu)
    # one sequence is near the cache's end, several are anywhere in its second half
    least = (cap - n) // 2 if seqs > 1 else cap - n
    s["starts"] = torch.randint(least, cap - n + 1, (seqs,), generator=gen, device="cuda", dtype=torch.int32)
    s["counts"] = torch.full((seqs,), n, device="cuda", dtype=torch.int32)
    if n > 1 and seqs > 1:
        s["counts"] = torch.randint(n // 2, n + 1, (seqs,), generator=gen, device="cuda", dtype=torch.int32)
    s["out"] = torch.zeros_like(s["q"])
    return s


# ------------------------------------------------------- the definition, in 64 bits

def _mask(c, p, j):
    """[rows, keys] of integer vectors p and j, by the definition."""
    p, j = p[:, None], j[None, :]
    gap = torch.div(j, c["chunk"], rounding_mode="floor") - torch.div(p, c["chunk"], rounding_mode="floor")
    ahead, back = gap > 0, gap < 0
    out = torch.zeros_like(ahead)
    if c["right"] >= 0:
        out |= ahead & (gap > c["right"])
    if c["left"] >= 0:
        out |= back & (-gap > c["left"])
    keep = j < c["sinks"]
    if c["right"] == 0:
        keep = keep & ~ahead
    return ~out | keep


def _exact_rows(c, q, k, p, j_end):
    """Scaled scores of some rows [heads, rows, D] with the keys [heads, tokens, D]
    that one of them sees, which keys those are, and what is seen."""
    j = torch.arange(j_end, device=q.device)
    seen = _mask(c, p, j)
    j = seen.any(0).nonzero().flatten()
    seen = seen[:, j]
    return torch.matmul(q, k[:, j].transpose(1, 2)) / math.sqrt(q.shape[-1]), j, seen


def _exact_attention(c, q, k, v, p, j_end):
    """(out, lse) of rows at positions p over the first j_end keys; [heads, rows, D]."""
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float64, device=q.device)
    for r in range(0, q.shape[1], 1024):
        sc, j, seen = _exact_rows(c, q[:, r:r + 1024], k, p[r:r + 1024], j_end)
        if j.numel() == 0:
            continue
        sc.masked_fill_(~seen, float("-inf"))
        norm = torch.logsumexp(sc, -1)
        some = torch.isfinite(norm)
        prob = torch.exp(sc - torch.where(some, norm, 0.0).unsqueeze(-1))
        out[:, r:r + 1024] = torch.matmul(prob, v[:, j])
        lse[:, r:r + 1024] = norm
    return out, lse


def _exact_rope(s):
    c = s["case"]
    w, B, S, H, D = c["w"], c["B"], c["S"], c["H"], c["D"]
    dims = _dims(c)
    R = sum(dims)
    x = s["x"].double()
    if c["mode"] in (1, -2):                                     # [B, S*w, H, D], whatever x's layout
        x = x.permute(1, 2, 0, 3, 4).reshape(B, S * w, H, D)
    else:
        x = x.permute(1, 0, 2, 3, 4).reshape(B, S * w, H, D)
    y = x.clone()
    pair = 0
    for a, d in enumerate(dims):
        at = s["positions"][a].double()
        for i in range(d // 2):
            angle = (at * math.exp(-2 * i / d * math.log(10000.0))).unsqueeze(-1)
            if c["inverse"]:
                angle = -angle
            u, z = (pair, pair + R // 2) if c["halves"] else (2 * pair, 2 * pair + 1)
            y[..., u] = x[..., u] * torch.cos(angle) - x[..., z] * torch.sin(angle)
            y[..., z] = x[..., u] * torch.sin(angle) + x[..., z] * torch.cos(angle)
            pair += 1
    if c["mode"] in (0, -2):
        y = y.view(B, S * w, w, H // w, D).permute(2, 0, 1, 3, 4)
    else:
        y = y.view(B, w, S, H, D).permute(1, 0, 2, 3, 4)
    return {"out": y.contiguous()}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return _exact_rope(s)
    q = s["q"]
    group = c["H"] // c["kv"]
    ranks, planes, rows, hl, D = q.shape
    if c["op"] == "cache":
        out = s["out"].double()
        for i in range(planes):
            start, count = int(s["starts"][i]), int(s["counts"][i])
            p = start + torch.arange(count, device=q.device)
            for r in range(ranks):
                kv = []
                for part in range(2):
                    sc = s["scales"][part, r, i].double()
                    d = torch.arange(D, device=sc.device) // BLOCK
                    x = (s["codes"][part, r, i].double() * sc[..., d]).to(q.dtype).double()   # as the type holds it
                    kv.append(x.transpose(0, 1).repeat_interleave(group, 0))
                o, _ = _exact_attention(c, q[r, i, :count].double().transpose(0, 1), *kv, p, start + count)
                out[r, i, :count] = o.transpose(0, 1)
        return {"out": out}
    counts = s["counts"].tolist() if c["counts"] else [rows] * planes
    if c["op"] == "attn":
        out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        lse = torch.full((ranks, planes, hl, rows), float("-inf"), dtype=torch.float64, device=q.device)
        for r in range(ranks):
            for b, n in enumerate(counts):
                Q = q[r, b, :n].double().transpose(0, 1)
                K, V = (x[r, b, :n].double().transpose(0, 1).repeat_interleave(group, 0) for x in (s["k"], s["v"]))
                o, lse[r, b, :, :n] = _exact_attention(c, Q, K, V, torch.arange(n, device=q.device), n)
                out[r, b, :n] = o.transpose(0, 1)
        return {"out": out, "lse": lse} if c["lse"] else {"out": out}
    dq = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    dk = torch.zeros(s["k"].shape, dtype=torch.float64, device=q.device)
    dv = torch.zeros_like(dk)
    for r in range(ranks):
        for b, n in enumerate(counts):
            for h in range(hl):
                Q, O, G = (x[r, b, :n, h].double() for x in (q, s["out"], s["dout"]))
                K, V = (x[r, b, :n, h // group].double() for x in (s["k"], s["v"]))
                delta = (O * G).sum(-1, keepdim=True)
                lse = s["lse"][r, b, h, :n].double()
                for t in range(0, n, 4096):
                    p = torch.arange(t, min(n, t + 4096), device=q.device)
                    sc, j, seen = _exact_rows(c, Q[None, p], K[None], p, n)
                    prob = torch.where(seen, torch.exp(sc[0] - lse[p, None]), 0.0)
                    ds = prob * (G[p] @ V[j].T - delta[p]) / math.sqrt(D)
                    dq[r, b, p, h] = ds @ K[j]
                    dk[r, b, j, h // group] += ds.T @ Q[p]
                    dv[r, b, j, h // group] += prob.T @ G[p]
    return {"dq": dq, "dk": dk, "dv": dv}
