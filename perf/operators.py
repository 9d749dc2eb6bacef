"""Timed cases of the operators that work on activations around the exchange.

Four operators of a sequence-parallel attention block on rank-stacked tensors
(P layout ``[w, B, S, H, D]``, A layout ``[w, B, S*w, H/w, D]``):

* ``norm``   RMS norm joined with the exchange (mode 0: norm, then exchange;
             mode 1: exchange, residual's addition, norm), the result in the
             input's type or in 8 bits with scales, optionally with an 8-bit
             checkpoint of what the backward pass needs;
* ``back``   its backward pass, from an 8-bit checkpoint or from the values;
* ``write``  the mode-0 exchange of new keys and values into an 8-bit cache;
* ``read``   positions of that cache, back in the type.

8 bits with scales: blocks of 32 values along D (a head's last block may be
shorter), e4m3 or e5m2 codes and one power-of-two scale (e8m0) per block, the
least one that no value of the block overflows.

``own`` selects between the plain form (elementary torch operations) and the
package's calls.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}            # largest value: 1.75 * 2**TOP
MANTISSA = {"e4m3": 3, "e5m2": 2}
LEAST = {"e4m3": -6, "e5m2": -14}        # exponent of the smallest normal value


# --------------------------------------------------------------------- cases

def listed():
    return [
        # forward of a video model's query norm over whole tokens, in training: the 75,600-token exchange
        dict(name="norm0_video_train", op="norm", mode=0, w=8, B=1, S=9450, H=40, D=128, type="bf16",
             head=False, residual=False, out="", save="e4m3"),
        # per-head query/key norm in inference, four batch planes of short sequences
        dict(name="norm0_planes_head", op="norm", mode=0, w=4, B=4, S=2048, H=16, D=64, type="fp16",
             head=True, residual=False, out="", save=""),
        # attention's output back on its tokens, with a residual, in 8 bits for an 8-bit projection
        dict(name="norm1_residual_8bit", op="norm", mode=1, w=4, B=1, S=1024, H=32, D=128, type="bf16",
             head=False, residual=True, out="e4m3", save=""),
        # single precision, odd sequence, a head that is no multiple of a block
        dict(name="norm1_odd_fp32", op="norm", mode=1, w=3, B=2, S=4681, H=12, D=80, type="fp32",
             head=False, residual=True, out="", save="e5m2"),
        # a few tokens: latency
        dict(name="norm0_tiny", op="norm", mode=0, w=2, B=1, S=8, H=4, D=16, type="bf16",
             head=False, residual=False, out="", save=""),
        # the backward pass of the first case, from its 8-bit checkpoint
        dict(name="back0_video_train", op="back", mode=0, w=8, B=1, S=9450, H=40, D=128, type="bf16",
             head=False, residual=False, save="e4m3"),
        # the backward pass after attention, per head, with the residual stream's gradient
        dict(name="back1_head_residual", op="back", mode=1, w=4, B=2, S=1531, H=16, D=64, type="fp16",
             head=True, residual=True, save="e5m2"),
        # the backward pass from the values themselves, single precision, odd sizes
        dict(name="back0_odd_fp32", op="back", mode=0, w=3, B=2, S=4681, H=12, D=80, type="fp32",
             head=False, residual=False, save=""),
        # prompts of different lengths into the cache
        dict(name="write_prompts", op="write", w=8, B=2, S=2048, H=16, D=128, type="bf16", fmt="e4m3",
             each=16384, cap=20000),
        # one new token for each of 32 sequences
        dict(name="write_token", op="write", w=8, B=1, S=4, H=8, D=128, type="bf16", fmt="e4m3",
             each=1, cap=2048),
        # a whole video's keys and values
        dict(name="read_long", op="read", w=8, H=40, D=128, type="bf16", fmt="e4m3", seqs=1, each=75600,
             cap=75600),
        # many short sequences of different lengths
        dict(name="read_ragged", op="read", w=4, H=16, D=72, type="fp16", fmt="e5m2", seqs=33, each=257,
             cap=515),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "back", "write", "read"])
    w = rng.choice([1, 2, 3, 4, 5, 8])
    D = rng.choice([16, 40, 64, 72, 80, 96, 128, 192, 256])
    H = w * _spread(rng, 1, max(1, 6144 // (w * D)))
    c = dict(op=op, w=w, H=H, D=D, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    values = 110_000_000 if c["type"] == "fp32" else 200_000_000
    tokens = _spread(rng, 16, max(16, min(75600, values // (H * D))))
    if op in ("norm", "back"):
        B = rng.choice([1, 1, 2, 3])
        c.update(mode=rng.choice([0, 1]), B=B, S=max(1, tokens // (w * B)), head=rng.random() < 0.4,
                 residual=rng.random() < 0.5, save=rng.choice(["", "e4m3", "e5m2"]))
        if op == "norm":
            c["out"] = rng.choice(["", "", "e4m3", "e5m2"])
    else:
        c["fmt"] = rng.choice(["e4m3", "e5m2"])
        if op == "write":
            B = rng.choice([1, 2, 3])
            one = rng.random() < 0.4
            S = max(1, (_spread(rng, 1, 512) if one else tokens) // (w * B))
            each = 1 if one else S * w
            c.update(B=B, S=S, each=each, cap=each + _spread(rng, 1, 2048 if each > 1 else 64))
        else:
            seqs = _spread(rng, 1, 64)
            each = max(1, tokens // seqs)
            c.update(seqs=seqs, each=each, cap=each + _spread(rng, 1, 999))
    return c


def _sizes(case):
    e = 4 if case["type"] == "fp32" else 2
    blocks = -(-case["D"] // BLOCK)
    return e, blocks


def work(case):
    e, blocks = _sizes(case)
    H, D = case["H"], case["D"]
    q = D + blocks                                             # bytes of one head in 8 bits
    if case["op"] in ("norm", "back"):
        rows = case["w"] * case["B"] * case["S"]
        n = rows * H * D
        stats = 4 * rows * (H if case["head"] else 1)
        weight = 4 * (D if case["head"] else H * D)
        if case["op"] == "norm":
            b = n * e + weight + (rows * H * q if case["out"] else n * e)
            b += 2 * n * e if case["residual"] else 0
            b += rows * H * q + stats if case["save"] else 0
            return {"bytes": b, "flops": 5 * n}
        b = 2 * n * e + 2 * weight + stats + (rows * H * q if case["save"] else n * e)
        if case["residual"]:
            b += n * e * (2 if case["mode"] == 1 else 1)       # the sum's gradient, and the residual's own
        return {"bytes": b, "flops": 9 * n}
    if case["op"] == "write":
        rows = case["w"] * case["B"] * case["S"]
        rows = int(rows * (0.75 if case["each"] > 1 else 1))   # the sequences' mean share
        return {"bytes": 2 * rows * H * (D * e + q), "flops": 4 * rows * H * D}
    rows = int(case["seqs"] * case["each"] * (1 if case["seqs"] == 1 else 0.75))
    return {"bytes": 2 * rows * H * (D * e + q), "flops": 2 * rows * H * D}


# -------------------------------------------------------------------- layouts

def _to_a(x, w):
    """P layout -> A layout, any trailing size."""
    j, B, S, H, d = x.shape
    return x.view(w, B, S, w, H // w, d).permute(3, 1, 0, 2, 4, 5).reshape(w, B, S * w, H // w, d)


def _to_p(x, w):
    """A layout -> P layout."""
    r, B, SG, hl, d = x.shape
    return x.view(w, B, w, SG // w, hl, d).permute(2, 1, 3, 0, 4, 5).reshape(w, B, SG // w, hl * w, d)


# ----------------------------------------------------------------- plain form

def _pow2(k):
    """2.0**k in 32 bits, k an int32 tensor in [-127, 127], from its bits."""
    bits = torch.where(k > -127, (k + 127) << 23, torch.full_like(k, 1 << 22))
    return bits.view(torch.float32)


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


def _dequantise(codes, scales):
    """32-bit values of codes [..., D] and scales [..., blocks]."""
    D = codes.shape[-1]
    s = _pow2(scales.view(torch.uint8).to(torch.int32) - 127)
    return codes.float() * s.repeat_interleave(BLOCK, -1)[..., :D]


def _mean(v, head):
    return v.mean(-1, keepdim=True) if head else v.mean((-2, -1), keepdim=True)


def _plain_norm(s):
    c, t = s["case"], TYPES[s["case"]["type"]]
    w, head, mode = c["w"], c["head"], c["mode"]
    h = s["x"] if mode == 0 else _to_p(s["x"], w)
    total = None
    if c["residual"]:
        total = (h.float() + s["residual"].float()).to(t)
        h = total
    h = h.float()
    rstd = 1.0 / torch.sqrt(_mean(h * h, head) + EPS)
    y = h * rstd * s["weight"].float().view(1, 1, 1, *((1,) if head else (c["H"],)), c["D"])
    got = {}
    if c["out"]:
        codes, scales = _quantise(y, c["out"])
        got["out"] = codes if mode else _to_a(codes.view(torch.uint8), w).view(codes.dtype)
        got["scales"] = scales if mode else _to_a(scales.view(torch.uint8), w).view(scales.dtype)
    else:
        y = y.to(t)
        got["out"] = y if mode else _to_a(y, w)
    if total is not None:
        got["sum"] = total
    if c["save"]:
        got["saved"], got["saved_scales"] = _quantise(h, c["save"])
        got["rstd"] = rstd.flatten(3 if head else 2)
    return got


def _plain_back(s):
    c, t = s["case"], TYPES[s["case"]["type"]]
    w, head, mode = c["w"], c["head"], c["mode"]
    if c["save"]:
        h = _dequantise(s["saved"], s["saved_scales"])
    else:
        h = (s["saved"] if mode == 0 or c["residual"] else _to_p(s["saved"], w)).float()
    dy = s["dy"].float() if mode else _to_p(s["dy"], w).float()
    rstd = s["rstd"].view(*s["rstd"].shape, *((1,) if head else (1, 1)))
    xh = h * rstd
    g = dy * s["weight"].float().view(1, 1, 1, *((1,) if head else (c["H"],)), c["D"])
    dh = rstd * (g - xh * _mean(g * xh, head))
    if c["residual"]:
        dh = dh + s["dsum"].float()
    dw = dy * xh
    dw = dw.view(-1, s["weight"].numel()).sum(0)
    dh = dh.to(t)
    got = {"dx": dh if mode == 0 else _to_a(dh, w), "dweight": dw}
    if c["residual"] and mode == 1:
        got["dresidual"] = dh
    return got


def _places(s):
    """Sequence, position and whether it is written, for every row of every sequence."""
    c = s["case"]
    t = torch.arange(c["each"], device=s["starts"].device)
    at = s["starts"].view(-1, 1) + t                           # within the capacity by construction
    return torch.arange(at.shape[0], device=at.device).view(-1, 1).expand_as(at), at, t < s["counts"].view(-1, 1)


def _plain_write(s):
    c = s["case"]
    seq, at, live = _places(s)
    n, each = at.shape
    live = live.view(1, n, each, 1, 1)
    for part, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantise(_to_a(x, c["w"]).float(), c["fmt"])
        for new, all_ in ((codes, s["codes"]), (scales, s["scales"])):
            new = new.view(torch.uint8)
            new = new.reshape(c["w"], n, each, *new.shape[-2:])
            to = all_[part].view(torch.uint8)
            to[:, seq, at] = torch.where(live, new, to[:, seq, at])
    return {"codes": s["codes"], "scales": s["scales"]}


def _plain_read(s):
    c, t = s["case"], TYPES[s["case"]["type"]]
    seq, at, live = _places(s)
    live = live.view(1, *live.shape, 1, 1)
    for part, out in enumerate((s["k_out"], s["v_out"])):
        codes = s["codes"][part].view(torch.uint8)[:, seq, at].view(s["codes"].dtype)
        scales = s["scales"][part].view(torch.uint8)[:, seq, at].view(s["scales"].dtype)
        out.copy_(torch.where(live, _dequantise(codes, scales).to(t), out))
    return {"k": s["k_out"], "v": s["v_out"]}


# ------------------------------------------------------------ the package's calls

def _own_norm(s):
    c = s["case"]
    if "plan" not in s:
        import ulysses_all_re_amd as ua
        s["plan"] = ua.Plan(c["w"], c["B"], c["S"], c["H"], c["D"], TYPES[c["type"]])
    r = s["plan"].norm_exchange(s["x"], s["weight"], c["mode"], residual=s.get("residual"), eps=EPS,
                                per_head=c["head"], out_dtype=FORMATS.get(c["out"]),
                                checkpoint=FORMATS.get(c["save"]), out=s.get("own_out"))
    s["own_out"] = r
    got = {"out": r.out}
    if c["out"]:
        got["scales"] = r.scales
    if c["residual"]:
        got["sum"] = r.sum
    if c["save"]:
        got.update(saved=r.saved, saved_scales=r.saved_scales, rstd=r.rstd)
    return got


def _own_back(s):
    c = s["case"]
    if "plan" not in s:
        import ulysses_all_re_amd as ua
        s["plan"] = ua.Plan(c["w"], c["B"], c["S"], c["H"], c["D"], TYPES[c["type"]])
    r = s["plan"].norm_exchange_backward(s["dy"], s["weight"], c["mode"], s["saved"], s["rstd"],
                                         saved_scales=s.get("saved_scales"), dsum=s.get("dsum"),
                                         residual=c["residual"], per_head=c["head"], out=s.get("own_out"))
    s["own_out"] = r
    got = {"dx": r.dx, "dweight": r.dweight}
    if c["residual"] and c["mode"] == 1:
        got["dresidual"] = r.dresidual
    return got


def _own_cache(s, B, S):
    if "cache" not in s:
        import ulysses_all_re_amd as ua
        c = s["case"]
        s["plan"] = ua.Plan(c["w"], B, S, c["H"], c["D"], TYPES[c["type"]])
        s["cache"] = ua.Cache.of(s["codes"], s["scales"])
    return s["plan"], s["cache"]


def _own_write(s):
    plan, cache = _own_cache(s, s["case"]["B"], s["case"]["S"])
    plan.cache_write(cache, s["k"], s["v"], s["starts"], s["counts"])
    return {"codes": cache.codes, "scales": cache.scales}


def _own_read(s):
    plan, cache = _own_cache(s, 1, 1)
    k, v = plan.cache_read(cache, s["case"]["each"], s["starts"], s["counts"], out=(s["k_out"], s["v_out"]))
    return {"k": k, "v": v}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _own_norm, "back": _own_back, "write": _own_write, "read": _own_read}[op](s)
    return {"norm": _plain_norm, "back": _plain_back, "write": _plain_write, "read": _plain_read}[op](s)


# --------------------------------------------------------------------- inputs

def _activations(shape, t, gen):
    """Values as a projection gives them: normal, some channels of a head much larger, tokens of different size."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= 0.3 + torch.rand(shape[:-2] + (1, 1), generator=gen, device="cuda")
    x *= torch.exp(0.7 * torch.randn(shape[-1], generator=gen, device="cuda"))
    return x.to(t)


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    c, t = dict(case), TYPES[case["type"]]
    w, H, D, op = c["w"], c["H"], c["D"], c["op"]
    s = {"case": c}
    if op in ("norm", "back"):
        p = (w, c["B"], c["S"], H, D)
        a = (w, c["B"], c["S"] * w, H // w, D)
        weight = 1 + 0.2 * torch.randn(D if c["head"] else H * D, generator=gen, device="cuda")
        s["weight"] = weight.to(t)
        if op == "norm":
            s["x"] = _activations(p if c["mode"] == 0 else a, t, gen)
            if c["residual"]:
                s["residual"] = _activations(p, t, gen)
            return s
        h = _activations(p, t, gen)
        s["dy"] = (torch.randn(a if c["mode"] == 0 else p, generator=gen, device="cuda") * 0.02).to(t)
        h32 = h.float()
        rstd = 1.0 / torch.sqrt(_mean(h32 * h32, c["head"]) + EPS)
        s["rstd"] = rstd.flatten(3 if c["head"] else 2)
        if c["save"]:
            s["saved"], s["saved_scales"] = _quantise(h32, c["save"])
        else:
            s["saved"] = h if c["mode"] == 0 or c["residual"] else _to_a(h, w)
        if c["residual"]:
            s["dsum"] = (torch.randn(p, generator=gen, device="cuda") * 0.02).to(t)
        return s
    n = c["B"] * c["S"] * w // c["each"] if op == "write" else c["seqs"]
    room = c["cap"] - c["each"]
    s["starts"] = torch.randint(0, room + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    s["counts"] = torch.full((n,), c["each"], device="cuda", dtype=torch.int32)
    if n > 1 and c["each"] > 1:
        least = c["each"] // 2
        s["counts"] = torch.randint(least, c["each"] + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
    nb = -(-D // BLOCK)
    hl = H // w
    if op == "write":
        # the cache holds earlier sequences' codes
        shape = (2, w, n, c["cap"], hl)
        s["codes"] = torch.randint(0, 120, shape + (D,), generator=gen, device="cuda",
                                   dtype=torch.uint8).view(FORMATS[c["fmt"]])
        s["scales"] = torch.randint(110, 130, shape + (nb,), generator=gen, device="cuda",
                                    dtype=torch.uint8).view(torch.float8_e8m0fnu)
        p = (w, c["B"], c["S"], H, D)
        s["k"], s["v"] = _activations(p, t, gen), _activations(p, t, gen)
        return s
    both = [_quantise(_activations((w, n, c["cap"], hl, D), t, gen).float(), c["fmt"]) for _ in range(2)]
    s["codes"] = torch.stack([q.view(torch.uint8) for q, _ in both]).view(FORMATS[c["fmt"]])
    s["scales"] = torch.stack([q.view(torch.uint8) for _, q in both]).view(torch.float8_e8m0fnu)
    s["k_out"] = torch.zeros((w, n, c["each"], hl, D), dtype=t, device="cuda")
    s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ------------------------------------------------------- the definition, in 64 bits

def _index_a(c):
    """A-layout places of the P layout's heads: rank, gathered token, head of the rank."""
    dev = "cuda"
    j = torch.arange(c["w"], device=dev).view(-1, 1, 1, 1)
    b = torch.arange(c["B"], device=dev).view(1, -1, 1, 1)
    i = torch.arange(c["S"], device=dev).view(1, 1, -1, 1)
    h = torch.arange(c["H"], device=dev).view(1, 1, 1, -1)
    hl = c["H"] // c["w"]
    return h // hl, b, j * c["S"] + i, h % hl


def _exact_codes(v, fmt):
    """The values of the codes, and the scales, of 64-bit values [..., D]."""
    codes, scales = torch.empty_like(v), []
    for lo in range(0, v.shape[-1], BLOCK):
        x = v[..., lo:lo + BLOCK]
        top = x.abs().amax(-1, keepdim=True)
        k = torch.ceil(torch.log2(top / (1.75 * 2.0 ** TOP[fmt])))
        # the logarithm may be off next to a whole number
        k = torch.where(top > 1.75 * torch.exp2(k + TOP[fmt]), k + 1, k)
        k = torch.where(top <= 1.75 * torch.exp2(k - 1 + TOP[fmt]), k - 1, k)
        k = torch.where(top == 0, torch.full_like(k, -127.0), k).clamp_min(-127.0)
        x = x * torch.exp2(-k)
        ex = torch.frexp(x)[1].to(torch.float64) - 1
        step = torch.exp2(ex.clamp_min(LEAST[fmt]) - MANTISSA[fmt])
        codes[..., lo:lo + BLOCK] = torch.round(x / step) * step
        scales.append(torch.exp2(k))
    return codes, torch.cat(scales, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    w = c["w"]
    if c["op"] in ("norm", "back"):
        at = _index_a(c)

        def scatter(v):
            out = v.new_empty(w, c["B"], c["S"] * w, c["H"] // w, v.shape[-1])
            out[at] = v
            return out

        dims = (4,) if c["head"] else (3, 4)
        count = c["D"] if c["head"] else c["H"] * c["D"]
        wt = s["weight"].double().expand(c["H"], c["D"]) if c["head"] else s["weight"].double().view(c["H"], c["D"])
    if c["op"] == "norm":
        h = (s["x"] if c["mode"] == 0 else s["x"][at]).double()
        got = {}
        if c["residual"]:
            got["sum"] = h + s["residual"].double()
            h = got["sum"].to(TYPES[c["type"]]).double()       # the sum is what the type holds of it
        rstd = (h.square().sum(dims, keepdim=True) / count + EPS).rsqrt()
        y = h * rstd * wt
        if c["out"]:
            y, sc = _exact_codes(y, c["out"])
            got["scales"] = sc if c["mode"] else scatter(sc)
        got["out"] = y if c["mode"] else scatter(y)
        if c["save"]:
            got["saved"], got["saved_scales"] = _exact_codes(h, c["save"])
            got["rstd"] = rstd.reshape(rstd.shape[:4] if c["head"] else rstd.shape[:3])
        return got
    if c["op"] == "back":
        if c["save"]:
            sc = s["saved_scales"].double()
            h = s["saved"].double() * sc[..., torch.arange(c["D"], device=sc.device) // BLOCK]
        else:
            h = (s["saved"] if c["mode"] == 0 or c["residual"] else s["saved"][at]).double()
        dy = (s["dy"] if c["mode"] == 1 else s["dy"][at]).double()
        rstd = s["rstd"].double()
        rstd = rstd[..., None] if c["head"] else rstd[..., None, None]
        xh = h * rstd
        dw = (dy * xh).sum((0, 1, 2))
        g = dy * wt
        dh = rstd * (g - xh * ((g * xh).sum(dims, keepdim=True) / count))
        if c["residual"]:
            dh += s["dsum"].double()
        got = {"dx": dh if c["mode"] == 0 else scatter(dh), "dweight": dw.sum(0) if c["head"] else dw.flatten()}
        if c["residual"] and c["mode"] == 1:
            got["dresidual"] = dh
        return got
    starts, counts = s["starts"].tolist(), s["counts"].tolist()
    if c["op"] == "write":
        codes, scales = s["codes"].double(), s["scales"].double()
        at = _index_a(c)
        for part, x in enumerate((s["k"], s["v"])):
            q, sc = _exact_codes(x.double(), c["fmt"])
            for new, all_ in ((q, codes), (sc, scales)):
                flat = new.new_empty(w, c["B"], c["S"] * w, c["H"] // w, new.shape[-1])
                flat[at] = new
                flat = flat.view(w, len(starts), c["each"], c["H"] // w, new.shape[-1])
                for i, (a, n) in enumerate(zip(starts, counts)):
                    all_[part, :, i, a:a + n] = flat[:, i, :n]
        return {"codes": codes, "scales": scales}
    got = {}
    for part, name in enumerate(("k", "v")):
        out = torch.zeros_like(s["k_out"], dtype=torch.float64)
        for i, (a, n) in enumerate(zip(starts, counts)):
            sc = s["scales"][part, :, i, a:a + n].double()
            d = torch.arange(c["D"], device=sc.device) // BLOCK
            out[:, i, :n] = s["codes"][part, :, i, a:a + n].double() * sc[..., d]
        got[name] = out
    return got
