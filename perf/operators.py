"""The transformer-block operators around the detection head, as they are measured: the calls, their plain forms and
their definitions in 64 bits.

Prompt rows become kernels in a few transformer blocks (projections with bias, activation, layer scale and residual;
queries and keys with norms and rotary positions; attention of the rows among themselves and over the query image's
patches), and the same operators carry the image and text towers in front of the head. Three operators:

  linear         out = residual + scale * act(x weight^T + bias)
  qk_norm_rope   RMS norm of every query and key head, then the rotation by positions on one to three axes
  attention      softmax(scale q k^T) v under a key mask and, for text, a causal one; several query heads may share a key head

Case fields: linear: rows, cin, cout, dt, odt (output type), act, scale, residual. qk_norm_rope: batch, rows, heads, kv (key
heads), d, axes, rot (rotated pairs of a head's d / 2), style (half: pairs (i, i + rot); pairs: (2 i, 2 i + 1)), norm, grid (what
the positions are), dt. attention: batch, q, k (rows), heads, kv, d, causal, mask (all, prefix: 5 to k valid rows, holes: each
key present or not, some batches with none), packed (one buffer of keys and values, or heads ahead of rows), dt.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_FLOPS = {"linear": 4.9e11, "qk_norm_rope": 2e9, "attention": 2.2e11}


def listed():
    return [
        # text features of one class's 17 keypoint names to the head's 2048 columns: the smallest product, latency bound
        {"name": "linear_text_17", "op": "linear", "rows": 17, "cin": 1280, "cout": 2048, "dt": "bf16", "odt": "bf16",
         "act": "none", "scale": False, "residual": False},
        # the prompt rows of 64 crops (80 each) through the first half of a feed-forward of width 1024
        {"name": "linear_rows_5120", "op": "linear", "rows": 5120, "cin": 1024, "cout": 1024, "dt": "bf16", "odt": "bf16",
         "act": "quick_gelu", "scale": False, "residual": False},
        # 64 crops of 24 x 24 patches through the wide half of a tower's feed-forward: the largest product
        {"name": "linear_patches_up", "op": "linear", "rows": 36864, "cin": 1280, "cout": 5120, "dt": "bf16",
         "odt": "bf16", "act": "gelu", "scale": False, "residual": False},
        # 16 crops of 576 patches and 5 extra tokens (an odd count) back down, with layer scale, onto the fp32 residual stream
        {"name": "linear_down_9296", "op": "linear", "rows": 9296, "cin": 4096, "cout": 1024, "dt": "bf16", "odt": "f32",
         "act": "none", "scale": True, "residual": True},
        # the fp32 rows of 80 prompt sets of 17, as pooling writes them
        {"name": "linear_rows_f32", "op": "linear", "rows": 1360, "cin": 1024, "cout": 1024, "dt": "f32", "odt": "f32",
         "act": "gelu", "scale": False, "residual": True},
        # the tokens of one keypoint name: the smallest call
        {"name": "rope_text_77", "op": "qk_norm_rope", "batch": 1, "rows": 77, "heads": 20, "kv": 20, "d": 64, "axes": 1,
         "rot": 32, "style": "half", "norm": True, "grid": "text", "dt": "bf16"},
        # 64 crops of 24 x 24 patches and 5 unrotated tokens, rotation alone, by rows and columns
        {"name": "rope_patches", "op": "qk_norm_rope", "batch": 64, "rows": 581, "heads": 20, "kv": 20, "d": 64, "axes": 2,
         "rot": 32, "style": "half", "norm": False, "grid": "patches", "dt": "bf16"},
        # two clips of 8 frames of 24 x 24 patches, three axes, fp32, heads of 80 that share keys
        {"name": "rope_frames_f32", "op": "qk_norm_rope", "batch": 2, "rows": 4608, "heads": 16, "kv": 4, "d": 80, "axes": 3,
         "rot": 40, "style": "pairs", "norm": True, "grid": "frames", "dt": "f32"},
        # one prompt row over the 48 x 48 patches of one crop
        {"name": "attention_row", "op": "attention", "batch": 1, "q": 1, "k": 2304, "heads": 16, "kv": 16, "d": 64,
         "causal": False, "mask": "all", "packed": True, "dt": "bf16"},
        # 80 prompt rows over the 576 patches of each of 64 crops
        {"name": "attention_cross", "op": "attention", "batch": 64, "q": 80, "k": 576, "heads": 16, "kv": 16, "d": 64,
         "causal": False, "mask": "all", "packed": True, "dt": "bf16"},
        # the patches of 8 crops of 48 x 48 and 5 extra tokens among themselves: the largest
        {"name": "attention_patches", "op": "attention", "batch": 8, "q": 2309, "k": 2309, "heads": 20, "kv": 20, "d": 64,
         "causal": False, "mask": "all", "packed": True, "dt": "bf16"},
        # the padded visual and text rows of 64 crops among themselves in fp32
        {"name": "attention_rows_f32", "op": "attention", "batch": 64, "q": 160, "k": 160, "heads": 16, "kv": 16, "d": 64,
         "causal": False, "mask": "prefix", "packed": False, "dt": "f32"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _cost(c):
    if c["op"] == "linear":
        return 2.0 * c["rows"] * c["cin"] * c["cout"]
    if c["op"] == "qk_norm_rope":
        return 10.0 * c["batch"] * c["rows"] * (c["heads"] + c["kv"]) * c["d"]
    return 4.0 * c["batch"] * c["heads"] * c["q"] * c["k"] * c["d"]


def draw(rng):
    op = rng.choice(["linear", "qk_norm_rope", "attention"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "linear":
        c = {"op": op, "rows": _spread(rng, 1, 36864), "cin": 8 * _spread(rng, 8, 640), "cout": 8 * _spread(rng, 8, 640),
             "dt": dt, "odt": dt if rng.random() < 0.7 else "f32", "act": rng.choice(["none", "relu", "gelu", "quick_gelu"]),
             "scale": rng.random() < 0.3, "residual": rng.random() < 0.5}
        size = "rows"
    else:
        heads = rng.choice([4, 8, 12, 16, 20])
        kv = rng.choice([n for n in range(1, heads + 1) if heads % n == 0 and n >= heads // 4])
        if op == "qk_norm_rope":
            d = rng.choice([32, 64, 64, 80, 96, 128])
            axes = rng.choice([1, 2, 2, 3])
            c = {"op": op, "batch": _spread(rng, 1, 64), "rows": _spread(rng, 1, 4613), "heads": heads, "kv": kv, "d": d,
                 "axes": axes, "rot": d // 2 if rng.random() < 0.7 else d // 4, "style": rng.choice(["half", "pairs"]),
                 "norm": rng.random() < 0.6, "grid": {1: "text", 2: "patches", 3: "frames"}[axes], "dt": dt}
        else:
            q = _spread(rng, 1, 2309)
            causal = rng.random() < 0.25
            c = {"op": op, "batch": _spread(rng, 1, 64), "q": q,
                 "k": max(q, _spread(rng, 1, 2309)) if causal else _spread(rng, 1, 4613), "heads": heads, "kv": kv,
                 "d": rng.choice([32, 64, 64, 72, 80, 96, 128]), "causal": causal,
                 "mask": rng.choice(["all", "prefix", "holes"]), "packed": rng.random() < 0.5, "dt": dt}
        size = "batch"
    while _cost(c) > MOST_FLOPS[op]:
        c[size] = max(1, c[size] // 2)
    return c


def _heads(buffer, batch, rows, heads, d, ahead):
    """[batch][rows][heads][d] over a buffer, with the heads beside one another in a row or ahead of the rows."""
    if ahead:
        return buffer.view(batch, heads, rows, d).transpose(1, 2)
    return buffer.view(batch, rows, heads, d)


def _positions(grid, rows, axes, rng):
    """[rows][axes] positions: token numbers, patch centres of a square in -1..1 behind unrotated tokens, or (frame, row, column)."""
    if grid == "text":
        # a batch's window into a long running position
        return (torch.arange(rows, device="cuda").float() + int(rng[0]))[:, None]
    if grid == "patches":
        side = max(1, int(math.isqrt(rows)))
        extra = rows - side * side
        at = (torch.arange(side, device="cuda").float() + 0.5) / side * 2 - 1
        pos = torch.stack(torch.meshgrid(at, at, indexing="ij"), -1).reshape(-1, 2)
        return torch.cat([torch.zeros(extra, 2, device="cuda"), pos])
    n = torch.arange(rows, device="cuda")
    return torch.stack([n // 576 + int(rng[0]), n % 576 // 24, n % 24], -1).float()


def _frequencies(grid, rot, axes):
    """(axis of each pair, radians per unit of position of each pair): the pairs are shared out among the axes in runs."""
    per = -(-rot // axes)
    n = torch.arange(rot, device="cuda")
    axis, step = n // per, (n % per).double() / per
    base = 100.0 if grid == "patches" else 10000.0
    freq = base ** -step
    return axis.to(torch.uint8), (2 * math.pi * freq if grid == "patches" else freq).float()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dt="f32", std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(DT[dt])

    s = {"case": c}
    if c["op"] == "linear":
        s["x"] = normal(c["rows"], c["cin"], dt=c["dt"])
        s["weight"] = normal(c["cout"], c["cin"], dt=c["dt"], std=c["cin"] ** -0.5)
        s["bias"] = normal(c["cout"], std=0.1)
        s["scale"] = torch.rand(c["cout"], generator=g, device="cuda") * 0.9 + 0.1 if c["scale"] else None
        s["residual"] = normal(c["rows"], c["cout"], dt=c["odt"]) if c["residual"] else None
        s["out"] = torch.empty(c["rows"], c["cout"], dtype=DT[c["odt"]], device="cuda")
    elif c["op"] == "qk_norm_rope":
        b, t, h, kv, d = (c[n] for n in ("batch", "rows", "heads", "kv", "d"))
        s["q"] = normal(b, t, h, d, dt=c["dt"])
        s["k"] = normal(b, t, kv, d, dt=c["dt"])
        s["q_weight"] = 1 + normal(d, std=0.1) if c["norm"] else None
        s["k_weight"] = 1 + normal(d, std=0.1) if c["norm"] else None
        first = torch.randint(0, 20000, (1,), generator=g, device="cuda").tolist()
        s["pos"] = _positions(c["grid"], t, c["axes"], first).contiguous()
        s["axis"], s["freq"] = _frequencies(c["grid"], c["rot"], c["axes"])
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
    else:
        b, tq, tk, h, kv, d = (c[n] for n in ("batch", "q", "k", "heads", "kv", "d"))
        s["q"] = _heads(normal(b * tq * h * d, dt=c["dt"], std=1.5), b, tq, h, d, not c["packed"])
        if c["packed"]:
            both = normal(b, tk, 2 * kv, d, dt=c["dt"])
            s["k"], s["v"] = both[:, :, :kv], both[:, :, kv:]
        else:
            s["k"] = _heads(normal(b * tk * kv * d, dt=c["dt"]), b, tk, kv, d, True)
            s["v"] = _heads(normal(b * tk * kv * d, dt=c["dt"]), b, tk, kv, d, True)
        s["mask"] = None
        if c["mask"] == "prefix":
            low = min(5, tk)
            count = torch.randint(low, tk + 1, (b, 1), generator=g, device="cuda")
            s["mask"] = (torch.arange(tk, device="cuda")[None] < count).to(torch.uint8)
        elif c["mask"] == "holes":
            share = torch.randint(0, 5, (b, 1), generator=g, device="cuda") / 4
            s["mask"] = (torch.rand(b, tk, generator=g, device="cuda") < share).to(torch.uint8)
        s["out"] = torch.empty(b, tq, h, d, dtype=DT[c["dt"]], device="cuda")
    return s


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["weight"].float().t() + s["bias"]
    if c["act"] == "relu":
        y = torch.clamp(y, min=0)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    elif c["act"] == "quick_gelu":
        y = y / (1 + torch.exp(-1.702 * y))
    if s["scale"] is not None:
        y = y * s["scale"]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DT[c["odt"]])


def _plain_rope(s):
    c = s["case"]
    rot, half = c["rot"], c["style"] == "half"
    angle = s["pos"].double()[:, s["axis"].long()] * s["freq"].double()     # [rows][rot]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    outs = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        y = x.float()
        if weight is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight
        turn, rest = y[..., :2 * rot], y[..., 2 * rot:]
        a, b = (turn[..., :rot], turn[..., rot:]) if half else (turn[..., 0::2], turn[..., 1::2])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        turned = torch.cat([ra, rb], -1) if half else torch.stack([ra, rb], -1).flatten(-2)
        outs.append(torch.cat([turned, rest], -1).to(x.dtype))
    return outs


def _plain_attention(s):
    c = s["case"]
    group = c["heads"] // c["kv"]
    q = s["q"].float().transpose(1, 2)                                      # [batch][heads][q][d]
    k = s["k"].float().transpose(1, 2).repeat_interleave(group, 1)
    v = s["v"].float().transpose(1, 2).repeat_interleave(group, 1)
    x = (q @ k.transpose(-1, -2)) * c["d"] ** -0.5
    hide = None
    if s["mask"] is not None:
        hide = (s["mask"] == 0)[:, None, None]
    if c["causal"]:
        i = torch.arange(c["q"], device=x.device)[:, None] + (c["k"] - c["q"])
        later = torch.arange(c["k"], device=x.device)[None] > i
        hide = later if hide is None else hide | later
    if hide is not None:
        x = torch.where(hide, -math.inf, x)
    top = torch.clamp(x.amax(-1, keepdim=True), min=-3e38)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    y = (p @ v) / torch.where(total == 0, 1.0, total)                       # rows whose mask leaves nothing: 0
    return y.transpose(1, 2).contiguous().to(DT[c["dt"]])


def run(state):
    s, c = state, state["case"]
    if own:
        from prompt_conditioned_keypoint_b200 import binding as gk
        dt = gk.GKD_BF16 if c["dt"] == "bf16" else gk.GKD_F32
        if c["op"] == "linear":
            act = {"none": gk.GKD_ACT_NONE, "relu": gk.GKD_ACT_RELU, "gelu": gk.GKD_ACT_GELU,
                   "quick_gelu": gk.GKD_ACT_QUICK_GELU}[c["act"]]
            gk.gkd_linear(s["x"], dt, c["rows"], c["cin"], c["cin"], s["weight"], c["cout"], s["bias"], act, s["scale"],
                          s["residual"], c["cout"], s["out"], gk.GKD_BF16 if c["odt"] == "bf16" else gk.GKD_F32, c["cout"])
            return s["out"]
        if c["op"] == "qk_norm_rope":
            gk.gkd_qk_norm_rope(s["q"], s["k"], dt, c["batch"], c["rows"], c["d"], s["q_weight"], s["k_weight"], 1e-6,
                                s["pos"], 0, c["axes"], s["axis"], s["freq"], c["rot"], c["style"] == "pairs", s["q_out"],
                                s["k_out"])
            return [s["q_out"], s["k_out"]]
        gk.gkd_attention(s["q"], s["k"], s["v"], dt, c["batch"], c["q"], c["k"], c["d"], c["d"] ** -0.5, c["causal"],
                         s["mask"], c["k"], s["out"])
        return s["out"]
    if c["op"] == "linear":
        return _plain_linear(s)
    return _plain_rope(s) if c["op"] == "qk_norm_rope" else _plain_attention(s)


def work(case):
    c = case
    size = 2 if c["dt"] == "bf16" else 4
    if c["op"] == "linear":
        osize = 2 if c["odt"] == "bf16" else 4
        outs = c["rows"] * c["cout"] * osize
        return {"bytes": (c["rows"] + c["cout"]) * c["cin"] * size + outs * (2 if c["residual"] else 1)
                + 4 * c["cout"] * (2 if c["scale"] else 1), "flops": 2 * c["rows"] * c["cin"] * c["cout"]}
    if c["op"] == "qk_norm_rope":
        n = c["batch"] * c["rows"] * (c["heads"] + c["kv"])
        return {"bytes": 2 * n * c["d"] * size + 4 * c["rows"] * c["axes"],
                "flops": n * (6 * c["rot"] + (4 * c["d"] if c["norm"] else 0))}
    # the keys that the mask leaves, as the inputs draw them: all, 5 to k, or one half
    share = 1.0 if c["mask"] == "all" else (0.5 + 0.5 * min(5, c["k"]) / c["k"]) if c["mask"] == "prefix" else 0.5
    pairs = c["q"] * c["k"] - (c["q"] * (c["q"] - 1) // 2 if c["causal"] else 0)
    return {"bytes": c["batch"] * c["d"] * size * (2 * c["q"] * c["heads"] + 2 * share * c["k"] * c["kv"])
            + (c["batch"] * c["k"] if c["mask"] != "all" else 0),
            "flops": 4 * c["batch"] * c["heads"] * share * pairs * c["d"]}


def _exact_linear(c, s):
    y = torch.addmm(s["bias"].double(), s["x"].double(), s["weight"].double().t())
    f = {"none": lambda z: z, "relu": lambda z: z * (z > 0), "quick_gelu": lambda z: z * torch.sigmoid(1.702 * z),
         "gelu": lambda z: z * torch.special.ndtr(z)}[c["act"]]
    y = f(y)
    if s["scale"] is not None:
        y = torch.einsum("tn,n->tn", y, s["scale"].double())
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_rope(c, s):
    n = c["rot"]
    freq = s["freq"].double()
    angle = sum((s["axis"] == a) * freq * s["pos"][:, a, None].double() for a in range(c["axes"]))
    turn = torch.polar(torch.ones_like(angle), angle)[None, :, None]        # unit complex numbers
    outs = []
    for x, weight in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        z = x.double().clone()
        if weight is not None:
            z = torch.einsum("bthd,bth,d->bthd", z, (z.square().sum(-1) / c["d"] + 1e-6).rsqrt(), weight.double())
        first, second = (slice(0, n), slice(n, 2 * n)) if c["style"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        w = torch.complex(z[..., first], z[..., second]) * turn
        z[..., first], z[..., second] = w.real, w.imag
        outs.append(z)
    return outs


def _exact_attention(c, s):
    group = c["heads"] // c["kv"]
    out = torch.zeros(c["batch"], c["q"], c["heads"], c["d"], dtype=torch.float64, device="cuda")
    reach = torch.arange(c["q"], device="cuda") + c["k"] - c["q"] if c["causal"] else None
    for b in range(c["batch"]):
        keep = torch.arange(c["k"], device="cuda") if s["mask"] is None else s["mask"][b].nonzero()[:, 0]
        if not len(keep):
            continue
        for h in range(c["heads"]):
            x = s["q"][b, :, h].double() @ s["k"][b, keep, h // group].double().t() / math.sqrt(c["d"])
            if reach is not None:
                x = x.masked_fill(keep[None] > reach[:, None], -math.inf)
            w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
            out[b, :, h] = w @ s["v"][b, keep, h // group].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"linear": _exact_linear, "qk_norm_rope": _exact_rope, "attention": _exact_attention}[case["op"]](case, s)
