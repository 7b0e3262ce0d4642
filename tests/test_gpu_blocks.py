"""GPU: the transformer-block operators against their definitions in 64 bits.

Tolerances. u = torch.finfo(type).eps / 2 is one rounding (bf16 2^-8, fp32 2^-24).
linear: one rounding of the result, u |y|; the sum of Cin products in fp32, in any
order and with truncation, is within (Cin + 16) 2^-23 of sum |x w| + |b|, which the
activation (slope at most 1.13) and the scale carry on; the epilogue's own fp32
operations (the exponential and erf are within 2^-20 of their value) add 2^-19
of |b| + |y| + |residual|.
qk_norm_rope: u |y|, and (D / 2 + 24) 2^-24 of |a| + |b| of the pair: the sum of
squares, the reciprocal root, the reduced angle (half a turn rounded to fp32) and
six operations.
attention: u |y|; the weights' rounding for the second product, u of sum p |v| /
sum p (bf16 only); a score off by d = (D + 8) 2^-23 scale sum |q k| changes every
weight by 2 d at most (numerator and sum); sums and exponentials, (Tk + 24) 2^-22.
"""
import math

import pytest
import torch

from prompt_conditioned_keypoint_b200 import binding as gk

pytestmark = pytest.mark.gpu
DT = {"bf16": (torch.bfloat16, gk.GKD_BF16), "f32": (torch.float32, gk.GKD_F32)}
ACTS = {"none": gk.GKD_ACT_NONE, "relu": gk.GKD_ACT_RELU, "gelu": gk.GKD_ACT_GELU, "quick_gelu": gk.GKD_ACT_QUICK_GELU}


def unit(dt):
    return torch.finfo(DT[dt][0]).eps / 2


def rand(seed, *shape, dt="f32", std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(DT[dt][0]).cuda()


def check(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape
    assert bool(torch.isfinite(got).all()), what
    over = ((got - ref).abs() - tol).max().item() if ref.numel() else -1.0
    assert over <= 0, f"{what}: {over:.3e} over the bound"


def settle():
    torch.cuda.synchronize()
    gk.gkd_check_device_error()


# ------------------------------------------------------------------ linear
def linear_ref(x, w, b, act, scale, res, odt):
    x, w = x.double(), w.double()
    y = x @ w.t()
    size = x.abs() @ w.abs().t()
    if b is not None:
        y, size = y + b.double(), size + b.double().abs()
    slack = (x.shape[1] + 16) * 2.0 ** -23 * 1.13 * size + 2.0 ** -19 * (size if b is None else b.double().abs())
    y = {"none": lambda z: z, "relu": torch.relu, "gelu": lambda z: 0.5 * z * (1 + torch.erf(z / math.sqrt(2))),
         "quick_gelu": lambda z: z * torch.sigmoid(1.702 * z)}[act](y)
    slack = slack + 2.0 ** -19 * y.abs()
    if scale is not None:
        y, slack = y * scale.double(), slack * scale.double().abs()
    if res is not None:
        y, slack = y + res.double(), slack + 2.0 ** -19 * res.double().abs()
    return y, unit(odt) * y.abs() + slack


LINEAR = [
    # T, Cin, Cout, dt, odt, act, bias, scale, residual
    (1, 8, 8, "bf16", "bf16", "none", True, False, False),
    (1, 1280, 2048, "bf16", "bf16", "none", True, False, False),
    (2, 72, 24, "bf16", "f32", "relu", False, True, True),
    (17, 1280, 520, "bf16", "bf16", "gelu", True, True, True),
    (31, 200, 136, "bf16", "f32", "quick_gelu", True, False, True),
    (64, 1024, 264, "bf16", "bf16", "none", False, False, False),
    (80, 1024, 1024, "bf16", "f32", "none", True, True, True),
    (127, 64, 128, "bf16", "bf16", "gelu", True, False, False),
    (128, 136, 256, "bf16", "bf16", "quick_gelu", True, True, False),
    (129, 520, 1288, "bf16", "f32", "gelu", True, False, True),
    (581, 1024, 1024, "bf16", "bf16", "none", True, True, True),
    (581, 4096, 200, "bf16", "f32", "none", True, False, False),
    (1360, 1096, 808, "bf16", "bf16", "relu", True, False, True),
    (2600, 320, 2056, "bf16", "bf16", "gelu", True, True, True),
    (5000, 1096, 1032, "bf16", "f32", "quick_gelu", True, True, True),
    (1, 8, 8, "f32", "f32", "none", True, False, False),
    (3, 1024, 40, "f32", "f32", "gelu", True, True, True),
    (17, 264, 1032, "f32", "f32", "quick_gelu", True, False, True),
    (80, 1024, 1024, "f32", "f32", "none", True, True, True),
    (200, 72, 136, "f32", "f32", "relu", False, False, False),
    (1360, 520, 520, "f32", "f32", "gelu", True, False, True),
    (3000, 200, 1000, "f32", "f32", "quick_gelu", True, True, True),
]

# every tile width of the kernel for many rows (256, 192 and 128 columns), several tiles per CTA, both output types,
# with and without a residual
LINEAR += [
    (4700, 264, 1024, "bf16", "bf16", "gelu", True, False, False),
    (9400, 72, 1000, "bf16", "bf16", "none", True, False, True),
    (4700, 1096, 1024, "bf16", "f32", "none", True, True, True),
    (9400, 520, 1024, "bf16", "f32", "relu", False, False, False),
    (5000, 200, 1032, "bf16", "bf16", "gelu", True, False, False),
    (5000, 1096, 1032, "bf16", "f32", "none", True, False, False),
    (1360, 520, 808, "bf16", "bf16", "quick_gelu", True, False, False),
    (1360, 1096, 808, "bf16", "f32", "none", True, True, True),
    (1400, 1096, 800, "bf16", "f32", "gelu", True, False, False),
    (20000, 64, 8, "bf16", "bf16", "none", True, True, True),
    (3, 8192, 24, "bf16", "f32", "none", True, False, False),
    (700, 9000, 72, "bf16", "f32", "none", True, False, True),
    (5, 65536, 16, "bf16", "bf16", "none", True, False, False),
    (5, 8, 65536, "bf16", "bf16", "none", True, False, False),
    (130, 4104, 136, "f32", "f32", "none", True, False, True),
]


def linear_case(T, Cin, Cout, dt, odt, act, bias, scale, res, seed=1):
    x, w = rand(seed, T, Cin, dt=dt), rand(seed + 1, Cout, Cin, dt=dt, std=Cin ** -0.5)
    b = rand(seed + 2, Cout) if bias else None
    s = rand(seed + 3, Cout) if scale else None
    r = rand(seed + 4, T, Cout, dt=odt) if res else None
    return x, w, b, s, r


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "-".join(str(v) for v in c))
def test_linear(case):
    T, Cin, Cout, dt, odt, act, *_ = case
    x, w, b, s, r = linear_case(*case)
    out = torch.full((T, Cout), 777.0, dtype=DT[odt][0], device="cuda")
    gk.gkd_linear(x, DT[dt][1], T, Cin, Cin, w, Cout, b, ACTS[act], s, r, Cout, out, DT[odt][1], Cout)
    settle()
    check(out, *linear_ref(x, w, b, act, s, r, odt), "linear")


@pytest.mark.parametrize("T,dt,odt", [(5, "bf16", "bf16"), (150, "bf16", "f32"), (4000, "bf16", "bf16"),
                                      (5, "f32", "f32"), (700, "f32", "f32")])
def test_linear_strides_and_residual_in_place(T, dt, odt):
    Cin, Cout = 200, 520
    wide = rand(5, T, Cin + 24, dt=dt)
    x = wide[:, 8:8 + Cin]
    _, w, b, s, _ = linear_case(T, Cin, Cout, dt, odt, "none", True, True, False)
    buf = rand(6, T + 2, Cout + 40, dt=odt)
    before = buf.clone()
    out = buf[1:T + 1, 16:16 + Cout]
    ref, tol = linear_ref(x, w, b, "none", s, before[1:T + 1, 16:16 + Cout], odt)
    gk.gkd_linear(x, DT[dt][1], T, Cin, Cin + 24, w, Cout, b, gk.GKD_ACT_NONE, s, out, Cout + 40, out, DT[odt][1],
                  Cout + 40)
    settle()
    check(out, ref, tol, "strided linear")
    buf[1:T + 1, 16:16 + Cout] = before[1:T + 1, 16:16 + Cout]
    assert torch.equal(buf, before)                       # nothing beside the output was touched


@pytest.mark.parametrize("T", [3, 300, 5000])
def test_linear_keeps_infinities_and_nan_to_their_own_rows(T):
    Cin, Cout = 136, 264
    x, w, b, _, _ = linear_case(T, Cin, Cout, "bf16", "bf16", "none", True, False, False)
    x[1, 3] = math.inf
    x[2] = math.nan
    out = torch.empty(T, Cout, dtype=torch.bfloat16, device="cuda")
    gk.gkd_linear(x, gk.GKD_BF16, T, Cin, Cin, w, Cout, b, gk.GKD_ACT_NONE, None, None, 0, out, gk.GKD_BF16, Cout)
    settle()
    assert bool(torch.isinf(out[1].float()).all()) and bool(torch.isnan(out[2].float()).all())
    rows = [i for i in range(T) if i not in (1, 2)]
    check(out[rows], *linear_ref(x[rows], w, b, "none", None, None, "bf16"), "other rows")


def test_linear_output_rows_past_32_bit_offsets():
    T, Cin, Cout, stride = 3, 64, 64, 2 ** 31 + 64
    x, w, b, _, _ = linear_case(T, Cin, Cout, "bf16", "bf16", "none", True, False, False)
    buf = torch.empty(2 * stride + Cout, dtype=torch.bfloat16, device="cuda")
    gk.gkd_linear(x, gk.GKD_BF16, T, Cin, Cin, w, Cout, b, gk.GKD_ACT_NONE, None, None, 0, buf, gk.GKD_BF16, stride)
    settle()
    out = torch.stack([buf[i * stride:i * stride + Cout] for i in range(T)])
    check(out, *linear_ref(x, w, b, "none", None, None, "bf16"), "far rows")


# ------------------------------------------------------------------ qk_norm_rope
def rope_ref(x, weight, eps, pos, axis, freq, pairs, inter):
    y = x.double()
    D = y.shape[-1]
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    size = y.abs()
    if pairs:
        angle = (pos.double()[..., axis.long()] * freq.double()).unsqueeze(-2)    # [B or 1][T][1][pairs]
        c, s = torch.cos(angle), torch.sin(angle)
        ia = torch.arange(pairs, device=y.device) * (2 if inter else 1)
        ib = ia + (1 if inter else pairs)
        a, b = y[..., ia], y[..., ib]
        y, size = y.clone(), size.clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, (D / 2 + 24) * 2.0 ** -24 * size


def positions(seed, B, T, axes, top):
    g = torch.Generator().manual_seed(seed)
    return ((torch.rand(B, T, axes, generator=g) * 2 - 1) * top).cuda()


ROPE = [
    # B, T, Hq, Hk, D, pairs, axes, interleaved, norm, dt, per-batch positions, largest position
    (1, 1, 1, 1, 8, 4, 1, 0, True, "bf16", False, 1.0),
    (1, 1, 20, 20, 64, 32, 2, 0, True, "f32", False, 1.0),
    (2, 77, 20, 20, 64, 32, 1, 0, True, "bf16", False, 1e5),
    (3, 29, 16, 4, 64, 32, 2, 1, True, "bf16", True, 30.0),
    (2, 31, 3, 1, 80, 40, 3, 0, False, "bf16", True, 1e3),
    (2, 31, 5, 5, 80, 20, 3, 1, True, "bf16", False, 1e3),
    (1, 50, 7, 2, 72, 36, 2, 0, True, "f32", False, 1e4),
    (2, 13, 16, 2, 128, 64, 3, 1, True, "f32", False, 1.6e7),
    (1, 9, 4, 4, 256, 128, 2, 0, True, "bf16", False, 10.0),
    (1, 9, 4, 4, 256, 16, 2, 0, True, "f32", False, 10.0),
    (2, 40, 8, 8, 64, 0, 1, 0, True, "bf16", False, 1.0),
    (4, 581, 20, 20, 64, 32, 2, 0, False, "bf16", False, 1.0),
    (1, 3, 1024, 1024, 8, 4, 1, 1, True, "bf16", False, 5.0),
    (2, 600, 16, 4, 96, 48, 3, 0, True, "f32", True, 100.0),
]


def rope_case(case, seed=11):
    B, T, Hq, Hk, D, pairs, axes, inter, norm, dt, per_batch, top = case
    q, k = rand(seed, B, T, Hq, D, dt=dt), rand(seed + 1, B, T, Hk, D, dt=dt)
    qw, kw = (1 + rand(seed + 2, D, std=0.2), 1 + rand(seed + 3, D, std=0.2)) if norm else (None, None)
    pos = positions(seed + 4, B if per_batch else 1, T, axes, top)
    pos[:, :min(2, T - 1)] = 0                             # unrotated tokens
    axis = (torch.arange(max(pairs, 1)) % axes).to(torch.uint8).cuda()
    freq = (10000.0 ** -(torch.arange(max(pairs, 1)).double() / max(pairs, 1))).float().cuda()
    return q, k, qw, kw, pos, T * axes if per_batch else 0, axis, freq


@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(v) for v in c))
def test_qk_norm_rope(case):
    B, T, Hq, Hk, D, pairs, axes, inter, norm, dt, *_ = case
    q, k, qw, kw, pos, pbs, axis, freq = rope_case(case)
    qo, ko = torch.full_like(q, 777.0), torch.full_like(k, 777.0)
    gk.gkd_qk_norm_rope(q, k, DT[dt][1], B, T, D, qw, kw, 1e-6, pos, pbs, axes, axis, freq, pairs, inter, qo, ko)
    settle()
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        ref, slack = rope_ref(x, w, 1e-6, pos, axis, freq, pairs, inter)
        check(o, ref, unit(dt) * ref.abs() + slack, "qk_norm_rope")
    if not norm and T > 2:
        assert torch.equal(qo[:, :2], q[:, :2])            # positions of 0 turn nothing


@pytest.mark.parametrize("dt,pairs", [("bf16", 32), ("bf16", 20), ("f32", 32)])
def test_qk_norm_rope_in_place_on_slices_and_other_layouts(dt, pairs):
    B, T, H, D = 3, 45, 6, 64
    packed = rand(3, B, T, 3 * H, D, dt=dt)
    before = packed.clone()
    q, k = packed[:, :, :H], packed[:, :, H:2 * H]
    qw, kw = 1 + rand(4, D, std=0.2), 1 + rand(5, D, std=0.2)
    pos, axis = positions(6, 1, T, 2, 20.0), (torch.arange(pairs) // (pairs // 2)).to(torch.uint8).cuda()
    freq = rand(7, pairs).abs()
    ahead = torch.full((B, H, T, D), 777.0, dtype=DT[dt][0], device="cuda").transpose(1, 2)
    refs = [rope_ref(x, w, 1e-5, pos, axis, freq, pairs, 0) for x, w in ((before[:, :, :H], qw), (before[:, :, H:2 * H], kw))]
    gk.gkd_qk_norm_rope(q, k, DT[dt][1], B, T, D, qw, kw, 1e-5, pos, 0, 2, axis, freq, pairs, 0, q, ahead)
    settle()
    for o, (ref, slack) in zip((q, ahead), refs):
        check(o, ref, unit(dt) * ref.abs() + slack, "in place / heads ahead")
    assert torch.equal(packed[:, :, H:], before[:, :, H:])  # keys (not in place) and values untouched
    gk.gkd_qk_norm_rope(k, None, DT[dt][1], B, T, D, kw, None, 1e-5, pos, 0, 2, axis, freq, pairs, 0, k, None)
    settle()
    assert torch.equal(k, ahead)                            # alone and beside queries: the same bits


def test_qk_norm_rope_zero_rows_and_out_of_range_axes():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos, freq = positions(1, 1, 4, 2, 3.0), torch.ones(32, device="cuda")
    w = torch.ones(64, device="cuda")
    axis = torch.full((32,), 200, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 777.0)
    gk.gkd_qk_norm_rope(q, None, gk.GKD_BF16, 1, 4, 64, w, None, 1e-6, pos, 0, 2, axis, freq, 32, 0, out, None)
    settle()
    assert not out.any()
    x = rand(2, 1, 4, 2, 64)
    gk.gkd_qk_norm_rope(x, None, gk.GKD_F32, 1, 4, 64, None, None, 0.0, pos, 0, 2, axis, freq, 32, 0, x.clone(), None)
    got = torch.empty_like(x)
    gk.gkd_qk_norm_rope(x, None, gk.GKD_F32, 1, 4, 64, None, None, 0.0, pos, 0, 2, axis, freq, 32, 0, got, None)
    settle()
    ref, slack = rope_ref(x, None, 0.0, pos, torch.zeros_like(axis), freq, 32, 0)
    check(got, ref, unit("f32") * ref.abs() + slack, "axis 0")


# ------------------------------------------------------------------ attention
def attention_ref(q, k, v, scale, causal, mask, dt):
    """The definition, with hidden keys and values left out altogether; and the bound beside it."""
    B, Tq, H, D = q.shape
    Tk, g = k.shape[1], H // k.shape[2]
    ref = torch.zeros(B, Tq, H, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(ref)
    u = unit(dt)
    row = torch.arange(Tq, device=q.device)[:, None] + (Tk - Tq)
    for b in range(B):
        keep = torch.arange(Tk, device=q.device)
        if mask is not None:
            keep = keep[mask[b if mask.shape[0] > 1 else 0] != 0]
        if not len(keep):
            continue
        for h in range(H):
            qq, kk, vv = q[b, :, h].double(), k[b, keep, h // g].double(), v[b, keep, h // g].double()
            s = scale * qq @ kk.t()
            if causal:
                s = s.masked_fill(keep[None] > row, -math.inf)
            p = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
            ref[b, :, h] = p @ vv
            d = ((D + 8) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().t())).amax(-1, keepdim=True)
            tol[b, :, h] = u * ref[b, :, h].abs() + ((u if dt == "bf16" else 0) + 2 * d + (Tk + 24) * 2.0 ** -22) * (p @ vv.abs())
    return ref, tol


def masks(kind, seed, B, T):
    if kind == "all":
        return None
    g = torch.Generator().manual_seed(seed)
    if kind == "prefix":
        n = torch.randint(0, T + 1, (B, 1), generator=g)
        n[0] = 0                                            # a batch without any key
        return (torch.arange(T)[None] < n).to(torch.uint8).cuda()
    if kind == "last":
        return (torch.arange(T)[None] == T - 1).to(torch.uint8).expand(B, T).contiguous().cuda()
    m = torch.rand(B, T, generator=g) < 0.4
    m[:, 64:200] = False                                    # whole tiles without a key
    return m.to(torch.uint8).cuda()


ATTENTION = [
    # B, Tq, Tk, H, Hk, D, dt, causal, mask
    (1, 1, 1, 1, 1, 8, "bf16", 0, "all"),
    (1, 1, 1, 1, 1, 64, "bf16", 1, "all"),
    (1, 1, 2304, 16, 16, 64, "bf16", 0, "all"),
    (1, 3, 4613, 4, 1, 128, "bf16", 0, "holes"),
    (2, 1, 700, 8, 2, 80, "bf16", 1, "prefix"),
    (3, 17, 17, 4, 4, 64, "bf16", 0, "prefix"),
    (3, 80, 576, 8, 4, 64, "bf16", 0, "holes"),
    (2, 77, 77, 20, 20, 64, "bf16", 1, "all"),
    (2, 127, 129, 3, 3, 72, "bf16", 1, "holes"),
    (2, 128, 128, 2, 2, 32, "bf16", 0, "last"),
    (1, 129, 127, 2, 1, 128, "bf16", 0, "all"),
    (2, 200, 65, 2, 2, 64, "bf16", 1, "all"),               # more queries than keys: the first rows see none
    (1, 581, 581, 4, 4, 64, "bf16", 0, "all"),
    (1, 581, 581, 4, 2, 96, "bf16", 1, "holes"),
    (2, 300, 1200, 4, 2, 128, "bf16", 1, "prefix"),
    (1, 1, 1, 1, 1, 8, "f32", 0, "all"),
    (1, 1, 2304, 16, 16, 64, "f32", 0, "all"),
    (3, 17, 17, 4, 4, 64, "f32", 0, "prefix"),
    (2, 160, 160, 4, 4, 64, "f32", 0, "holes"),
    (2, 77, 77, 6, 3, 80, "f32", 1, "holes"),
    (2, 200, 65, 2, 2, 32, "f32", 1, "all"),
    (1, 130, 300, 4, 1, 128, "f32", 1, "last"),
    (1, 581, 581, 2, 2, 96, "f32", 0, "all"),
]

# many key tiles per CTA, so that every ring turns over, whole and partial tiles mixed
ATTENTION += [
    (4, 300, 3001, 6, 2, 64, "bf16", 0, "holes"),
    (4, 300, 3001, 6, 6, 128, "bf16", 0, "holes"),
    (8, 700, 900, 8, 8, 80, "bf16", 1, "holes"),
    (8, 700, 900, 8, 4, 64, "bf16", 1, "all"),
    (2, 129, 2049, 16, 4, 128, "bf16", 0, "prefix"),
    (4, 300, 1500, 6, 2, 64, "f32", 0, "holes"),
    (4, 300, 1500, 6, 6, 128, "f32", 0, "holes"),
    (8, 400, 500, 8, 4, 72, "f32", 1, "holes"),
    (1, 5, 3001, 4, 4, 128, "f32", 0, "prefix"),
]


def attention_case(case, seed=21):
    B, Tq, Tk, H, Hk, D, dt, causal, kind = case
    q = rand(seed, B, Tq, H, D, dt=dt, std=2.0)
    k, v = rand(seed + 1, B, Tk, Hk, D, dt=dt), rand(seed + 2, B, Tk, Hk, D, dt=dt)
    return q, k, v, masks(kind, seed + 3, B, Tk)


# few keys: each size of that kernel and both sides of it, rows behind a tile, shared heads, more queries than keys
ATTENTION += [(2, q, k, 4, hk, D, "f32", causal, kind)
              for q, k, hk, D, causal, kind in [
                  (1, 1, 4, 64, 0, "prefix"), (65, 2, 2, 8, 0, "holes"), (131, 3, 2, 64, 0, "all"), (64, 7, 4, 24, 0, "last"),
                  (200, 8, 1, 128, 1, "all"), (33, 9, 4, 72, 0, "holes"), (17, 16, 4, 16, 1, "holes"), (17, 17, 2, 64, 1, "prefix"),
                  (300, 17, 4, 104, 0, "holes"), (5, 24, 1, 128, 1, "prefix"), (129, 24, 4, 64, 0, "all"), (129, 25, 4, 64, 0, "all"),
                  (40, 32, 2, 64, 1, "holes"), (70, 33, 4, 128, 0, "holes")]]

# few rows: one alone, shared heads, both sides of the rule, keys from one turn of a group to several CTAs' shares
ATTENTION += [(2, q, k, 4, hk, D, "f32", causal, kind)
              for q, k, hk, D, causal, kind in [
                  (1, 25, 4, 64, 0, "prefix"), (1, 64, 4, 128, 1, "holes"), (1, 65, 4, 8, 0, "last"), (1, 4613, 4, 64, 0, "holes"),
                  (1, 5000, 4, 104, 0, "prefix"), (1, 700, 1, 64, 0, "holes"), (2, 255, 4, 64, 1, "all"), (3, 256, 2, 72, 0, "holes"),
                  (5, 4358, 4, 64, 0, "holes"), (7, 2049, 1, 128, 1, "prefix"), (16, 300, 4, 64, 1, "holes"), (16, 1111, 4, 96, 0, "all"),
                  (17, 300, 4, 64, 1, "holes")]]
ATTENTION += [(300, 5, 333, 4, 2, 64, "f32", 1, "holes"), (300, 1, 333, 4, 4, 128, "f32", 0, "holes")]


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "-".join(str(v) for v in c))
def test_attention(case):
    B, Tq, Tk, H, Hk, D, dt, causal, kind = case
    q, k, v, mask = attention_case(case)
    out = torch.full_like(q, 777.0)
    ref, tol = attention_ref(q, k, v, D ** -0.5, causal, mask, dt)
    if mask is not None:                                    # what the mask hides may hold anything
        hidden = mask == 0
        k[hidden], v[hidden] = math.nan, math.inf
        v[:, ::2][hidden[:, ::2]] = math.nan
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, D ** -0.5, causal, mask, Tk, out)
    settle()
    check(out, ref, tol, "attention")
    none = tol.sum((2, 3)) == 0                             # rows without a key
    assert not out[none].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_on_slices_other_layouts_and_shared_keys(dt):
    B, Tq, Tk, H, D = 3, 70, 150, 6, 64
    q = rand(1, B, H, Tq, D, dt=dt).transpose(1, 2)
    kv = rand(2, Tk, 2 * H + 1, D, dt=dt)
    k, v = kv[:, :H].expand(B, -1, -1, -1), kv[:, H:2 * H].expand(B, -1, -1, -1)      # batch stride 0
    mask = masks("holes", 3, 1, Tk)
    buf = torch.full((B, Tq + 2, H + 1, D), 777.0, dtype=DT[dt][0], device="cuda")
    out = buf[:, 1:-1, :H]
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, 0.1, 0, mask, 0, out)
    settle()
    check(out, *attention_ref(q, k, v, 0.1, 0, mask, dt), "shared keys")
    out.fill_(777.0)
    assert bool((buf == 777.0).all())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_extreme_scores(dt):
    """Scores of hundreds: the running maximum moves by more than the exponent's range between key tiles."""
    B, Tq, Tk, H, D = 1, 100, 600, 2, 64
    q, k, v = rand(1, B, Tq, H, D, dt=dt, std=8.0), rand(2, B, Tk, H, D, dt=dt, std=4.0), rand(3, B, Tk, H, D, dt=dt)
    k[:, 300:] *= 4
    out = torch.empty_like(q)
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, 1.0, 0, None, 0, out)
    settle()
    check(out, *attention_ref(q, k, v, 1.0, 0, None, dt), "extreme scores")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_without_keys_writes_zeros(dt):
    out = torch.full((2, 5, 3, 64), 777.0, dtype=DT[dt][0], device="cuda")
    q = rand(1, 2, 5, 3, 64, dt=dt)
    gk.gkd_attention(q, gk.GkdHeads(None, 0, 0, 0, 3), gk.GkdHeads(None, 0, 0, 0, 3), DT[dt][1], 2, 5, 0, 64, 1.0, 0, None,
                     0, out)
    settle()
    assert not out.any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_keys_past_32_bit_offsets(dt):
    Tk, D, stride = 5, 64, 2 ** 29 + 64
    buf = torch.empty((Tk - 1) * stride + D, dtype=DT[dt][0], device="cuda")
    rows, v = rand(1, Tk, D, dt=dt), rand(2, 1, Tk, 1, D, dt=dt)
    k = buf.as_strided((1, Tk, 1, D), (0, stride, D, 1))
    k[0, :, 0] = rows
    q, out = rand(3, 1, 3, 1, D, dt=dt, std=3.0), torch.empty(1, 3, 1, D, dtype=DT[dt][0], device="cuda")
    gk.gkd_attention(q, k, v, DT[dt][1], 1, 3, Tk, D, 0.5, 0, None, 0, out)
    settle()
    check(out, *attention_ref(q, rows[None, :, None], v, 0.5, 0, None, dt), "far keys")


@pytest.mark.parametrize("Tq", [1, 3, 40])
def test_attention_many_keys_past_32_bit_offsets(Tq):
    Tk, D, stride = 30, 64, 2 ** 27 + 64
    buf = torch.empty((Tk - 1) * stride + D, device="cuda")
    rows, k = rand(1, Tk, D, dt="f32"), rand(2, 1, Tk, 1, D, dt="f32")
    v = buf.as_strided((1, Tk, 1, D), (0, stride, D, 1))
    v[0, :, 0] = rows
    q, out = rand(3, 1, Tq, 1, D, dt="f32", std=3.0), torch.empty(1, Tq, 1, D, device="cuda")
    gk.gkd_attention(q, k, v, DT["f32"][1], 1, Tq, Tk, D, 0.5, 0, None, 0, out)
    settle()
    check(out, *attention_ref(q, k, rows[None, :, None], 0.5, 0, None, "f32"), "far values")


@pytest.mark.parametrize("Tk", [3, 16, 24])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_over_few_keys_on_slices_with_nan(dt, Tk):
    """Strided views and one set of keys for all batches; NaN and infinities reach only the rows that meet them."""
    B, Tq, H, D = 3, 70, 4, 64
    base = rand(1, B, Tq + 3, H + 2, D + 16, dt=dt)
    q = base[:, 2:Tq + 2, 1:H + 1, 8:D + 8]
    kv = rand(2, 1, 2, H, Tk, D, dt=dt)                                             # heads outside, rows inside
    k, v = (kv[:, i].transpose(1, 2)[:, :, :2].expand(B, -1, -1, -1) for i in range(2))
    ref, tol = attention_ref(q, k, v, 0.1, 1, None, dt)
    last = Tq - 1                                                                   # the row that sees the last key
    q[0, last - 1, 0, 3], q[1, last, 1, ::2] = math.nan, math.inf
    kv[0, 0, 1, Tk - 1, 5] = math.nan                                               # seen by the last row of heads 2 and 3
    bad = torch.zeros(B, Tq, H, dtype=torch.bool, device="cuda")
    bad[0, last - 1, 0] = bad[1, last, 1] = True
    bad[:, last, 2:] = True
    buf = torch.full((B, Tq + 2, H + 1, D), 777.0, dtype=DT[dt][0], device="cuda")
    out = buf[:, 1:-1, :H]
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, 0.1, 1, None, 0, out)
    settle()
    assert bool(torch.isnan(out[bad]).all())
    check(out[~bad], ref[~bad], tol[~bad], "other rows")
    assert not out[:, :Tq - Tk].any()                                               # rows without a key
    out.fill_(777.0)
    assert bool((buf == 777.0).all())


@pytest.mark.parametrize("Tq,Hk", [(1, 4), (1, 2), (6, 2), (16, 4)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_of_few_rows_on_slices_with_nan(dt, Tq, Hk):
    B, Tk, H, D = 3, 1500, 4, 64
    q = rand(1, B, Tq + 3, H + 2, D + 16, dt=dt)[:, 2:Tq + 2, 1:H + 1, 8:D + 8]
    k, v = (rand(i, 1, Hk, Tk, D, dt=dt).transpose(1, 2).expand(B, -1, -1, -1) for i in (2, 3))
    ref, tol = attention_ref(q, k, v, 0.1, 1, None, dt)
    bad = torch.zeros(B, Tq, H, dtype=torch.bool, device="cuda")
    q[0, 0, 0, 3], q[1, Tq - 1, 1, ::2] = math.nan, math.inf
    bad[0, 0, 0] = bad[1, Tq - 1, 1] = True
    k[0, Tk - 1, Hk - 1, 5] = math.nan                                              # seen by the last row of the last heads
    bad[:, Tq - 1, H - H // Hk:] = True
    buf = torch.full((B, Tq + 2, H + 1, D), 777.0, dtype=DT[dt][0], device="cuda")
    out = buf[:, 1:-1, :H]
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, 0.1, 1, None, 0, out)
    settle()
    assert bool(torch.isnan(out[bad]).all())
    check(out[~bad], ref[~bad], tol[~bad], "other rows")
    out.fill_(777.0)
    assert bool((buf == 777.0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_keeps_nan_to_the_rows_that_see_it(dt, D):
    B, Tq, Tk, H = 2, 150, 200, 2
    q, k, v = rand(1, B, Tq, H, D, dt=dt), rand(2, B, Tk, H, D, dt=dt), rand(3, B, Tk, H, D, dt=dt)
    ref, tol = attention_ref(q, k, v, 0.1, 1, None, dt)
    q[0, 3, 0] = math.nan                                   # a query: its own row
    k[1, 120, 1, 5] = math.nan                              # a key: the rows that see it (causal: from 70 on)
    q[0, 9, 1, 0] = math.inf                                # infinite scores: the row
    out = torch.empty_like(q)
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, 0.1, 1, None, 0, out)
    settle()
    bad = torch.zeros(B, Tq, H, dtype=torch.bool, device="cuda")
    bad[0, 3, 0] = bad[0, 9, 1] = True
    bad[1, 70:, 1] = True
    assert bool(torch.isnan(out[bad]).all())
    check(out[~bad], ref[~bad], tol[~bad], "other rows")


@pytest.mark.parametrize("D", [40, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [0, 1])
def test_attention_keeps_nan_to_its_row_where_shares_have_no_key(dt, D, causal):
    """Fewer key tiles than the CTAs that share a query tile (the first rows of a causal call, a mask that
    leaves the first keys): a share without a key adds nothing to any row, whatever Q holds."""
    B, T, H = 1, 1024, 2
    q, k, v = rand(11, B, T, H, D, dt=dt), rand(12, B, T, H, D, dt=dt), rand(13, B, T, H, D, dt=dt)
    mask = None
    if not causal:
        mask = torch.zeros(B, T, dtype=torch.uint8, device="cuda")
        mask[:, :40] = 1
    ref, tol = attention_ref(q, k, v, 0.1, causal, mask, dt)
    bad = torch.zeros(B, T, H, dtype=torch.bool, device="cuda")
    for first in (5, 64, 127, 300):
        q[:, first] = math.nan
        q[:, first + 3, :, ::2] = math.inf
        bad[:, first] = bad[:, first + 3] = True
    for _ in range(20):
        out = torch.full_like(q, 7.0)
        gk.gkd_attention(q, k, v, DT[dt][1], B, T, T, D, 0.1, causal, mask, T if mask is not None else 0, out)
        settle()
        assert bool(torch.isnan(out[bad]).all())
        check(out[~bad], ref[~bad], tol[~bad], "other rows")


# ------------------------------------------------------------------ all of them
def ours(seed, dt, T):
    """One pass of each operator on fresh buffers; returns a callable and its outputs."""
    lc = linear_case(T, 136, 264, dt, dt, "gelu", True, True, True, seed)
    lo = torch.empty(T, 264, dtype=DT[dt][0], device="cuda")
    rc = rope_case((2, T, 4, 2, 64, 32, 2, 0, True, dt, False, 9.0), seed)
    ro = [torch.empty_like(rc[0]), torch.empty_like(rc[1])]
    ac = attention_case((2, T, 333, 4, 2, 64, dt, 0, "holes"), seed)
    ao = torch.empty_like(ac[0])

    def run(stream=None):
        x, w, b, s, r = lc
        gk.gkd_linear(x, DT[dt][1], T, 136, 136, w, 264, b, gk.GKD_ACT_GELU, s, r, 264, lo, DT[dt][1], 264, stream)
        q, k, qw, kw, pos, pbs, axis, freq = rc
        gk.gkd_qk_norm_rope(q, k, DT[dt][1], 2, T, 64, qw, kw, 1e-6, pos, pbs, 2, axis, freq, 32, 0, *ro, stream)
        gk.gkd_attention(*ac[:3], DT[dt][1], 2, T, 333, 64, 0.125, 0, ac[3], 333, ao, stream)
    return run, [lo, *ro, ao]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 90, 700])
def test_repeats_streams_and_graphs_give_the_same_bits(dt, T):
    runs = [ours(31 + i, dt, T) for i in range(2)]
    first = []
    for run, outs in runs:
        run()
        torch.cuda.synchronize()
        first.append([o.clone() for o in outs])
    for _, outs in runs:
        for o in outs:
            o.fill_(777.0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]           # two at once
    for _ in range(5):
        for (run, _), st in zip(runs, streams):
            run(st)
    settle()
    for (_, outs), want in zip(runs, first):
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for run, outs in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
        for o in outs:
            o.fill_(777.0)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    settle()
    for (_, outs), want in zip(runs, first):
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_host_pointers_are_refused():
    x = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(gk.GkdError):
        gk.gkd_linear(x, gk.GKD_BF16, 8, 64, 64, x.cuda(), 8, None, 0, None, None, 0, x.cuda(), gk.GKD_BF16, 8, stream=0)


def test_prompt_rows_to_keypoints():
    """A kernel generator's block on the prompt rows of a batch, in the order it is used: projections, norms and
    positions, attention over the query patches, output projection onto the residual rows, feed-forward; then the
    head's own steps on the refined rows."""
    B, K, h, w, C, H, D, F = 3, 20, 8, 8, 128, 2, 64, 256
    feat = rand(1, B, h * w, C, dt="bf16")
    rows = rand(2, B * K, C)
    wq, wkv, wo = (rand(3 + i, n, C, dt="bf16", std=C ** -0.5) for i, n in enumerate((H * D, 2 * H * D, C)))
    w1, w2 = rand(6, F, C, dt="bf16", std=C ** -0.5), rand(7, C, F, dt="bf16", std=F ** -0.5)
    qn, kn = 1 + rand(8, D, std=0.1), 1 + rand(9, D, std=0.1)
    at = (torch.arange(8).float() + 0.5) / 4 - 1
    pos = torch.stack(torch.meshgrid(at, at, indexing="ij"), -1).reshape(-1, 2).cuda()
    axis, freq = (torch.arange(32) // 16).to(torch.uint8).cuda(), (6.28 * 100.0 ** -(torch.arange(32) % 16 / 16)).cuda()
    mask = (torch.arange(K)[None] < torch.tensor([[20], [7], [1]])).to(torch.uint8).cuda()

    def bf(*s):
        return torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    x, q, kv, y, hid = rows.bfloat16(), bf(B, K, H, D), bf(B, h * w, 2 * H, D), bf(B, K, H, D), bf(B * K, F)
    N, BF, F4 = gk.GKD_ACT_NONE, gk.GKD_BF16, gk.GKD_F32
    out = rows.clone()
    gk.gkd_linear(x, BF, B * K, C, C, wq, H * D, None, N, None, None, 0, q, BF, H * D)
    gk.gkd_linear(feat, BF, B * h * w, C, C, wkv, 2 * H * D, None, N, None, None, 0, kv, BF, 2 * H * D)
    k, v = kv[:, :, :H], kv[:, :, H:]
    gk.gkd_qk_norm_rope(q, None, BF, B, K, D, qn, None, 1e-6, None, 0, 1, None, None, 0, 0, q, None)
    gk.gkd_qk_norm_rope(k, None, BF, B, h * w, D, kn, None, 1e-6, pos, 0, 2, axis, freq, 32, 0, k, None)
    gk.gkd_attention(q, k, v, BF, B, K, h * w, D, D ** -0.5, 0, None, 0, y)
    gk.gkd_linear(y, BF, B * K, H * D, H * D, wo, C, None, N, None, out, C, out, F4, C)
    x2 = out.bfloat16()
    gk.gkd_linear(x2, BF, B * K, C, C, w1, F, None, gk.GKD_ACT_GELU, None, None, 0, hid, BF, F)
    gk.gkd_linear(hid, BF, B * K, F, F, w2, C, None, N, None, out, C, out, F4, C)
    khat = bf(B, 1, K, C)
    xy, score = torch.empty(B, K, 2, device="cuda"), torch.empty(B, K, device="cuda")
    idx, valid = torch.empty(B, K, dtype=torch.int32, device="cuda"), torch.empty(B, K, dtype=torch.uint8, device="cuda")
    scratch = torch.empty(B, K, dtype=torch.int64, device="cuda")
    gk.gkd_norm_kernels(out, mask, B, 1, K, C, 1e-12, BF, khat)
    gk.gkd_heatmap_decode(feat, BF, B, h, w, C, 4, khat, BF, K * C, mask, K, 1, K, scratch, xy, score, idx, valid)
    settle()

    # the same in 64 bits without the roundings in between: they are some 2^-8 each, and a row's norm averages them
    d = torch.float64
    qr = (x.to(d) @ wq.to(d).t()).view(B, K, H, D)
    kvr = (feat.reshape(-1, C).to(d) @ wkv.to(d).t()).view(B, h * w, 2 * H, D)
    qr, _ = rope_ref(qr, qn, 1e-6, None, None, None, 0, 0)
    kr, _ = rope_ref(kvr[:, :, :H], kn, 1e-6, pos, axis, freq, 32, 0)
    yr, _ = attention_ref(qr, kr, kvr[:, :, H:], D ** -0.5, 0, None, "bf16")
    r1 = rows.to(d) + yr.reshape(B * K, -1) @ wo.to(d).t()
    a = r1 @ w1.to(d).t()
    r2 = r1 + (0.5 * a * (1 + torch.erf(a / math.sqrt(2)))) @ w2.to(d).t()
    rel = ((out.to(d) - r2).norm(dim=-1) / r2.norm(dim=-1)).max().item()
    assert rel <= 3 * unit("bf16"), rel                     # six roundings of at most 2^-8, independent: sqrt(6) of them
    assert torch.equal(valid, mask)
    assert bool((score[mask == 0] == 0).all()) and bool((idx[mask == 0] == -1).all()) and bool((idx[mask == 1] >= 0).all())
