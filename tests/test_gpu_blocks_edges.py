"""GPU: the transformer-block operators at the ends of what their header allows: the longest row count, infinite and
very large scores, long sums, waits that run out."""
import math

import pytest
import torch

from prompt_conditioned_keypoint_b200 import binding as gk
from test_gpu_blocks import DT, check, linear_ref, rand, settle, unit

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ rows
def test_linear_of_two_billion_rows():
    """2^31 - 1 rows: tile counts and row numbers next to the end of 32 bits."""
    T, C = 2 ** 31 - 1, 8
    torch.cuda.empty_cache()                                # 69 GB follow
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda").normal_()
    out = torch.full((T, C), 777.0, dtype=torch.bfloat16, device="cuda")
    w, b = rand(1, C, C, dt="bf16", std=C ** -0.5), rand(2, C)
    gk.gkd_linear(x, gk.GKD_BF16, T, C, C, w, C, b, gk.GKD_ACT_RELU, None, None, 0, out, gk.GKD_BF16, C)
    settle()
    for first in (0, 2 ** 28 - 150, 2 ** 30 - 150, T - 300):
        rows = slice(first, first + 300)
        check(out[rows], *linear_ref(x[rows], w, b, "relu", None, None, "bf16"), f"rows from {first}")
    del x, out
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ long sums
@pytest.mark.parametrize("T,Cin,Cout", [(5, 1024, 136), (64, 8192, 136), (200, 4096, 1032), (5, 65536, 136), (128, 65536, 1408),
                                        (40, 32768, 2056), (16, 65536, 9472), (70, 65528, 9472)])
def test_linear_fp32_output_of_long_sums_does_not_drift(T, Cin, Cout):
    """Sums of positive products: an accumulator of 512 channels loses 5e-7 by the tensor core's truncation, the mean over
    many results of what the fp32 additions behind it do is far below that. 2^-20 is 9.5e-7; 1024 channels lose more."""
    x = (rand(1, T, Cin).abs() + 0.5).bfloat16()
    w = torch.empty(Cout, Cin, device="cuda").uniform_(0.5, 1.5, generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    out = torch.empty(T, Cout, device="cuda")
    gk.gkd_linear(x, gk.GKD_BF16, T, Cin, Cin, w, Cout, None, gk.GKD_ACT_NONE, None, None, 0, out, gk.GKD_F32, Cout)
    settle()
    part = slice(0, min(Cout, 1408))
    ref = x.double() @ w[part].double().t()
    off = (out[:, part].double() - ref) / ref
    assert abs(off.mean().item()) <= 2.0 ** -20
    # every step of an accumulator (32 of them) and every addition off by a whole unit of the sum so far, which averages half
    assert off.abs().max().item() <= (16.5 + Cin / 512 / 4) * 2.0 ** -23


# ------------------------------------------------------------------ infinite scores
# Every attention kernel: fp32 by its rules for keys and rows, bf16 by the width of a head; with one CTA per query tile
# and with clusters that share the keys.
KERNELS = [
    # B, Tq, Tk, H, Hk, D, dt
    (3, 40, 3, 2, 2, 64, "f32"), (3, 70, 24, 2, 1, 128, "f32"),
    (3, 1, 40, 2, 2, 64, "f32"), (3, 1, 1500, 2, 2, 128, "f32"), (3, 5, 300, 4, 2, 64, "f32"), (3, 16, 900, 2, 1, 128, "f32"),
    (3, 40, 100, 2, 2, 64, "f32"), (3, 200, 700, 2, 1, 64, "f32"), (3, 150, 1000, 2, 2, 128, "f32"), (90, 130, 90, 2, 2, 72, "f32"),
    (3, 1, 40, 2, 2, 64, "bf16"), (3, 40, 100, 2, 1, 64, "bf16"), (3, 150, 1000, 2, 2, 64, "bf16"), (3, 17, 1500, 2, 2, 128, "bf16"),
    (90, 130, 90, 4, 2, 80, "bf16"), (90, 260, 130, 4, 2, 64, "bf16"),
]


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("case", KERNELS, ids=lambda c: "-".join(str(v) for v in c))
def test_attention_where_scores_are_minus_infinity(case, causal):
    """A visible key whose score is -inf has no weight beside others; a row that sees only such keys is NaN (0 / 0 by the
    definition), not 0 as a row without a key."""
    B, Tq, Tk, H, Hk, D, dt = case
    q, k, v = rand(1, B, Tq, H, D, dt=dt), rand(2, B, Tk, Hk, D, dt=dt), rand(3, B, Tk, Hk, D, dt=dt)
    mask = (torch.rand(B, Tk, generator=torch.Generator().manual_seed(4)) < 0.7).to(torch.uint8).cuda()
    low = torch.zeros(Tk, dtype=torch.bool, device="cuda")
    low[:max(1, Tk // 3)] = True                            # these keys' scores overflow for every other row
    low[Tk // 2] = True
    mask[:, Tk // 2] = mask[:, Tk - 1] = 1
    mask[1] = low.to(torch.uint8)                           # a batch that sees nothing else
    mask[2] = 0                                             # and one that sees no key
    q[..., 0] = 0
    q[:, ::2, :, 0] = 2.0 ** 100                            # the product with -2^100 is -inf, with 0 it is 0
    k[..., 0] = torch.where(low, -2.0 ** 100, 0.0)[None, :, None].to(k.dtype)
    out = torch.full_like(q, 777.0)
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, D ** -0.5, causal, mask, Tk, out)
    settle()

    qs, ks = q.double(), k.double().repeat_interleave(H // Hk, 2)
    big = qs[..., 0] > 0                                    # [B][Tq][H]
    qs, ks = qs.clone(), ks.clone()
    qs[..., 0] = 0
    s = torch.einsum("bihd,bjhd->bhij", qs, ks) * D ** -0.5
    seen = (mask != 0)[:, None, None].expand(B, H, Tq, Tk)
    if causal:
        seen = seen & (torch.arange(Tk, device="cuda")[None] <= torch.arange(Tq, device="cuda")[:, None] + (Tk - Tq))
    finite = seen & ~(big.permute(0, 2, 1)[..., None] & low)
    p = torch.nan_to_num(torch.softmax(s.masked_fill(~finite, -math.inf), -1), nan=0.0)
    vs = v.double().repeat_interleave(H // Hk, 2)
    ref = torch.einsum("bhij,bjhd->bihd", p, vs)
    size = torch.einsum("bhij,bjhd->bihd", p, vs.abs())
    d = (D + 8) * 2.0 ** -23 * D ** -0.5 * torch.einsum("bihd,bjhd->bhij", qs.abs(), ks.abs()).amax(-1).permute(0, 2, 1)
    tol = unit(dt) * ref.abs() + ((unit(dt) if dt == "bf16" else 0) + 2 * d[..., None] + (Tk + 24) * 2.0 ** -22) * size
    none, nan = ~seen.any(-1), seen.any(-1) & ~finite.any(-1)
    none, nan = none.permute(0, 2, 1), nan.permute(0, 2, 1)
    assert bool(nan.any()) and bool(none.any())
    assert bool(torch.isnan(out[nan]).all()), "rows whose scores are all -inf"
    assert not out[none].any(), "rows without a key"
    rest = ~(nan | none)
    check(out[rest], ref[rest], tol[rest], "other rows")


@pytest.mark.parametrize("case", KERNELS, ids=lambda c: "-".join(str(v) for v in c))
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_scores_beyond_32_bits(case, sign):
    """Finite scores of some 2^37 of either sign: neighbours are thousands apart, so that a row is its best key's value
    (the mean of two, where the key stands twice)."""
    B, Tq, Tk, H, Hk, D, dt = case
    q, k, v = (rand(i, *s, dt=dt) for i, s in ((1, (B, Tq, H, D)), (2, (B, Tk, Hk, D)), (3, (B, Tk, Hk, D))))
    q, k = q * 2.0 ** 17, k * 2.0 ** 17
    if sign < 0:                                            # the best of a row is far below 0
        q, k = q.abs(), -k.abs()
    k[:, Tk - 1] = k[:, 0]
    out = torch.full_like(q, 777.0)
    gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, 1.0, 0, None, 0, out)
    settle()
    s = torch.einsum("bihd,bjhd->bhij", q.double(), k.double().repeat_interleave(H // Hk, 2))
    vs = v.double().repeat_interleave(H // Hk, 2)
    # the keys 0 and Tk - 1 count as one
    best, at = s[..., :-1].topk(2 if Tk > 2 else 1, -1)
    slack = (D + 8) * 2.0 ** -23 * torch.einsum("bihd,bjhd->bhij", q.double().abs(), k.double().abs().repeat_interleave(H // Hk, 2)).amax(-1)
    clear = best[..., 0] - best[..., 1] > 2 * slack + 200   # rounding does not change the order, and 2^-288 is nothing
    assert clear.double().mean().item() > 0.9
    win = at[..., 0].permute(0, 2, 1)                       # [B][Tq][H]
    ref = torch.gather(vs, 1, win[..., None].expand(B, Tq, H, D))
    ref = torch.where((win == 0)[..., None], (ref + vs[:, Tk - 1:Tk]) / 2, ref)
    clear = clear.permute(0, 2, 1)
    check(out[clear], ref[clear], (unit(dt) * ref.abs() + 2.0 ** -22 * (vs.abs().amax(1, keepdim=True)))[clear], "best key's value")


# ------------------------------------------------------------------ waits that run out
def linear_call(T, Cin, Cout, dt, odt, res):
    x, w, b = rand(1, T, Cin, dt=dt), rand(2, Cout, Cin, dt=dt, std=Cin ** -0.5), rand(3, Cout)
    r = rand(4, T, Cout, dt=odt) if res else None
    out = torch.empty(T, Cout, dtype=DT[odt][0], device="cuda")

    def call():
        gk.gkd_linear(x, DT[dt][1], T, Cin, Cin, w, Cout, b, gk.GKD_ACT_GELU, None, r, Cout, out, DT[odt][1], Cout)
        return out
    return call


def attention_call(B, Tq, Tk, H, Hk, D, dt, causal, masked):
    q, k, v = (rand(i, *s, dt=dt) for i, s in ((1, (B, Tq, H, D)), (2, (B, Tk, Hk, D)), (3, (B, Tk, Hk, D))))
    mask = (torch.rand(B, Tk, generator=torch.Generator().manual_seed(4)) < 0.7).to(torch.uint8).cuda() if masked else None
    out = torch.empty_like(q)

    def call():
        gk.gkd_attention(q, k, v, DT[dt][1], B, Tq, Tk, D, D ** -0.5, causal, mask, Tk, out)
        return out
    return call


WAITS = [
    # the kernel for many rows (each width, both output types, a residual on its way), the one for few (alone, in clusters)
    (linear_call, 5000, 72, 1032, "bf16", "bf16", True), (linear_call, 1360, 520, 808, "bf16", "f32", True),
    (linear_call, 9400, 520, 1024, "bf16", "f32", False), (linear_call, 17, 1280, 2048, "bf16", "bf16", False),
    (linear_call, 64, 8192, 136, "bf16", "f32", True), (linear_call, 200, 128, 1032, "bf16", "bf16", True),
    (linear_call, 17, 1280, 520, "f32", "f32", True), (linear_call, 1360, 264, 1024, "f32", "f32", False),
    # heads of one and two chunks, with and without a mask, one CTA and clusters per query tile
    (attention_call, 2, 300, 300, 8, 4, 64, "bf16", 0, False), (attention_call, 2, 300, 300, 8, 8, 128, "bf16", 1, True),
    (attention_call, 1, 1, 2304, 4, 4, 64, "bf16", 0, True), (attention_call, 1, 130, 1500, 2, 1, 128, "bf16", 0, False),
    (attention_call, 2, 300, 300, 8, 4, 64, "f32", 0, False), (attention_call, 2, 300, 300, 8, 8, 128, "f32", 1, True),
    (attention_call, 1, 40, 2304, 4, 4, 64, "f32", 0, True), (attention_call, 1, 130, 1500, 2, 1, 128, "f32", 0, False),
]


@pytest.mark.parametrize("case", WAITS, ids=lambda c: "-".join(str(v) for v in (c[0].__name__, *c[1:])))
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(case):
    call = case[0](*case[1:])
    want = call().clone()
    settle()
    gk.gkd_set_wait_timeout_ms(50)
    try:
        gk.gkd_debug_set_flags(gk.DEBUG_SKIP_PRODUCER_ARRIVE)
        call()
        with pytest.raises(gk.GkdError) as e:
            gk.gkd_check_device_error()
        assert e.value.status == gk.GKD_ERR_TIMEOUT
    finally:
        gk.gkd_debug_set_flags(0)
        gk.gkd_set_wait_timeout_ms(2000)
    call().fill_(777.0)
    got = call()
    settle()
    assert torch.equal(got, want)
