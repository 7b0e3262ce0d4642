"""GPU: fp32 gkd_attention and gkd_linear on inputs that need every product of their split operands, against bounds that
the loss of one breaks (test_blocks_accuracy.py shows that on the CPU), and the range that gkd_blocks.h gives."""
import math

import block_accuracy as A
import pytest
import torch

from prompt_conditioned_keypoint_b200 import binding as gk
from test_gpu_blocks import DT, attention_ref, check, rand, settle

pytestmark = pytest.mark.gpu
# tensor cores with one CTA per query tile and with clusters; up to 24 keys; up to 16 rows
SHAPES = [(1, 300, 100), (90, 130, 70), (1, 40, 1500), (2, 70, 20), (2, 1, 700), (2, 9, 300)]


def attention(q, k, v, scale, mask=None):
    B, Tq, _, D = q.shape
    Tk = k.shape[1]
    out = torch.full((B, Tq, 1, D), 777.0, device="cuda")
    gk.gkd_attention(q.cuda(), k.cuda(), v.cuda(), gk.GKD_F32, B, Tq, Tk, D, scale, 0, None if mask is None else mask.cuda(), Tk,
                     out)
    settle()
    return out


@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("B,Tq,Tk", SHAPES)
@pytest.mark.parametrize("term", A.TERMS)
def test_attention_scores_have_every_product(term, B, Tq, Tk, D):
    q, k, v, scale, ref, tol = A.score_case(term, B, Tq, Tk, D)
    check(attention(q, k, v, scale), ref.cuda(), tol.cuda(), f"product {term}")


@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("B,Tq,Tk", SHAPES)
def test_attention_outputs_have_every_product(B, Tq, Tk, D):
    for first, second in ((0, 1), (3, Tk - 5), (Tk - 1, 2)):
        q, k, v, mask, scale, ref, tol = A.output_case(B, Tq, Tk, D, first, second)
        check(attention(q, k, v, scale, mask), ref.cuda(), tol.cuda(), f"keys {first}, {second}")


@pytest.mark.parametrize("T,Cin,Cout", [(1, 8, 8), (3, 64, 40), (17, 1024, 136), (80, 4104, 1024), (130, 4104, 136), (300, 520, 520),
                                        (2000, 1024, 1024)])
def test_linear_has_every_product(T, Cin, Cout):
    x, w, ref, tol = A.linear_case(T, Cin, Cout)
    out = torch.full((T, Cout), 777.0, device="cuda")
    gk.gkd_linear(x.cuda(), gk.GKD_F32, T, Cin, Cin, w.cuda(), Cout, None, gk.GKD_ACT_NONE, None, None, 0, out, gk.GKD_F32, Cout)
    settle()
    check(out, ref.cuda(), tol.cuda(), "positive sums")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,Tk", [(40, 100), (150, 1000), (40, 24), (5, 300), (1, 300)])
def test_attention_values_near_the_end_of_the_range(Tq, Tk, dt, D):
    """Values of one sign up to 2^127 / Tk, for bf16 2^119 / Tk: their weighted sum, before its division, stays finite."""
    q, k, v = (rand(i, 1, n, 2, D, dt=dt) for i, n in ((1, Tq), (2, Tk), (3, Tk)))
    v = (v.abs() / v.abs().max()).to(v.dtype)
    ref, tol = attention_ref(q, k, v, D ** -0.5, 0, None, dt)
    big = 2.0 ** ((127 if dt == "f32" else 119) - math.ceil(math.log2(Tk)))
    out = torch.empty_like(q)
    gk.gkd_attention(q, k, v * big, DT[dt][1], 1, Tq, Tk, D, D ** -0.5, 0, None, 0, out)
    settle()
    check(out.double() / big, ref, tol, "large values")


@pytest.mark.parametrize("T", [3, 300])
def test_linear_keeps_an_infinity_to_its_own_row_and_column(T):
    """fp32: an infinity in x or weight makes its row or column infinite or NaN; the rest does not see it."""
    Cin, Cout = 136, 264
    x, w, ref, tol = (t.cuda() for t in A.linear_case(T, Cin, Cout))
    x[1, 3], w[7, 5], w[9, 100] = math.inf, math.nan, -math.inf
    out = torch.empty(T, Cout, device="cuda")
    gk.gkd_linear(x, gk.GKD_F32, T, Cin, Cin, w, Cout, None, gk.GKD_ACT_NONE, None, None, 0, out, gk.GKD_F32, Cout)
    settle()
    rows = [i for i in range(T) if i != 1]
    cols = [i for i in range(Cout) if i not in (7, 9)]
    assert not torch.isfinite(out[1]).any() and not torch.isfinite(out[:, [7, 9]]).any()
    check(out[rows][:, cols], ref[rows][:, cols], tol[rows][:, cols], "the rest")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Tq,Tk,Hk", [(12, 100, 8), (13, 30, 8), (13, 49, 2), (16, 128, 2), (16, 129, 2), (16, 192, 8), (14, 193, 8),
                                      (16, 256, 8), (15, 257, 8)])
def test_attention_of_up_to_16_rows_in_a_batch_that_fills_the_gpu(Tq, Tk, Hk, D):
    """Both kernels that take 13 to 16 rows, and each end of the rule between them."""
    B, H = 40, 8
    q, k, v = rand(1, B, Tq, H, D, std=2.0), rand(2, B, Tk, Hk, D), rand(3, B, Tk, Hk, D)
    mask = (torch.rand(B, Tk, generator=torch.Generator().manual_seed(4)) < 0.6).to(torch.uint8).cuda()
    mask[3] = 0
    ref, tol = attention_ref(q, k, v, D ** -0.5, 1, mask, "f32")
    k[mask == 0], v[mask == 0] = math.nan, math.inf
    out = torch.full_like(q, 777.0)
    gk.gkd_attention(q, k, v, gk.GKD_F32, B, Tq, Tk, D, D ** -0.5, 1, mask, Tk, out)
    settle()
    check(out, ref, tol, "up to 16 rows")
    assert not out[3].any()
