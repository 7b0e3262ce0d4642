"""GPU: the transformer-block operators at the ends of what their header allows: the longest row count, infinite and
very large scores, long sums, waits that run out."""
import pytest
import torch

from prompt_conditioned_keypoint_b200 import binding as gk
from test_gpu_blocks import check, linear_ref, rand, settle

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
