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
