"""Inputs that show every product of the fp32 operators' split operands, their exact results, and bounds that the loss of
one product breaks. Used on the CPU with a model of the split products (test_blocks_accuracy.py) and on the GPU with the
kernels (test_gpu_blocks_accuracy.py).

gkd_attention, fp32: x = b0 + b1 + b2 in bf16 and the products (i, j) with i + j <= 2. gkd_linear, fp32: x = hi + lo in TF32
and the products hi hi, hi lo, lo hi.
"""
from __future__ import annotations

import torch

TERMS = [(0, 0), (1, 0), (0, 1), (1, 1), (2, 0), (0, 2)]
E, F = 2.0 ** -9, 2.0 ** -18
# (elements of a query, elements of a key): their products cancel but for planes (i, j) of one pair. 1 + E has the planes
# 1, E and 1 + E + F the planes 1, E, F (half a step of bf16 at 1 is 2^-8, at E 2^-17).
GROUPS = {
    (0, 0): ([1.0], [1.0], 1.0),
    (1, 0): ([1 + E, 1.0], [1.0, -1.0], E),
    (0, 1): ([1.0, 1.0], [1 + E, -1.0], E),
    (1, 1): ([1 + E, 1.0, 2 * E], [1 + E, -1.0, -1.0], F),
    (2, 0): ([1 + E + F, 1 + E], [1.0, -1.0], F),
    (0, 2): ([1.0, 1.0], [1 + E + F, -(1 + E)], F),
}


def planes(x):
    out = []
    for _ in range(3):
        out.append(x.bfloat16().to(x.dtype))
        x = x - out[-1]
    return out


def split_product(a, b, terms):
    """a b^T in 64 bits from the plane products in `terms`."""
    pa, pb = ([p.double() for p in planes(x.float())] for x in (a, b))
    return sum(pa[i] @ pb[j].transpose(-1, -2) for i, j in terms)


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def score_case(term, B, Tq, Tk, D):
    """q, k, v [B][rows][1][D] and a scale: scores of 0 to 4 that the products of `term` alone make (n of D / length pairs
    at key j; every third row at a half and a quarter). The reference in 64 bits; and the bound.

    All plane products and their sums are multiples of 2^-18 below 2^6, so exact in 24 bits; the exponents (up to
    6) are off by 6 (2^-24 each for the rounded log2 e, its product with the scale, the fused multiply-add and the
    offset), some 2^-20 of a weight; ex2 2^-22; sums (Tk + 24) 2^-22, as for any input. Scores without `term` are 0."""
    qs, ks, unit = GROUPS[term]
    n = D // len(qs)
    q = torch.zeros(B, Tq, 1, D)
    q[..., :n * len(qs)] = torch.tensor(qs).repeat(n)
    q *= (2.0 ** -(torch.arange(Tq) % 3))[None, :, None, None]
    count = (torch.arange(Tk) * 7) % (n + 1)
    live = (torch.arange(n)[None] < count[:, None]).float()
    k = torch.zeros(B, Tk, 1, D)
    k[..., :n * len(ks)] = (live[..., None] * torch.tensor(ks)).flatten(1)[None, :, None]
    v = _rand(5, B, Tk, 1, D)
    scale = 4.0 / (n * unit)
    p = torch.softmax(scale * (q.double()[:, :, 0] @ k.double()[:, :, 0].transpose(-1, -2)), -1)
    ref = (p @ v.double()[:, :, 0])[:, :, None]
    tol = 2.0 ** -24 * ref.abs() + (2.0 ** -19 + (Tk + 24) * 2.0 ** -22) * (p @ v.double().abs()[:, :, 0])[:, :, None]
    return q, k, v, scale, ref, tol


def output_case(B, Tq, Tk, D, first, second):
    """q, k, v, a mask that leaves two keys, a scale: key `first` has score 0 and value 0, key `second` score -x (24 random
    bits of 0..1, another one in each row) and a random value, so that the output is v p / (1 + p), p = exp(-x).

    The bound is 2^-19 of the result: exponents 5 2^-24 (three roundings of numbers below 1.5, times ln 2, and an
    offset's), two ex2 at 2^-22, the sum, the division and the products 6 2^-24, what the six products leave out 2^-25, the
    tensor core's truncation 3 2^-24: some 22 2^-24. A lost product of third planes takes up to 2^-17 of a result, that
    of second planes up to 2^-16."""
    x = torch.rand(B, Tq, generator=torch.Generator().manual_seed(6))
    q, k, v = torch.zeros(B, Tq, 1, D), torch.zeros(B, Tk, 1, D), _rand(7, B, Tk, 1, D)
    q[:, :, 0, 0] = x
    k[:, second, 0, 0] = -1.0
    v[:, first] = 0
    mask = torch.zeros(B, Tk, dtype=torch.uint8)
    mask[:, first] = mask[:, second] = 1
    p = torch.exp(-x.double())
    ref = (p / (1 + p))[:, :, None, None] * v.double()[:, second][:, None]
    return q, k, v, mask, 1.0, ref, 2.0 ** -19 * ref.abs()


def linear_case(T, Cin, Cout):
    """x, weight of positive numbers, the result, and the bound: accumulators of 32 channels, each step of four of them
    off by a unit (2^-23) of a sum that grows, 2.5 units; an addition in fp32 per accumulator, 2^-24 of a sum that
    grows; lo lo, up to 2^-20; the roundings of lo, 2^-21; the epilogue's 2^-24. TF32 without a lo part is off by some 2^-12."""
    g = torch.Generator().manual_seed(8)
    x, w = torch.rand(T, Cin, generator=g) + 0.5, torch.rand(Cout, Cin, generator=g) + 0.5
    ref = x.double() @ w.double().t()
    return x, w, ref, (5 + Cin / 64 + 16 + 8 + 1) * 2.0 ** -24 * ref
