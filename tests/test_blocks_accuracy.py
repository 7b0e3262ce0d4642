"""CPU: the accuracy cases of the fp32 operators tell every split product from none: a model with all of them stays within
the bounds that the kernels are held to, and one that lacks any of them does not."""
import block_accuracy as A
import pytest
import torch


@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("term", A.TERMS)
def test_every_product_of_the_scores_is_seen(term, D):
    q, k, v, scale, ref, tol = A.score_case(term, 1, 20, 70, D)

    def attend(terms):
        s = scale * A.split_product(q[:, :, 0], k[:, :, 0], terms)
        return (torch.softmax(s, -1) @ v.double()[:, :, 0])[:, :, None]
    assert bool(((attend(A.TERMS) - ref).abs() <= tol / 100).all())
    without = (attend([t for t in A.TERMS if t != term]) - ref).abs()
    assert bool((without > 100 * tol).any())


def test_every_product_of_the_weights_is_seen():
    q, k, v, mask, scale, ref, tol = A.output_case(1, 200, 100, 64, 3, 90)
    p = torch.exp(scale * (q.double()[:, :, 0] @ k.double()[:, :, 0].transpose(-1, -2))) * mask[0]
    total = p.sum(-1, keepdim=True)

    def output(terms):
        return (A.split_product(p, v[:, :, 0].transpose(-1, -2).contiguous(), terms) / total)[:, :, None]
    # what a float holds of p is 2^-24 of it
    assert bool(((output(A.TERMS) - ref).abs() <= tol / 8).all())
    for term in A.TERMS:
        without = (output([t for t in A.TERMS if t != term]) - ref).abs()
        assert bool((without > 1.5 * tol).any()), term


@pytest.mark.parametrize("Cin", [8, 520, 4104])
def test_every_product_of_the_linear_layer_is_seen(Cin):
    x, w, ref, tol = A.linear_case(9, Cin, 16)

    def parts(t):                                           # TF32 has 11 bits; lo's rounding is left out
        hi = (t.view(torch.int32) & -8192).view(torch.float32)
        return hi.double(), (t - hi).double()
    (xh, xl), (wh, wl) = parts(x), parts(w)
    terms = [xh @ wh.t(), xh @ wl.t(), xl @ wh.t()]
    assert bool(((sum(terms) - ref).abs() <= tol).all())
    for lost in range(3):
        assert bool(((sum(terms) - terms[lost] - ref).abs() > 5 * tol).all())


def test_a_scale_whose_base_2_form_overflows_is_refused():
    from prompt_conditioned_keypoint_b200 import binding as gk
    v = gk.GkdHeads(0x10000, 1 << 12, 1 << 8, 64, 4)
    for scale, refused in ((2.0 ** 127, True), (3e38, True), (1.7e38, False), (1e-44, False)):
        status = gk.lib.gkd_attention(v, v, v, gk.GKD_F32, 2, 3, 5, 64, scale, 0, None, 5, v, None)
        assert ("scale" in gk.gkd_last_error()) == refused and status in (gk.GKD_ERR_CUDA, gk.GKD_ERR_ARG)
