"""The transformer-block operators: declared, exported, and bad calls rejected on
the host before CUDA is touched (runs without a GPU)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from prompt_conditioned_keypoint_b200 import binding as gk

L = gk.lib
OK, ARG, SHAPE, DTYPE, ALIGN = gk.GKD_OK, gk.GKD_ERR_ARG, gk.GKD_ERR_SHAPE, gk.GKD_ERR_DTYPE, gk.GKD_ERR_ALIGN
F32, BF16 = gk.GKD_F32, gk.GKD_BF16
REACHED = (gk.GKD_ERR_CUDA, ARG)   # past every host check: stopped at the pointer query of the stand-in pointer
P, MIS = 0x10000, 0x10004


def test_every_declared_operator_is_exported_and_bound():
    header = os.path.join(os.path.dirname(gk.HEADER_PATH), "gkd_blocks.h")
    with open(header) as f:
        names = re.findall(r"GKD_API\s+[\w\s\*]+?\b(gkd_\w+)\s*\(", f.read())
    assert sorted(names) == ["gkd_attention", "gkd_linear", "gkd_qk_norm_rope"]
    out = subprocess.run(["nm", "-D", "--defined-only", gk.LIB_PATH], capture_output=True, text=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    for n in names:
        assert n in exported and callable(getattr(gk, n))


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "use.c"
    src.write_text('#include "gkd_blocks.h"\nint main(void) { gkd_heads h = {0}; return h.heads + GKD_ACT_NONE; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.dirname(gk.HEADER_PATH),
                        str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def linear(x=P, dt=BF16, T=4, Cin=64, xs=64, w=P, Cout=32, bias=P, act=0, scale=None, res=None, rs=32, out=P, odt=BF16,
           os_=32):
    return L.gkd_linear(x, dt, T, Cin, xs, w, Cout, bias, act, scale, res, rs, out, odt, os_, None)


def test_linear_refusals():
    assert linear(dt=3) == ARG and linear(odt=-1) == ARG and linear(act=4) == ARG and linear(act=-1) == ARG
    assert linear(dt=F32, odt=BF16) == DTYPE
    assert linear(T=-1) == SHAPE and linear(Cin=0) == SHAPE and linear(Cin=12, xs=12) == SHAPE
    assert linear(Cin=65544, xs=65544) == SHAPE and linear(Cout=4) == SHAPE and linear(Cout=65544, os_=65544) == SHAPE
    assert linear(xs=56) == SHAPE and linear(os_=24) == SHAPE and linear(res=P, rs=24) == SHAPE
    assert linear(xs=1 << 40) == SHAPE
    assert linear(x=None) == ARG and linear(w=None) == ARG and linear(out=None) == ARG
    assert "out" in gk.gkd_last_error()
    assert linear(x=MIS) == ALIGN and linear(w=MIS) == ALIGN and linear(out=MIS) == ALIGN and linear(res=MIS) == ALIGN
    assert linear(bias=MIS) == ALIGN and linear(scale=MIS) == ALIGN
    assert linear(xs=68) == ALIGN and linear(os_=36) == ALIGN and linear(res=P, rs=36) == ALIGN
    assert linear(dt=F32, odt=F32, xs=68, os_=36) in REACHED         # 16-byte multiples in fp32
    assert linear(T=1, xs=0, os_=0) in REACHED                       # one row has no stride
    assert linear(T=0, x=None, w=None, out=None) == OK


def view(data=P, b=1 << 12, r=1 << 8, h=64, heads=4):
    return gk.GkdHeads(data, b, r, h, heads)


def rope(q="v", k="v", dt=BF16, B=2, T=3, D=64, qw=None, kw=None, eps=1e-6, pos=P, pbs=0, axes=2, axis=P, freq=P, pairs=32,
         inter=0, qo="v", ko="v"):
    q, k, qo, ko = (view() if v == "v" else v for v in (q, k, qo, ko))
    return L.gkd_qk_norm_rope(q, k, dt, B, T, D, qw, kw, eps, pos, pbs, axes, axis, freq, pairs, inter, qo, ko, None)


def test_qk_norm_rope_refusals():
    assert rope(dt=2) == ARG and rope(inter=2) == ARG
    assert rope(B=-1) == SHAPE and rope(B=65536) == SHAPE and rope(T=-1) == SHAPE
    assert rope(D=0) == SHAPE and rope(D=60) == SHAPE and rope(D=264) == SHAPE
    assert rope(axes=0) == SHAPE and rope(axes=4) == SHAPE and rope(pbs=-1) == SHAPE
    assert rope(pairs=-4) == SHAPE and rope(pairs=36) == SHAPE and rope(pairs=6) == SHAPE
    assert rope(q=None) == ARG and rope(qo=None) == ARG and rope(k=None) == ARG and rope(ko=None) == ARG
    assert rope(k=None, ko=None) in REACHED
    assert rope(qo=view(heads=3)) == SHAPE and rope(ko=view(heads=8)) == SHAPE
    assert rope(q=view(heads=0), qo=view(heads=0)) == SHAPE and rope(q=view(heads=1025), qo=view(heads=1025)) == SHAPE
    assert rope(qw=P) == ARG and rope(kw=P) == ARG
    assert rope(qw=P, kw=P, eps=0.0) == ARG and rope(qw=P, kw=P, eps=float("nan")) == ARG
    assert rope(eps=0.0) in REACHED                                  # no norm, no eps
    assert rope(pos=None) == ARG and rope(axis=None) == ARG and rope(freq=None) == ARG
    assert rope(pairs=0, pos=None, axis=None, freq=None) in REACHED
    assert rope(pos=P + 2) == ALIGN and rope(qw=P + 1, kw=P) == ALIGN
    assert rope(q=view(data=MIS)) == ALIGN and rope(k=view(data=None)) == ARG
    assert rope(q=view(r=260)) == ALIGN and rope(q=view(h=32)) == SHAPE and rope(q=view(b=-64)) == SHAPE
    assert rope(qo=view(b=0)) == SHAPE                               # an output is not shared by the batch
    assert rope(q=view(b=0)) in REACHED                              # an input may be
    assert rope(q=view(b=3), T=1, B=1) in REACHED                    # strides of axes of size 1 are not looked at
    assert rope(q=view(h=1 << 40)) == SHAPE
    assert rope(B=0, pos=None, axis=None, freq=None) == OK and rope(T=0, q=view(data=None)) == OK


def attention(q="v", k="v", v="v", dt=BF16, B=2, Tq=3, Tk=5, D=64, scale=0.125, causal=0, mask=None, mbs=5, out="v"):
    q, k, v, out = (view() if x == "v" else x for x in (q, k, v, out))
    return L.gkd_attention(q, k, v, dt, B, Tq, Tk, D, scale, causal, mask, mbs, out, None)


def test_attention_refusals():
    assert attention(dt=5) == ARG and attention(causal=2) == ARG
    assert attention(scale=0.0) == ARG and attention(scale=-1.0) == ARG
    assert attention(scale=float("inf")) == ARG and attention(scale=float("nan")) == ARG
    assert attention(B=-1) == SHAPE and attention(B=65536) == SHAPE and attention(Tq=-1) == SHAPE and attention(Tk=-1) == SHAPE
    assert attention(Tk=2 ** 31 - 1) == SHAPE
    assert attention(D=4) == SHAPE and attention(D=68) == SHAPE and attention(D=136) == SHAPE and attention(mbs=-1) == SHAPE
    for name in ("q", "k", "v", "out"):
        assert attention(**{name: None}) == ARG and attention(**{name: view(data=None)}) == ARG
        assert attention(**{name: view(data=MIS)}) == ALIGN and attention(**{name: view(r=260)}) == ALIGN
        assert attention(**{name: view(r=60)}) == SHAPE
    assert attention(k=view(heads=3), v=view(heads=3)) == SHAPE      # 3 does not divide 4
    assert attention(k=view(heads=2)) == SHAPE and attention(out=view(heads=2)) == SHAPE
    assert attention(k=view(heads=2), v=view(heads=2)) in REACHED
    assert attention(k=view(b=0), v=view(b=0)) in REACHED and attention(out=view(b=0)) == SHAPE
    assert attention(B=65535, Tq=1 << 21, q=view(heads=1024, b=64, r=64), out=view(heads=1024, b=64, r=64)) == SHAPE
    assert attention(B=0) == OK and attention(Tq=0) == OK
    assert attention(Tk=0, k=view(data=None), v=view(data=None)) in REACHED


def test_views_follow_a_tensors_strides():
    t = torch.zeros(2, 5, 12, 64)
    v = gk.gkd_heads(t[:, 1:, 4:8])
    assert (v.batch_stride, v.row_stride, v.head_stride, v.heads) == (5 * 12 * 64, 12 * 64, 64, 4)
    assert v.data == t.data_ptr() + 4 * (12 * 64 + 4 * 64)
    assert gk.gkd_heads(v) is v and gk.gkd_heads(None) is None
    ahead = torch.zeros(2, 4, 5, 64).transpose(1, 2)
    v = gk.gkd_heads(ahead)
    assert (v.row_stride, v.head_stride, v.heads) == (64, 5 * 64, 4)
    for bad in (torch.zeros(2, 5, 64), torch.zeros(2, 5, 64, 4).transpose(2, 3)):
        with pytest.raises(gk.GkdError):
            gk.gkd_heads(bad)


def test_binding_raises_with_the_librarys_message():
    x = torch.zeros(4, 64)
    with pytest.raises(gk.GkdError) as e:
        gk.gkd_linear(x, F32, 4, 60, 60, x, 32, None, gk.GKD_ACT_NONE, None, None, 0, x, F32, 32, stream=0)
    assert e.value.status == SHAPE and "Cin=60" in str(e.value)
    assert ctypes.sizeof(gk.GkdHeads) == 40


def test_block_calls_follow_the_first_tensors_device(monkeypatch):
    class OnDevice:
        device = torch.device("cuda", 3)

    monkeypatch.setattr(gk, "_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(gk, "_stream", lambda s, ref=None: -1 if s is None else s)
    assert gk._stream_fast(None, OnDevice()) == 1003
    assert gk._stream_fast(77, OnDevice()) == 77
    assert gk._stream_fast(None, torch.zeros(4)) == -1 and gk._stream_fast(None, 12345) == -1 and gk._stream_fast(None) == -1
