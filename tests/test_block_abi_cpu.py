"""Refusals of the attention-block operators without a GPU: the C interface
with fake addresses (validation never reads them), and the tensor calls."""
import ctypes

import pytest
import torch

import deformable_attention_sampling_b200 as dcnb
from deformable_attention_sampling_b200 import build as dcn_build

OK, BAD, UNSUP, ALIGN = (dcnb.DCN_OK, dcnb.DCN_ERR_INVALID_ARG, dcnb.DCN_ERR_UNSUPPORTED,
                         dcnb.DCN_ERR_MISALIGNED)
BF16 = 2
# fake device addresses 16 GiB apart
P = [0x7F0000000000 + (i << 34) for i in range(20)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    dcn_build.build()
    return dcnb.library()


def ints(values):
    return (ctypes.c_int * max(len(values), 1))(*values)


def rope(lib, grad, **kw):
    a = dict(x=P[0], pos=P[1], freqs=P[2], go=P[3], out=P[4], gpos=P[5], pairs=(8, 8), N=2, L=7,
             M=4, D=32, A=2, images=2, x_image=7 * 128, x_row=128, inter=0, inv=0, dtype=BF16)
    a.update(kw)
    pairs = None if a["pairs"] is None else ints(a["pairs"])
    tail = (a["N"], a["L"], a["M"], a["D"], a["A"], a["images"], a["x_image"], a["x_row"],
            a["inter"], a["inv"], a["dtype"], None)
    if grad:
        return lib.axial_rope_backward(a["x"], a["pos"], a["freqs"], a["go"], a["out"], a["gpos"],
                                       pairs, *tail)
    return lib.axial_rope_forward(a["x"], a["pos"], a["freqs"], a["out"], pairs, *tail)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), BAD), (dict(N=-1), BAD), (dict(L=-1), BAD), (dict(M=0), BAD), (dict(D=0), BAD),
    (dict(A=0), BAD), (dict(A=5, pairs=(1,) * 5), UNSUP), (dict(pairs=None), BAD),
    (dict(pairs=(9, 8)), BAD),                       # 34 channels of 32
    (dict(pairs=(-1, 8)), BAD), (dict(images=3), BAD), (dict(inter=2), BAD), (dict(inv=-1), BAD),
    (dict(x_row=127), BAD), (dict(x_image=-1), BAD),
    (dict(D=1024, pairs=(200, 200), x_row=4096), UNSUP),            # 400 pairs
    (dict(M=1 << 20, x_row=1 << 25), UNSUP), (dict(N=1 << 20, L=1 << 12, images=1), UNSUP),
    (dict(x=None), BAD), (dict(pos=None), BAD), (dict(freqs=None), BAD), (dict(out=None), BAD),
    (dict(x=P[0] + 1), ALIGN), (dict(pos=P[1] + 2), ALIGN), (dict(out=P[4] + 1), ALIGN),
    (dict(out=P[0] + 2), BAD), (dict(out=P[1]), BAD), (dict(out=P[2]), BAD),
    (dict(N=0, images=1), OK), (dict(L=0, x=None, out=None), OK),
])
def test_axial_rope_refusals(lib, grad, change, status):
    before = dcnb.dcn_launch_count()
    assert rope(lib, grad, **change) == status
    assert dcnb.dcn_launch_count() == before


@pytest.mark.parametrize("change,status", [
    (dict(go=None), BAD), (dict(out=P[3]), BAD), (dict(gpos=P[4]), BAD), (dict(gpos=P[1]), BAD),
    (dict(gpos=P[5] + 2), ALIGN), (dict(out=P[0]), BAD)])      # no in-place gradient
def test_axial_rope_gradient_refusals(lib, change, status):
    assert rope(lib, True, **change) == status


def test_axial_rope_in_place_needs_dense_tokens(lib):
    assert rope(lib, False, out=P[0], x_row=256, x_image=7 * 256) == BAD


def join(lib, **kw):
    a = dict(x=P[0], y=P[1], scale=P[2], gate=P[3], pw=P[4], pb=P[5], qw=P[6], qb=P[7], z=P[8],
             h=P[9], N=2, L=5, C=64, flags=6, eps=1e-6, dtype=BF16)
    a.update(kw)
    return lib.norm_residual_forward(*(a[k] for k in ("x", "y", "scale", "gate", "pw", "pb", "qw",
                                                      "qb", "z", "h", "N", "L", "C", "flags",
                                                      "eps", "dtype")), None)


def join_grad(lib, **kw):
    a = dict(y=P[0], z=P[1], gz=P[2], gh=P[3], scale=P[4], gate=P[5], pw=P[6], pb=P[7], qw=P[8],
             gx=P[9], gy=P[10], gs=P[11], gg=P[12], gpw=P[13], gpb=P[14], gqw=P[15], gqb=P[16],
             ws=P[17], ws_bytes=1 << 30, N=2, L=5, C=64, flags=6, eps=1e-6, dtype=BF16)
    a.update(kw)
    return lib.norm_residual_backward(
        *(a[k] for k in ("y", "z", "gz", "gh", "scale", "gate", "pw", "pb", "qw", "gx", "gy", "gs",
                         "gg", "gpw", "gpb", "gqw", "gqb", "ws", "ws_bytes", "N", "L", "C",
                         "flags", "eps", "dtype")), None)


@pytest.mark.parametrize("call", [join, join_grad])
@pytest.mark.parametrize("change,status", [
    (dict(dtype=-1), BAD), (dict(N=-1), BAD), (dict(L=-2), BAD), (dict(C=0), BAD),
    (dict(flags=8), BAD), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(C=8193), UNSUP), (dict(N=1 << 16, L=1 << 16), UNSUP),
    (dict(flags=4), BAD),                       # factors of a norm that is off
    (dict(flags=2), BAD), (dict(y=None), BAD), (dict(z=None), BAD),
    (dict(y=P[0] + 1), ALIGN), (dict(gate=P[5] + 1), ALIGN),
])
def test_norm_residual_refusals(lib, call, change, status):
    before = dcnb.dcn_launch_count()
    assert call(lib, **change) == status
    assert dcnb.dcn_launch_count() == before


@pytest.mark.parametrize("change", [dict(x=None), dict(h=None), dict(z=P[1]), dict(h=P[0]),
                                    dict(h=P[8] + 16), dict(z=P[0] + 2), dict(z=P[3])])
def test_norm_residual_forward_pointers(lib, change):
    assert join(lib, **change) == BAD


@pytest.mark.parametrize("change,status", [
    (dict(gz=None), BAD), (dict(gh=None), BAD), (dict(gx=None), BAD), (dict(gy=None), BAD),
    (dict(ws=None), BAD), (dict(ws_bytes=64), BAD), (dict(ws=P[17] + 8), ALIGN),
    (dict(gate=None), BAD),                     # its gradient asked for without it
    (dict(gx=P[2]), BAD), (dict(gy=P[9]), BAD), (dict(gs=P[11] + 1), ALIGN), (dict(ws=P[0]), BAD)])
def test_norm_residual_backward_pointers(lib, change, status):
    assert join_grad(lib, **change) == status


def test_norm_residual_empty_forward(lib):
    assert join(lib, N=0) == OK
    assert join(lib, L=0, x=None, y=None, z=None, h=None) == OK
    size = dcnb.norm_residual_backward_workspace_size
    assert size(0, 5, 64, 1, BF16) == 0 and size(2, 5, 64, 0, BF16) > 0
    assert size(2, 5, 8193, 0, BF16) == UNSUP and size(2, 5, 64, 2, BF16) == BAD


def attn(lib, grad=False, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], lam=P[3], mask=P[4], lengths=P[5], out=P[6], maps=P[7],
             lse=P[8], go=P[9], gq=P[10], gk=P[11], gv=P[12], gl=P[13], ws=P[14],
             ws_bytes=1 << 33, N=2, Lq=9, Lk=70, M=4, Mk=2, D=64, Dv=128, scale=0.125, causal=1,
             dtype=BF16)
    a.update(kw)
    tail = [a[k] for k in ("ws", "ws_bytes", "N", "Lq", "Lk", "M", "Mk", "D", "Dv")]
    qr, kr, vr = a["M"] * 2 * a["D"], a["Mk"] * 2 * a["D"], a["Mk"] * a["Dv"]
    tail += [a.get(k, d) for k, d in (("q_image", a["Lq"] * qr), ("q_row", qr),
                                      ("k_image", a["Lk"] * kr), ("k_row", kr),
                                      ("v_image", a["Lk"] * vr), ("v_row", vr))]
    tail += [a["scale"], a["causal"], a["dtype"], None]
    head = [a[k] for k in ("q", "k", "v", "lam", "mask", "lengths")]
    if grad:
        return lib.diff_attn_backward(*head, a["maps"], a["lse"], a["go"], a["gq"], a["gk"], a["gv"], a["gl"], *tail)
    return lib.diff_attn_forward(*head, a["out"], a["maps"], a["lse"], *tail)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(dtype=9), BAD), (dict(N=-1), BAD), (dict(Lq=-1), BAD), (dict(Lk=-1), BAD),
    (dict(M=0), BAD), (dict(Mk=0), BAD), (dict(M=5), BAD), (dict(D=0), BAD), (dict(Dv=0), BAD),
    (dict(causal=2), BAD), (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD),
    (dict(q_image=-1), BAD), (dict(q_row=511), BAD), (dict(k_row=255), BAD), (dict(v_row=0), BAD),
    (dict(D=129), UNSUP), (dict(Dv=257), UNSUP), (dict(N=40000, Lq=1, Lk=1), UNSUP),
    (dict(Lk=2147483647, Lq=1), UNSUP), (dict(Lq=1 << 30), UNSUP),
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(lam=None), BAD),
    (dict(q=P[0] + 1), ALIGN), (dict(lengths=P[5] + 2), ALIGN),
    (dict(lse=P[8] + 2), ALIGN), (dict(ws=P[14] + 8), ALIGN), (dict(maps=P[7] + 2), ALIGN),
])
def test_diff_attn_refusals(lib, grad, change, status):
    before = dcnb.dcn_launch_count()
    assert attn(lib, grad, **change) == status
    assert dcnb.dcn_launch_count() == before


@pytest.mark.parametrize("change", [
    dict(out=None), dict(maps=None), dict(lse=None), dict(out=P[0] + 64), dict(out=P[1]),
    dict(maps=P[6]),
    dict(lse=P[4]), dict(out=P[3])])
def test_diff_attn_forward_pointers(lib, change):
    assert attn(lib, **change) == BAD


@pytest.mark.parametrize("change", [
    dict(go=None), dict(gq=None), dict(gk=None), dict(gv=None), dict(gl=None), dict(maps=None),
    dict(lse=None), dict(ws=None), dict(ws_bytes=16), dict(gq=P[0]), dict(gk=P[2] + 16),
    dict(gv=P[9]), dict(gl=P[8]), dict(gq=P[11]), dict(ws=P[7])])
def test_diff_attn_backward_pointers(lib, change):
    assert attn(lib, True, **change) == BAD


def test_diff_attn_split_needs_its_workspace(lib):
    big = dict(N=1, Lq=1, Lk=8192, Mk=1, M=4)
    need = dcnb.diff_attn_forward_workspace_size(1, 1, 8192, 4, 1, 64, 128, BF16)
    assert need > 0
    assert attn(lib, ws=None, **big) == BAD
    assert attn(lib, ws_bytes=need - 1, **big) == BAD
    assert attn(lib, ws=P[0], **big) == BAD
    assert attn(lib, N=0) == OK and attn(lib, Lq=0, q=None, out=None) == OK


@pytest.mark.parametrize("call", [
    lambda t: dcnb.axial_rope(t(1, 2, 3, 4), t(1, 2, 1), t(2), (2,)),                    # not on a GPU
    lambda t: dcnb.axial_rope(t(2, 3, 4), t(1, 2, 1), t(2), (2,)),
    lambda t: dcnb.axial_rope(t(1, 2, 3, 4), t(1, 2, 1), t(2), (1,)),
    lambda t: dcnb.axial_rope(t(1, 2, 3, 4), t(1, 2, 1), t(3), (3,)),
    lambda t: dcnb.axial_rope(t(1, 2, 3, 4), t(1, 2, 1).double(), t(2), (2,)),
    lambda t: dcnb.axial_rope(t(1, 2, 3, 4), t(3, 2, 1), t(2), (2,)),
    lambda t: dcnb.norm_residual(t(1, 2, 8), t(1, 2, 8)),
    lambda t: dcnb.norm_residual(t(1, 2, 8), t(1, 2, 8), norm="batch"),
    lambda t: dcnb.norm_residual(t(2, 8), t(2, 8)),
    lambda t: dcnb.norm_residual_grad(t(1, 2, 8), t(1, 2, 8), t(1, 2, 8)),
    lambda t: dcnb.diff_attn(t(1, 2, 3, 2, 4), t(1, 2, 3, 2, 4), t(1, 2, 3, 4), t(3)),
    lambda t: dcnb.diff_attn(t(1, 2, 3, 2, 4), t(1, 2, 2, 2, 4), t(1, 2, 2, 4), t(3)),
    lambda t: dcnb.diff_attn(t(1, 2, 3, 4), t(1, 2, 3, 4), t(1, 2, 3, 4), t(3)),
])
def test_tensor_calls_refuse(call):
    with pytest.raises(ValueError):
        call(lambda *s: torch.zeros(s))
