"""Refusals and host-only calls of the wide appearance network's operators.  No GPU work is issued (CPU only): every
call here is refused before its first launch, or has nothing to do."""
import ctypes

import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs

OK, P = rs.RS_OK, ctypes.c_void_p(0x10000)
BAD, SMALL = rs.RS_ERR_INVALID_ARG, rs.RS_ERR_WORKSPACE
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return rs.lib()


NORM = dict(rows=4, cols=256, dtype=0, x=P, xs=256, r=None, rs=0, w=P, eps=1e-6, sum=None, sums=0, y=None, ys=0, q=P,
            qs=256, sc=P, rstd=None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(cols=16385, xs=20000, qs=20000), dict(dtype=3), dict(dtype=-1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(x=ODD), dict(xs=255), dict(w=None), dict(w=ODD),
    dict(r=P, rs=255), dict(r=ODD, rs=256), dict(sum=P, sums=300), dict(sum=P, sums=10), dict(y=P, ys=100),
    dict(q=None), dict(sc=None), dict(q=None, sc=None), dict(qs=250), dict(qs=264), dict(q=ctypes.c_void_p(0x10008)),
    dict(rstd=ODD)])
def test_norm_forward_refusals(L, change):
    a = NORM | change
    assert L.rs_rms_norm_fwd(*a.values(), None) == BAD


def test_norm_forward_of_no_rows(L):
    assert L.rs_rms_norm_fwd(*(NORM | dict(rows=0, x=None, q=None, sc=None, w=None)).values(), None) == OK


def test_norm_backward_refusals(L):
    need = rs.rs_rms_norm_bwd_workspace_size(4, 256)
    assert need > 0
    base = dict(rows=4, cols=256, dtype=2, s=P, ss=256, w=P, rstd=P, dy=P, dys=256, ds=None, dss=0, dx=P, dxs=256, dw=P,
                ws=P, bytes=need)
    call = lambda **c: L.rs_rms_norm_bwd(*(base | c).values(), None)
    for c in (dict(rows=-1), dict(cols=0), dict(cols=20000), dict(dtype=5), dict(s=None), dict(ss=1), dict(w=ODD),
              dict(rstd=None), dict(dy=None), dict(dys=255), dict(ds=P, dss=3), dict(dx=None), dict(dxs=255), dict(dw=ODD),
              dict(ws=None), dict(ws=ODD), dict(dys=300)):
        assert call(**c) == BAD, c
    assert call(bytes=need - 1) == SMALL
    assert call(rows=0, dw=None) == OK
    assert rs.rs_rms_norm_bwd_workspace_size(-1, 5) == 0 and rs.rs_rms_norm_bwd_workspace_size(5, 0) == 0


def test_quantize_refusals(L):
    base = dict(rows=4, cols=256, dtype=0, x=P, xs=256, relu=None, relus=0, q=P, qs=256, sc=P, qt=P, qts=16, sct=P)
    call = lambda **c: L.rs_quantize_fp8(*(base | c).values(), None)
    for c in (dict(rows=-1), dict(cols=-1), dict(dtype=9), dict(x=None), dict(x=ODD), dict(xs=255), dict(relu=P, relus=1),
              dict(relu=ODD, relus=256), dict(q=None), dict(sc=None), dict(qs=255), dict(qt=None), dict(sct=ODD), dict(qts=8),
              dict(q=None, sc=None, qt=None, sct=None), dict(q=ODD)):
        assert call(**c) == BAD, c
    assert call(rows=0) == OK and call(cols=0) == OK
    del base["relu"], base["relus"]
    assert L.rs_quantize_fp8_blocks(*(base | dict(qts=8)).values(), None) == BAD
    assert L.rs_quantize_fp8_blocks(*(base | dict(rows=0)).values(), None) == OK


def test_matmul_refusals(L):
    need = rs.rs_matmul_fp8_workspace_size(64, 256, 128)
    base = dict(m=64, n=256, k=128, a=P, as_=128, sa=P, b=P, bs=128, sb=P, rows=128, relu=0, dt=0, out=P, os=256, ws=P,
                bytes=max(need, 1))
    call = lambda **c: L.rs_matmul_fp8(*(base | c).values(), None)
    for c in (dict(m=-1), dict(n=-1), dict(k=-1), dict(a=None), dict(a=ODD), dict(as_=120), dict(as_=136), dict(sa=None),
              dict(b=None), dict(bs=100), dict(sb=ODD), dict(rows=64), dict(dt=3), dict(out=None), dict(out=ODD), dict(os=255)):
        assert call(**c) == BAD, c
    assert call(m=0) == OK and call(n=0) == OK
    big = rs.rs_matmul_fp8_workspace_size(512, 256, 160000)
    if big:
        more = dict(m=512, k=160000, as_=160000, bs=160000)
        assert call(**more, bytes=big - 1) == SMALL and call(**more, ws=None, bytes=big) == BAD


def test_clip_refusals(L):
    need = rs.rs_grad_norm_workspace_size(2)
    assert 0 < need <= rs.rs_grad_norm_workspace_size(1000)
    assert L.rs_grad_norm_workspace_size(-1) == 0

    def call(max_norm=1.0, norm=P, ws=P, bytes=need, n=2, null=False, **c):
        t = (rs.rs_grad_tensor * 2)()
        for e in t:
            e.d_grad, e.d_out, e.count, e.dtype, e.activation = 0x10000, 0x20000, 10, 0, 0
        for k, v in c.items():
            setattr(t[1], k, v)
        return (L.rs_grad_clip(None if null else t, n, max_norm, norm, ws, bytes, None),
                L.rs_grad_norm(None if null else t, n, norm, ws, bytes, None) if c or null or norm is not P or ws is not P
                or bytes < need or n < 0 else BAD)

    for c in (dict(n=-1), dict(null=True), dict(norm=None), dict(norm=ODD), dict(ws=None), dict(ws=ODD), dict(dtype=4),
              dict(activation=3), dict(activation=-1), dict(d_grad=None), dict(d_grad=0x10002), dict(activation=1),
              dict(count=1 << 50)):
        assert call(**c) == (BAD, BAD), c
    assert call(d_out=0x20001, bytes=0)[0] == BAD
    for m in (0.0, -1.0, float("nan")):
        assert call(max_norm=m)[0] == BAD
    assert call(bytes=need - 1) == (SMALL, SMALL)


def test_clipped_adam_refusals(L):
    need = rs.rs_grad_norm_workspace_size(1)
    seg = (rs.rs_adam_segment * 1)()
    s = seg[0]
    s.d_param = s.d_grad = s.d_m = s.d_v = 0x10000
    s.count, s.lr, s.activation = 10, 0.01, 0
    call = lambda step=1, b1=0.9, eps=1e-15, limit=1.0, norm=P, ws=P, bytes=need, n=1: L.rs_adam_step_clipped(
        seg, n, b1, 0.999, eps, step, limit, norm, ws, bytes, None)
    for c in (dict(step=0), dict(b1=1.0), dict(eps=0.0), dict(limit=0.0), dict(limit=float("nan")), dict(norm=None),
              dict(ws=None), dict(n=17), dict(n=-1)):
        assert call(**c) == BAD, c
    assert call(bytes=need - 1) == SMALL
    s.activation = 3
    assert call() == BAD


def test_binding_refuses_what_it_cannot_describe(L):
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        rs.rs_rms_norm_fwd(x, torch.ones(8))
    with pytest.raises(TypeError):
        rs.rs_quantize_fp8(x.int())
    with pytest.raises(TypeError):
        rs.GradTable([rs.GradTensor(torch.zeros(4, dtype=torch.int32))])
    with pytest.raises(TypeError):
        rs.GradTable([rs.GradTensor(torch.zeros(4))])
