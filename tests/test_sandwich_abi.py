"""Refusals and host-only calls of the sandwich norm and of the 8-bit checkpoints.  No GPU work is issued (CPU only): every
call here is refused before its first launch, or has nothing to do."""
import ctypes

import pytest
import torch

from gaussian_splatting_tile_gb300 import build_lib, rs

OK, P, Q = rs.RS_OK, 0x10000, 0x20000
BAD, SMALL = rs.RS_ERR_INVALID_ARG, rs.RS_ERR_WORKSPACE
ODD = 0x10001
ref = ctypes.byref


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return rs.lib()


BLOCK = dict(rows=4, cols=256, dtype=0, gate_cols=256, d_x=P, x_stride=256, d_x_scales=None, d_r=P, r_stride=256,
             d_r_scales=None, d_gate=P, gate_stride=256, d_gate_scales=None, d_residual_scale=P, d_post_weight=P,
             d_pre_weight=P)
KEPT = BLOCK | dict(d_x_scales=P, d_r_scales=P, d_gate_scales=P)
FORM = rs.rs_fp8_matrix(P, 256, P)
BAD_BLOCKS = [dict(rows=-1), dict(cols=0), dict(cols=16385, x_stride=20000, r_stride=20000, gate_stride=20000), dict(dtype=3),
              dict(dtype=-1), dict(gate_cols=2), dict(gate_cols=-1), dict(d_x=None), dict(d_x=ODD), dict(x_stride=255),
              dict(d_r=None), dict(d_r=ODD), dict(r_stride=1), dict(d_gate=None), dict(gate_stride=255),
              dict(d_residual_scale=ODD), dict(d_post_weight=None), dict(d_post_weight=ODD), dict(d_pre_weight=None),
              dict(d_x_scales=P), dict(d_r_scales=P), dict(d_gate_scales=P), dict(gate_cols=1, gate_stride=0),
              dict(gate_cols=1, d_gate_scales=P)]


@pytest.mark.parametrize("change", BAD_BLOCKS)
def test_operands_refused_both_ways(L, change):
    out = ref(rs.rs_sandwich_out(q=FORM))
    b = ref(rs.rs_sandwich(**(BLOCK | change)))
    assert L.rs_sandwich_norm_fwd(b, 1e-6, out, None) == BAD
    grads = ref(rs.rs_sandwich_grads(d_rstd_r=P, d_rstd_s=P, d_dL_dy=P, dy_stride=256, d_dL_dx=Q, dx_stride=256, d_dL_dr=P,
                                     dr_stride=256))
    assert L.rs_sandwich_norm_bwd(b, grads, None, 0, None) == BAD


@pytest.mark.parametrize("change", [dict(d_x=0x10008), dict(x_stride=250), dict(x_stride=264), dict(r_stride=128),
                                    dict(gate_stride=8), dict(d_r_scales=None), dict(d_x_scales=None),
                                    dict(d_gate_scales=None), dict(gate_cols=1), dict(d_x_scales=ODD)])
def test_kept_operands_refused(L, change):
    b = ref(rs.rs_sandwich(**(KEPT | change)))
    grads = ref(rs.rs_sandwich_grads(d_rstd_r=P, d_rstd_s=P, d_dL_dy=P, dy_stride=256, d_dL_dx=Q, dx_stride=256, d_dL_dr=P,
                                     dr_stride=256))
    assert L.rs_sandwich_norm_bwd(b, grads, None, 0, None) == BAD


def test_forward_refusals(L):
    def call(eps=1e-6, block=BLOCK, **out):
        return L.rs_sandwich_norm_fwd(ref(rs.rs_sandwich(**block)), eps, ref(rs.rs_sandwich_out(**({"q": FORM} | out))), None)

    F = rs.rs_fp8_matrix
    for c in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(block=KEPT), dict(q=F()),
              dict(q=F(P, 256, None)), dict(q=F(None, 0, P)), dict(q=F(P, 250, P)), dict(q=F(0x10008, 256, P)),
              dict(kept_x=F(P, 256, None)), dict(kept_r=F(P, 240, P)), dict(kept_gate=F(P, 256, ODD)),
              dict(d_sum=P, sum_stride=300), dict(d_sum=Q, sum_stride=255), dict(d_sum=ODD, sum_stride=256),
              dict(d_y=P, y_stride=100), dict(d_rstd_r=ODD), dict(d_rstd_s=ODD),
              dict(block=BLOCK | dict(gate_cols=1), kept_gate=FORM), dict(block=BLOCK | dict(gate_cols=0), kept_gate=FORM)):
        assert call(**c) == BAD, c
    assert L.rs_sandwich_norm_fwd(None, 1e-6, ref(rs.rs_sandwich_out(q=FORM)), None) == BAD
    assert L.rs_sandwich_norm_fwd(ref(rs.rs_sandwich(**BLOCK)), 1e-6, None, None) == BAD
    none = dict.fromkeys([k for k in BLOCK if k.startswith("d_")])
    assert call(block=BLOCK | none | dict(rows=0, gate_cols=0), q=F()) == OK


def test_backward_refusals(L):
    need = rs.rs_sandwich_norm_bwd_workspace_size(4, 256)
    assert need > 0 and rs.rs_sandwich_norm_bwd_workspace_size(-1, 5) == 0
    assert rs.rs_sandwich_norm_bwd_workspace_size(5, 0) == 0 and rs.rs_sandwich_norm_bwd_workspace_size(5, 16385) == 0
    base = dict(d_rstd_r=P, d_rstd_s=P, d_dL_dy=P, dy_stride=256, d_dL_dsum=Q, dsum_stride=256, d_dL_dx=P, dx_stride=256,
                d_dL_dr=Q, dr_stride=256, d_dL_dgate=0x30000, dgate_stride=256, d_dL_dpost_weight=P)

    def call(block=BLOCK, ws=P, bytes=need, **c):
        return L.rs_sandwich_norm_bwd(ref(rs.rs_sandwich(**block)), ref(rs.rs_sandwich_grads(**(base | c))), ws, bytes, None)

    for c in (dict(d_rstd_r=None), dict(d_rstd_s=ODD), dict(d_dL_dy=None), dict(dy_stride=255), dict(d_dL_dsum=ODD),
              dict(dsum_stride=1), dict(d_dL_dx=None), dict(dx_stride=300), dict(d_dL_dr=None), dict(d_dL_dr=P),
              dict(dr_stride=257), dict(d_dL_dgate=P), dict(d_dL_dgate=Q), dict(dgate_stride=200), dict(d_dL_dgate=ODD),
              dict(block=BLOCK | dict(gate_cols=0)), dict(block=BLOCK | dict(gate_cols=1), d_dL_dgate=P, dgate_stride=256),
              dict(d_dL_dpost_weight=ODD), dict(d_dL_dpre_weight=ODD), dict(d_dL_dresidual_scale=ODD), dict(ws=None),
              dict(ws=ODD)):
        assert call(**c) == BAD, c
    assert call(bytes=need - 1) == SMALL
    assert L.rs_sandwich_norm_bwd(None, ref(rs.rs_sandwich_grads(**base)), P, need, None) == BAD
    assert L.rs_sandwich_norm_bwd(ref(rs.rs_sandwich(**BLOCK)), None, P, need, None) == BAD
    assert call(block=BLOCK | dict(rows=0), d_dL_dpost_weight=None) == OK


def test_relu8_refusals(L):
    base = dict(rows=4, cols=256, dtype=0, x=P, xs=256, relu=P, relus=256, q=P, qs=256, sc=P, qt=P, qts=16, sct=P)
    call = lambda **c: L.rs_quantize_fp8_relu8(*(base | c).values(), None)
    for c in (dict(rows=-1), dict(cols=-1), dict(dtype=9), dict(x=None), dict(x=ODD), dict(xs=255), dict(relu=None),
              dict(relu=0x10008), dict(relus=250), dict(relus=128), dict(q=None), dict(sc=None), dict(qs=255), dict(qt=None),
              dict(sct=ODD), dict(qts=8), dict(q=None, sc=None, qt=None, sct=None)):
        assert call(**c) == BAD, c
    assert call(rows=0) == OK and call(cols=0) == OK


def test_transpose_refusals(L):
    base = dict(rows=4, cols=256, q=P, qs=256, sc=P, qt=P, qts=16, sct=P)
    call = lambda **c: L.rs_transpose_fp8(*(base | c).values(), None)
    for c in (dict(rows=-1), dict(cols=-1), dict(q=None), dict(q=0x10008), dict(qs=255), dict(qs=128), dict(sc=None), dict(sc=ODD),
              dict(qt=None), dict(qts=8), dict(qts=0), dict(sct=None), dict(sct=ODD)):
        assert call(**c) == BAD, c
    assert call(rows=0) == OK and call(cols=0) == OK


def test_matmul_q_refusals(L):
    need = rs.rs_matmul_fp8_q_workspace_size(64, 256, 1280)
    assert need >= 64 * 256 * 4
    base = dict(m=64, n=256, k=1280, a=P, as_=1280, sa=P, b=P, bs=1280, sb=P, rows=128, relu=0, q=P, qs=256, sc=P, ws=P,
                bytes=need)
    call = lambda **c: L.rs_matmul_fp8_q(*(base | c).values(), None)
    for c in (dict(m=-1), dict(n=-1), dict(k=-1), dict(a=None), dict(a=ODD), dict(as_=1264), dict(as_=1288), dict(sa=None),
              dict(b=None), dict(bs=100), dict(sb=ODD), dict(rows=64), dict(q=None), dict(q=0x10008), dict(qs=255), dict(qs=240),
              dict(sc=None), dict(sc=ODD), dict(ws=None), dict(ws=ODD), dict(m=0x7ffffc01)):
        assert call(**c) == BAD, c
    assert call(bytes=need - 1) == SMALL
    assert call(m=0) == OK and call(n=0) == OK
    assert rs.rs_matmul_fp8_q_workspace_size(0, 5, 5) == 0 and rs.rs_matmul_fp8_q_workspace_size(160000, 512, 512) == 0


def test_binding_refuses_what_it_cannot_describe(L):
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(TypeError):
        rs.rs_sandwich_norm_fwd(x, x, w, w)
    with pytest.raises(TypeError):
        rs.rs_sandwich_norm_fwd(x.int(), x, w, w)
    for gate in (torch.zeros(4, 2), torch.zeros(3, 8), torch.zeros(4)):
        with pytest.raises(ValueError):
            rs.rs_sandwich_norm_fwd(x, x, w, w, gate=gate)
    with pytest.raises(TypeError):
        rs.rs_transpose_fp8(x, w, x.t(), w)
    with pytest.raises(TypeError):
        rs.rs_quantize_fp8_relu8(x, x)


def test_packed_structures_are_the_declared_ones():
    names = lambda c: [n for n, _ in c._fields_]
    count = lambda c: sum(3 if t is rs.rs_fp8_matrix else 1 for _, t in c._fields_)
    for cls, pack, ints in ((rs.rs_sandwich, rs._SANDWICH, 4), (rs.rs_sandwich_out, rs._SANDWICH_OUT, 0),
                            (rs.rs_sandwich_grads, rs._SANDWICH_GRADS, 0)):
        values = list(range(1, count(cls) + 1))
        raw = pack(*values)
        assert len(raw) == ctypes.sizeof(cls)
        got = cls.from_buffer_copy(raw)
        flat = []
        for n in names(cls):
            v = getattr(got, n)
            flat += [v.d_q, v.stride, v.d_scales] if isinstance(v, rs.rs_fp8_matrix) else [v]
        assert flat == values
