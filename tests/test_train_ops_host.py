"""Refusals of the training operators' entry points (no GPU: the pointers are fake, nothing is launched)."""
import ctypes
import math

import pytest

import fully_sharded_gb300 as fs

A, B, C, D, E, F, G = (0x10000000 * (i + 1) for i in range(7))  # far apart
lib = fs._lib


def norm_args(**over):
    a = dict(rows=4, cols=100, x_stride=100, residual_stride=100, h_stride=100, y_stride=100, dtype=1, gain_dtype=1,
             y_dtype=1, group=0, eps=1e-6)
    a.update(over)
    return fs.RmsNormArgs(**a)


@pytest.mark.parametrize("over,pointers", [
    (dict(cols=0), {}), (dict(cols=(1 << 30) + 1), {}), (dict(rows=-1), {}), (dict(x_stride=99), {}),
    (dict(y_stride=0), {}), (dict(dtype=2), {}), (dict(dtype=7), {}), (dict(gain_dtype=2), {}), (dict(y_dtype=0), {}),
    (dict(group=128), {}), (dict(y_dtype=2, group=48), {}), (dict(y_dtype=2), {}), (dict(eps=0.0), {}),
    (dict(eps=-1.0), {}), (dict(eps=math.inf), {}), (dict(eps=math.nan), {}), (dict(eps=1e-60), {}),
    ({}, dict(x=None)), ({}, dict(y=None)), ({}, dict(gain=None)), ({}, dict(x=A + 1)), ({}, dict(residual=F)),
    ({}, dict(h_out=F)), ({}, dict(scales=G)), (dict(h_stride=99), dict(residual=F, h_out=G)),
    ({}, dict(rstd=G + 2)), (dict(rows=1 << 60, x_stride=1 << 40, y_stride=1 << 40), {}),
])
def test_rmsnorm_refuses(over, pointers):
    p = dict(x=A, residual=None, gain=B, h_out=None, y=C, scales=None, rstd=None)
    p.update(pointers)
    assert lib.fsdp_rmsnorm(ctypes.byref(norm_args(**over)), p["x"], p["residual"], p["gain"], p["h_out"], p["y"],
                            p["scales"], p["rstd"], None) == fs.FSDP_EINVAL


@pytest.mark.parametrize("pointers", [
    dict(y=A + 2), dict(y=A - 200), dict(h_out=A + 798), dict(h_out=C), dict(y=B), dict(rstd=C + 4), dict(rstd=A),
    dict(h_out=D + 2),
])
def test_rmsnorm_refuses_overlaps(pointers):
    p = dict(x=A, residual=D, gain=B, h_out=E, y=C, scales=None, rstd=None)
    p.update(pointers)
    a = norm_args(x_stride=104, y_stride=100) if pointers.get("y") == A + 2 else norm_args()
    assert lib.fsdp_rmsnorm(ctypes.byref(a), p["x"], p["residual"], p["gain"], p["h_out"], p["y"], p["scales"],
                            p["rstd"], None) == fs.FSDP_EALIAS


def bwd(over=None, pointers=None, ws_bytes=1 << 20):
    a = dict(rows=4, cols=100, dy_stride=100, h_stride=100, dh_stride=100, dx_stride=100, dtype=1, gain_dtype=1)
    a.update(over or {})
    p = dict(dy=A, h=B, gain=C, rstd=D, dh=None, dx=E, dgain=F, ws=G)
    p.update(pointers or {})
    return lib.fsdp_rmsnorm_backward(ctypes.byref(fs.RmsNormBackwardArgs(**a)), p["dy"], p["h"], p["gain"], p["rstd"],
                                     p["dh"], p["dx"], p["dgain"], p["ws"], ws_bytes, None)


def test_rmsnorm_backward_refuses():
    for over in (dict(cols=0), dict(rows=-2), dict(h_stride=5), dict(dx_stride=99), dict(dtype=2), dict(gain_dtype=3)):
        assert bwd(over) == fs.FSDP_EINVAL
    for k in ("dy", "h", "gain", "rstd", "dx", "dgain", "ws"):
        assert bwd(pointers={k: None}) == fs.FSDP_EINVAL
    assert bwd(pointers=dict(dgain=F + 1)) == fs.FSDP_EINVAL
    assert bwd(ws_bytes=fs.fsdp_rmsnorm_backward_workspace(4, 100) - 1) == fs.FSDP_EWORKSPACE
    for p in (dict(dx=B), dict(dx=A + 2), dict(dgain=C), dict(dgain=E + 10), dict(ws=A), dict(ws=E), dict(dx=D)):
        assert bwd(pointers=p) == fs.FSDP_EALIAS
    with pytest.raises(fs.FsdpError):
        fs.fsdp_rmsnorm_backward_workspace(4, 0)


def matrix(source=A, out=B, rows=10, cols=20, source_stride=20, out_stride=20, dtype=0):
    return fs.MatrixArgs(source, out, rows, cols, source_stride, out_stride, dtype)


def ns(matrices, hyper=None, ws=G, ws_bytes=1 << 24, n=None):
    array = (fs.MatrixArgs * max(1, len(matrices)))(*matrices)
    return lib.fsdp_newton_schulz(array, len(matrices) if n is None else n, fs._byref_or_none(hyper), ws, ws_bytes, None)


def test_newton_schulz_refuses():
    for bad in (dict(source=None), dict(out=None), dict(rows=-1), dict(cols=-1), dict(source_stride=19),
                dict(out_stride=3), dict(dtype=2), dict(source=A + 2), dict(out=B + 1), dict(rows=1 << 31)):
        assert ns([matrix(**bad)]) == fs.FSDP_EINVAL
    for h in (fs.NewtonSchulz(steps=0), fs.NewtonSchulz(steps=33), fs.NewtonSchulz(terms=2), fs.NewtonSchulz(eps=0.0),
              fs.NewtonSchulz(eps=math.nan), fs.NewtonSchulz(coefficients=(math.nan, 0, 0)),
              fs.NewtonSchulz(coefficients=(9.0, 0.0, 0.0)), fs.NewtonSchulz(coefficients=(3.0, -61.0, 60.0)),
              fs.NewtonSchulz(steps=3, coefficients=(2.0, 0.0, 0.0)), fs.NewtonSchulz(coefficients=(3.0, 3.0, 3.0))):
        assert ns([matrix()], h) == fs.FSDP_EINVAL
    assert ns([matrix()], n=-1) == fs.FSDP_EINVAL
    assert ns([matrix()], ws=None) == fs.FSDP_EINVAL
    assert ns([matrix()], ws_bytes=16) == fs.FSDP_EWORKSPACE
    for pair in ([matrix(out=A)], [matrix(out=A + 4)], [matrix(), matrix(source=C)], [matrix(), matrix(source=B, out=C)],
                 [matrix(), matrix(source=C, out=A + 100)]):
        assert ns(pair) == fs.FSDP_EALIAS
    assert ns([matrix()], ws=A) == fs.FSDP_EALIAS
    assert ns([matrix()], ws=B + 64) == fs.FSDP_EALIAS
    # nothing to do is no error, and launches nothing
    assert ns([]) == fs.FSDP_OK and ns([matrix(rows=0), matrix(cols=0)], ws=None, ws_bytes=0) == fs.FSDP_OK


def test_newton_schulz_accepts_usual_coefficients():
    array = (fs.MatrixArgs * 1)(matrix())
    n = ctypes.c_int64(0)
    for co in (None, (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (3.0, -3.2, 1.2)):
        h = fs.NewtonSchulz(steps=7, coefficients=co)
        assert lib.fsdp_newton_schulz_workspace(array, 1, ctypes.byref(h), ctypes.byref(n)) == fs.FSDP_OK
        assert n.value > 0
    with pytest.raises(ValueError):
        fs.NewtonSchulz(steps=3, coefficients=[(1.5, -0.5, 0.0)] * 2)


def muon_unit(tensors=((8, 6, 1.0), (4, 0, 0.0)), world=2, factor=None, **over):
    layout, _ = fs.fsdp_flatten_layout([52] + [0] * (len(tensors) - 1), world, factor)
    base = dict(grads=[A, B], master=[C, C + 4096], exp_avg=[D, D + 4096], exp_avg_sq=[E, E + 4096], full_out=F)
    base.update(over)
    return fs.MuonUnit(layout, [fs.MuonTensor(*t) for t in tensors], **base)


def muon_step(unit, muon=None, ws=G, ws_bytes=1 << 24):
    return lib.fsdp_muon_step(ctypes.byref(unit.args), ctypes.byref(muon or fs.Muon()), ws, ws_bytes, None)


def test_muon_refuses():
    for tensors in (((8, 6, 1.0), (5, 0, 0.0)), ((8, 6, 1.0), (3, 0, 0.0)), ((-8, -6, 1.0), (4, 0, 0.0)),
                    ((8, 6, math.nan), (4, 0, 0.0)), ((1 << 62, 1 << 62, 1.0), (4, 0, 0.0)), ((52, 0, 0.0), (1, 1, 1.0))):
        assert muon_step(muon_unit(tensors)) == fs.FSDP_EINVAL
    assert muon_step(muon_unit(factor=1)) == fs.FSDP_EINVAL
    for m in (fs.Muon(lr=math.nan), fs.Muon(weight_decay=math.inf), fs.Muon(momentum=1.0), fs.Muon(momentum=-0.1),
              fs.Muon(adam=fs.AdamHyper(step=0)), fs.Muon(newton_schulz=fs.NewtonSchulz(terms=5))):
        assert muon_step(muon_unit(), m) == fs.FSDP_EINVAL
    for over in (dict(grads=[A, None]), dict(master=[None, C]), dict(full_out=None), dict(grads=[A, B + 1]),
                 dict(exp_avg=[D + 2, D + 4096]), dict(full_out=F + 1)):
        assert muon_step(muon_unit(**over)) == fs.FSDP_EINVAL
    assert muon_step(muon_unit(), ws=None) == fs.FSDP_EINVAL
    assert muon_step(muon_unit(), ws_bytes=8) == fs.FSDP_EWORKSPACE
    for over in (dict(grads=[A, F]), dict(master=[C, C]), dict(full_out=E), dict(exp_avg=[C, D])):
        assert muon_step(muon_unit(**over)) == fs.FSDP_EALIAS
    for ws in (A, B, C, C + 4096, D, E, F):
        assert muon_step(muon_unit(), ws=ws) == fs.FSDP_EALIAS


def test_binding_refuses_wrong_counts():
    layout, _ = fs.fsdp_flatten_layout([48, 4], 2)
    args = dict(grads=[A, B], master=[C, C], exp_avg=[D, D], exp_avg_sq=[E, E], full_out=F)
    with pytest.raises(ValueError):
        fs.MuonUnit(layout, [fs.MuonTensor(8, 6)], **args)
    with pytest.raises(ValueError):
        fs.MuonUnit(layout, [fs.MuonTensor(8, 6), fs.MuonTensor(4)], **dict(args, master=[C]))
    with pytest.raises(ValueError):
        fs.NewtonSchulzBatch([1, 2], [1])
