"""Host-side checks of rarn_gated_add_rms_norm: argument errors come before
anything touches a GPU.  CPU only: the addresses are fake."""
import ctypes

import pytest

import residual_add_rmsnorm_gb300 as rarn
from residual_add_rmsnorm_gb300 import build as rbuild

OK, INVALID, UNSUPPORTED, ALIAS, CUDA = 0, 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 2
T, H = 8, 64


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rarn.library()


def at(i):
    """The i-th fake allocation, 16 TiB apart."""
    return (i + 1) << 44


def rows(i, stride=H, dt=BF16):
    return rarn.Rows(at(i), stride, dt)


def gate(data=at(6), stride=H, n=T, index=None):
    return ctypes.byref(rarn.Gate(data, stride, n, index))


def call(lib, **kw):
    d = dict(y=rows(0), h=rows(1), x=rows(2), r=rows(3), xg=at(4), g=at(5), gate=gate(), scale=1.0,
             rscale=1.0, T=T, H=H, eps=1e-6)
    d.update(kw)
    return lib.rarn_gated_add_rms_norm(d["y"], d["h"], d["x"], d["r"], d["xg"], d["g"], d["gate"],
                                       d["scale"], d["rscale"], d["T"], d["H"], d["eps"], None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=(1 << 24) + 1), UNSUPPORTED),
    (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID),
    (dict(scale=INF), INVALID), (dict(scale=NAN), INVALID), (dict(rscale=-INF), INVALID),
    (dict(g=None), INVALID), (dict(g=at(5) + 1), INVALID), (dict(xg=at(4) + 1), INVALID),
    (dict(y=rows(0, dt=7)), INVALID), (dict(y=rows(0, dt=F16)), UNSUPPORTED),
    (dict(r=rows(3, dt=F16), h=rows(1, dt=F16)), UNSUPPORTED),
    (dict(r=rows(3, dt=F32)), UNSUPPORTED), (dict(x=rows(2, stride=H - 1)), INVALID),
    (dict(x=rows(2, stride=1 << 40)), UNSUPPORTED), (dict(x=rarn.Rows(None, H, BF16)), INVALID),
    (dict(x=rarn.Rows(at(2) + 1, H, BF16)), INVALID),
    (dict(gate=gate(n=3)), INVALID), (dict(gate=gate(n=0)), INVALID),
    (dict(gate=gate(data=None)), INVALID), (dict(gate=gate(stride=3)), INVALID),
    (dict(gate=gate(n=3, index=at(7) + 2)), INVALID),
    # overlaps: outputs with each other, with inputs they may not be, in part
    (dict(y=rows(1)), ALIAS), (dict(y=rows(3)), ALIAS), (dict(h=rows(2)), ALIAS),
    (dict(h=rarn.Rows(at(3) + 2, H, BF16)), ALIAS), (dict(y=rarn.Rows(at(2) + 2, H, BF16)), ALIAS),
    (dict(x=rows(2, H), y=rows(2, H + 8)), ALIAS), (dict(g=at(0) + 16), ALIAS),
    (dict(xg=at(1) + 16), ALIAS), (dict(gate=gate(data=at(0))), ALIAS),
    (dict(gate=gate(n=3, index=at(1))), ALIAS),
])
def test_refusals(lib, kw, want):
    assert call(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(), dict(gate=None), dict(xg=None), dict(y=rows(2)), dict(h=rows(3)),
    dict(gate=gate(n=1, stride=0)), dict(gate=gate(n=5, index=at(7))),
    dict(r=rows(3, dt=F32), h=rows(1, dt=F32)),
    dict(T=1, x=rows(2, stride=0), gate=gate(n=1)), dict(eps=0.0),
])
def test_sound_calls_pass_the_checks(lib, kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a device")
    assert call(lib, **kw) == CUDA


def test_no_rows_is_a_no_op(lib):
    assert call(lib, T=0, x=rarn.Rows(None, H, BF16), gate=gate(n=1)) == OK


def test_the_binding_refuses():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        rarn.gated_add_rms_norm(x, x, x[0], x[0], 1e-6)
    with pytest.raises(ValueError):
        rarn.gated_add_rms_norm(x[0], x, x[0], x[0], 1e-6)
    for kw in (dict(gate=x), dict(out=x), dict(residual_out=x)):
        with pytest.raises((TypeError, ValueError)):
            rarn.gated_add_rms_norm(x, x, x[0], x[0], 1e-6, **kw)
