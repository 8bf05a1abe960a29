"""Host-side checks of the rotation by positions of several axes, and the order
of its sections.  CPU only: the addresses are fake."""
import ctypes

import pytest

import residual_add_rmsnorm_gb300 as rarn
from residual_add_rmsnorm_gb300 import build as rbuild
from test_kv_host import ALIAS, C, CUDA, INVALID, OK, UNSUPPORTED, at


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rarn.library()


def rotation(axes=3, stride=8, pairs=(0,) * 10 + (1,) * 11 + (2,) * 11, **kw):
    d = dict(cos_sin=at(10), positions=at(11), table_rows=100, rot_dim=64, style=0)
    d.update(kw)
    r = rarn.Rotation(d["cos_sin"], d["positions"], d["table_rows"], d["rot_dim"], d["style"])
    m = None if pairs is None else (ctypes.c_uint8 * len(pairs))(*pairs)
    x = rarn.RotationAxes(r, axes, stride, None if m is None else ctypes.addressof(m))
    x.keep = m
    return x


def rope(lib, rot, **kw):
    d = dict(q_out=C.heads(0, C.Hq), T=C.T)
    d.update(kw)
    return lib.rarn_qk_norm_rope_axes(d["q_out"], C.heads(1, C.Hk), C.heads(2, C.Hq),
                                      C.heads(3, C.Hk), at(4), at(5),
                                      None if rot is None else ctypes.byref(rot), d["T"], C.D,
                                      C.eps, None)


def fused(lib, rot, **kw):
    return lib.rarn_qk_norm_rope_axes_kv_write(
        C.heads(0, C.Hq), C.cache(**kw), C.heads(2, C.Hq), C.heads(3, C.Hk), C.heads(6, C.Hk),
        at(4), at(5), None if rot is None else ctypes.byref(rot), at(7), C.T, C.eps, None)


@pytest.mark.parametrize("call", [rope, fused])
@pytest.mark.parametrize("kw,want", [
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(stride=-1), INVALID),
    (dict(stride=1 << 40), UNSUPPORTED), (dict(pairs=None), INVALID),
    (dict(axes=2), INVALID), (dict(pairs=(0,) * 31 + (3,)), INVALID),
    (dict(rot_dim=63), INVALID), (dict(positions=None), INVALID), (dict(style=2), INVALID),
    (dict(table_rows=0), INVALID), (dict(positions=at(11) + 4), INVALID),
])
def test_refusals(lib, call, kw, want):
    assert call(lib, rotation(**kw)) == want


@pytest.mark.parametrize("call", [rope, fused])
def test_no_rotation_is_refused(lib, call):
    assert call(lib, None) == INVALID


def test_every_axis_counts_for_overlaps(lib):
    # q_out begins inside the third axis's positions
    r = rotation(stride=1 << 20)
    bad = C.heads(0, C.Hq, data=at(11) + 2 * (8 << 20))
    assert rope(lib, r, q_out=bad) == ALIAS


def test_sound_calls_pass_the_checks(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a device")
    for r in (rotation(), rotation(axes=1, pairs=(0,) * 32), rotation(stride=0),
              rotation(axes=4, pairs=(3, 2, 1, 0) * 8)):
        assert rope(lib, r) == CUDA
        assert fused(lib, r) == CUDA
    assert rope(lib, rotation(positions=None), T=0) == OK


@pytest.mark.parametrize("sections,order,want", [
    ((1, 2, 3), "blocks", [0, 1, 1, 2, 2, 2]), ((2, 2, 2), "cyclic", [0, 1, 2, 0, 1, 2]),
    ((4, 1, 2), "cyclic", [0, 1, 2, 0, 2, 0, 0]), ((0, 3), "cyclic", [1, 1, 1]),
    ((24, 20, 20), "cyclic", [0, 1, 2] * 20 + [0] * 4),
])
def test_the_order_of_sections(sections, order, want):
    assert list(rarn._axis_map(sum(sections), sections, order)) == want
