"""Host-side checks of rarn_verify_drafts: argument errors come before anything touches
a GPU.  CPU only: the addresses are fake."""
import ctypes

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
import step_ref as R
from residual_add_rmsnorm_gb300 import build as rbuild

OK, INVALID, UNSUPPORTED, ALIAS, CUDA = 0, 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 2
N, B, V, MOST = 12, 3, 100, 4


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rarn.library()


def at(i):
    """The i-th fake allocation, 16 TiB apart."""
    return (i + 1) << 44


def rows(i, stride=V, dt=F32):
    return rarn.Rows(at(i), stride, dt)


def call(lib, **kw):
    d = dict(new=at(0), path=at(1), lengths=at(2), p=rows(3), q=rows(4), tokens=at(5), parents=None,
             starts=at(7), u=at(8), v=at(9), B=B, N=N, V=V, most=MOST)
    d.update(kw)
    q = None if d["q"] is None else ctypes.byref(d["q"])
    return lib.rarn_verify_drafts(d["new"], d["path"], d["lengths"], d["p"], q, d["tokens"],
                                  d["parents"], d["starts"], d["u"], d["v"], d["B"], d["N"],
                                  d["V"], d["most"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(most=-1), INVALID),
    (dict(V=(1 << 20) + 1), UNSUPPORTED), (dict(most=1 << 24), UNSUPPORTED),
    (dict(N=1 << 31), UNSUPPORTED), (dict(B=(1 << 20) + 1), UNSUPPORTED),
    (dict(p=rows(3, dt=5)), INVALID), (dict(p=rows(3, dt=BF16)), UNSUPPORTED),
    (dict(parents=at(6)), UNSUPPORTED), (dict(p=rows(3, stride=V - 1)), INVALID),
    (dict(q=rows(4, stride=-V)), INVALID), (dict(p=rows(3, stride=1 << 40)), UNSUPPORTED),
    (dict(p=rarn.Rows(None, V, F32)), INVALID), (dict(q=rarn.Rows(at(4) + 2, V, F32)), INVALID),
    (dict(new=None), INVALID), (dict(path=None), INVALID), (dict(lengths=None), INVALID),
    (dict(tokens=None), INVALID), (dict(starts=None), INVALID), (dict(u=None), INVALID),
    (dict(v=None), INVALID), (dict(new=at(0) + 4), INVALID), (dict(tokens=at(5) + 4), INVALID),
    (dict(u=at(8) + 2), INVALID), (dict(q=None, parents=at(6) + 2), INVALID),
    (dict(path=at(0) + 8), ALIAS), (dict(lengths=at(1) + 4), ALIAS), (dict(new=at(3)), ALIAS),
    (dict(path=at(4) + 400), ALIAS), (dict(lengths=at(7) + 4), ALIAS), (dict(new=at(5)), ALIAS),
    (dict(q=None, parents=at(1)), ALIAS), (dict(lengths=at(9)), ALIAS), (dict(path=at(8)), ALIAS),
    (dict(B=0), OK),
])
def test_refusals(lib, kw, want):
    assert call(lib, **kw) == want


def test_sound_calls_pass_the_checks(lib):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a device")
    for kw in (dict(), dict(q=None), dict(q=None, parents=at(6)), dict(most=0),
               dict(N=0, p=rarn.Rows(None, V, F32), q=None, tokens=None, u=None),
               dict(N=1, p=rows(3, 0), q=rows(4, 0)), dict(p=rows(3, dt=F16), q=rows(4, dt=F16))):
        assert call(lib, **kw) == CUDA


def test_the_binding_refuses():
    x = torch.zeros(3, 4)
    i = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        rarn.verify_drafts(x, i, i, x[0], x[0], 2)
    with pytest.raises(ValueError):
        rarn.verify_drafts(x[0], i, i, x[0], x[0], 2)


def test_the_definition_on_worked_examples():
    """Hand-worked: p = (1/2, 1/4, 1/4)."""
    p = torch.tensor([[0.5, 0.25, 0.25]] * 3)
    u, v = torch.tensor([0.6, 0.3, 0.0]), torch.tensor([0.5])
    # 0.6 >= 1/2: token 0 is refused; what is left is (0, 1/4, 1/4), half of it reached at 2
    assert R.verify(p, [0, 0, 0], [0, 3], u, v, 2) == ([[2, -1, -1]], [[0, -1, -1]], [1])
    # drawn from q = (1, 0, 0): 0.6 * 1 < 1/2 fails; max(p - q, 0) = (0, 1/4, 1/4)
    q = torch.tensor([[1.0, 0.0, 0.0]] * 3)
    assert R.verify(p, [0, 0, 0], [0, 3], u, v, 2, q) == ([[2, -1, -1]], [[0, -1, -1]], [1])
    # a tree: token 0 takes 0 .. 1/2, token 2 takes 1/2 .. 3/4; below it 0.0 accepts nothing
    # (no children), so p itself is drawn at row 2
    assert R.verify(p, [0, 0, 2], [0, 3], u, v, 2, None, [-1, 0, 0]) == \
        ([[2, 1, -1]], [[0, 2, -1]], [2])
