"""Host-side checks of rarn_kv_step, rarn_kv_trim and rarn_kv_cache_compact: argument
errors come before anything touches a GPU.  CPU only: the addresses are fake."""
import ctypes

import pytest

import residual_add_rmsnorm_gb300 as rarn
import step_ref as R
from residual_add_rmsnorm_gb300 import build as rbuild
from test_kv_host import ALIAS, C, CUDA, INVALID, OK, UNSUPPORTED, at


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rarn.library()


def pages(**kw):
    d = dict(page_table=at(0), table_stride=10, table_width=10, held=at(1), free_pages=at(2),
             free_count=at(3), ticket=at(4), sequences=6, num_pages=60, page_size=16)
    d.update(kw)
    return ctypes.byref(rarn.KvPagesDesc(*[d[f] for f, _ in rarn.KvPagesDesc._fields_]))


def step(lib, p=None, **kw):
    d = dict(ctx=at(5), new=at(6), starts=at(7), slots=at(8), positions=at(9), served=at(10),
             tokens=100)
    d.update(kw)
    return lib.rarn_kv_step(p or pages(), d["ctx"], d["new"], d["starts"], d["slots"],
                            d["positions"], d["served"], d["tokens"], None)


def trim(lib, p=None, lens=at(5)):
    return lib.rarn_kv_trim(p or pages(), lens, None)


def compact(lib, **kw):
    d = dict(cache=C.cache(), table=at(0), stride=4, width=4, ctx=at(5), path=at(6), lengths=at(7),
             B=3, W=8)
    d.update(kw)
    return lib.rarn_kv_cache_compact(d["cache"], d["table"], d["stride"], d["width"], d["ctx"],
                                     d["path"], d["lengths"], d["B"], d["W"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(page_table=None), INVALID), (dict(held=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(free_count=None), INVALID), (dict(ticket=None), INVALID), (dict(held=at(1) + 2), INVALID),
    (dict(table_stride=9), INVALID), (dict(table_width=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(sequences=-1), INVALID), (dict(table_stride=-10), INVALID),
    (dict(sequences=8193), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED),
    (dict(page_size=(1 << 20) + 1), UNSUPPORTED), (dict(table_stride=1 << 40), UNSUPPORTED),
    (dict(table_width=1 << 28, table_stride=1 << 28), UNSUPPORTED),
    (dict(held=at(0)), ALIAS), (dict(free_pages=at(0) + 16), ALIAS), (dict(ticket=at(3)), ALIAS),
])
def test_pages_are_checked(lib, kw, want):
    assert step(lib, pages(**kw)) == want
    assert trim(lib, pages(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), UNSUPPORTED), (dict(ctx=None), INVALID),
    (dict(new=at(6) + 1), INVALID), (dict(starts=None), INVALID), (dict(served=None), INVALID),
    (dict(slots=None), INVALID), (dict(positions=at(9) + 4), INVALID),
    (dict(slots=at(9)), ALIAS), (dict(starts=at(5)), ALIAS), (dict(new=at(2)), ALIAS),
    (dict(served=at(7) + 24), ALIAS), (dict(ctx=at(0) + 4), ALIAS),
])
def test_step_refuses(lib, kw, want):
    assert step(lib, **kw) == want


def test_trim_refuses(lib):
    assert trim(lib, None, None) == INVALID
    assert trim(lib, None, at(5) + 1) == INVALID
    assert trim(lib, None, at(1)) == ALIAS
    assert lib.rarn_kv_trim(None, at(5), None) == INVALID
    assert trim(lib, pages(sequences=0)) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(cache=None), INVALID), (dict(B=-1), INVALID), (dict(W=-1), INVALID),
    (dict(W=(1 << 24) + 1), UNSUPPORTED), (dict(ctx=None), INVALID), (dict(path=None), INVALID),
    (dict(lengths=at(7) + 2), INVALID), (dict(table=None), INVALID),
    (dict(stride=1 << 40), UNSUPPORTED), (dict(cache=C.cache(head_dim=40)), UNSUPPORTED),
    (dict(path=at(12)), ALIAS), (dict(table=at(13)), ALIAS), (dict(lengths=at(14)), ALIAS),
    (dict(cache=C.cache(v=at(12))), ALIAS), (dict(B=0), OK), (dict(W=1), OK), (dict(W=0), OK),
])
def test_compact_refuses(lib, kw, want):
    assert compact(lib, **kw) == want


def test_sound_calls_pass_the_checks(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a device")
    for p in (pages(), pages(sequences=8192), pages(sequences=1, table_stride=0)):
        assert step(lib, p) == CUDA and trim(lib, p) == CUDA
    assert step(lib, tokens=0, slots=None, positions=None) == CUDA
    for kw in (dict(), dict(cache=C.cache(scale_mode=0)), dict(B=1, stride=0)):
        assert compact(lib, **kw) == CUDA


def test_the_model_gives_back_what_it_took():
    m = R.Pages(2, 4, 6, 4)
    before = list(m.free)
    assert m.step([0, 0], [5, 9], 20) == ([0, 5, 14], [0, 1, 2, 3, 4, 8, 9, 10, 11, 12, 13, 14, 15,
                                                       16] + [-1] * 6,
                                          [*range(5), *range(9)] + [0] * 6, 2, False)
    assert m.table() == [[0, 1, -1, -1], [2, 3, 4, -1]]
    m.trim([0, 0])
    assert m.free == before
