"""What the rotation takes as positions: tensors of the call's device and nothing else, an
address least of all.  CPU only: the launch is replaced, nothing reaches a GPU."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn

T, HQ, HK, D = 1, 4, 2, 32


class Here(torch.Tensor):
    """A tensor on the device that the binding asks for."""

    def get_device(self):
        return self.device.index


def here(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Here)


@pytest.fixture
def launches(monkeypatch):
    got = []
    monkeypatch.setattr(rarn, "_on", lambda *a: got.append(a))
    return got


class Cache:
    device, heads, head_dim, _ref = torch.device("cpu"), HK, D, None


def rope(positions, **kw):
    rarn.qk_norm_rope(here(T, HQ, D), here(T, HK, D), here(D), here(D), 1e-6, here(100, D),
                      positions, q_out=here(T, HQ, D), k_out=here(T, HK, D), **kw)


def write(positions, **kw):
    rarn.qk_norm_rope_kv_write(here(T, HQ, D), here(T, HK, D), here(T, HK, D), here(D), here(D),
                               1e-6, here(100, D), positions, Cache, here(T, dtype=torch.int64),
                               q_out=here(T, HQ, D), **kw)


@pytest.mark.parametrize("call", [rope, write])
def test_a_tensor_is_taken(call, launches):
    call(here(T, dtype=torch.int64))
    call(here(2, T, dtype=torch.int64), sections=(8, 8))
    assert len(launches) == 2


@pytest.mark.parametrize("call", [rope, write])
@pytest.mark.parametrize("sections", [None, (8, 8)])
@pytest.mark.parametrize("positions", [16, 4096, 0, True, 16.0, [16], None])
def test_nothing_else_is(call, sections, positions, launches):
    with pytest.raises((TypeError, ValueError)):
        call(positions, sections=sections)
    assert not launches


@pytest.mark.parametrize("call", [rope, write])
def test_nor_a_tensor_of_another_kind(call, launches):
    for positions in (here(T, dtype=torch.int32), here(T + 1, dtype=torch.int64)):
        with pytest.raises((TypeError, ValueError)):
            call(positions)
    assert not launches
