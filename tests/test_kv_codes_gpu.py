"""GPU tests of the codes that the 8-bit cache gets with one scale for all,
bit for bit: the binary32 quotient x / scale, rounded once more to nearest
even."""
import pytest
import torch

import kv_ref as R
import residual_add_rmsnorm_gb300 as rarn
from test_kv_gpu import DT, make_cache, rows_at

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def want_codes(x, scale, fmt):
    u = (x.float() / torch.tensor(scale)).clamp(-R.MAXF[fmt], R.MAXF[fmt])
    return u.to(R.CODE[fmt]).view(torch.uint8)


@pytest.mark.parametrize("scale", [1.0, 7.0, 3.0, 0.1, 448.0, 2.0 ** -126, 2.0 ** -130, 1e-41,
                                   3e38])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f16", 64), ("f32", 64), ("bf16", 48)])
def test_every_quotient(dt, D, fmt, scale):
    """All finite values of a 16-bit type (as many binary32 ones around them),
    ties and zeros among them, by the vector kernel and by the one that goes
    element by element."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.float16 if dt == "f16" else torch.bfloat16).float()
    x = x[torch.isfinite(x)]
    if dt == "f32":
        x = torch.cat([x, x * (1 + 2.0 ** -9), x * 1.7])
        x = x[torch.isfinite(x)]
    T = len(x) // D
    x = x[:T * D].view(T, 1, D).to(DT[dt])
    v = x.flip(0)
    page = 16
    cache = make_cache(T // page + 1, page, 1, D, fmt, "tensor", "heads")
    cache.k_scale.fill_(scale)
    cache.v_scale.fill_(scale)
    slots = torch.arange(T)
    pad = 0 if D == 64 else 1                     # rows off their 16-byte boundaries
    wide = torch.zeros(T, 2, D + pad, dtype=DT[dt], device="cuda")
    wide[:, :1, :D], wide[:, 1:, :D] = x.cuda(), v.cuda()
    rarn.kv_cache_write(wide[:, :1, :D], wide[:, 1:, :D], cache, slots.cuda())
    for codes, src in ((cache.k, x), (cache.v, v)):
        assert torch.equal(rows_at(codes, slots, page), want_codes(src, scale, fmt))
    assert rarn.watchdog() == 0
