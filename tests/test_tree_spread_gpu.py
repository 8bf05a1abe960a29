"""GPU tests of the attention over caches whose scales are spread over many
powers of two, with a bound that says something: key by key (kv_bounds)."""
import pytest
import torch

import kv_bounds
import kv_ref as R
import residual_add_rmsnorm_gb300 as rarn
from test_kv_gpu import rows_at
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


# new tokens, heads to a key head, D, format, type: blocks of 8 and 16 rows,
# tiles of 128 and 256
SIZES = [(2, 4, 128, "e4m3", "bf16"), (5, 3, 128, "e5m2", "f16"), (4, 3, 192, "e4m3", "bf16"),
         (3, 2, 96, "e4m3", "f16"), (2, 2, 256, "e5m2", "bf16"), (16, 4, 128, "e4m3", "bf16"),
         (20, 2, 64, "e5m2", "bf16"), (33, 4, 128, "e4m3", "bf16"), (40, 4, 64, "e4m3", "f16")]


@pytest.mark.parametrize("n,G,D,fmt,dt", SIZES)
@pytest.mark.parametrize("spread", ["values", "keys", "both", "steps"])
def test_spread_scales(n, G, D, fmt, dt, spread):
    ctx = 500
    c = Case([ctx], [n], 2 * G, 2, D, fmt=fmt, dt=dt, seed=60)
    L = ctx + n
    at = c.slots(0, L)
    page, slot = (at // 16).cuda(), (at % 16).cuda()
    g = torch.Generator().manual_seed(n + D)
    wide = torch.exp(2 * torch.randn(2, L, 2, generator=g)).cuda()
    if spread in ("values", "both"):
        c.cache.v_scale[page, :, slot] *= wide[0]
    if spread in ("keys", "both"):
        c.cache.k_scale[page, :, slot] *= wide[1].clamp_max(20.0)
    if spread == "steps":      # value scales that rise 2^6 every 128 keys, and fall again
        step = torch.tensor([0, 6, 12, 3], device="cuda")[torch.arange(L, device="cuda") // 128 % 4]
        c.cache.v_scale[page, :, slot] *= torch.exp2(step.float())[:, None]
    if dt == "f16":            # results that binary16 holds
        c.cache.v_scale *= 2.0 ** -12
    out = c.run()
    assert rarn.watchdog() == 0
    codes = [R.decode(rows_at(t, at, 16), fmt) for t in (c.cache.k, c.cache.v)]
    scales = [rows_at(t, at, 16).to(R.F64) for t in (c.cache.k_scale, c.cache.v_scale)]
    want, tol, mag = kv_bounds.attention(c.q, codes[0], scales[0], codes[1], scales[1],
                                         c.visible(0), D ** -0.5)
    # a case whose bound lets anything pass is no test
    assert (tol / mag).median() <= 2.0 ** -6
    assert ((tol / mag) <= 2.0 ** -4).double().mean() >= 0.9
    R.check_attention(out.cpu(), want, tol)
    assert torch.equal(c.run(out=torch.zeros_like(out)), out)
