"""GPU tests of the codes that the 8-bit cache gets with a scale per row, bit for bit on the
values (which nothing is done to before): (x * (1 / max|x|)) * largest code, in binary32, and
the same whether written alone, with one position or with positions of several axes."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn

pytestmark = pytest.mark.gpu

CODE = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


@pytest.mark.parametrize("T,D", [(1, 128), (128, 128), (517, 96), (33, 80)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_values_codes(T, D, dt, fmt):
    g = torch.Generator().manual_seed(T)
    Hq, H, page = 4, 3, 16
    q, k, v = (torch.randn(T, n, D, generator=g).to(dt).cuda() for n in (Hq, H, H))
    gamma = torch.ones(D, dtype=dt, device="cuda")
    angle = torch.rand(100, D // 2, generator=g)
    table = torch.cat([angle.cos(), angle.sin()], 1).cuda()
    at = torch.arange(T, device="cuda") % 100
    slots = torch.randperm(T, generator=g).cuda()
    caches = [rarn.KVCache.empty(T // page + 1, page, H, D, fmt) for _ in range(3)]
    rarn.kv_cache_write(k, v, caches[0], slots)
    rarn.qk_norm_rope_kv_write(q, k, v, gamma, gamma, 1e-6, table, at, caches[1], slots)
    rarn.qk_norm_rope_kv_write(q, k, v, gamma, gamma, 1e-6, table, torch.stack([at, at]),
                               caches[2], slots, sections=(D // 4, D // 4),
                               section_order="cyclic")
    code, top = CODE[fmt]
    x = v.float().cpu()     # where torch's division by a number is one
    most = x.abs().amax(-1, keepdim=True)
    want = ((x * (1 / most)) * top).clamp(-top, top).to(code).view(torch.uint8)
    for c in caches:
        got = c.v[slots // page, :, slots % page].cpu()
        assert torch.equal(got, want)
        got = c.v_scale[slots // page, :, slots % page].cpu()
        assert torch.equal(got, (most / top)[..., 0])
    # one position on every axis is one position
    assert torch.equal(caches[1].k, caches[2].k)
    assert torch.equal(caches[1].k_scale, caches[2].k_scale)
