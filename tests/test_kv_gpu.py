"""GPU tests of the per-head norm and rotation and of the 8-bit cache's write
and read, against binary64 (kv_ref)."""
import pytest
import torch

import kv_ref as R
import residual_add_rmsnorm_gb300 as rarn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
INDEX_BIT = 16


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def gen(seed):
    return torch.Generator().manual_seed(seed)


def table_of(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=R.F64) / rot)
    a = torch.arange(rows, dtype=R.F64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def packed(T, Hq, Hk, D, dt, g, pad=0):
    """q, k, v as slices of one [T, heads, D + pad] projection, on the host."""
    x = torch.randn(T, Hq + 2 * Hk, D + pad, generator=g)
    x = (x * torch.exp(torch.randn(T, 1, 1, generator=g))).to(dt)
    return x


def split(x, Hq, Hk, D):
    x = x[..., :D]
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


# T, Hq, Hk, D, rot, pad: vector and element-wise kernels, groups of every size,
# lanes left over, one token, odd everything
ROPE = [
    (1, 32, 8, 128, 128, 0), (3, 5, 5, 64, 32, 0), (17, 40, 8, 96, 64, 0), (33, 7, 1, 192, 192, 8),
    (5, 3, 2, 256, 64, 0), (2, 2, 1, 512, 512, 0), (9, 3, 3, 80, 16, 0), (1000, 16, 4, 128, 128, 0),
    (4, 3, 1, 20, 10, 0), (6, 2, 2, 1, 0, 0), (7, 2, 1, 129, 128, 3), (3, 2, 2, 1000, 6, 0),
    (11, 4, 2, 128, 64, 1), (2, 1, 1, 2, 2, 0), (300, 64, 8, 128, 0, 0),
]


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,pad", ROPE)
def test_norm_rope(T, Hq, Hk, D, rot, pad, dt, style):
    g = gen(T + 31 * D + rot)
    x = packed(T, Hq, Hk, D, DT[dt], g, pad)
    qg, kg = ((torch.rand(D, generator=g) + 0.5).to(DT[dt]) for _ in range(2))
    table = table_of(5000, rot) if rot else None
    pos = torch.randint(0, 5000, (T,), generator=g) if rot else None
    q, k, _ = split(x, Hq, Hk, D)
    dq, dk, _ = split(x.cuda(), Hq, Hk, D)
    got = rarn.qk_norm_rope(dq, dk, qg.cuda(), kg.cuda(), EPS,
                            None if table is None else table.cuda(),
                            None if pos is None else pos.cuda(), style=style)
    torch.cuda.synchronize()
    for n, y, src, gamma in (("q", got[0], q, qg), ("k", got[1], k, kg)):
        want, mag = R.rotate(R.norm(src, gamma, EPS), table, pos, style)
        R.check_rows(y.cpu(), want, mag, n)
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("D", [128, 36])
@pytest.mark.parametrize("which", ["q", "k", "none"])
def test_a_missing_gamma_leaves_its_norm_out(which, D):
    g = gen(D)
    q, k = (torch.randn(5, 3, D, generator=g).to(torch.bfloat16) for _ in range(2))
    gamma = (torch.rand(D, generator=g) + 0.5).to(torch.bfloat16)
    table, pos = table_of(64, 32), torch.arange(5)
    qg, kg = (gamma if which == n else None for n in "qk")
    out = rarn.qk_norm_rope(q.cuda(), k.cuda(), None if qg is None else qg.cuda(),
                            None if kg is None else kg.cuda(), EPS, table.cuda(), pos.cuda())
    for y, x, gm in ((out[0], q, qg), (out[1], k, kg)):
        want, mag = R.rotate(R.norm(x, gm, EPS), table, pos, "half")
        R.check_rows(y.cpu(), want, mag)


@pytest.mark.parametrize("D,pad", [(128, 0), (72, 1)])
def test_in_place_in_the_packed_projection(D, pad):
    T, Hq, Hk = 21, 6, 2
    g = gen(4)
    x = packed(T, Hq, Hk, D, torch.bfloat16, g, pad)
    gamma = torch.ones(D, dtype=torch.bfloat16)
    table, pos = table_of(100, 64), torch.arange(T) * 3
    d = x.cuda()
    dq, dk, _ = split(d, Hq, Hk, D)
    apart = rarn.qk_norm_rope(dq, dk, gamma.cuda(), gamma.cuda(), EPS, table.cuda(), pos.cuda())
    rarn.qk_norm_rope(dq, dk, gamma.cuda(), gamma.cuda(), EPS, table.cuda(), pos.cuda(),
                      q_out=dq, k_out=dk)
    assert torch.equal(dq, apart[0]) and torch.equal(dk, apart[1])
    # the values and the padding stay as they were
    rest = d.cpu()
    assert torch.equal(rest[:, Hq + Hk:], x[:, Hq + Hk:])
    assert torch.equal(rest[..., D:], x[..., D:])


def test_head_major_matrices():
    T, H, D = 19, 4, 64
    g = gen(9)
    q, k = (torch.randn(H, T, D, generator=g).to(torch.float16) for _ in range(2))
    gamma = torch.ones(D, dtype=torch.float16)
    table, pos = table_of(100, D), torch.arange(T)
    out = torch.empty(H, T, D, dtype=torch.float16, device="cuda")
    rarn.qk_norm_rope(q.cuda().transpose(0, 1), k.cuda().transpose(0, 1), gamma.cuda(),
                      gamma.cuda(), EPS, table.cuda(), pos.cuda(), q_out=out.transpose(0, 1))
    want, mag = R.rotate(R.norm(q.transpose(0, 1), gamma, EPS), table, pos, "half")
    R.check_rows(out.cpu().transpose(0, 1), want, mag)


@pytest.mark.parametrize("D", [128, 20])
def test_positions_outside_the_table(D):
    T, H = 6, 3
    q = torch.randn(T, H, D, generator=gen(1)).to(torch.bfloat16).cuda()
    gamma = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([0, -1, 15, 16, 1 << 40, 3], device="cuda")
    qo, ko = (torch.full_like(q, -7.0) for _ in range(2))
    rarn.qk_norm_rope(q, q, gamma, gamma, EPS, table_of(16, 16).cuda(), pos, q_out=qo, k_out=ko)
    assert rarn.watchdog() == INDEX_BIT
    for o in (qo, ko):
        assert (o[[1, 3, 4]] == -7.0).all() and not (o[[0, 2, 5]] == -7.0).all(-1).any()


def test_special_rows():
    """Zero rows stay zero, NaN and infinities stay in their own head."""
    q = torch.randn(4, 2, 128, generator=gen(2))
    q[1, 0] = 0.0
    q[2, 1, 5] = float("nan")
    q[3, 0, 7] = float("inf")
    q = q.to(torch.bfloat16)
    gamma = torch.ones(128, dtype=torch.bfloat16)
    out, _ = rarn.qk_norm_rope(q.cuda(), q.cuda(), gamma.cuda(), gamma.cuda(), EPS)
    out = out.cpu()
    assert (out[1, 0] == 0).all() and torch.isnan(out[2, 1]).all()
    assert torch.isnan(out[3, 0, 7]) and (out[3, 0, :7] == 0).all()
    keep = torch.ones(4, 2, dtype=torch.bool)
    keep[2, 1] = keep[3, 0] = False
    want = R.norm(q, gamma, EPS)
    R.check_rows(out[keep], want[keep], want[keep].abs())


# --------------------------------------------------------------------------
# the cache
# --------------------------------------------------------------------------

def make_cache(pages, page, H, D, fmt, mode, layout, fill=0x35):
    """A cache in one of three layouts, its codes and scales filled."""
    if layout == "heads":      # [pages, heads, page, D], keys and values apart
        k, v = (torch.full((pages, H, page, D), fill, dtype=torch.uint8, device="cuda")
                for _ in range(2))
    elif layout == "tokens":   # [pages, page, heads, D]
        k, v = (torch.full((pages, page, H, D), fill, dtype=torch.uint8,
                           device="cuda").transpose(1, 2) for _ in range(2))
    else:                      # one pool, keys and values by pages, rows padded
        pool = torch.full((pages, 2, H, page, D + 16), fill, dtype=torch.uint8, device="cuda")
        k, v = pool[:, 0, :, :, :D], pool[:, 1, :, :, :D]
    if mode == "row":
        if layout == "tokens":
            ks, vs = (torch.full((pages, page, H), 3.0, device="cuda").transpose(1, 2)
                      for _ in range(2))
        elif layout == "pool":
            both = torch.full((pages, 2, H, page), 3.0, device="cuda")
            ks, vs = both[:, 0], both[:, 1]
        else:
            ks, vs = (torch.full((pages, H, page), 3.0, device="cuda") for _ in range(2))
    else:
        ks = torch.full((1,), 4.0 / R.MAXF[fmt], device="cuda")
        vs = torch.full((1,), 0.25, device="cuda")
    return rarn.KVCache(k, v, ks, vs, fmt, mode)


def rows_at(t, slots, page):
    """[pages, heads, page, ...] -> [len(slots), heads, ...] on the host."""
    return t.cpu().transpose(1, 2)[slots // page, slots % page]


WRITE = [  # T, H, D, page, layout
    (1, 8, 128, 16, "heads"), (37, 2, 64, 16, "tokens"), (50, 3, 96, 24, "pool"),
    (300, 4, 192, 1, "heads"), (65, 1, 256, 64, "pool"), (20, 5, 16, 8, "tokens"),
    (9, 2, 48, 3, "heads"), (6, 2, 80, 7, "pool"),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,mode", [("e4m3", "row"), ("e5m2", "row"), ("e4m3", "tensor"),
                                      ("e5m2", "tensor")])
@pytest.mark.parametrize("T,H,D,page,layout", WRITE)
def test_cache_write(T, H, D, page, layout, fmt, mode, dt):
    g = gen(T * D)
    pages = T // page + 3
    cache = make_cache(pages, page, H, D, fmt, mode, layout)
    x = packed(T, 0, H, D, DT[dt], g, 8 if T % 2 else 0)
    x[T // 2, 0] = 0.0                                  # a key row of zeros
    k, v = x[:, :H, :D], x[:, H:, :D]
    slots = torch.randperm(pages * page, generator=g)[:T]
    skip = torch.rand(T, generator=g) < 0.2
    slots = torch.where(skip, torch.tensor(-1), slots)
    d = x.cuda()
    rarn.kv_cache_write(d[:, :H, :D], d[:, H:, :D], cache, slots.cuda())
    torch.cuda.synchronize()
    at = slots[~skip]
    for n, codes, scale, src in (("k", cache.k, cache.k_scale, k),
                                 ("v", cache.v, cache.v_scale, v)):
        want = src[~skip].to(R.F64)
        s = rows_at(scale, at, page) if mode == "row" else scale.cpu()
        R.check_codes(rows_at(codes, at, page), s, want, want.abs(), fmt, mode, n)
        # every other slot as it was
        rest = torch.ones(pages * page, dtype=torch.bool)
        rest[at] = False
        rest = rest.nonzero()[:, 0]
        assert (rows_at(codes, rest, page) == 0x35).all()
        if mode == "row":
            assert (rows_at(scale, rest, page) == 3.0).all()
    if layout == "pool":
        assert (cache.k._base.cpu()[..., D:] == 0x35).all()
    assert rarn.watchdog() == 0


def test_slots_past_the_cache():
    cache = make_cache(2, 4, 1, 64, "e4m3", "row", "heads")
    k = torch.randn(4, 1, 64, generator=gen(3)).cuda()
    rarn.kv_cache_write(k, k, cache, torch.tensor([8, 1, 1 << 50, -5], device="cuda"))
    assert rarn.watchdog() == INDEX_BIT
    assert (rows_at(cache.k, torch.tensor([0, 2, 3, 4, 5, 6, 7]), 4) == 0x35).all()
    assert not (rows_at(cache.k, torch.tensor([1]), 4) == 0x35).all()


def test_extreme_rows():
    """Tiny, huge and subnormal magnitudes keep a finite scale and full codes."""
    g = gen(8)
    x = torch.randn(5, 1, 64, generator=g)
    x = x * torch.tensor([1e-38, 1e-41, 1e30, 1e38, 1.0])[:, None, None]
    cache = make_cache(2, 4, 1, 64, "e4m3", "row", "heads")
    rarn.kv_cache_write(x.cuda(), x.cuda(), cache, torch.arange(5, device="cuda"))
    codes = R.decode(rows_at(cache.k, torch.arange(5), 4), "e4m3")
    assert (codes.abs().amax(-1) == 448).all()
    s = rows_at(cache.k_scale, torch.arange(5), 4).to(R.F64)
    assert torch.isfinite(s).all()
    # the smallest scales are subnormal: their own step is 2^-149
    err = (codes * s[..., None] - x.to(R.F64)).abs()
    u = x.to(R.F64) / s[..., None]
    assert (err <= s[..., None] * (R.half_step(u, "e4m3") + 2.0 ** -18 * u.abs()) +
            448 * 2.0 ** -150).all()


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("fmt,mode", [("e4m3", "row"), ("e5m2", "tensor")])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,dt", [
    (1, 32, 8, 128, 128, "bf16"), (70, 5, 5, 64, 32, "f16"), (33, 28, 4, 96, 96, "bf16"),
    (600, 40, 8, 128, 64, "bf16"), (5, 16, 1, 256, 256, "f32"), (8, 3, 1, 80, 10, "bf16"),
])
def test_fused_write(T, Hq, Hk, D, rot, dt, fmt, mode, style):
    g = gen(T + D)
    page = 16
    pages = T // page + 2
    x = packed(T, Hq, Hk, D, DT[dt], g)
    qg, kg = ((torch.rand(D, generator=g) + 0.5).to(DT[dt]) for _ in range(2))
    table, pos = table_of(4096, rot), torch.randint(0, 4096, (T,), generator=g)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[T // 3] = -1 if T > 1 else slots[0]
    cache = make_cache(pages, page, Hk, D, fmt, mode, "heads")
    dq, dk, dv = split(x.cuda(), Hq, Hk, D)
    args = (qg.cuda(), kg.cuda(), EPS, table.cuda(), pos.cuda())
    q = rarn.qk_norm_rope_kv_write(dq, dk, dv, *args, cache, slots.cuda(), style=style)
    assert torch.equal(q, rarn.qk_norm_rope(dq, dk, *args, style=style)[0])
    live = slots >= 0
    _, k, v = split(x, Hq, Hk, D)
    want, mag = R.rotate(R.norm(k, kg, EPS), table, pos, style)
    for n, codes, scale, w, m in (("k", cache.k, cache.k_scale, want, mag),
                                  ("v", cache.v, cache.v_scale, v.to(R.F64), v.to(R.F64).abs())):
        s = rows_at(scale, slots[live], page) if mode == "row" else scale.cpu()
        R.check_codes(rows_at(codes, slots[live], page), s, w[live], m[live], fmt, mode, n)
    assert rarn.watchdog() == 0


READ = [  # lengths, H, D, page, layout, first row, rows behind
    ([1], 8, 128, 16, "heads", 0, 0), ([5, 0, 17, 33], 2, 64, 16, "tokens", 0, 3),
    ([100, 3], 3, 96, 24, "pool", 2, 1), ([0, 0, 4], 1, 256, 1, "heads", 0, 20),
    ([257, 64, 63, 65], 4, 192, 64, "heads", 1, 0), ([9, 40], 5, 16, 7, "tokens", 0, 1),
]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt,mode", [("e4m3", "row"), ("e5m2", "row"), ("e4m3", "tensor")])
@pytest.mark.parametrize("lens,H,D,page,layout,first,behind", READ)
def test_cache_read(lens, H, D, page, layout, first, behind, fmt, mode, dt):
    g = gen(sum(lens))
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    cache = make_cache(pages, page, H, D, fmt, mode, layout)
    fill_random(cache, g)
    table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=g)
    n = 0
    for b, c in enumerate(need):
        table[b, :c] = order[n:n + c].to(torch.int32)
        n += c
    starts = torch.tensor([first + sum(lens[:b]) for b in range(len(lens) + 1)],
                          dtype=torch.int32)
    rows = first + sum(lens) + behind
    # outputs side by side in one buffer, rows wider than needed
    buf = torch.full((rows, 2 * H, D + 8), -7.0, dtype=DT[dt], device="cuda")
    ko, vo = buf[:, :H, :D], buf[:, H:, :D]
    rarn.kv_cache_read(cache, table.cuda()[:, :], starts.cuda(), ko, vo)
    for codes, scale, out in ((cache.k, cache.k_scale, ko), (cache.v, cache.v_scale, vo)):
        out = out.cpu()
        for b, c in enumerate(lens):
            j = torch.arange(c)
            slots = table[b].long()[j // page] * page + j % page
            x = R.decode(rows_at(codes, slots, page), fmt)
            x = x * (rows_at(scale, slots, page).to(R.F64)[..., None] if mode == "row"
                     else float(scale))
            got = out[starts[b]:starts[b + 1]].to(R.F64)
            tol = (R.half(DT[dt]) + 2.0 ** -23) * x.abs() + R.smallest(DT[dt])
            assert ((got - x).abs() <= tol).all()
    host = buf.cpu()
    assert (host[..., D:] == -7.0).all()
    assert (host[:first] == -7.0).all() and (host[first + sum(lens):] == -7.0).all()
    assert rarn.watchdog() == 0


def fill_random(cache, g, spread=1.0):
    """Random finite codes and scales."""
    for codes in (cache.k, cache.v):
        x = torch.randn(codes.shape, generator=g) * (R.MAXF[cache.fmt] / 4)
        c = x.clamp(-R.MAXF[cache.fmt], R.MAXF[cache.fmt]).to(R.CODE[cache.fmt])
        codes.copy_(c.view(torch.uint8))
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.exp(spread * torch.randn(s.shape, generator=g)) * 4 / R.MAXF[cache.fmt])


def test_read_of_missing_pages():
    cache = make_cache(3, 4, 1, 64, "e4m3", "row", "heads")
    table = torch.tensor([[0, 3, -1, 2]], dtype=torch.int32, device="cuda")
    out = [torch.full((20, 1, 64), -7.0, device="cuda") for _ in range(2)]
    rarn.kv_cache_read(cache, table, torch.tensor([0, 18], dtype=torch.int32, device="cuda"),
                       *out)
    assert rarn.watchdog() == INDEX_BIT
    for o in out:
        assert (o[4:12] == 0).all() and (o[16:18] == 0).all() and (o[18:] == -7.0).all()
        assert (o[:4] != 0).all() and (o[12:16] != 0).all()


def test_offsets_past_32_bits():
    """A pool whose pages lie more than 4 GiB apart."""
    stride = (1 << 32) + (1 << 20)
    buf = torch.zeros(2 * stride + 4096, dtype=torch.uint8, device="cuda")
    k = buf.as_strided((3, 1, 4, 64), (stride, 256, 64, 1))
    v = buf.as_strided((3, 1, 4, 64), (stride, 256, 64, 1), 1024)
    ks, vs = (torch.ones(3, 1, 4, device="cuda") for _ in range(2))
    cache = rarn.KVCache(k, v, ks, vs)
    x = torch.randn(12, 2, 64, generator=gen(5)).to(torch.bfloat16)
    rarn.kv_cache_write(x[:, :1].cuda(), x[:, 1:].cuda(), cache, torch.arange(12, device="cuda"))
    out = [torch.empty(12, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rarn.kv_cache_read(cache, torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"),
                       torch.tensor([0, 12], dtype=torch.int32, device="cuda"), *out)
    for o, src in zip(out, (x[:, :1], x[:, 1:])):
        want = src.to(R.F64)
        most = want.abs().amax(-1, keepdim=True)
        assert ((o.cpu().to(R.F64) - want).abs() <= most * 2.0 ** -4).all()
    q = torch.randn(1, 2, 64, generator=gen(6)).to(torch.bfloat16)
    got = rarn.tree_attention(q.cuda(), cache, torch.tensor([[0, 1, 2]], dtype=torch.int32,
                                                            device="cuda"),
                              torch.tensor([11], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    kk, vv = (R.decode(rows_at(c, torch.arange(12), 4), "e4m3") *
              rows_at(s, torch.arange(12), 4).to(R.F64)[..., None]
              for c, s in ((k, ks), (v, vs)))
    want, tol = R.attention(q, kk, vv, torch.ones(1, 12, dtype=torch.bool), 64 ** -0.5)
    R.check_attention(got.cpu(), want, tol)


def test_binding_refusals():
    x = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    cache = rarn.KVCache.empty(2, 4, 3, 64)
    slots = torch.arange(2, device="cuda")
    with pytest.raises(ValueError):
        rarn.qk_norm_rope(x, x[:1], None, None, EPS)
    with pytest.raises(ValueError):
        rarn.qk_norm_rope(x.cpu(), x.cpu(), None, None, EPS)
    with pytest.raises(TypeError):
        rarn.qk_norm_rope(x, x.float(), None, None, EPS)
    with pytest.raises(ValueError):
        rarn.qk_norm_rope(x, x, None, None, EPS, table_of(4, 64).cuda())
    with pytest.raises(ValueError):
        rarn.qk_norm_rope(x, x, None, None, EPS, style="other")
    with pytest.raises(TypeError):
        rarn.kv_cache_write(x, x, cache, slots.int())
    with pytest.raises(ValueError):
        rarn.kv_cache_write(x, x, cache, torch.arange(3, device="cuda"))
    with pytest.raises(ValueError):
        rarn.kv_cache_write(x[:, :2], x, cache, slots)
    with pytest.raises(TypeError):
        rarn.KVCache(cache.k.float(), cache.v, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        rarn.KVCache(cache.k, cache.v, cache.k_scale, cache.v_scale, scale_mode="tensor")
    with pytest.raises(rarn.RarnError):
        rarn.qk_norm_rope(x, x, None, None, -1.0)
