"""GPU tests of the rotation by positions of several axes, against binary64."""
import pytest
import torch

import kv_ref as R
import residual_add_rmsnorm_gb300 as rarn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
INDEX_BIT = 16
ROWS = 700


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def table_of(rows, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=R.F64) / rot)
    a = torch.arange(rows, dtype=R.F64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def axes_of(sections, order):
    """Each pair's axis, from the sections' description."""
    if order == "blocks":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    turns = sorted((i, a) for a, n in enumerate(sections) for i in range(n))
    return [a for _, a in turns]


def flat(table, positions, axes):
    """A table of one row a token, in which every pair has its own axis's angles."""
    h = table.shape[1] // 2
    row = positions[torch.tensor(axes)].t()         # [T, pairs]
    i = torch.arange(h)
    return torch.cat([table[row, i], table[row, h + i]], 1)


# T, Hq, Hk, D, rot, sections, pad: fours of one axis and of several, lanes of two
# axes, the element-wise kernel, an axis without pairs, one axis, four
CASES = [
    (1, 32, 8, 128, 128, (16, 24, 24), 0), (37, 5, 2, 128, 128, (64,), 0),
    (19, 8, 1, 128, 64, (10, 11, 11), 0), (300, 64, 8, 128, 128, (22, 21, 21), 0),
    (9, 3, 3, 80, 80, (10, 15, 15), 0), (6, 4, 2, 96, 64, (0, 20, 12), 0),
    (5, 2, 1, 64, 32, (4, 4, 4, 4), 0), (7, 2, 1, 129, 126, (13, 30, 20), 0),
    (11, 4, 2, 128, 128, (16, 24, 24), 3), (3, 2, 2, 1000, 1000, (100, 200, 200), 0),
    (2, 1, 1, 2, 2, (1, 0), 0), (4, 3, 1, 256, 256, (1, 126, 1), 0),
    (3, 2, 1, 512, 512, (56, 200), 0),
]


@pytest.mark.parametrize("order", ["blocks", "cyclic"])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,sections,pad", CASES)
def test_axes(T, Hq, Hk, D, rot, sections, pad, dt, style, order):
    g = torch.Generator().manual_seed(T + D + rot)
    x = torch.randn(T, Hq + Hk, D + pad, generator=g).to(DT[dt])
    q, k = x[:, :Hq, :D], x[:, Hq:, :D]
    qg, kg = ((torch.rand(D, generator=g) + 0.5).to(DT[dt]) for _ in range(2))
    table = table_of(ROWS, rot)
    pos = torch.randint(0, ROWS, (len(sections), T), generator=g)
    d = x.cuda()
    got = rarn.qk_norm_rope(d[:, :Hq, :D], d[:, Hq:, :D], qg.cuda(), kg.cuda(), EPS, table.cuda(),
                            pos.cuda(), style=style, sections=sections, section_order=order)
    own = flat(table, pos, axes_of(sections, order))
    for y, src, gamma in ((got[0], q, qg), (got[1], k, kg)):
        want, mag = R.rotate(R.norm(src, gamma, EPS), own, torch.arange(T), style)
        R.check_rows(y.cpu(), want, mag)
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("D", [128, 80, 100])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_equal_positions_are_the_one_axis_form(D, dt):
    T = 50
    g = torch.Generator().manual_seed(D)
    q, k = (torch.randn(T, 4, D, generator=g).to(DT[dt]).cuda() for _ in range(2))
    gm = torch.ones(D, dtype=DT[dt], device="cuda")
    table = table_of(ROWS, D).cuda()
    one = torch.randint(0, ROWS, (T,), generator=g).cuda()
    want = rarn.qk_norm_rope(q, k, gm, gm, EPS, table, one)
    n = D // 2
    for order in rarn.SECTION_ORDERS:
        got = rarn.qk_norm_rope(q, k, gm, gm, EPS, table, one.expand(3, T).contiguous(),
                                sections=(n - 2 * (n // 3), n // 3, n // 3), section_order=order)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # the axes' rows at any distance, none at all among them
        got = rarn.qk_norm_rope(q, k, gm, gm, EPS, table, one.expand(3, T),
                                sections=(n - 2 * (n // 3), n // 3, n // 3), section_order=order)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("mode", ["row", "tensor"])
@pytest.mark.parametrize("D,page", [(128, 16), (80, 7)])
def test_with_the_cache_write(D, page, mode):
    """Queries as without a cache; keys and values as from a table of each token's own."""
    T, Hq, Hk, sections = 45, 6, 2, (D // 2 - 2 * (D // 5), D // 5, D // 5)
    g = torch.Generator().manual_seed(D)
    x = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(torch.bfloat16).cuda()
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    gm = (torch.rand(D, generator=g) + 0.5).to(torch.bfloat16).cuda()
    table, pos = table_of(ROWS, D), torch.randint(0, ROWS, (3, T), generator=g)
    slots = torch.randperm(10 * page, generator=g)[:T].cuda()
    slots[3] = -1
    own = flat(table, pos, axes_of(sections, "cyclic")).cuda()
    caches = [rarn.KVCache.empty(10, page, Hk, D, scale_mode=mode, k_scale=0.02, v_scale=0.02)
              for _ in range(2)]
    a = rarn.qk_norm_rope_kv_write(q, k, v, gm, gm, EPS, table.cuda(), pos.cuda(), caches[0], slots,
                                   sections=sections, section_order="cyclic")
    b = rarn.qk_norm_rope_kv_write(q, k, v, gm, gm, EPS, own, torch.arange(T).cuda(), caches[1],
                                   slots)
    assert torch.equal(a, b)
    for n in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(caches[0], n), getattr(caches[1], n))
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("D", [64, 36])
def test_a_position_outside_leaves_its_token(D):
    T, rows = 9, 20
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn(T, 2, D, generator=g).to(torch.float16).cuda() for _ in range(2))
    gm = torch.ones(D, dtype=torch.float16, device="cuda")
    table = table_of(rows, D).cuda()
    pos = torch.randint(0, rows, (3, T), generator=g)
    good = pos.clone()
    pos[0, 1], pos[1, 4], pos[2, 8] = rows, -1, 2 ** 62
    n = D // 2
    sections = (n - 2 * (n // 3), n // 3, n // 3)
    out = [torch.full_like(q, 7.0) for _ in range(2)]
    rarn.qk_norm_rope(q, k, gm, gm, EPS, table, pos.cuda(), q_out=out[0], k_out=out[1],
                      sections=sections)
    want = rarn.qk_norm_rope(q, k, gm, gm, EPS, table, good.cuda(), sections=sections)
    ok = torch.ones(T, dtype=torch.bool, device="cuda")
    ok[[1, 4, 8]] = False
    for o, w in zip(out, want):
        assert (o[~ok] == 7.0).all() and torch.equal(o[ok], w[ok])
    assert rarn.watchdog() == INDEX_BIT


def test_in_a_graph_with_positions_that_change():
    T, D = 20, 128
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn(T, 2, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    gm = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    table = table_of(ROWS, D).cuda()
    pos = torch.zeros(3, T, dtype=torch.int64, device="cuda")
    out = [torch.empty_like(q) for _ in range(2)]
    s = (16, 24, 24)
    rarn.qk_norm_rope(q, k, gm, gm, EPS, table, pos, sections=s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rarn.qk_norm_rope(q, k, gm, gm, EPS, table, pos, q_out=out[0], k_out=out[1], sections=s)
    for seed in (3, 4):
        pos.copy_(torch.randint(0, ROWS, (3, T), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        want = rarn.qk_norm_rope(q, k, gm, gm, EPS, table, pos, sections=s)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_the_binding_refuses():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    gm, table = q[0, 0], torch.zeros(8, 64, device="cuda")
    pos = torch.zeros(3, 4, dtype=torch.int64, device="cuda")
    sound = dict(sections=(8, 12, 12))

    def call(table=table, pos=pos, **kw):
        rarn.qk_norm_rope(q, q.clone(), gm, gm, EPS, table, pos, **kw)

    call(**sound)
    for kw in (dict(sections=(8, 12, 11)), dict(sections=(33, -1, 0)), dict(sections=()),
               dict(sections=(16, 16)), dict(sections=(8, 12, 12), section_order="mixed"),
               dict(pos=pos[:2], **sound), dict(pos=pos[0], **sound), dict(pos=None, **sound),
               dict(pos=torch.zeros(4, 3, dtype=torch.int64, device="cuda").t(), **sound),
               dict(table=None, **sound)):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(TypeError):
        call(pos=pos.int(), **sound)
    with pytest.raises(rarn.RarnError):     # five axes
        call(pos=torch.zeros(5, 4, dtype=torch.int64, device="cuda"), sections=(8, 8, 8, 4, 4))
