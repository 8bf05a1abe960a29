"""GPU tests of the norms around a block (gated_add_rms_norm) against binary64."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
import step_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
INDEX_BIT = 16


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def inputs(T, H, dt, wide, gates, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H + pad, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dt)
    r = (2 * torch.randn(T, H + pad, generator=g)).to(torch.float32 if wide else dt)
    xg, gm = ((torch.rand(H, generator=g) + 0.5).to(dt) for _ in range(2))
    gate = torch.randn(gates, H + pad, generator=g).to(dt) if gates else None
    return x, r, xg, gm, gate


# rows of a warp, a CTA, several rounds of CTAs, longer than registers, odd, one element
SHAPES = [(1, 4096), (1, 1), (3, 7), (2, 256), (700, 512), (5, 1000), (33, 1024), (19, 1591),
          (300, 1592), (4, 2048), (700, 4096), (17, 5120), (1300, 5120), (9, 8192), (400, 8192),
          (2, 16384), (320, 16384), (2, 20000), (3, 40000), (1, 131072), (2500, 64), (5000, 128),
          (320, 32768), (13000, 2048), (3000, 1024)]


@pytest.mark.parametrize("kind", ["bf16", "bf16w", "f16", "f16w", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_shapes(T, H, kind):
    dt, wide = DT[kind.rstrip("w")], kind.endswith("w")
    gates = [0, 1, T, min(T, 5)][(T + H + len(kind)) % 4]
    x, r, xg, gm, gate = inputs(T, H, dt, wide, gates, T * 7 + H)
    index = None
    if gates not in (0, 1, T):
        index = (torch.arange(T) * 3 % gates).to(torch.int32)
    full = None if gate is None else gate[index.long()] if index is not None else gate.expand(T, H)
    h = torch.empty_like(r, device="cuda")
    y = rarn.gated_add_rms_norm(x.cuda(), r.cuda(), xg.cuda(), gm.cuda(), EPS,
                                gate=None if gate is None else gate.cuda(),
                                gate_index=None if index is None else index.cuda(), scale=0.5,
                                residual_scale=1.25, residual_out=h)
    R.check_block(y.cpu(), h.cpu(), x, r, xg, gm, EPS, full, 0.5, 1.25)
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("H", [64, 1001, 1024, 4096, 8192, 33000])
@pytest.mark.parametrize("gates", [0, 6])
@pytest.mark.parametrize("post", [False, True])
def test_in_place_equals_apart(H, gates, post):
    T, dt = 6, torch.bfloat16
    x, r, xg, gm, gate = (v.cuda() if v is not None else None
                          for v in inputs(T, H, dt, False, gates, H))
    xg = xg if post else None
    h = torch.empty_like(r)
    y = rarn.gated_add_rms_norm(x, r, xg, gm, EPS, gate=gate, residual_out=h)
    R.check_block(y.cpu(), h.cpu(), x.cpu(), r.cpu(), None if xg is None else xg.cpu(), gm.cpu(),
                  EPS, None if gate is None else gate.cpu())
    x2, r2 = x.clone(), r.clone()
    got = rarn.gated_add_rms_norm(x2, r2, xg, gm, EPS, gate=gate, out=x2)
    assert got is x2 and torch.equal(x2, y) and torch.equal(r2, h)


def test_without_post_norm_and_gate_it_is_the_fused_form():
    """With n = x and scales of one, h is bit for bit that of fused_add_rms_norm."""
    for T, H in ((1, 4096), (40, 8192), (9, 1000)):
        x, r, _, gm, _ = inputs(T, H, torch.bfloat16, False, 0, H)
        ra, rb = r.cuda(), r.cuda()
        rarn.fused_add_rms_norm(x.cuda(), ra, gm.cuda(), EPS)
        rarn.gated_add_rms_norm(x.cuda(), rb, None, gm.cuda(), EPS)
        assert torch.equal(ra, rb)


@pytest.mark.parametrize("H,pad", [(256, 8), (1024, 3), (5120, 16), (8192, 8), (1000, 1)])
def test_strided_rows_and_their_padding(H, pad):
    T, dt = 37, torch.float16
    x, r, xg, gm, gate = inputs(T, H, dt, False, T, H, pad)
    dx, dr, dg = x.cuda(), r.cuda(), gate.cuda()
    out = torch.full((T, H + 2 * pad), 7.0, dtype=dt, device="cuda")
    rarn.gated_add_rms_norm(dx[:, :H], dr[:, :H], xg.cuda(), gm.cuda(), EPS, gate=dg[:, :H],
                            out=out[:, :H])
    h = dr.cpu()
    R.check_block(out.cpu()[:, :H], h[:, :H], x[:, :H], r[:, :H], xg, gm, EPS, gate[:, :H])
    assert torch.equal(h[:, H:], r[:, H:]) and torch.equal(dx.cpu(), x)
    assert (out[:, H:] == 7.0).all()


def test_misaligned_base():
    T, H = 5, 512
    x, r, xg, gm, _ = inputs(T, H, torch.bfloat16, False, 0, 3)
    for shift in ("x", "r", "gamma", "out"):
        def at(v, n):
            if n != shift:
                return v.cuda()
            b = torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")
            b[1:] = v.flatten().cuda()
            return b[1:].view(v.shape)
        dr = at(r, "r")
        y = rarn.gated_add_rms_norm(at(x, "x"), dr, xg.cuda(), at(gm, "gamma"), EPS,
                                    out=at(x, "out"))
        R.check_block(y.cpu(), dr.cpu(), x, r, xg, gm, EPS)


@pytest.mark.parametrize("H", [128, 4096, 8192, 999])
def test_indices_outside_leave_their_rows(H):
    T, dt = 50, torch.bfloat16
    x, r, xg, gm, gate = inputs(T, H, dt, False, 3, H)
    index = (torch.arange(T) % 3).to(torch.int32)
    index[4], index[7], index[49] = -1, 3, 2 ** 31 - 1
    dr = r.cuda()
    out = torch.full((T, H), 7.0, dtype=dt, device="cuda")
    rarn.gated_add_rms_norm(x.cuda(), dr, xg.cuda(), gm.cuda(), EPS, gate=gate.cuda(),
                            gate_index=index.cuda(), out=out)
    ok = torch.ones(T, dtype=torch.bool)
    ok[[4, 7, 49]] = False
    h, y = dr.cpu(), out.cpu()
    assert torch.equal(h[~ok], r[~ok]) and (y[~ok] == 7.0).all()
    R.check_block(y[ok], h[ok], x[ok], r[ok], xg, gm, EPS, gate[index[ok].long()])
    assert rarn.watchdog() == INDEX_BIT


@pytest.mark.parametrize("H", [256, 4096])
def test_zeros_infinities_and_nan(H):
    x, r, xg, gm, gate = inputs(6, H, torch.float32, False, 6, 5)
    x[0] = 0                    # a block that gives nothing: h = r
    x[1], r[1] = 0, 0           # a row of zeros
    x[2, 3] = float("nan")
    r[3, 5] = float("inf")      # h infinite there: the row's y is 0, and inf * 0
    gate[4] = 0
    dr = r.cuda()
    y = rarn.gated_add_rms_norm(x.cuda(), dr, xg.cuda(), gm.cuda(), EPS, gate=gate.cuda())
    y, h = y.cpu(), dr.cpu()
    assert torch.equal(h[0], r[0]) and torch.equal(h[4], r[4])
    assert (y[1] == 0).all() and (h[1] == 0).all()
    assert torch.isnan(h[2]).all() and torch.isnan(y[2]).all()
    assert torch.isinf(h[3, 5]) and torch.isnan(y[3, 5])
    others = torch.arange(H) != 5
    assert (y[3, others] == 0).all()
    R.check_block(y[5:], h[5:], x[5:], r[5:], xg, gm, EPS, gate[5:])


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gm = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    assert rarn.gated_add_rms_norm(x, x.clone(), gm, gm, EPS).shape == (0, 64)


@pytest.mark.parametrize("T,H", [(3, 4096), (2000, 1024), (20, 1001)])
def test_the_same_bits_every_time_on_streams_and_in_graphs(T, H):
    x, r, xg, gm, gate = (v.cuda() for v in inputs(T, H, torch.bfloat16, True, T, 11))
    h, y = torch.empty_like(r), torch.empty_like(x)
    rarn.gated_add_rms_norm(x, r, xg, gm, EPS, gate=gate, residual_out=h, out=y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h2, y2 = torch.empty_like(h), torch.empty_like(y)
    with torch.cuda.stream(s):
        rarn.gated_add_rms_norm(x, r, xg, gm, EPS, gate=gate, residual_out=h2, out=y2)
    s.synchronize()
    assert torch.equal(h, h2) and torch.equal(y, y2)
    g = torch.cuda.CUDAGraph()
    h2.zero_(), y2.zero_()
    with torch.cuda.graph(g):
        rarn.gated_add_rms_norm(x, r, xg, gm, EPS, gate=gate, residual_out=h2, out=y2)
        rarn.gated_add_rms_norm(y2, h2, xg, gm, EPS, residual_out=h2, out=y2)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    rarn.gated_add_rms_norm(y, h, xg, gm, EPS, out=y)
    assert torch.equal(h, h2) and torch.equal(y, y2)


@pytest.mark.parametrize("H", [4096, 999])
def test_rows_far_apart(H):
    """Rows whose offsets pass 2^31 elements."""
    T, ld, dt = 3, (1 << 30) + 8, torch.bfloat16
    x, r, xg, gm, gate = inputs(T, H, dt, False, T, H)
    far = []
    for v in (x, r, gate, torch.zeros_like(x)):
        d = torch.empty((T - 1) * ld + H, dtype=dt, device="cuda").as_strided((T, H), (ld, 1))
        d.copy_(v)
        far.append(d)
    rarn.gated_add_rms_norm(far[0], far[1], xg.cuda(), gm.cuda(), EPS, gate=far[2], out=far[3])
    R.check_block(far[3].cpu(), far[1].cpu(), x, r, xg, gm, EPS, gate)


def test_two_streams_at_once():
    T, H = 3000, 4096
    ins = [[v.cuda() for v in inputs(T, H, torch.bfloat16, False, T, s)] for s in (1, 2)]
    want = []
    for x, r, xg, gm, gate in ins:
        h = torch.empty_like(r)
        want.append((rarn.gated_add_rms_norm(x, r, xg, gm, EPS, gate=gate, residual_out=h), h))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [(torch.empty_like(y), torch.empty_like(h)) for y, h in want]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (x, r, xg, gm, gate), (y, h) in zip(streams, ins, got):
            with torch.cuda.stream(s):
                rarn.gated_add_rms_norm(x, r, xg, gm, EPS, gate=gate, residual_out=h, out=y)
    torch.cuda.synchronize()
    for (y, h), (y2, h2) in zip(want, got):
        assert torch.equal(y, y2) and torch.equal(h, h2)
