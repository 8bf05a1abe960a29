"""GPU tests of the attention of drafted tokens over the 8-bit cache, against
binary64 over the cache's own dequantised values (kv_ref)."""
import pytest
import torch

import kv_ref as R
import residual_add_rmsnorm_gb300 as rarn
from test_kv_gpu import DT, fill_random, gen, make_cache, rows_at, table_of

pytestmark = pytest.mark.gpu

INDEX_BIT = 16


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


class Case:
    """Sequences over a cache with stale NaN codes in every unused slot."""

    def __init__(self, ctx, new, Hq, Hk, D, page=16, dt="bf16", fmt="e4m3", mode="row",
                 layout="heads", seed=0, mask="tree", first=0, behind=0, spread=1.0, gain=1.0):
        g = gen(seed + sum(ctx) + 7 * sum(new))
        self.ctx, self.new, self.page, self.dt = ctx, new, page, DT[dt]
        self.Hq, self.Hk, self.D, self.fmt, self.mode = Hq, Hk, D, fmt, mode
        both = [a + b for a, b in zip(ctx, new)]
        need = [-(-n // page) for n in both]
        pages = sum(need) + 2
        self.cache = make_cache(pages, page, Hk, D, fmt, mode, layout)
        fill_random(self.cache, g, spread)
        self.table = torch.full((len(ctx), max(need) + 1), -1, dtype=torch.int32)
        order = torch.randperm(pages, generator=g)
        at, used = 0, torch.zeros(pages * page, dtype=torch.bool)
        for b, c in enumerate(need):
            self.table[b, :c] = order[at:at + c].to(torch.int32)
            used[self.slots(b, both[b])] = True
            at += c
        unused = (~used).nonzero()[:, 0].cuda()
        for t in (self.cache.k, self.cache.v):  # what earlier sequences left
            t.transpose(1, 2)[unused // page, unused % page] = 0x7f if fmt == "e4m3" else 0x7e
        self.first = first
        rows = first + sum(new) + behind
        self.q = (gain * torch.randn(rows, Hq, D, generator=g)).to(self.dt)
        self.starts = torch.tensor([first + sum(new[:b]) for b in range(len(new) + 1)],
                                   dtype=torch.int32)
        self.mask = self.bits = None
        if mask != "chain":
            words = max(1, -(-max(new) // 32)) + (1 if seed % 2 else 0)
            self.bits = torch.zeros(rows, 32 * words, dtype=torch.bool)
            for b, n in enumerate(new):
                s = int(self.starts[b])
                for i in range(n):
                    if mask == "tree":
                        if i:
                            parent = int(torch.randint(0, i, (1,), generator=g))
                            self.bits[s + i] = self.bits[s + parent]
                        self.bits[s + i, i] = True
                    elif mask == "random":
                        self.bits[s + i, :n] = torch.rand(n, generator=g) < 0.5
                        self.bits[s + i, n:] = True  # past the sequence: names no one
            w = (self.bits.view(rows, words, 32).long() << torch.arange(32)).sum(-1)
            self.mask = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)

    def slots(self, b, n):
        j = torch.arange(n)
        return self.table[b].long()[j // self.page] * self.page + j % self.page

    def visible(self, b):
        n, c = self.new[b], self.ctx[b]
        drafted = torch.tril(torch.ones(n, n, dtype=torch.bool))
        if self.bits is not None:
            s = int(self.starts[b])
            drafted = self.bits[s:s + n, :n]
            if n > drafted.shape[1]:
                drafted = torch.cat([drafted, torch.zeros(n, n - drafted.shape[1],
                                                          dtype=torch.bool)], 1)
        return torch.cat([torch.ones(n, c, dtype=torch.bool), drafted], 1)

    def values(self, t, s, b, n):
        at = self.slots(b, n)
        x = R.decode(rows_at(t, at, self.page), self.fmt)
        return x * (rows_at(s, at, self.page).to(R.F64)[..., None] if self.mode == "row"
                    else float(s))

    def run(self, out=None, **kw):
        return rarn.tree_attention(self.q.cuda(), self.cache, self.table.cuda(),
                                   torch.tensor(self.ctx, dtype=torch.int32, device="cuda"),
                                   self.starts.cuda(),
                                   mask=None if self.mask is None else self.mask.cuda(), out=out,
                                   **kw)

    def check(self, got, scale=None):
        got = got.cpu()
        c = self.cache
        for b, n in enumerate(self.new):
            L = self.ctx[b] + n
            if n == 0:
                continue
            k = self.values(c.k, c.k_scale, b, L)
            v = self.values(c.v, c.v_scale, b, L)
            s = int(self.starts[b])
            at = self.slots(b, L)
            codes = R.decode(rows_at(c.v, at, self.page), self.fmt).abs()
            codes *= (rows_at(c.v_scale, at, self.page).to(R.F64).abs().amax(0)[None, :, None]
                      if self.mode == "row" else float(c.v_scale))
            want, tol = R.attention(self.q[s:s + n], k, v, self.visible(b),
                                    self.D ** -0.5 if scale is None else scale, codes)
            R.check_attention(got[s:s + n], want, tol, f"sequence {b}")


CASES = {
    "one": dict(ctx=[0], new=[1], Hq=8, Hk=8, D=64),
    "one token": dict(ctx=[700], new=[1], Hq=32, Hk=8, D=128),
    "decode": dict(ctx=[1, 63, 64, 65, 500, 0, 130], new=[1] * 7, Hq=16, Hk=2, D=128,
                   mask="chain"),
    "decode f16": dict(ctx=[300, 17], new=[1, 1], Hq=5, Hk=5, D=96, dt="f16"),
    "ragged trees": dict(ctx=[100, 0, 37, 260, 5], new=[7, 12, 1, 0, 33], Hq=12, Hk=4, D=64),
    "random masks": dict(ctx=[40, 0, 0, 15], new=[9, 8, 1, 31], Hq=8, Hk=4, D=128,
                         mask="random", seed=1),
    "chain": dict(ctx=[50, 0], new=[40, 70], Hq=4, Hk=2, D=64, mask="chain"),
    "wide tree": dict(ctx=[90], new=[100], Hq=10, Hk=2, D=128, page=24),
    "five heads to one": dict(ctx=[1000, 129], new=[8, 5], Hq=40, Hk=8, D=128, fmt="e5m2",
                              mode="tensor", dt="f16", page=64),
    "one key head": dict(ctx=[333], new=[6], Hq=16, Hk=1, D=192),
    "D 256": dict(ctx=[200, 31], new=[5, 3], Hq=8, Hk=2, D=256, fmt="e5m2"),
    "D 96 e5m2": dict(ctx=[150, 16], new=[16, 2], Hq=8, Hk=4, D=96, fmt="e5m2", layout="pool"),
    "page 1": dict(ctx=[77, 3], new=[4, 2], Hq=4, Hk=4, D=64, page=1, layout="tokens"),
    "page 7": dict(ctx=[77, 13], new=[10, 2], Hq=6, Hk=2, D=128, page=7, layout="pool"),
    "page 128": dict(ctx=[130, 127, 128], new=[3, 1, 2], Hq=8, Hk=1, D=128, page=128),
    "rows around": dict(ctx=[60, 9], new=[3, 4], Hq=8, Hk=2, D=64, first=2, behind=3),
    "spread scales": dict(ctx=[400], new=[16], Hq=8, Hk=2, D=128, spread=4.0),
    "sharp": dict(ctx=[500, 90], new=[2, 20], Hq=8, Hk=2, D=128, gain=6.0),
    "many": dict(ctx=[i % 50 for i in range(300)], new=[1 + i % 3 for i in range(300)], Hq=4,
                 Hk=2, D=64),
    "long": dict(ctx=[9000], new=[4], Hq=4, Hk=2, D=64),
    "group of 64": dict(ctx=[210], new=[3], Hq=64, Hk=1, D=64),
    # segments of one tile among segments of several, several to a CTA
    "short and long": dict(ctx=[(37 * i) % 390 for i in range(250)],
                           new=[9 + i % 4 for i in range(250)], Hq=4, Hk=2, D=64),
    "256 rows": dict(ctx=[700, 10, 0, 129], new=[40, 33, 64, 1], Hq=16, Hk=2, D=128),
    "more than 256 rows": dict(ctx=[260], new=[90], Hq=8, Hk=1, D=64, fmt="e5m2"),
    "spread scales, many rows": dict(ctx=[600], new=[20], Hq=8, Hk=2, D=128, spread=4.0),
    "sharp, many rows": dict(ctx=[900], new=[40], Hq=16, Hk=2, D=128, gain=6.0, mode="tensor"),
    "f16, many rows": dict(ctx=[300, 44], new=[30, 17], Hq=8, Hk=4, D=128, dt="f16", page=24),
    "group of 3": dict(ctx=[45, 600], new=[11, 23], Hq=9, Hk=3, D=192, dt="f16"),
    "D 192, 16 rows": dict(ctx=[45, 600], new=[11, 23], Hq=12, Hk=3, D=192, dt="f16", page=7),
    "D 192, 16 rows, e5m2": dict(ctx=[300], new=[30], Hq=8, Hk=2, D=192, fmt="e5m2"),
}


@pytest.mark.parametrize("name", CASES)
def test_tree_attention(name):
    c = Case(**CASES[name])
    out = torch.full(c.q.shape, -7.0, dtype=c.dt, device="cuda")
    c.run(out=out)
    assert rarn.watchdog() == 0
    c.check(out)
    used = torch.zeros(c.q.shape[0], dtype=torch.bool)
    used[int(c.starts[0]):int(c.starts[-1])] = True
    assert (out.cpu()[~used] == -7.0).all()
    # the same bits again, in a workspace that holds something else
    n = rarn.tree_attention_workspace_bytes(c.q.shape[0], len(c.ctx), c.Hq, c.Hk, c.D)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.run(out=out.clone(), workspace=ws), out)


def test_strided_queries_and_outputs():
    c = Case([70, 3], [5, 2], 8, 2, 64)
    wide = torch.zeros(7, 12, 64, dtype=torch.bfloat16)
    wide[:, :8] = c.q
    out = torch.full((8, 7, 72), -7.0, dtype=torch.bfloat16, device="cuda")
    got = rarn.tree_attention(wide.cuda()[:, :8], c.cache, c.table.cuda(),
                              torch.tensor(c.ctx, dtype=torch.int32, device="cuda"),
                              c.starts.cuda(), mask=c.mask.cuda(),
                              out=out.transpose(0, 1)[..., :64])
    c.check(got)
    assert (out[..., 64:] == -7.0).all()


def test_scale_and_narrow_masks():
    c = Case([20], [40], 4, 2, 64, mask="random")
    c.mask = c.mask[:, :1].contiguous()          # bits of drafted tokens 32 .. 39 are not there
    c.bits = c.bits[:, :32]
    c.check(c.run(scale=0.3), scale=0.3)


def test_rows_that_see_nothing():
    c = Case([0, 0], [3, 40], 8, 2, 128, mask="random")
    c.bits[1] = False
    c.mask[1] = 0
    c.bits[5:, :] = False
    c.mask[5:] = 0
    got = c.run()
    assert (got[1] == 0).all() and (got[5:] == 0).all()
    c.check(got)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("n,D", [(5, 128), (20, 128), (40, 64), (6, 256)])
def test_values_that_are_not_finite(n, D, fmt):
    """NaN in a drafted token's key or value reaches the rows that see it, and
    no other."""
    c = Case([30], [n], 8, 2, D, fmt=fmt, seed=2)
    nan = 0x7f if fmt == "e4m3" else 0x7e
    slots = c.slots(0, 30 + n)
    at = slots[30 + n - 2].item()                # a leaf: few rows see it
    c.cache.v[at // 16, 0, at % 16, 3] = nan
    at = slots[30 + n - 1].item()
    c.cache.k[at // 16, 1, at % 16, 0] = nan
    if fmt == "e5m2":
        at = slots[30].item()
        c.cache.v[at // 16, 1, at % 16, 9] = 0x7c    # +inf in the root's value
    got = c.run()
    assert torch.isnan(got[n - 1, 4:]).all() and not torch.isnan(got[n - 1, :4, 4:]).any()
    # rows that see no such value are as if it were not there
    vis = c.visible(0)
    clean = Case([30], [n], 8, 2, D, fmt=fmt, seed=2)
    want, tol = R.attention(c.q, *(clean.values(t, s, 0, 30 + n) for t, s in (
        (clean.cache.k, clean.cache.k_scale), (clean.cache.v, clean.cache.v_scale))),
        vis, D ** -0.5)
    ok = ~vis[:, -2] & ~vis[:, -1] & (~vis[:, 30] if fmt == "e5m2" else True)
    R.check_attention(got.cpu()[ok], want[ok], tol[ok])
    sees = vis[:, -2]
    assert torch.isnan(got.cpu()[sees][:, :4, 3]).all()
    if fmt == "e5m2":
        # +inf, or NaN where the weight is 0 in binary32: scores here reach 117 under their
        # row's largest (row 13, head 5), and exp(-117) = 1.6e-51 < 2^-149
        sees = vis[:, 30] & ~vis[:, -1]
        x = got.cpu()[sees][:, 4:, 9]
        k = c.values(c.cache.k, c.cache.k_scale, 0, 30 + n)[:, 1]
        s = torch.einsum("ihd,jd->ihj", c.q[sees][:, 4:].to(R.F64), k) * D ** -0.5
        s = s.masked_fill(~vis[sees][:, None], float("-inf"))
        kept = s[..., 30] - s.amax(-1) > -100        # exp(-100) = 3.7e-44 > 2^-149
        assert torch.isinf(x[kept]).all() and not torch.isfinite(x).any()


def test_scales_that_are_not_finite():
    c = Case([20], [6], 4, 1, 64, seed=4)
    slots = c.slots(0, 26)
    at = slots[25].item()
    c.cache.v_scale[at // 16, 0, at % 16] = float("inf")
    at = slots[24].item()
    c.cache.k_scale[at // 16, 0, at % 16] = float("nan")
    got, vis = c.run().cpu(), c.visible(0)
    clean = Case([20], [6], 4, 1, 64, seed=4)
    ok = ~vis[:, 24] & ~vis[:, 25]
    full = clean.run().cpu()
    R.check_attention(got[ok], full[ok].to(R.F64), torch.full_like(full[ok], 2.0 ** -7,
                                                                   dtype=R.F64))
    assert torch.isnan(got[vis[:, 24]]).all()
    assert not torch.isfinite(got[vis[:, 25]]).any()


def test_zero_scales_and_infinite_queries():
    c = Case([40], [3], 4, 2, 64, seed=6)
    c.cache.v_scale.zero_()
    c.q[1, 2, 5] = float("inf")
    got = c.run().cpu()
    assert torch.isnan(got[1, 2]).all()
    got[1, 2] = 0
    assert (got == 0).all()


def test_missing_pages_are_hidden():
    c = Case([100, 40], [4, 4], 8, 2, 64, mask="chain")
    full = c.table.clone()
    c.table[0, 2] = -1
    c.table[1, 1] = 1 << 30
    got = c.run().cpu()
    assert rarn.watchdog() == INDEX_BIT
    c.table = full
    for b in range(2):
        L = c.ctx[b] + 4
        vis = c.visible(b)
        vis[:, 32:48] &= b != 0
        vis[:, 16:32] &= b != 1
        k, v = (c.values(t, s, b, L) for t, s in ((c.cache.k, c.cache.k_scale),
                                                  (c.cache.v, c.cache.v_scale)))
        s = int(c.starts[b])
        want, tol = R.attention(c.q[s:s + 4], k, v, vis, 64 ** -0.5)
        R.check_attention(got[s:s + 4], want, tol)


def test_a_table_too_narrow_hides_the_rest():
    c = Case([60], [4], 4, 2, 64, mask="chain")
    full = c.table.clone()
    c.table = c.table[:, :2].contiguous()
    got = c.run().cpu()
    c.table = full
    vis = c.visible(0)
    vis[:, 32:] = False
    k, v = (c.values(t, s, 0, 64) for t, s in ((c.cache.k, c.cache.k_scale),
                                               (c.cache.v, c.cache.v_scale)))
    R.check_attention(got, *R.attention(c.q, k, v, vis, 64 ** -0.5))


def test_starts_that_fall():
    c = Case([20, 20], [4, 4], 4, 2, 64)
    out = torch.full(c.q.shape, -7.0, dtype=c.dt, device="cuda")
    c.starts = torch.tensor([0, 4, 2], dtype=torch.int32)
    c.run(out=out)                                # the second sequence is empty
    assert (out[4:] == -7.0).all() and not (out[:4] == -7.0).any()
    n = 40
    c = Case([20] * n, [4] * n, 4, 2, 64)
    out = torch.full(c.q.shape, -7.0, dtype=c.dt, device="cuda")
    c.starts = torch.tensor([0, 4 * n] * (n // 2) + [0], dtype=torch.int32)
    rarn.watchdog(clear=True)
    c.run(out=out)                                # they name more rows than there are
    assert rarn.watchdog() == INDEX_BIT and (out == -7.0).all()


def test_a_captured_call_follows_the_lengths():
    c = Case([300, 200], [6, 5], 8, 2, 128)
    q, table, mask = c.q.cuda(), c.table.cuda(), c.mask.cuda()
    ctx = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    n = rarn.tree_attention_workspace_bytes(11, 2, 8, 2, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)

    def call():
        rarn.tree_attention(q, c.cache, table, ctx, starts, mask=mask, out=out, workspace=ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    ctx.copy_(torch.tensor(c.ctx, dtype=torch.int32))
    starts.copy_(c.starts)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out)
    eager = out.clone()
    out.zero_()
    for _ in range(3):
        graph.replay()
    assert torch.equal(out, eager)


def test_two_streams_with_a_workspace_each():
    cases = [Case([900, 40], [8, 3], 8, 2, 128, seed=s) for s in (10, 20)]
    streams = [torch.cuda.Stream() for _ in cases]
    args = []
    for c in cases:
        args.append(dict(q=c.q.cuda(), page_table=c.table.cuda(),
                         context_lens=torch.tensor(c.ctx, dtype=torch.int32, device="cuda"),
                         starts=c.starts.cuda(), mask=c.mask.cuda(), cache=c.cache,
                         out=torch.zeros(c.q.shape, dtype=c.dt, device="cuda"),
                         workspace=torch.empty(rarn.tree_attention_workspace_bytes(
                             11, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a in zip(streams, args):
            with torch.cuda.stream(s):
                rarn.tree_attention(**a)
    torch.cuda.synchronize()
    for c, a in zip(cases, args):
        c.check(a["out"])


def test_decode_steps_with_the_library():
    """Prefill and decode steps as a model makes them: norm, projection, per-head
    norm and rotation into the cache, attention over it, output projection with
    the residual add and norm; against the same steps in binary64 over the
    cache's own codes."""
    g = gen(77)
    T, Hq, Hk, D, page = 21, 8, 2, 64, 16
    H = Hq * D
    bf = torch.bfloat16
    dev = "cuda"
    wqkv = (torch.randn(H, (Hq + 2 * Hk) * D, generator=g) / H ** 0.5).to(bf).to(dev)
    wo = (torch.randn(H, H, generator=g) / H ** 0.5).to(bf).to(dev)
    g1, g2 = ((torch.rand(H, generator=g) + 0.5).to(bf).to(dev) for _ in range(2))
    qg, kg = ((torch.rand(D, generator=g) + 0.5).to(bf).to(dev) for _ in range(2))
    table = table_of(64, D).to(dev)
    cache = rarn.KVCache.empty(4, page, Hk, D)
    pages = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=dev)
    x = torch.randn(T, H, generator=g).to(bf).to(dev)
    residual = torch.zeros(T, H, dtype=bf, device=dev)
    done = 0
    for n in (15, 1, 1, 4):                      # a prompt, two tokens, a drafted chain
        rows = slice(done, done + n)
        y = rarn.fused_add_rms_norm(x[rows].contiguous(), residual[rows], g1, 1e-6)
        qkv = (y @ wqkv).view(n, Hq + 2 * Hk, D)
        pos = torch.arange(done, done + n, device=dev)
        slots = pages[0].long()[pos // page] * page + pos % page
        q = rarn.qk_norm_rope_kv_write(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], qg, kg,
                                       1e-6, table, pos, cache, slots)
        o = rarn.tree_attention(q, cache, pages,
                                torch.tensor([done], dtype=torch.int32, device=dev),
                                torch.tensor([0, n], dtype=torch.int32, device=dev))
        r = residual[rows].clone()
        z = rarn.gemm_add_rms_norm(o.view(n, H), wo, r, g2, 1e-6)
        # the steps' own definitions in binary64
        want, mag = R.rotate(R.norm(qkv[:, :Hq].cpu(), qg.cpu(), 1e-6), table.cpu(), pos.cpu(),
                             "half")
        R.check_rows(q.cpu(), want, mag)
        at = (pages[0].long().cpu()[torch.arange(done + n) // page] * page +
              torch.arange(done + n) % page)
        kk, vv = (R.decode(rows_at(t, at, page), "e4m3") *
                  rows_at(s, at, page).to(R.F64)[..., None]
                  for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        vis = torch.arange(done + n)[None] <= torch.arange(done, done + n)[:, None]
        R.check_attention(o.cpu(), *R.attention(q.cpu(), kk, vv, vis, D ** -0.5))
        h = (o.view(n, H).cpu().to(R.F64) @ wo.cpu().to(R.F64).T +
             residual[rows].cpu().to(R.F64))
        # h: a binary32 sum of H + 1 terms, one rounding
        terms = (o.view(n, H).cpu().to(R.F64).abs() @ wo.cpu().to(R.F64).abs().T +
                 residual[rows].cpu().to(R.F64).abs())
        assert ((r.cpu().to(R.F64) - h).abs() <= 2.0 ** -8 * h.abs() +
                H * 2.0 ** -22 * terms + 1e-30).all()
        zz = R.norm(r.cpu(), g2.cpu(), 1e-6)
        R.check_rows(z.cpu(), zz, zz.abs())
        # the cache holds the normalised, rotated keys and the values
        want, mag = R.rotate(R.norm(qkv[:, Hq:Hq + Hk].cpu(), kg.cpu(), 1e-6), table.cpu(),
                             pos.cpu(), "half")
        new = at[done:]
        R.check_codes(rows_at(cache.k, new, page), rows_at(cache.k_scale, new, page), want, mag,
                      "e4m3", "row")
        done += n
    out = [torch.empty(done, Hk, D, dtype=bf, device=dev) for _ in range(2)]
    rarn.kv_cache_read(cache, pages, torch.tensor([0, done], dtype=torch.int32, device=dev), *out)
    assert ((out[1].cpu().to(R.F64) - vv).abs() <= 2.0 ** -8 * vv.abs()).all()
    assert rarn.watchdog() == 0


# Rows enough for the tensor-memory kernel: its box sizes, both pipelines' ways
# of sharing rows, types, head sizes, and segments of one tile among others.
MANY_ROWS = {
    "short and long": dict(ctx=[(37 * i) % 390 for i in range(250)],
                           new=[17 + i % 4 for i in range(250)], Hq=4, Hk=2, D=64),
    "short and long, 256 rows": dict(ctx=[(61 * i) % 700 for i in range(60)],
                                     new=[66 + i % 9 for i in range(60)], Hq=4, Hk=2, D=128),
    "page 8": dict(ctx=[300, 7], new=[30, 21], Hq=8, Hk=2, D=128, page=8, layout="tokens"),
    "page 40": dict(ctx=[333], new=[33], Hq=8, Hk=2, D=64, page=40, layout="pool"),
    "page 96": dict(ctx=[200, 95, 96], new=[9, 30, 17], Hq=8, Hk=2, D=128, page=96),
    "page 128": dict(ctx=[130, 127, 128], new=[30, 10, 20], Hq=8, Hk=1, D=128, page=128),
    "page 256": dict(ctx=[130, 500], new=[30, 12], Hq=8, Hk=2, D=64, page=256, layout="pool"),
    "f16, 256 rows": dict(ctx=[2000, 31], new=[40, 21], Hq=16, Hk=2, D=128, dt="f16"),
    "f16, 256 rows, D 64, e5m2": dict(ctx=[700, 0, 90], new=[30, 41, 20], Hq=16, Hk=2, D=64,
                                      dt="f16", fmt="e5m2", page=32),
    "e5m2, 256 rows, one scale": dict(ctx=[1300], new=[64], Hq=10, Hk=2, D=128, fmt="e5m2",
                                      mode="tensor", page=64),
    "long": dict(ctx=[9000], new=[20], Hq=4, Hk=2, D=64),
    "long, 256 rows": dict(ctx=[9000], new=[50], Hq=8, Hk=2, D=128, page=64),
}


@pytest.mark.parametrize("name", MANY_ROWS)
def test_many_rows(name):
    c = Case(**MANY_ROWS[name])
    assert rarn.plan_tree_attention(c.q.shape[0], len(c.ctx), c.Hq, c.Hk, c.D,
                                    c.page).startswith("tree.tiles")
    out = c.run()
    assert rarn.watchdog() == 0
    c.check(out)
    assert torch.equal(c.run(out=torch.zeros_like(out)), out)


@pytest.mark.parametrize("n,G,D,dt", [(2, 4, 128, "bf16"), (20, 2, 128, "bf16"),
                                      (20, 2, 64, "f16"), (40, 4, 128, "f16"),
                                      (40, 4, 64, "bf16")])
def test_scores_that_keep_growing(n, G, D, dt):
    """Keys whose scales rise along the context, so that each row's largest
    score moves up again and again, within a tile and from tile to tile."""
    c = Case([900], [n], 2 * G, 2, D, dt=dt, seed=8)
    L = 900 + n
    at = c.slots(0, L).cuda()
    grow = torch.linspace(0.2, 5.0, L, device="cuda")
    c.cache.k_scale[at // 16, :, at % 16] *= grow[:, None]
    c.check(c.run())


@pytest.mark.parametrize("n", [20, 80])
def test_missing_pages_are_hidden_from_many_rows(n):
    c = Case([300, 40], [n, 4], 4, 2, 128, mask="chain")
    full = c.table.clone()
    c.table[0, 2] = -1
    c.table[0, 9] = 1 << 30
    got = c.run().cpu()
    assert rarn.watchdog() == INDEX_BIT
    c.table = full
    vis = c.visible(0)
    vis[:, 32:48] = vis[:, 144:160] = False
    k, v = (c.values(t, s, 0, 300 + n) for t, s in ((c.cache.k, c.cache.k_scale),
                                                    (c.cache.v, c.cache.v_scale)))
    R.check_attention(got[:n], *R.attention(c.q[:n], k, v, vis, 128 ** -0.5))


@pytest.mark.parametrize("n", [20, 70])
def test_graphs_of_many_rows_on_two_streams(n):
    """Two captured calls with a workspace each, replayed at once, their
    lengths changed after the capture."""
    cases = [Case([900 - 7 * i, 40], [n, 3 + i], 8, 2, 128, seed=10 * i) for i in (1, 2)]
    made = []
    for c in cases:
        N = c.q.shape[0]
        a = dict(q=c.q.cuda(), page_table=c.table.cuda(), cache=c.cache,
                 context_lens=torch.tensor([3, 5], dtype=torch.int32, device="cuda"),
                 starts=torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"),
                 mask=c.mask.cuda(), out=torch.zeros(c.q.shape, dtype=c.dt, device="cuda"),
                 workspace=torch.empty(rarn.tree_attention_workspace_bytes(N, 2, 8, 2, 128),
                                       dtype=torch.uint8, device="cuda"))
        rarn.tree_attention(**a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rarn.tree_attention(**a)
        a["context_lens"].copy_(torch.tensor(c.ctx, dtype=torch.int32))
        a["starts"].copy_(c.starts)
        made.append((c, a, g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for _, _, g, s in made:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert rarn.watchdog() == 0
    for c, a, _, _ in made:
        c.check(a["out"])
