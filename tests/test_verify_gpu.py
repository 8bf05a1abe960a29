"""GPU tests of the verification of drafted tokens (verify_drafts) against binary64."""
import random

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
import step_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INDEX_BIT = 16


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def starts_of(rows):
    at = [0]
    for n in rows:
        at.append(at[-1] + n)
    return at


def run(probs, tokens, starts, u, v, most, q=None, parents=None, **kw):
    def dev(x, dt):
        return torch.tensor(x, dtype=dt, device="cuda")
    got = rarn.verify_drafts(probs.cuda(), dev(tokens, torch.int64), dev(starts, torch.int32),
                             u.cuda(), v.cuda(), most,
                             draft_probs=None if q is None else q.cuda(),
                             parents=None if parents is None else dev(parents, torch.int32), **kw)
    return tuple(x.tolist() for x in got)


def inputs(rows, V, dt, kind, seed, sharp=2.5):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    N = sum(rows)
    logits = sharp * torch.randn(N, V, generator=g)
    probs = torch.softmax(logits, -1).to(dt)
    near = logits + 0.7 * torch.randn(N, V, generator=g)
    parents, above, rank = [], [], []
    for b, n in enumerate(rows):
        mine = [-1 if i == 0 else r.randrange(max(0, i - 5), i) if kind == "tree" else i - 1
                for i in range(n)]
        above += [len(parents) + max(p, 0) for p in mine]
        rank += [mine[:i].count(p) for i, p in enumerate(mine)]
        parents += mine
    q = None
    if kind == "drawn":
        q = torch.softmax(near, -1).to(dt)[above]
        tokens = torch.multinomial(q.float(), 1, generator=g)[:, 0].tolist()
    else:
        best = near.topk(min(V, max(rank) + 1), -1).indices
        tokens = [int(best[a, min(k, best.shape[1] - 1)]) for a, k in zip(above, rank)]
    u, v = torch.rand(N, generator=g), torch.rand(len(rows), generator=g)
    return probs, tokens, starts_of(rows), u, v, q, parents if kind == "tree" else None


# rows of each sequence and the vocabulary: one token, one sequence, clusters of every
# size, odd vocabularies, a group's ends, sequences without rows
SHAPES = [([1], 1), ([5], 2), ([3, 0, 7, 1], 50257), ([6], 32000), ([4, 1, 5], 1023),
          ([2, 9], 1024), ([3, 3], 1025), ([12] * 3, 5000), ([2, 1, 3] * 30, 8200),
          ([3] * 200, 1000), ([2, 4] * 260, 333), ([64], 2000), ([40, 33, 50], 128256),
          ([2], 1 << 20), ([1, 2] * 40, 40001)]


@pytest.mark.parametrize("kind", ["drawn", "chosen", "tree"])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shapes(shape, dt, kind):
    rows, V = SHAPES[shape]
    probs, tokens, starts, u, v, q, parents = inputs(rows, V, DT[dt], kind, shape)
    for most in {max(max(rows) - 1, 0), 3}:
        want = R.verify(probs, tokens, starts, u, v, most, q, parents)
        assert run(probs, tokens, starts, u, v, most, q, parents) == want
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("kind", ["drawn", "chosen", "tree"])
@pytest.mark.parametrize("sharp", [0.0, 0.5, 12.0])
def test_flat_and_peaked_rows(kind, sharp):
    rows = [9] * 12
    for V in (997, 32000):
        probs, tokens, starts, u, v, q, parents = inputs(rows, V, torch.float32, kind, 5, sharp)
        want = R.verify(probs, tokens, starts, u, v, 8, q, parents)
        assert run(probs, tokens, starts, u, v, 8, q, parents) == want
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("kind", ["drawn", "tree"])
def test_the_largest_tree_and_long_chains(kind):
    rows = [1024, 3] if kind == "tree" else [3000, 3]
    probs, tokens, starts, u, v, q, parents = inputs(rows, 50, torch.float32, kind, 8, 6.0)
    if kind == "drawn":     # all accepted: as far as the path is long
        q = probs[[max(i - 1, 0) for i in range(3003)]]
        tokens = q.argmax(-1).tolist()
        u = u * 0.99
    for most in (5, 1023, 4000):
        want = R.verify(probs, tokens, starts, u, v, most, q, parents)
        assert run(probs, tokens, starts, u, v, most, q, parents) == want
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("V", [7, 2500])
def test_all_accepted_all_refused_and_nothing_left(V):
    probs = torch.softmax(torch.randn(4, V, generator=torch.Generator().manual_seed(V)), -1)
    top = probs.argmax(-1).tolist()
    tokens, starts = [0] + top[:3], [0, 4]
    one, zero = torch.zeros(4), torch.full((4,), 0.999999)
    v = torch.tensor([0.5])
    assert run(probs, tokens, starts, one, v, 3)[2] == [4]
    got = run(probs, tokens, starts, zero, v, 3)
    assert got[2] == [1] and got == R.verify(probs, tokens, starts, zero, v, 3)
    # the draft's distribution covers the target's everywhere: refused, p itself is drawn
    q = (probs * 1.5)[[0, 0, 1, 2]]
    want = R.verify(probs, tokens, starts, zero, v, 3, q)
    assert run(probs, tokens, starts, zero, v, 3, q) == want and want[2] == [1]
    # one token has everything: below it nothing is left without it
    sure = torch.zeros(2, V)
    sure[:, 3] = 1
    got = run(sure, [0, 3], [0, 2], torch.tensor([0.5, 0.5]), v, 0)
    assert got == ([[3]], [[0]], [1])
    assert rarn.watchdog() == 0


def test_a_token_drafted_twice_counts_once():
    p = torch.tensor([[0.25, 0.25, 0.5, 0.0], *[[0.25] * 4] * 4])
    tokens, parents = [0, 1, 1, 2, 3], [-1, 0, 0, 0, 0]
    for number, row in ((0.0, 1), (0.2499, 1), (0.25, 3), (0.7499, 3), (0.75, None), (0.99, None)):
        u = torch.full((5,), number)
        got = run(p, tokens, [0, 5], u, torch.tensor([0.9]), 2, None, parents)
        assert got == R.verify(p, tokens, [0, 5], u, torch.tensor([0.9]), 2, None, parents)
        assert got[2] == [1 if row is None else 2]
        if row is None:
            assert got[0][0][0] == 0    # all but token 0 were tried
        else:
            assert got[1][0][1] == row
    assert rarn.watchdog() == 0


def test_borders_of_the_draw():
    """Weights that binary32 sums would lose: the draw is that of the exact sums."""
    V = 4096
    p = torch.full((1, V), 2.0 ** -40)
    p[0, 0], p[0, V - 1] = 0.5, 0.25
    total = 0.75 + (V - 2) * 2.0 ** -40
    for v, x in ((0.0, 0), (0.5 / total * (1 - 2.0 ** -22), 0),
                 (0.99999994, V - 1), ((0.5 + 2.0 ** -29) / total, None)):
        vt = torch.tensor([v], dtype=torch.float32)
        got = run(p, [0], [0, 1], torch.zeros(1), vt, 0)[0][0][0]
        want = R.verify(p, [0], [0, 1], torch.zeros(1), vt, 0)[0][0][0]
        assert got == want and (x is None or got == x)
    # tokens without weight are never drawn
    p = torch.zeros(1, 3000)
    p[0, [5, 2047, 2999]] = torch.tensor([0.25, 0.5, 0.25])
    for v, x in ((0.0, 5), (0.2499, 5), (0.25, 2047), (0.7499, 2047), (0.75, 2999), (0.999, 2999)):
        assert run(p, [0], [0, 1], torch.zeros(1), torch.tensor([v]), 0)[0] == [[x]]
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("kind", ["drawn", "tree"])
def test_the_first_token_has_the_targets_distribution(kind):
    """Over a grid of random numbers, and over the draft's own distribution, the first
    new token comes as often as the target says."""
    K, V = 64, 5
    p = torch.tensor([0.40, 0.05, 0.25, 0.20, 0.10])
    q = torch.tensor([0.10, 0.30, 0.25, 0.05, 0.30])
    grid = (torch.arange(K) + 0.5) / K
    u, v = torch.meshgrid(grid, grid, indexing="ij")
    u, v = u.flatten(), v.flatten()
    n, freq = K * K, torch.zeros(V, dtype=torch.float64)
    cases = [([x], float(q[x])) for x in range(V)] if kind == "drawn" else [([3, 0, 1], 1.0)]
    for drafts, weight in cases:
        m = 1 + len(drafts)
        out = run(p.expand(n * m, V).contiguous(), [0, *drafts] * n, list(range(0, n * m + 1, m)),
                  u.repeat_interleave(m), v, 1,
                  q.expand(n * m, V).contiguous() if kind == "drawn" else None,
                  None if kind == "drawn" else [-1, 0, 0, 0] * n)
        first = torch.tensor([t[0] for t in out[0]])
        freq += weight * torch.bincount(first, minlength=V).double() / n
    # a border moves a grid of K points by one at most, in each of two numbers
    assert (freq - p.double()).abs().max() <= 2 / K
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_and_misaligned_rows(dt):
    rows, V = [5, 4], 3000
    for kind in ("drawn", "tree"):
        probs, tokens, starts, u, v, q, parents = inputs(rows, V, DT[dt], kind, 4)
        want = R.verify(probs, tokens, starts, u, v, 4, q, parents)
        for pad, shift in ((8, 0), (3, 0), (8, 1)):
            def place(x):
                if x is None:
                    return None
                b = torch.full((sum(rows), V + pad + 8), 9.0, dtype=x.dtype)
                b[:, shift:shift + V] = x
                return b.cuda()[:, shift:shift + V]
            assert run(place(probs), tokens, starts, u, v, 4, place(q), parents) == want
    assert rarn.watchdog() == 0


def test_indices_outside():
    probs, tokens, starts, u, v, _, _ = inputs([4, 4], 100, torch.float32, "chosen", 6)
    u = torch.zeros(8)
    tokens[2] = 100             # accepted up to it; nothing is refused in its place
    got = run(probs, tokens, starts, u, v, 3)
    assert got == R.verify(probs, tokens, starts, u, v, 3) and got[2] == [2, 4]
    assert rarn.watchdog() == INDEX_BIT
    tokens[2] = -5
    assert run(probs, tokens, starts, u, v, 3, probs)[2] == [2, 4]
    assert rarn.watchdog() == INDEX_BIT
    for parent in (-1, 2, 3, 10 ** 6):      # row 2 is then no one's child
        tokens[2] = 1
        parents = [-1, 0, parent, 1] * 2
        got = run(probs, tokens, starts, u, v, 3, None, parents)
        want = R.verify(probs, tokens, starts, u, v, 3, None, [-1, 0, -1, 1] * 2)
        assert got == want
        assert rarn.watchdog() == INDEX_BIT
    for bad in ([-1, 4, 8], [0, 9, 8], [0, 4, 9], [5, 4, 8]):
        got = run(probs, [1] * 8, bad, u, v, 3)
        for b in range(2):
            if not 0 <= bad[b] <= bad[b + 1] <= 8:
                assert got[2][b] == 0 and got[0][b] == [-1] * 4 and got[1][b] == [-1] * 4
        assert rarn.watchdog() == INDEX_BIT
    big = torch.full((1025, 4), 0.25)
    got = run(big, [0] * 1025, [0, 1025], torch.zeros(1025), v[:1], 2, None, [-1] + [0] * 1024)
    assert got[2] == [0] and rarn.watchdog() == INDEX_BIT


def test_rows_that_are_no_distribution():
    V, z = 3000, torch.zeros(1)
    for p in (torch.zeros(1, V), torch.ones(1, V), torch.full((1, V), float("nan")),
              torch.full((1, V), float("inf")), torch.full((1, V), -1.0),
              torch.full((1, V), 2.0 / V + 1e-6)):
        for dt in DT.values():
            assert run(p.to(dt), [0], [0, 1], z, z + 0.5, 0) == ([[-1]], [[0]], [1])
            assert rarn.watchdog() == INDEX_BIT
    # NaN and negative values weigh nothing
    p = torch.full((1, V), float("nan"))
    p[0, 7], p[0, 9], p[0, 2222] = 0.5, -3.0, 0.5
    assert run(p, [0], [0, 1], z, z + 0.6, 0)[0] == [[2222]]
    assert rarn.watchdog() == 0


def test_no_sequences_and_no_rows():
    e = torch.empty(0, 10, device="cuda")
    got = run(e, [], [0], torch.empty(0), torch.empty(0), 2)
    assert got == ([], [], [])
    got = run(e, [], [0, 0, 0], torch.empty(0), torch.zeros(2), 1)
    assert got == ([[-1, -1]] * 2, [[-1, -1]] * 2, [0, 0])


def test_in_a_graph_and_on_a_stream():
    rows, V = [5] * 9, 5000
    a = inputs(rows, V, torch.float32, "drawn", 1)
    b = inputs(rows, V, torch.float32, "drawn", 2)
    dev = [x.cuda() if torch.is_tensor(x) else torch.tensor(x, device="cuda") for x in
           (a[0], a[1], a[3], a[4], a[5])]
    st = torch.tensor(a[2], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = rarn.verify_drafts(dev[0], dev[1], st, dev[2], dev[3], 4, draft_probs=dev[4])
    torch.cuda.current_stream().wait_stream(s)
    assert tuple(x.tolist() for x in out) == R.verify(*a[:5], 4, a[5])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rarn.verify_drafts(dev[0], dev[1], st, dev[2], dev[3], 4, draft_probs=dev[4],
                           new_tokens=out[0], path=out[1], lengths=out[2])
    for x, y in zip(dev, (b[0], torch.tensor(b[1]), b[3], b[4], b[5])):
        x.copy_(y)
    graph.replay()
    assert tuple(x.tolist() for x in out) == R.verify(*b[:5], 4, b[5])


def test_rows_far_apart():
    """Probabilities whose offsets pass 2^31 elements, of p and of q."""
    rows, V, ld = [3], 5000, (1 << 30) + 8
    for kind in ("drawn", "tree"):
        probs, tokens, starts, u, v, q, parents = inputs(rows, V, torch.bfloat16, kind, 3)
        want = R.verify(probs, tokens, starts, u, v, 2, q, parents)
        far = []
        for x in (probs, q):
            if x is None:
                far.append(None)
                continue
            d = torch.empty(2 * ld + V, dtype=x.dtype, device="cuda").as_strided((3, V), (ld, 1))
            d.copy_(x)
            far.append(d)
        assert run(far[0], tokens, starts, u, v, 2, far[1], parents) == want
        del far


def test_two_streams_at_once():
    ins = [inputs([4] * 40, 20000, torch.float32, "drawn", s) for s in (1, 2)]
    dev = [[x.cuda() if torch.is_tensor(x) else torch.tensor(x, device="cuda") for x in
            (i[0], i[1], i[3], i[4], i[5])] for i in ins]
    st = torch.tensor(ins[0][2], dtype=torch.int32, device="cuda")
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                d = dev[k]
                outs[k].append(rarn.verify_drafts(d[0], d[1], st, d[2], d[3], 3, draft_probs=d[4]))
    torch.cuda.synchronize()
    for i, got in zip(ins, outs):
        want = R.verify(*i[:5], 3, i[5])
        assert all(tuple(x.tolist() for x in g) == want for g in got)
