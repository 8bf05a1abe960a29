"""GPU tests of a step's pages and slots (kv_step, kv_trim) against a model on the host,
and of the cache's tidying (kv_cache_compact)."""
import random

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
import step_ref as R

pytestmark = pytest.mark.gpu

INDEX_BIT = 16


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make(B, width, num, page, seed=0, stride=None):
    free = list(range(num))
    random.Random(seed).shuffle(free)
    table = torch.full((B, stride or width), -1, dtype=torch.int32, device="cuda")[:, :width]
    pages = rarn.KVPages(table, ints([0] * B), ints(free), ints([num]), page)
    return pages, R.Pages(B, width, num, page, free)


def same_state(pages, model):
    assert pages.page_table.tolist() == model.table()
    assert pages.held.tolist() == [len(h) for h in model.has]
    n = int(pages.free_count)
    assert n == len(model.free) and pages.free_pages.tolist()[:n] == model.free
    assert int(pages._ticket) == 0


def check_step(pages, model, context, new, tokens, served=None):
    got = rarn.kv_step(pages, ints(context), ints(new), tokens)
    want = model.step(context, new, tokens)
    for g, w in zip(got, want[:3]):
        assert g.tolist() == w
    assert int(got[3]) == want[3] and (served is None or served == want[3])
    same_state(pages, model)
    return want


# sequences, width, page size, largest prompt: one CTA and several, a sequence to a
# thread and many, pages of one slot and odd ones
RUNS = [(1, 4, 1, 3), (1, 1, 16, 5), (3, 9, 16, 40), (7, 50, 7, 100), (64, 20, 16, 90),
        (256, 70, 16, 300), (300, 12, 24, 60), (1000, 6, 8, 20), (8192, 3, 4, 5)]


@pytest.mark.parametrize("B,width,page,prompt", RUNS)
def test_a_run_of_steps_and_trims(B, width, page, prompt):
    r = random.Random(B + width)
    num = B * width
    pages, model = make(B, width, num, page, B, width + 3)
    lens = [0] * B
    most = width * page
    for turn in range(6 if B < 1000 else 3):
        new = [min(most - n, r.randint(1, prompt) if n == 0 or r.random() < 0.2
                   else r.randint(0, 4)) for n in lens]
        tokens = sum(new) + r.choice([0, 1, 77])
        want = check_step(pages, model, lens, new, tokens, served=B)
        assert not want[4]
        # some drafts are refused, some sequences end
        lens = [0 if r.random() < 0.1 else n + (k if r.random() < 0.5 else r.randint(0, k))
                for n, k in zip(lens, new)]
        if turn % 3 != 2:       # surplus pages may also be kept for the next step
            rarn.kv_trim(pages, ints(lens))
            model.trim(lens)
            same_state(pages, model)
    rarn.kv_trim(pages, ints([0] * B))
    model.trim([0] * B)
    same_state(pages, model)
    assert int(pages.free_count) == num and sorted(pages.free_pages.tolist()) == list(range(num))
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("B", [1, 40, 700])
def test_a_trim_undoes_a_step(B):
    pages, model = make(B, 30, B * 30, 8, 1)
    r = random.Random(B)
    context = [r.randint(0, 100) for _ in range(B)]
    check_step(pages, model, [0] * B, context, sum(context))
    before = [t.clone() for t in (pages.page_table, pages.held, pages.free_pages, pages.free_count)]
    first = rarn.kv_step(pages, ints(context), ints([100] * B), 100 * B)
    rarn.kv_trim(pages, ints(context))
    after = (pages.page_table, pages.held, pages.free_pages, pages.free_count)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    again = rarn.kv_step(pages, ints(context), ints([100] * B), 100 * B)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_pages_and_rows_run_out():
    # five free pages of four slots: sequence 2 would need the sixth; the fourth, which
    # needs none, stands behind it
    pages, model = make(4, 8, 5, 4)
    check_step(pages, model, [0, 0, 0, 0], [8, 4, 9, 0], 64, served=2)
    # the same with room, then out of rows
    rarn.kv_trim(pages, ints([0] * 4))
    model.trim([0] * 4)
    check_step(pages, model, [0, 0, 0, 0], [3, 3, 3, 3], 8, served=2)
    check_step(pages, model, [3, 3, 0, 0], [1, 2, 3, 1], 7, served=4)
    check_step(pages, model, [4, 5, 3, 1], [1, 0, 0, 0], 0, served=0)
    check_step(pages, model, [4, 5, 3, 1], [0, 0, 0, 0], 0, served=4)
    assert rarn.watchdog() == 0


def test_lengths_that_make_no_sense_leave_their_sequence():
    bad = [(-1, 3), (0, -2), (5, 1), (0, 33), (2 ** 31 - 1, 2 ** 31 - 1), (0, 2 ** 31 - 1)]
    for c, n in bad:
        pages, model = make(3, 4, 20, 8)
        check_step(pages, model, [0, 0, 0], [7, 0, 9], 30)
        assert rarn.watchdog() == 0
        want = check_step(pages, model, [7, c, 9], [3, n, 2], 30, served=3)
        assert want[4] and want[0] == [0, 3, 3, 5]
        assert rarn.watchdog() == INDEX_BIT
    # an idle sequence's context is not looked at
    pages, model = make(2, 4, 20, 8)
    check_step(pages, model, [-9, 0], [0, 3], 8, served=2)
    assert rarn.watchdog() == 0


def test_a_page_outside_gets_no_slot():
    pages, model = make(2, 4, 8, 4)
    check_step(pages, model, [0, 0], [6, 5], 16)
    pages.page_table[0, 1] = 8
    pages.free_pages[3] = -7        # the next one taken
    starts, slots, positions, served = rarn.kv_step(pages, ints([6, 5]), ints([2, 4]), 8)
    assert slots.tolist()[0] == -1 and slots.tolist()[1] == -1
    assert positions.tolist() == [6, 7, 5, 6, 7, 8, 0, 0] and int(served) == 2
    assert slots.tolist()[2] >= 0 and slots.tolist()[5] == -1
    assert rarn.watchdog() == INDEX_BIT


def test_a_count_outside_serves_what_needs_no_page():
    pages, model = make(2, 4, 8, 4)
    check_step(pages, model, [0, 0], [6, 5], 16)
    for count in (-1, 9):
        pages.free_count.fill_(count)
        starts, slots, _, served = rarn.kv_step(pages, ints([6, 5]), ints([2, 4]), 8)
        assert starts.tolist() == [0, 2, 2] and int(served) == 1 and min(slots.tolist()[:2]) >= 0
        assert int(pages.free_count) == count and rarn.watchdog() == INDEX_BIT
        held = pages.held.clone()
        rarn.kv_trim(pages, ints([0, 0]))
        assert torch.equal(held, pages.held) and rarn.watchdog() == INDEX_BIT


def test_trim_keeps_what_it_cannot_read():
    pages, model = make(3, 4, 12, 4)
    check_step(pages, model, [0, 0, 0], [9, 9, 9], 30)
    rarn.kv_trim(pages, ints([2, -1, 100]))
    model.trim([2, -1, 100])
    same_state(pages, model)
    assert rarn.watchdog() == INDEX_BIT
    # more pages than there are: nothing is done
    pages.free_count.fill_(12)
    table = pages.page_table.clone()
    rarn.kv_trim(pages, ints([0, 0, 0]))
    assert torch.equal(table, pages.page_table) and int(pages.free_count) == 12
    assert rarn.watchdog() == INDEX_BIT


def test_steps_in_a_graph():
    B, page = 20, 4
    pages, model = make(B, 30, B * 30, page)
    context, new = ints([0] * B), ints([0] * B)
    out = rarn.kv_step(pages, context, new, 64)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rarn.kv_step(pages, context, new, 64, *out)
        context.add_(new)
        rarn.kv_trim(pages, context)
    lens, r = [0] * B, random.Random(3)
    for _ in range(5):
        n = [r.randint(0, 3) for _ in lens]
        new.copy_(ints(n))
        graph.replay()
        want = model.step(lens, n, 64)
        for g, w in zip(out, want[:3]):
            assert g.tolist() == w
        lens = [a + b for a, b in zip(lens, n)]
        model.trim(lens)
        same_state(pages, model)


def cache_of(pages, page, H, D, fmt, mode, layout, g):
    if layout == "tokens":      # tokens before heads, as other pools lie
        shape, back = (pages, page, H, D), (0, 2, 1, 3)
    else:
        shape, back = (pages, H, page, D), (0, 1, 2, 3)
    k, v = (torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda().permute(back)
            for _ in range(2))
    if mode == "row":
        ks, vs = (torch.rand(pages, H, page, generator=g).cuda() for _ in range(2))
    else:
        ks, vs = (torch.ones(1, device="cuda") for _ in range(2))
    return rarn.KVCache(k, v, ks, vs, fmt=fmt, scale_mode=mode)


def moved(cache, table, context, paths):
    """Copies of the cache's tensors with the rows moved, one after another."""
    page = cache.page_size
    out = {}
    for n in ("k", "v", "k_scale", "v_scale"):
        x = getattr(cache, n).cpu().clone()
        if x.dim() > 1:
            old = x.clone()
            for b, path in enumerate(paths):
                for j in range(1, len(path)):
                    s, d = context[b] + path[j], context[b] + j
                    x[table[b][d // page], :, d % page] = old[table[b][s // page], :, s % page]
        out[n] = x
    return out


def compact_case(B, nodes, H, D, page, fmt, mode, layout, seed, W=None):
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    context = [r.randint(0, 50) for _ in range(B)]
    paths = [[0] + sorted(r.sample(range(1, nodes), r.randint(0, min(nodes - 1, 40))))
             for _ in range(B)]
    need = [-(-(c + nodes) // page) for c in context]
    order = list(range(sum(need) + 2))
    r.shuffle(order)
    table = [[order.pop() for _ in range(n)] for n in need]
    width = max(need)
    cache = cache_of(sum(need) + 2, page, H, D, fmt, mode, layout, g)
    W = W or max(len(p) for p in paths) + 1
    return (cache, table, context, paths, ints([t + [-1] * (width - len(t)) for t in table]),
            ints(context), ints([p + [-1] * (W - len(p)) for p in paths]),
            ints([len(p) for p in paths]))


# sources that are targets of others, whole rows of columns to a thread, several
# batches of rows, one page a row
COMPACT = [(1, 16, 8, 128, 16, "e4m3", "row", "heads"), (5, 5, 2, 64, 1, "e5m2", "row", "tokens"),
           (17, 64, 1, 16, 7, "e4m3", "tensor", "heads"),
           (3, 100, 5, 80, 24, "e4m3", "row", "heads"),
           (40, 9, 16, 256, 16, "e5m2", "tensor", "tokens"),
           (4, 2, 3, 48, 5, "e4m3", "row", "tokens"),
           (2, 300, 8, 128, 64, "e4m3", "row", "heads")]


@pytest.mark.parametrize("B,nodes,H,D,page,fmt,mode,layout", COMPACT)
def test_compact(B, nodes, H, D, page, fmt, mode, layout):
    for seed in range(3):
        cache, table, context, paths, t, c, p, n = compact_case(B, nodes, H, D, page, fmt, mode,
                                                                layout, seed)
        want = moved(cache, table, context, paths)
        rarn.kv_cache_compact(cache, t, c, p, n)
        for name, w in want.items():
            assert torch.equal(getattr(cache, name).cpu(), w), name
    assert rarn.watchdog() == 0


def test_compact_refuses_what_does_not_rise_or_lies_outside():
    for spoil in ("fall", "same", "start", "page", "far", "length", "context"):
        cache, table, context, paths, t, c, p, n = compact_case(4, 60, 2, 32, 8, "e4m3", "row",
                                                                "heads", 9, W=41)
        paths[1] = [0, 2, 5, 6, 9, 20]
        p[1] = ints(paths[1] + [-1] * 35)
        n[1] = 6
        left = {"fall": 3, "same": 2, "start": 1}.get(spoil)
        if spoil == "fall":
            p[1, 3] = 4
        elif spoil == "same":
            p[1, 2] = 2
        elif spoil == "start":
            p[1, 0] = -1
        elif spoil == "page":
            t[1, (context[1] + 20) // 8] = 10 ** 6
            left = 5
        elif spoil == "far":
            p[1, 5] = 2 ** 31 - 1
            left = 5
        elif spoil == "length":     # beyond the path's end, which falls
            n[1] = 10 ** 6
            left = 6
        else:
            c[1] = -1
            left = 1
        paths[1] = paths[1][:left]
        want = moved(cache, table, context, paths)
        rarn.kv_cache_compact(cache, t, c, p, n)
        for name, w in want.items():
            assert torch.equal(getattr(cache, name).cpu(), w), (spoil, name)
        assert rarn.watchdog() == INDEX_BIT, spoil


def test_compact_without_work():
    cache, table, context, paths, t, c, p, n = compact_case(3, 9, 2, 32, 8, "e4m3", "row", "heads",
                                                            2)
    before = cache.k.clone()
    rarn.kv_cache_compact(cache, t, c, p, torch.zeros_like(n))
    rarn.kv_cache_compact(cache, t, c, p[:, :1].contiguous(), torch.ones_like(n))
    rarn.kv_cache_compact(cache, t[:0], c[:0], p[:0], n[:0])
    assert torch.equal(before, cache.k) and rarn.watchdog() == 0


def test_compact_pages_far_apart():
    """Pages whose offsets pass 2^31 bytes."""
    pages, H, page, D, ld = 3, 2, 4, 32, (1 << 30) + 16
    g = torch.Generator().manual_seed(1)
    kv = []
    for _ in range(2):
        d = torch.empty((pages - 1) * ld + H * page * D, dtype=torch.uint8, device="cuda")
        d = d.as_strided((pages, H, page, D), (ld, page * D, D, 1))
        d.copy_(torch.randint(0, 256, (pages, H, page, D), generator=g, dtype=torch.uint8))
        kv.append(d)
    s = [torch.rand(pages, H, page, generator=g).cuda() for _ in range(2)]
    cache = rarn.KVCache(*kv, *s)
    want = moved(cache, [[0, 2, 1]], [1], [[0, 3, 5, 10]])
    rarn.kv_cache_compact(cache, ints([[0, 2, 1]]), ints([1]), ints([[0, 3, 5, 10]]), ints([4]))
    for name, w in want.items():
        assert torch.equal(getattr(cache, name).cpu(), w), name
    assert rarn.watchdog() == 0


def test_pages_made_on_one_stream_are_used_on_another():
    s = torch.cuda.Stream()
    for _ in range(20):
        pages, model = make(300, 12, 3600, 16)
        torch.cuda.synchronize()
        held = torch.full((300,), 100, dtype=torch.int32, device="cuda")
        zero = torch.zeros_like(held)
        s.wait_stream(torch.cuda.current_stream())
        pages = rarn.KVPages(pages.page_table, pages.held, pages.free_pages, pages.free_count, 16)
        with torch.cuda.stream(s):
            out = rarn.kv_step(pages, zero, held, 30000)
        s.synchronize()
        want = model.step([0] * 300, [100] * 300, 30000)
        assert out[0].tolist() == want[0] and out[1].tolist() == want[1]
        same_state(pages, model)
