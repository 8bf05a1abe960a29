"""Timed cases of a serving step of drafted tokens: page tables and slots from the
sequences' lengths, per-head norms with positions of several axes (and the cache's
write), the norms before and after a block with its gate and residual scale, the
verification of the drafts, and the cache's tidying after it.

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU
from a seed, ``run`` makes one pass: through the package's entry points where
``own`` is true, in plain torch (binary32, binary64 for sums that decide a whole
number, one rounding at the end) otherwise.  ``exact`` is the same definition
in binary64.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
POSITIONS = 16384


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _block(name, T, H, gates, dt, wide, post, scale):
    return {"name": name, "op": "block", "T": T, "H": H, "gates": gates, "dt": dt, "wide": wide,
            "post": post, "scale": scale}


def _axes(name, T, Hq, Hk, D, rot, dt, style, order, axes, fmt, mode, page):
    return {"name": name, "op": "axes", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot, "dt": dt,
            "style": style, "order": order, "axes": axes, "fmt": fmt, "mode": mode, "page": page}


def _step(name, B, context, new, page, lens):
    return {"name": name, "op": "step", "B": B, "context": context, "new": new, "page": page,
            "lens": lens}


def _verify(name, B, rows, V, dt, drafted, tree, lens):
    return {"name": name, "op": "verify", "B": B, "rows": rows, "V": V, "dt": dt,
            "drafted": drafted, "tree": tree, "lens": lens}


def _compact(name, B, rows, Hk, D, fmt, mode, page, lens):
    return {"name": name, "op": "compact", "B": B, "rows": rows, "Hk": Hk, "D": D, "fmt": fmt,
            "mode": mode, "page": page, "lens": lens}


def listed():
    return [
        # the norms around a block for one decoded token: latency
        _block("block_1", 1, 4096, 0, "bf16", False, True, 1.0),
        # a mixed batch of odd length, a modulating gate for each of nine requests, a binary32
        # residual stream
        _block("block_517_gates", 517, 5120, 9, "bf16", True, True, 0.5),
        # a long prefill batch, one learned gate for all tokens
        _block("block_16384", 16384, 5120, 1, "bf16", False, True, 0.22),
        # a decode batch of a model of images and text: three axes in blocks, cache written
        _axes("axes_write_128", 128, 32, 8, 128, 128, "bf16", "half", "blocks", 3, "e4m3", "row",
              16),
        # a video's prompt, axes taken in turn, queries and keys only
        _axes("axes_8192", 8192, 64, 8, 128, 128, "bf16", "half", "cyclic", 3, "", "", 0),
        # a small decode batch: a token or two each, now and then a page
        _step("step_8", 8, 2000, 2, 16, 1),
        # a large batch of prompts and decodes
        _step("step_256", 256, 4096, 1024, 16, 2),
        # one sequence's chain of four drafts, deterministic draft model
        _verify("verify_1", 1, 5, 32000, "f32", False, False, 3),
        # a batch of chains drafted by sampling: target and draft probabilities
        _verify("verify_64", 64, 6, 128256, "f32", True, False, 4),
        # trees of up to 32 tokens, an odd vocabulary, 16-bit probabilities
        _verify("verify_tree_16", 16, 32, 50257, "bf16", False, True, 5),
        # one tree's accepted tokens moved together
        _compact("compact_1", 1, 16, 8, 128, "e4m3", "row", 16, 6),
        # the same for a large batch of wide trees
        _compact("compact_256", 256, 64, 8, 128, "e4m3", "row", 16, 7),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["block", "axes", "step", "verify", "verify", "compact"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    fmt, mode = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["row", "row", "tensor"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    lens = rng.randrange(1 << 20)
    if op == "block":
        H = rng.choice([512, 1000, 1592, 2048, 4096, 5120, 7168, 8192, 16384, rng.randint(1, 9000)])
        T = _log(rng, 1, min(16384, (1 << 25) // H))
        gates = rng.choice([0, 1, T, min(T, 7), min(T, 64)])
        c = _block("", T, H, gates, dt, dt != "f32" and rng.random() < 0.3, rng.random() < 0.8,
                   rng.choice([1.0, 0.5, 0.22]))
    elif op == "axes":
        Hq, Hk = rng.choice([(32, 8), (64, 8), (40, 8), (28, 4), (16, 16), (16, 1), (5, 5)])
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rot = rng.choice([D, D, D // 2 // 8 * 8, 32])
        write = rng.random() < 0.5
        T = _log(rng, 1, min(8192, (1 << 25) // ((Hq + 2 * Hk) * D)))
        c = _axes("", T, Hq, Hk, D, rot, dt, rng.choice(["half", "interleaved"]),
                  rng.choice(["blocks", "cyclic"]), rng.choice([2, 3, 3, 4]),
                  *((fmt, mode, page) if write else ("", "", 0)))
    elif op == "step":
        B = _log(rng, 1, 256)
        c = _step("", B, _log(rng, 1, 4096), _log(rng, 1, min(4096, (1 << 18) // B)), page, lens)
    elif op == "verify":
        tree = rng.random() < 0.4
        rows = rng.randint(1, 48) if tree else rng.randint(1, 12)
        V = rng.choice([32000, 50257, 102400, 128256, 151936, rng.randint(2, 99999)])
        B = _log(rng, 1, max(1, min(256, (1 << 25) // (rows * V))))
        c = _verify("", B, rows, V, dt, not tree and rng.random() < 0.6, tree, lens)
    else:
        Hk, D = rng.choice([1, 2, 4, 8, 8, 16]), rng.choice([64, 80, 128, 128, 256])
        rows = rng.randint(3, 64)
        c = _compact("", _log(rng, 1, min(256, (1 << 25) // (rows * Hk * D))), rows, Hk, D, fmt,
                     mode, page, lens)
    del c["name"]
    return c


def _counts(c, most, salt, least=1):
    """A number for each sequence, `least` to `most`, the largest there."""
    r = random.Random(c["lens"] + salt)
    got = [most if b == 0 else r.randint(min(least, most), most) for b in range(c["B"])]
    r.shuffle(got)
    return got


def _news(c):
    """New tokens of each sequence: most decode one or two, one in eight brings a prompt."""
    r = random.Random(c["lens"] + 9)
    few = min(2, c["new"])
    got = [c["new"] if b == 0 else r.randint(1, c["new"]) if r.random() < 0.125
           else r.randint(0, few) for b in range(c["B"])]
    r.shuffle(got)
    return got


def _paths(c):
    """Kept rows of each sequence's tree: row 0, then rows behind those that they move to (a
    tree laid level by level whose first branches were refused)."""
    r = random.Random(c["lens"] + 11)
    got = []
    for n in _counts(c, c["rows"], 10, 3):
        m = r.randint(1, max(1, min(7, (n - 1) // 2)))
        got.append([0] + sorted(r.sample(range(m + 1, n), min(m, n - m - 1))))
    return got


def work(case):
    c = case
    if c["op"] == "block":
        T, H, s, w = c["T"], c["H"], SIZES[c["dt"]], 4 if c["wide"] else SIZES[c["dt"]]
        n = 2 * T * H * (s + w) + (c["gates"] + 2) * H * s
        return {"bytes": n + (4 * T if 1 < c["gates"] < T else 0), "flops": 10 * T * H}
    if c["op"] == "axes":
        T, D, Hq, Hk, s = c["T"], c["D"], c["Hq"], c["Hk"], SIZES[c["dt"]]
        n = 2 * T * Hq * D * s + T * (c["rot"] * 4 + 8 * c["axes"]) + 2 * D * s
        if not c["fmt"]:
            return {"bytes": n + 2 * T * Hk * D * s, "flops": 8 * T * (Hq + Hk) * D}
        n += 2 * T * Hk * (D * (s + 1) + (4 if c["mode"] == "row" else 0)) + 8 * T
        return {"bytes": n, "flops": 8 * T * (Hq + 2 * Hk) * D}
    if c["op"] == "step":
        new, page = sum(_news(c)), c["page"]
        return {"bytes": 20 * c["B"] + 16 * new + 16 * (new // page), "flops": 4 * new}
    if c["op"] == "verify":
        s = SIZES[c["dt"]]
        n = sum(_counts(c, c["rows"], 1))
        return {"bytes": c["B"] * c["V"] * s * (2 if c["drafted"] else 1) + n * (8 + 4 + 2 * s),
                "flops": 2 * c["B"] * c["V"]}
    moved = sum(len(p) - 1 for p in _paths(c))
    row = 2 * c["Hk"] * (c["D"] + (4 if c["mode"] == "row" else 0))
    return {"bytes": 2 * moved * row + 8 * moved + 12 * c["B"], "flops": 0}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _sections(c):
    """Pairs of each axis: a quarter to the first (time), the rest shared."""
    n, axes = c["rot"] // 2, c["axes"]
    if axes == 2:
        return (n // 2, n - n // 2)
    first = n // 4
    rest = (n - first) // (axes - 1)
    return (n - rest * (axes - 1),) + (rest,) * (axes - 1)


def _axis_of_pair(c):
    """The axis of each pair: block after block, or the axes in turn while they have pairs."""
    left = list(_sections(c))
    if c["order"] == "blocks":
        return [a for a, n in enumerate(left) for _ in range(n)]
    got = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                got.append(a)
                left[a] -= 1
    return got


def _cache(c, pages, g, filled):
    """An 8-bit cache of `pages` pages; `filled`: of random codes and scales."""
    shape, got = (pages, c["Hk"], c["page"], c["D"]), {}
    for n in "kv":
        if filled:      # finite codes of either format
            got[n] = torch.randint(0, 120, shape, device="cuda", generator=g, dtype=torch.uint8)
        else:
            got[n] = torch.zeros(shape, dtype=torch.uint8, device="cuda")
        if c["mode"] == "tensor":
            got[n + "_scale"] = torch.full((1,), 8.0 / LARGEST[c["fmt"]], device="cuda")
        elif filled:
            got[n + "_scale"] = torch.rand(shape[:3], device="cuda", generator=g) + 0.1
        else:
            got[n + "_scale"] = torch.ones(shape[:3], device="cuda")
    return got


def _table(need, width, g):
    """Pages of each sequence in an order of their own, [B, width]; unused entries are -1."""
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    rows = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    rows[torch.arange(width, device="cuda")[None] < _ints(need)[:, None]] = order
    return rows


def prepare(case, seed):
    c, g = case, _generator(seed)
    return {"block": _prepare_block, "axes": _prepare_axes, "step": _prepare_step,
            "verify": _prepare_verify, "compact": _prepare_compact}[c["op"]](c, g, {"case": c})


def _prepare_block(c, g, s):
    T, H, dt = c["T"], c["H"], TYPES[c["dt"]]
    wide = torch.float32 if c["wide"] else dt

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    # a block's output: rows of different sizes; the stream it joins
    s["x"] = (normal(T, H) * torch.exp(normal(T, 1))).to(dt)
    s["residual"] = (2.0 * normal(T, H)).to(wide)
    for n in ("x_gamma", "gamma"):
        s[n] = (torch.rand(H, device="cuda", generator=g) + 0.5).to(dt)
    if not c["post"]:
        s["x_gamma"] = None
    s["gate"] = (0.5 * normal(c["gates"], H)).to(dt) if c["gates"] else None
    if 1 < c["gates"] < T:
        s["gate_index"] = (torch.arange(T, device="cuda") * c["gates"] // T).to(torch.int32)
    else:
        s["gate_index"] = None
    s["h"] = torch.empty(T, H, dtype=wide, device="cuda")
    s["out"] = torch.empty(T, H, dtype=dt, device="cuda")
    return s


def _prepare_axes(c, g, s):
    T, Hq, Hk, D, dt = c["T"], c["Hq"], c["Hk"], c["D"], TYPES[c["dt"]]
    qkv = torch.randn(T, Hq + 2 * Hk, D, device="cuda", generator=g)
    qkv = (qkv * torch.exp(torch.randn(T, 1, 1, device="cuda", generator=g) * 0.5)).to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    for n in ("q_gamma", "k_gamma"):
        s[n] = (torch.rand(D, device="cuda", generator=g) + 0.5).to(dt)
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    a = torch.arange(POSITIONS, device="cuda", dtype=torch.float64)[:, None] * f
    s["table"] = torch.cat([a.cos(), a.sin()], 1).float()
    # patches of frames of 24 rows of 32, behind a text of some length
    t = torch.arange(T, device="cuda")
    first = torch.randint(0, 4000, (1,), device="cuda", generator=g)
    grid = [t // 768, t // 32 % 24, t % 32, t % 7]
    s["positions"] = torch.stack([first + x for x in grid[:c["axes"]]]).contiguous()
    s["pairs"] = _ints(_axis_of_pair(c), torch.int64)
    s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    s["k_out"] = torch.empty(T, Hk, D, dtype=dt, device="cuda")
    if c["fmt"]:
        pages = -(-T // c["page"]) + 2
        s["cache"] = _cache(c, pages, g, False)
        order = torch.randperm(pages, device="cuda", generator=g)
        s["slots"] = order[t // c["page"]] * c["page"] + t % c["page"]
    return s


def _prepare_step(c, g, s):
    ctx, new, page = _counts(c, c["context"], 8), _news(c), c["page"]
    held = [-(-n // page) for n in ctx]
    need = [-(-(a + n) // page) - h if n else 0 for a, n, h in zip(ctx, new, held)]
    s["width"] = max(h + n for h, n in zip(held, need)) + 1
    pages = sum(held) + sum(need) + 5
    table = _table(held, s["width"], g)
    free = sum(held) + torch.randperm(pages - sum(held), generator=g, device="cuda")
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    s["free"][:free.numel()] = free.to(torch.int32)
    s["count"] = _ints([free.numel()])
    s["table"], s["held"] = table, _ints(held)
    s["context_lens"], s["new_lens"] = _ints(ctx), _ints(new)
    s["tokens"] = -(-sum(new) // 64) * 64 or 64      # the step's rows, padded as a graph has them
    s["starts"] = torch.empty(c["B"] + 1, dtype=torch.int32, device="cuda")
    s["served"] = torch.empty(1, dtype=torch.int32, device="cuda")
    s["slots"] = torch.empty(s["tokens"], dtype=torch.int64, device="cuda")
    s["positions"] = torch.empty(s["tokens"], dtype=torch.int64, device="cuda")
    return s


def _prepare_verify(c, g, s):
    rows, V, dt = _counts(c, c["rows"], 1), c["V"], TYPES[c["dt"]]
    N, B = sum(rows), c["B"]
    s["starts"] = _starts(rows)
    logits = 2.5 * torch.randn(N, V, device="cuda", generator=g)
    s["probs"] = torch.softmax(logits, -1).to(dt)
    logits += 0.7 * torch.randn(N, V, device="cuda", generator=g)
    r = random.Random(c["lens"] + 2)
    parents = [[-1 if i == 0 else r.randrange(max(0, i - 6), i) if c["tree"] else i - 1
                for i in range(n)] for n in rows]
    at = [i - p if p >= 0 else 0 for row in parents for i, p in enumerate(row)]
    above = torch.arange(N, device="cuda") - _ints(at, torch.int64)  # each row's parent's row
    if c["drafted"]:
        q = torch.softmax(logits, -1).to(dt)[above]     # row i: what row i's token was drawn from
        s["draft_probs"] = q
        s["tokens"] = torch.multinomial(q.float(), 1, generator=g)[:, 0]
    else:                                               # a parent's most likely tokens in turn
        s["draft_probs"] = None
        rank = [row[:i].count(p) for row in parents for i, p in enumerate(row)]
        best = logits.topk(min(V, max(rank) + 1), -1).indices
        s["tokens"] = best[above, _ints(rank, torch.int64).clamp_max(best.shape[1] - 1)]
    del logits
    s["parents"] = _ints([p for row in parents for p in row]) if c["tree"] else None
    s["uniforms"] = torch.rand(N, device="cuda", generator=g)
    s["final_uniforms"] = torch.rand(B, device="cuda", generator=g)
    s["most"] = min(c["rows"] - 1, 8)
    W = s["most"] + 1
    s["new_tokens"] = torch.empty(B, W, dtype=torch.int64, device="cuda")
    s["path"] = torch.empty(B, W, dtype=torch.int32, device="cuda")
    s["lengths"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


def _prepare_compact(c, g, s):
    paths, page = _paths(c), c["page"]
    ctx, rows = _counts(c, 300, 12), _counts(c, c["rows"], 10, 3)
    need = [-(-(a + n) // page) for a, n in zip(ctx, rows)]
    s["cache"] = _cache(c, sum(need), g, True)
    s["block_table"] = _table(need, max(need), g)
    s["context_lens"] = _ints(ctx)
    W = max(len(p) for p in paths)
    s["path"] = _ints([p + [-1] * (W - len(p)) for p in paths])
    s["lengths"] = _ints([len(p) for p in paths])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _norm(x, gamma):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()


def _block_pass(s, c):
    n = s["x"].float() if s["x_gamma"] is None else _norm(s["x"], s["x_gamma"])
    if s["gate"] is not None:
        n = n * (s["gate"] if s["gate_index"] is None else s["gate"][s["gate_index"].long()]).float()
    h = (s["residual"].float() + c["scale"] * n).to(s["residual"].dtype)
    return h, _norm(h, s["gamma"]).to(s["x"].dtype)


def _rotate(x, table, positions, pairs, style):
    half = pairs.numel()
    i = torch.arange(half, device="cuda")
    row = positions[pairs].t()                          # [T, half]: each pair's own position
    cos, sin = table[row, i][:, None], table[row, half + i][:, None]
    if style == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _store(x, slots, cache, n, c):
    """Rows of x quantised into the cache's slots."""
    top = LARGEST[c["fmt"]]
    page, at = slots // c["page"], slots % c["page"]
    if c["mode"] == "row":
        most = x.abs().amax(-1)
        scale = torch.where(most > 0, most / top, torch.ones_like(most))
        cache[n + "_scale"][page, :, at] = scale
        u = x / scale[..., None]
    else:
        u = x / cache[n + "_scale"]
    cache[n][page, :, at] = u.clamp(-top, top).to(CODES[c["fmt"]]).view(torch.uint8)


def _cached(s, c):
    n = s["cache"]
    got = {"k": n["k"].view(CODES[c["fmt"]]), "v": n["v"].view(CODES[c["fmt"]])}
    if c["mode"] == "row":
        got.update(k_scale=n["k_scale"], v_scale=n["v_scale"])
    return got


def _axes_pass(s, c):
    q, k = (_rotate(_norm(s[n], s[n + "_gamma"]), s["table"], s["positions"], s["pairs"],
                    c["style"]) for n in "qk")
    dt = s["q"].dtype
    if not c["fmt"]:
        return {"q": q.to(dt), "k": k.to(dt)}
    _store(k, s["slots"], s["cache"], "k", c)
    _store(s["v"].float(), s["slots"], s["cache"], "v", c)
    return {"q": q.to(dt), **{"cache_" + n: x for n, x in _cached(s, c).items()}}


def _step_pass(s, c):
    """The step's pages, slots and positions; then its new tokens are taken back (all drafts
    refused) and their pages returned, so that a pass ends as it began."""
    page, tokens = c["page"], s["tokens"]
    ctx, new, held = (s[n].long() for n in ("context_lens", "new_lens", "held"))
    free, count, table = s["free"], s["count"].long(), s["table"]
    B, width = table.shape
    need = torch.where(new > 0, (ctx + new + page - 1) // page - held, 0).clamp_min(0)
    fits = (new.cumsum(0) <= tokens) & (need.cumsum(0) <= count)
    served = fits.long().cumprod(0)
    new, need = new * served, need * served
    ends = new.cumsum(0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    j = torch.arange(width, device="cuda")
    order = (need.cumsum(0) - need - held)[:, None] + j
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None])
    table = torch.where(fresh, free[(count - 1 - order).clamp(0, free.numel() - 1)], table)
    row = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(ends, row, right=True).clamp_max(B - 1)
    live = row < ends[-1]
    pos = torch.where(live, ctx[b] + row - starts[b], 0)
    slots = torch.where(live, table[b, pos // page].long() * page + pos % page, -1)
    held, count = held + need, count - need.sum()

    keep = torch.minimum(held, (ctx + page - 1) // page)
    gone = held - keep
    order = (gone.cumsum(0) - gone - keep)[:, None] + j
    back = (j >= keep[:, None]) & (j < held[:, None])
    count = count + gone.sum()
    at = torch.where(back, count - 1 - order, free.numel())
    longer = torch.cat([free, free[:1]])                # one more for what does not go back
    longer[at.flatten()] = table.flatten()
    s["free"].copy_(longer[:-1])
    s["table"].copy_(torch.where(back, -1, table))
    s["held"].copy_(keep)
    s["count"].copy_(count)
    return {"starts": starts.int(), "slots": slots, "positions": pos,
            "served": served.sum().int().view(1), "table": s["table"], "held": s["held"],
            "free": s["free"], "count": s["count"]}


def _verify_pass(s, c):
    starts, n, V = s["starts"].long(), c["rows"], c["V"]
    N, B, W = s["probs"].shape[0], c["B"], s["most"] + 1
    i = torch.arange(n, device="cuda")
    rows = (starts[:-1, None] + i).clamp_max(N - 1)
    live = i < (starts[1:] - starts[:-1])[:, None]
    drafts = live & (i > 0)
    tok = s["tokens"][rows]
    up = (s["parents"].long()[rows] if c["tree"] else (i - 1).expand(B, n)).clamp(0, n - 1)
    above = rows.gather(1, up)
    p, u = s["probs"][above, tok].double(), s["uniforms"][above].double()
    if c["drafted"]:
        taken = u * s["draft_probs"][rows, tok].double() < p
    else:
        # a row's earlier siblings take the numbers below its own
        earlier = (up[:, :, None] == up[:, None]) & (i[None] < i[:, None]) & drafts[:, None]
        again = (earlier & (tok[:, :, None] == tok[:, None])).any(-1)
        p = torch.where(again, 0.0, p)
        low = (earlier * p[:, None]).sum(-1)
        taken = (low <= u) & (u < low + p)
    ok = (taken & drafts) | (live & (i == 0))
    jump = up
    for _ in range(n.bit_length()):                     # every row above accepted too
        ok = ok & ok.gather(1, jump)
        jump = jump.gather(1, jump)
    deep = ok.sum(-1)
    length = deep.clamp_max(W)
    rank = ok.cumsum(-1) - 1
    path = torch.full((B, W + 1), -1, device="cuda")
    path.scatter_(1, torch.where(ok & (rank < W), rank, W), i.expand(B, n))
    path = path[:, :W]
    j = torch.arange(W, device="cuda")
    path = torch.where(j < length[:, None], path, -1)
    last = path.gather(1, length[:, None] - 1)[:, 0]
    full = s["probs"][starts[:-1] + last].double()
    refused = drafts & (up == last[:, None]) & (deep < W)[:, None]
    if c["drafted"]:
        child = rows.gather(1, (last + 1).clamp_max(n - 1)[:, None])[:, 0]
        rest = (full - s["draft_probs"][child].double()).clamp_min(0.0)
        weight = torch.where(refused.any(-1)[:, None], rest, full)
    else:
        weight = torch.cat([full, full[:, :1]], 1)      # one more for what is not refused
        weight.scatter_(1, torch.where(refused, tok, V), 0.0)
        weight = weight[:, :V]
    weight = torch.where(weight.sum(-1, keepdim=True) > 0, weight, full)
    total = weight.cumsum(-1)
    drawn = (total <= s["final_uniforms"].double()[:, None] * total[:, -1:]).sum(-1)
    follow = path.clamp_min(0)[:, 1:]
    new = torch.cat([tok.gather(1, follow), tok[:, :1]], 1)
    new = torch.where(j == length[:, None] - 1, drawn[:, None], new)
    new = torch.where(j < length[:, None], new, -1)
    return {"new_tokens": new, "path": path.int(), "lengths": length.int()}


def _compact_pass(s, c):
    page, path = c["page"], s["path"].long()
    j = torch.arange(path.shape[1], device="cuda")
    moved = (j < s["lengths"][:, None]) & (j > 0)
    ctx = s["context_lens"].long()[:, None]
    table = s["block_table"].long()

    def place(t):
        return table.gather(1, t // page).flatten(), (t % page).flatten()

    # what does not move stays on its sequence's first row
    source = place(ctx + torch.where(moved, path, 0))
    target = place(ctx + torch.where(moved, j, 0))
    for x in s["cache"].values():
        if x.dim() > 1:
            x[target[0], :, target[1]] = x[source[0], :, source[1]]
    return _cached(s, c)


def _through_package(s, c):
    import residual_add_rmsnorm_gb300 as rarn
    op = c["op"]
    if op == "block":
        y = rarn.gated_add_rms_norm(s["x"], s["residual"], s["x_gamma"], s["gamma"], EPS,
                                    gate=s["gate"], gate_index=s["gate_index"], scale=c["scale"],
                                    out=s["out"], residual_out=s["h"])
        return s["h"], y
    if op == "step":
        if "pages" not in s:                            # the program's pages, made once
            s["pages"] = rarn.KVPages(s["table"], s["held"], s["free"], s["count"], c["page"])
        rarn.kv_step(s["pages"], s["context_lens"], s["new_lens"], s["tokens"],
                     starts=s["starts"], slots=s["slots"], positions=s["positions"],
                     served=s["served"])
        rarn.kv_trim(s["pages"], s["context_lens"])
        return {n: s[n] for n in ("starts", "slots", "positions", "served", "table", "held",
                                  "free", "count")}
    if op == "verify":
        new, path, lengths = rarn.verify_drafts(
            s["probs"], s["tokens"], s["starts"], s["uniforms"], s["final_uniforms"], s["most"],
            draft_probs=s["draft_probs"], parents=s["parents"], new_tokens=s["new_tokens"],
            path=s["path"], lengths=s["lengths"])
        return {"new_tokens": new, "path": path, "lengths": lengths}
    if "cache" in s and "handle" not in s:              # the program's cache object, made once
        n = s["cache"]
        s["handle"] = rarn.KVCache(n["k"], n["v"], n["k_scale"], n["v_scale"], fmt=c["fmt"],
                                   scale_mode=c["mode"])
    if op == "compact":
        rarn.kv_cache_compact(s["handle"], s["block_table"], s["context_lens"], s["path"],
                              s["lengths"])
        return _cached(s, c)
    if "sections" not in s:                             # the model's, known from its start
        s["sections"] = _sections(c)
    if not c["fmt"]:
        q, k = rarn.qk_norm_rope(s["q"], s["k"], s["q_gamma"], s["k_gamma"], EPS, s["table"],
                                 s["positions"], style=c["style"], q_out=s["q_out"],
                                 k_out=s["k_out"], sections=s["sections"],
                                 section_order=c["order"])
        return {"q": q, "k": k}
    q = rarn.qk_norm_rope_kv_write(s["q"], s["k"], s["v"], s["q_gamma"], s["k_gamma"], EPS,
                                   s["table"], s["positions"], s["handle"], s["slots"],
                                   style=c["style"], q_out=s["q_out"], sections=s["sections"],
                                   section_order=c["order"])
    return {"q": q, **{"cache_" + n: x for n, x in _cached(s, c).items()}}


def run(state):
    s, c = state, state["case"]
    if own:
        return _through_package(s, c)
    return {"block": _block_pass, "axes": _axes_pass, "step": _step_pass, "verify": _verify_pass,
            "compact": _compact_pass}[c["op"]](s, c)


# --------------------------------------------------------------------------
# the definition in binary64
# --------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    return {"block": _exact_block, "axes": _exact_axes, "step": _exact_step,
            "verify": _exact_verify, "compact": _exact_compact}[c["op"]](s, c)


def _exact_block(s, c):
    f64 = torch.float64
    x = s["x"].to(f64)
    if s["x_gamma"] is not None:
        x = x / (x.square().sum(-1, keepdim=True) / c["H"] + EPS).sqrt() * s["x_gamma"].to(f64)
    if s["gate"] is not None:
        g = s["gate"].to(f64)
        x = x * (g.expand_as(x) if c["gates"] in (1, c["T"]) else g.index_select(0, s["gate_index"]))
    h = s["residual"].to(f64) + c["scale"] * x
    r = h.to(s["residual"].dtype).to(f64)   # the norm is that of the stored stream
    return h, r / (r.square().sum(-1, keepdim=True) / c["H"] + EPS).sqrt() * s["gamma"].to(f64)


def _exact_axes(s, c):
    f64, half = torch.float64, c["rot"] // 2
    axis = _axis_of_pair(c)
    table = s["table"].to(f64)
    angle = torch.stack([torch.complex(table[:, i], table[:, half + i])[s["positions"][axis[i]]]
                         for i in range(half)], -1).unsqueeze(1)
    first, second = ((slice(0, half), slice(half, 2 * half)) if c["style"] == "half"
                     else (slice(0, 2 * half, 2), slice(1, 2 * half, 2)))

    def turned(x, gamma):
        x = x.to(f64)
        y = x / (x.square().sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * gamma.to(f64)
        w = torch.complex(y[..., first], y[..., second]) * angle
        out = y.clone()
        out[..., first], out[..., second] = w.real, w.imag
        return out

    q, k = turned(s["q"], s["q_gamma"]), turned(s["k"], s["k_gamma"])
    if not c["fmt"]:
        return {"q": q, "k": k}
    top, got, cache = LARGEST[c["fmt"]], {"q": q}, s["cache"]
    for n, x in (("k", k), ("v", s["v"].to(f64))):
        scale = cache[n + "_scale"].to(f64)
        flat = cache[n].view(CODES[c["fmt"]]).float().to(f64).transpose(1, 2).flatten(0, 1)
        if c["mode"] == "row":
            most = x.abs().max(-1).values
            by = torch.where(most == 0, 1.0, most / top)
            per = scale.transpose(1, 2).flatten(0, 1)
            per[s["slots"]] = by
            got["cache_" + n + "_scale"] = per.view(-1, c["page"], c["Hk"]).transpose(1, 2)
            x = x / by.unsqueeze(-1)
        else:
            x = (x / scale).clamp(-top, top)
        flat[s["slots"]] = x
        # before rounding to codes; half a step of e5m2 is too wide for that to say anything
        got["cache_" + n] = (flat.view(-1, c["page"], c["Hk"], c["D"]).transpose(1, 2)
                             if c["fmt"] == "e4m3" else None)
    return got


def _exact_step(s, c):
    """Sequence by sequence on the host."""
    ctx, new, page = s["context_lens"].tolist(), s["new_lens"].tolist(), c["page"]
    free, count = s["free"].tolist(), s["count"].item()
    starts, slots, positions = [0], [], []
    for b, row in enumerate(s["table"].tolist()):
        mine = [x for x in row if x >= 0]
        for t in range(ctx[b], ctx[b] + new[b]):
            if t // page == len(mine):
                count -= 1
                mine.append(free[count])
            positions.append(t)
            slots.append(mine[t // page] * page + t % page)
        starts.append(len(slots))
    pad = s["tokens"] - len(slots)
    return {"starts": _ints(starts), "slots": _ints(slots + [-1] * pad, torch.int64),
            "positions": _ints(positions + [0] * pad, torch.int64), "served": _ints([c["B"]]),
            "table": s["table"], "held": s["held"], "free": s["free"], "count": s["count"]}


def _exact_verify(s, c):
    """Sequence by sequence: down the accepted rows, then the draw."""
    f64, W = torch.float64, s["most"] + 1
    starts, tokens = s["starts"].tolist(), s["tokens"].tolist()
    u, last_u = s["uniforms"].tolist(), s["final_uniforms"].tolist()
    above = s["parents"].tolist() if c["tree"] else None
    new, paths, lengths = [], [], []
    for b in range(c["B"]):
        lo, hi = starts[b], starts[b + 1]
        at, path = lo, [0]
        while True:
            kids = [r for r in range(at + 1, hi)
                    if (lo + above[r] if above else r - 1) == at] if len(path) < W else []
            p = s["probs"][at].to(f64)
            left, low, step = p.clone(), 0.0, None
            for r in kids:
                if c["drafted"]:
                    q = s["draft_probs"][r].to(f64)
                    good = u[at] * q[tokens[r]].item() < p[tokens[r]].item()
                    left = torch.relu(p - q)
                else:
                    mass = left[tokens[r]].item()
                    good = low <= u[at] < low + mass
                    low += mass
                    left[tokens[r]] = 0.0
                if good:
                    step = r
                    break
            if step is None:
                break
            at = step
            path.append(at - lo)
        if not kids or not left.any():
            left = p
        total = left.cumsum(0)
        drawn = torch.searchsorted(total, total[-1] * last_u[b], right=True).item()
        pad = [-1] * (W - len(path))
        new.append([tokens[lo + r] for r in path[1:]] + [drawn] + pad)
        paths.append(path + pad)
        lengths.append(len(path))
    return {"new_tokens": _ints(new, torch.int64), "path": _ints(paths), "lengths": _ints(lengths)}


def _exact_compact(s, c):
    """The codes' values and scales, row by row."""
    page, cache = c["page"], s["cache"]
    table, ctx = s["block_table"].tolist(), s["context_lens"].tolist()
    goes, comes = [], []
    for b, path in enumerate(_paths(c)):
        for j in range(1, len(path)):
            for t, to in ((ctx[b] + j, goes), (ctx[b] + path[j], comes)):
                to.append(table[b][t // page] * page + t % page)
    got = {}
    for n, x in cache.items():
        if x.dim() == 1:
            continue
        x = (x.view(CODES[c["fmt"]]).float() if x.dtype == torch.uint8 else x).to(torch.float64)
        flat = x.transpose(1, 2).flatten(0, 1)
        flat[_ints(goes, torch.int64)] = flat[_ints(comes, torch.int64)]
        got[n] = flat.view(-1, page, *x.shape[1:2], *x.shape[3:]).transpose(1, 2)
    return got
