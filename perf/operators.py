"""Timed cases of the attention-side operators: per-head norms of queries and
keys with the position rotation, the 8-bit key / value cache (written, read
back), and attention of drafted tokens over it.

Each case is a dict of plain values; ``prepare`` makes its inputs on the GPU
from a seed, ``run`` makes one pass: through the package's entry points where
``own`` is true, in plain torch (binary32, one rounding at the end) otherwise.
``exact`` is the same definition in binary64.
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


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _rope(name, T, Hq, Hk, D, rot, dt, style):
    return {"name": name, "op": "norm_rope", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
            "dt": dt, "style": style}


def _write(name, T, Hq, Hk, D, rot, dt, style, fmt, mode, page, fused):
    return {"name": name, "op": "write", "T": T, "Hq": Hq, "Hk": Hk, "D": D, "rot": rot,
            "dt": dt, "style": style, "fmt": fmt, "mode": mode, "page": page, "fused": fused}


def _read(name, B, most, Hk, D, dt, fmt, mode, page, lens):
    return {"name": name, "op": "read", "B": B, "most": most, "Hk": Hk, "D": D, "dt": dt,
            "fmt": fmt, "mode": mode, "page": page, "lens": lens}


def _tree(name, B, most, nodes, Hq, Hk, D, dt, fmt, mode, page, lens):
    return {"name": name, "op": "tree", "B": B, "most": most, "nodes": nodes, "Hq": Hq,
            "Hk": Hk, "D": D, "dt": dt, "fmt": fmt, "mode": mode, "page": page, "lens": lens}


def listed():
    return [
        # one token of a decode step: launch latency
        _rope("norm_rope_1", 1, 32, 8, 128, 128, "bf16", "half"),
        # an odd prompt on a partly rotated, interleaved model in binary16
        _rope("norm_rope_517_part", 517, 40, 8, 96, 64, "f16", "interleaved"),
        # a long prefill batch
        _rope("norm_rope_8192", 8192, 64, 8, 128, 128, "bf16", "half"),
        # a decode batch's keys and values into the cache, one scale for all
        _write("write_64", 64, 0, 8, 128, 0, "bf16", "half", "e4m3", "tensor", 16, False),
        # the same step with the norms and the rotation in the pass, a scale per row
        _write("norm_rope_write_128", 128, 40, 8, 128, 128, "bf16", "half", "e4m3", "row", 16,
               True),
        # a long prefill batch written as it is normalised
        _write("norm_rope_write_8192", 8192, 64, 8, 128, 128, "bf16", "half", "e4m3", "row", 16,
               True),
        # a few short prefixes read back before a prompt's next chunk
        _read("read_7", 7, 600, 8, 128, "bf16", "e4m3", "row", 16, 1),
        # long prefixes of a whole batch
        _read("read_32", 32, 4096, 8, 128, "bf16", "e4m3", "row", 16, 2),
        # one sequence, one token: latency
        _tree("tree_decode_1", 1, 1000, 1, 32, 8, 128, "bf16", "e4m3", "row", 16, 3),
        # an ordinary decode batch of ragged lengths, one token each
        _tree("tree_decode_64", 64, 8192, 1, 32, 8, 128, "bf16", "e4m3", "row", 16, 4),
        # drafted trees of up to 32 tokens over ragged contexts
        _tree("tree_16x32", 16, 8192, 32, 64, 8, 128, "bf16", "e4m3", "row", 16, 5),
        # a small tree over one very long context, five query heads to a key head
        _tree("tree_long", 1, 131072, 8, 40, 8, 128, "f16", "e5m2", "tensor", 64, 6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["norm_rope", "write", "read", "tree", "tree"])
    D = rng.choice([64, 96, 128, 128, 192, 256])
    Hq, Hk = rng.choice([(32, 8), (64, 8), (40, 8), (28, 4), (16, 16), (16, 1), (16, 2), (5, 5)])
    dt = rng.choice(["bf16", "bf16", "f16"])
    fmt, mode = rng.choice(["e4m3", "e4m3", "e5m2"]), rng.choice(["row", "row", "tensor"])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    style = rng.choice(["half", "interleaved"])
    rot = rng.choice([D, D, D // 2, D // 2, 32])
    lens = rng.randrange(1 << 20)
    if op == "norm_rope":
        T = _log(rng, 1, min(8192, (1 << 26) // ((Hq + Hk) * D)))
        c = _rope("", T, Hq, Hk, D, rot, rng.choice([dt, dt, "f32"]), style)
    elif op == "write":
        fused = rng.random() < 0.7
        T = _log(rng, 1, min(8192, (1 << 26) // ((Hq + 2 * Hk) * D)))
        c = _write("", T, Hq if fused else 0, Hk, D, rot if fused else 0, dt, style, fmt, mode,
                   page, fused)
    elif op == "read":
        B = _log(rng, 1, 64)
        c = _read("", B, _log(rng, 1, min(32768, (1 << 27) // (B * Hk * D))), Hk, D, dt, fmt,
                  mode, page, lens)
    else:
        nodes = rng.choice([1, _log(rng, 1, 64)])
        B = _log(rng, 1, max(1, min(64, 4096 // (nodes * max(1, Hq // 16)))))
        cap = min((1 << 28) // (B * Hk * D), (1 << 34) // (B * Hq * nodes * D))
        c = _tree("", B, _log(rng, 1, min(65536, max(16, cap))), nodes, Hq, Hk, D, dt, fmt, mode,
                  page, lens)
    del c["name"]
    return c


def _lengths(c):
    """Cached tokens of each sequence: from one to the case's most, the longest there."""
    r = random.Random(c["lens"])
    got = [c["most"] if b == 0 else max(1, round(c["most"] * r.random())) for b in range(c["B"])]
    r.shuffle(got)
    return got


def _drafted(c):
    """Drafted tokens of each sequence."""
    r = random.Random(c["lens"] + 1)
    n = c["nodes"]
    return [n if b == 0 else r.randint((n + 1) // 2, n) for b in range(c["B"])]


def work(case):
    c = case
    D, Hk = c["D"], c["Hk"]
    if c["op"] in ("norm_rope", "write"):
        T, Hq, s = c["T"], c["Hq"], SIZES[c["dt"]]
        table = T * (c["rot"] * 4 + 8) if c["rot"] else 0
        n = T * Hq * D * s * 2 + table
        if c["op"] == "norm_rope":
            n += T * Hk * D * s * 2 + 2 * D * s
        else:
            n += 2 * T * Hk * D * (s + 1) + T * 8 + (2 * T * Hk * 4 if c["mode"] == "row" else 8)
            n += 2 * D * s if c["fused"] else 0
        return {"bytes": n, "flops": 8 * T * (Hq + 2 * Hk) * D}
    row = 2 * Hk * (D + (4 if c["mode"] == "row" else 0))
    if c["op"] == "read":
        n = sum(_lengths(c))
        return {"bytes": n * (row + 2 * Hk * D * SIZES[c["dt"]]), "flops": 2 * n * Hk * D}
    ctx, new, Hq = _lengths(c), _drafted(c), c["Hq"]
    total = sum(ctx) + sum(new)
    return {"bytes": total * row + 4 * total // c["page"] + 2 * sum(new) * Hq * D * SIZES[c["dt"]],
            "flops": 4 * D * Hq * sum(n * (a + n) for a, n in zip(ctx, new))}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _table(positions, rot):
    """cos and sin of the rotation's angles, [positions, rot] binary32 (formed in binary64)."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _pages_for(counts, page):
    return sum(-(-n // page) for n in counts)


def _cache(c, pages, g, filled):
    """An 8-bit cache of `pages` pages; `filled`: of normal keys and values, quantised."""
    Hk, D, page, fmt = c["Hk"], c["D"], c["page"], c["fmt"]
    got = {}
    for n in "kv":
        if not filled:
            got[n] = torch.zeros(pages, Hk, page, D, dtype=torch.uint8, device="cuda")
            got[n + "_scale"] = (torch.ones(pages, Hk, page, device="cuda") if c["mode"] == "row"
                                 else torch.full((1,), 8.0 / LARGEST[fmt], device="cuda"))
            continue
        x = torch.randn(pages, Hk, page, D, device="cuda", generator=g, dtype=torch.bfloat16)
        if c["mode"] == "row":
            s = x.abs().amax(-1).float().clamp_min(1e-20) / LARGEST[fmt]
            per = s[..., None]
        else:
            s = torch.full((1,), 6.0 / LARGEST[fmt], device="cuda")
            per = s
        u = (x / per).clamp_(-LARGEST[fmt], LARGEST[fmt])
        got[n], got[n + "_scale"] = u.to(CODES[fmt]).view(torch.uint8), s
        del x, u
    return got


def _block_table(counts, page, g):
    """Pages of each sequence in an order of their own, [B, most]; unused entries are -1."""
    need = [-(-n // page) for n in counts]
    order = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    rows = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    where = torch.arange(max(need), device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    rows[where] = order
    return rows


def _masks(new, g_seed):
    """A random tree for each sequence as ancestor bits, [sum, words] int32: a drafted token
    sees itself and its ancestors."""
    r = random.Random(g_seed)
    words = -(-max(new) // 32)
    rows = []
    for n in new:
        seen = []
        for i in range(n):
            parent = r.randrange(max(0, i - 6), i) if i else -1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        rows += seen
    signed = [[(v >> 32 * w & 0xffffffff) - ((v >> 32 * w & 0x80000000) << 1)
               for w in range(words)] for v in rows]
    return torch.tensor(signed, dtype=torch.int32, device="cuda")


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, g = case, _generator(seed)
    Hk, D, dt = c["Hk"], c["D"], TYPES[c["dt"]]
    s = {"case": c}
    if c["op"] in ("norm_rope", "write"):
        # the rows of a packed projection: each head's query, key and value side by side
        T, Hq = c["T"], c["Hq"]
        qkv = torch.randn(T, Hq + 2 * Hk, D, device="cuda", generator=g)
        qkv = (qkv * torch.exp(torch.randn(T, 1, 1, device="cuda", generator=g) * 0.5)).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
        for n in ("q_gamma", "k_gamma"):
            s[n] = (torch.rand(D, device="cuda", generator=g) + 0.5).to(dt)
        if c["rot"]:
            s["table"] = _table(16384, c["rot"])
            s["positions"] = torch.randint(0, 16384 - T, (1,), device="cuda", generator=g) + \
                torch.arange(T, device="cuda")
        s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
        s["k_out"] = torch.empty(T, Hk, D, dtype=dt, device="cuda")
        if c["op"] == "write":
            pages = -(-T // c["page"]) + 2
            s["cache"] = _cache(c, pages, g, False)
            order = torch.randperm(pages, device="cuda", generator=g)
            t = torch.arange(T, device="cuda")
            s["slots"] = order[t // c["page"]] * c["page"] + t % c["page"]
        return s
    ctx = _lengths(c)
    new = _drafted(c) if c["op"] == "tree" else [0] * c["B"]
    both = [a + b for a, b in zip(ctx, new)]
    s["cache"] = _cache(c, _pages_for(both, c["page"]), g, True)
    s["block_table"] = _block_table(both, c["page"], g)
    if c["op"] == "read":
        s["starts"] = _starts(ctx)
        n = sum(ctx)
        s["k_out"] = torch.empty(n, Hk, D, dtype=dt, device="cuda")
        s["v_out"] = torch.empty(n, Hk, D, dtype=dt, device="cuda")
        return s
    s["context_lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["starts"] = _starts(new)
    s["q"] = (1.5 * torch.randn(sum(new), c["Hq"], D, device="cuda", generator=g)).to(dt)
    s["mask"] = _masks(new, seed) if max(new) > 1 else None
    s["out"] = torch.empty_like(s["q"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _norm(x, gamma):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()


def _rotate(x, table, positions, style):
    rot = table.shape[1]
    cs = table[positions][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if style == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


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


def _values(cache, n, page, at, c):
    """The numbers in the cache's slots, binary32: [..., heads, D]."""
    x = cache[n][page, :, at].view(CODES[c["fmt"]]).float()
    s = cache[n + "_scale"]
    return x * (s[page, :, at][..., None] if c["mode"] == "row" else s)


def _attend(s, c):
    """softmax(q k^T / sqrt(D) + mask) v: sequences and drafted tokens padded to the longest."""
    B, Hk, D = c["B"], c["Hk"], c["D"]
    G = c["Hq"] // Hk
    ctx, starts = s["context_lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    n, L = c["nodes"], c["most"] + c["nodes"]
    i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    pages = s["block_table"].long()
    page = pages[:, (j // c["page"]).clamp_max(pages.shape[1] - 1)].clamp_min(0)
    at = (j % c["page"]).expand(B, L)
    rows = (starts[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(B, n, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, D)
    k = _values(s["cache"], "k", page, at, c).permute(0, 2, 3, 1)
    w = (q @ k).view(B, Hk, G, n, L) / math.sqrt(D)
    del k
    past = j[None] - ctx[:, None]                   # [B, L]: which drafted token, < 0: context
    seen = (past < 0)[:, None].expand(B, n, L)
    if s["mask"] is None:
        seen = seen | (past == 0)[:, None]
    else:
        bit = past.clamp(0, n - 1)
        words = s["mask"][rows].long()              # [B, n, words]
        word = words.gather(2, (bit // 32)[:, None].expand(B, n, L))
        live = (past >= 0) & (past < new[:, None])
        seen = seen | (((word >> (bit % 32)[:, None]) & 1 > 0) & live[:, None])
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(w - w.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _values(s["cache"], "v", page, at, c).permute(0, 2, 1, 3)
    o = (p.view(B, Hk, G * n, L) @ v).view(B, Hk, G, n, D).permute(0, 3, 1, 2, 4)
    return o.reshape(B, n, c["Hq"], D)[i < new[:, None]].to(s["q"].dtype)


def _through_package(s, c):
    import residual_add_rmsnorm_gb300 as rarn
    op = c["op"]
    if op == "norm_rope":
        return rarn.qk_norm_rope(s["q"], s["k"], s["q_gamma"], s["k_gamma"], EPS, s["table"],
                                 s["positions"], style=c["style"], q_out=s["q_out"],
                                 k_out=s["k_out"])
    if "handle" not in s:                           # the program's cache object, made once
        n = s["cache"]
        s["handle"] = rarn.KVCache(n["k"], n["v"], n["k_scale"], n["v_scale"], fmt=c["fmt"],
                                   scale_mode=c["mode"])
    cache = s["handle"]
    if op == "write":
        if c["fused"]:
            rarn.qk_norm_rope_kv_write(s["q"], s["k"], s["v"], s["q_gamma"], s["k_gamma"], EPS,
                                       s["table"], s["positions"], cache, s["slots"],
                                       style=c["style"], q_out=s["q_out"])
        else:
            rarn.kv_cache_write(s["k"], s["v"], cache, s["slots"])
        return _written(s, s["q_out"])
    if op == "read":
        return rarn.kv_cache_read(cache, s["block_table"], s["starts"], s["k_out"], s["v_out"])
    if "workspace" not in s:                        # kept by the program from call to call
        n = rarn.tree_attention_workspace_bytes(s["q"].shape[0], c["B"], c["Hq"], c["Hk"], c["D"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return rarn.tree_attention(s["q"], cache, s["block_table"], s["context_lens"], s["starts"],
                               mask=s["mask"], out=s["out"], workspace=s["workspace"])


def _written(s, q):
    c, n = s["case"], s["cache"]
    got = {"k": n["k"].view(CODES[c["fmt"]]), "v": n["v"].view(CODES[c["fmt"]])}
    if c["mode"] == "row":
        got.update(k_scale=n["k_scale"], v_scale=n["v_scale"])
    if c["fused"]:
        got["q"] = q
    return got


def run(state):
    s, c = state, state["case"]
    if own:
        return _through_package(s, c)
    op, dt = c["op"], TYPES[c["dt"]]
    if op == "norm_rope":
        return tuple(_rotate(_norm(s[n], s[n + "_gamma"]), s["table"], s["positions"],
                             c["style"]).to(dt) for n in "qk")
    if op == "write":
        k, q = s["k"].float(), None
        if c["fused"]:
            k = _rotate(_norm(s["k"], s["k_gamma"]), s["table"], s["positions"], c["style"])
            q = _rotate(_norm(s["q"], s["q_gamma"]), s["table"], s["positions"],
                        c["style"]).to(dt)
        _store(k, s["slots"], s["cache"], "k", c)
        _store(s["v"].float(), s["slots"], s["cache"], "v", c)
        return _written(s, q)
    if op == "read":
        starts = s["starts"].long()
        t = torch.arange(s["k_out"].shape[0], device="cuda")
        b = torch.searchsorted(starts[1:], t, right=True)
        j = t - starts[b]
        page = s["block_table"].long()[b, j // c["page"]]
        return tuple(_values(s["cache"], n, page, j % c["page"], c).to(dt) for n in "kv")
    return _attend(s, c)


# --------------------------------------------------------------------------
# the definition in binary64
# --------------------------------------------------------------------------

def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e12:
        return None
    s = prepare(c, seed)
    f64 = torch.float64

    def turned(x, gamma):
        x = x.to(f64)
        y = x / (x.square().sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * gamma.to(f64)
        r = c["rot"]
        angle = s["table"].to(f64).index_select(0, s["positions"]).unsqueeze(1)
        z = torch.complex(angle[..., :r // 2], angle[..., r // 2:])
        out = y.clone()
        first, second = ((slice(0, r // 2), slice(r // 2, r)) if c["style"] == "half"
                         else (slice(0, r, 2), slice(1, r, 2)))
        w = torch.complex(y[..., first], y[..., second]) * z
        out[..., first], out[..., second] = w.real, w.imag
        return out

    if c["op"] == "norm_rope":
        return turned(s["q"], s["q_gamma"]), turned(s["k"], s["k_gamma"])
    cache = s["cache"]
    if c["op"] == "write":
        top, got = LARGEST[c["fmt"]], {}
        rows = {"k": turned(s["k"], s["k_gamma"]) if c["fused"] else s["k"].to(f64),
                "v": s["v"].to(f64)}
        for n, x in rows.items():
            scale = cache[n + "_scale"].to(f64)
            codes = cache[n].view(CODES[c["fmt"]]).float().to(f64)
            flat = codes.transpose(1, 2).flatten(0, 1)
            if c["mode"] == "row":
                most = x.abs().max(-1).values
                by = torch.where(most == 0, 1.0, most / top)
                per = scale.transpose(1, 2).flatten(0, 1)
                per[s["slots"]] = by
                got[n + "_scale"] = per.view(-1, c["page"], c["Hk"]).transpose(1, 2)
                x = x / by.unsqueeze(-1)
            else:
                x = (x / scale).clamp(-top, top)
            flat[s["slots"]] = x
            # before rounding to codes; half a step of e5m2 is too wide for that to say anything
            got[n] = (flat.view(-1, c["page"], c["Hk"], c["D"]).transpose(1, 2)
                      if c["fmt"] == "e4m3" else None)
        if c["fused"]:
            got["q"] = turned(s["q"], s["q_gamma"])
        return got if any(x is not None for x in got.values()) else None

    def rows_of(n, b, count):
        j = torch.arange(count, device="cuda")
        slot = s["block_table"][b].long()[j // c["page"]] * c["page"] + j % c["page"]
        x = cache[n].transpose(1, 2).flatten(0, 1)[slot].view(CODES[c["fmt"]]).float().to(f64)
        if c["mode"] == "tensor":
            return x * cache[n + "_scale"].to(f64)
        return x * cache[n + "_scale"].transpose(1, 2).flatten(0, 1)[slot].to(f64).unsqueeze(-1)

    ctx = _lengths(c)
    if c["op"] == "read":
        return tuple(torch.cat([rows_of(n, b, m) for b, m in enumerate(ctx)]) for n in "kv")
    got, at = [], 0
    for b, (a, n) in enumerate(zip(ctx, _drafted(c))):
        k, v = rows_of("k", b, a + n), rows_of("v", b, a + n)
        bias = torch.zeros(n, a + n, dtype=f64, device="cuda")
        if s["mask"] is not None:
            bits = s["mask"][at:at + n]
            for j in range(n):
                hidden = (bits[:, j // 32] >> j % 32) & 1 == 0
                bias[hidden, a + j] = -math.inf
        q = s["q"][at:at + n].to(f64)
        out = torch.empty(n, c["Hq"], c["D"], dtype=f64, device="cuda")
        for h in range(c["Hq"]):
            hk = h // (c["Hq"] // c["Hk"])
            p = torch.softmax(q[:, h] @ k[:, hk].T * c["D"] ** -0.5 + bias, -1)
            out[:, h] = p @ v[:, hk]
        got.append(out)
        at += n
    return torch.cat(got)
