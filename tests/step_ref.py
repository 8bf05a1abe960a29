"""Binary64 definitions of a step's operators on CPU tensors, and the error
bounds that their GPU tests use.

Bounds (h(t) = eps(t) / 2, a type's half step; u = 2^-24):
  * gated norms.  A row sum of squares: a thread's run of k = ceil(H / 32) terms at
    most, a tree of at most 10 levels, one product and one sum: (k + 14) u; its
    reciprocal root half of that and 2^-22; the products with x, gamma, gate and
    scale, residual_scale's and the sum 8 u.  In all E = (k / 2 + 24) u times the
    magnitudes |residual_scale r| + |scale gate n|, then one rounding to the
    residual's type.  y is compared with the norm of the h that the kernel stored:
    E |y|, then one rounding.
"""
from __future__ import annotations

import torch

F64 = torch.float64


def half(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half the smallest subnormal step."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def norm(x, gamma, eps):
    x = x.to(F64)
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.to(F64)


def row_error(H):
    return ((H + 31) // 32 / 2 + 24) * 2.0 ** -24


def check_block(y, h, x, residual, x_gamma, gamma, eps, gate=None, scale=1.0, residual_scale=1.0,
                what=""):
    """y and h (what came of the call, on the host) against the formulas; gate: [T, H] or None."""
    H = x.shape[1]
    n = x.to(F64) if x_gamma is None else norm(x, x_gamma, eps)
    if gate is not None:
        n = n * gate.to(F64)
    a, b = residual_scale * residual.to(F64), scale * n
    want, err = a + b, row_error(H)
    bound = half(h.dtype) * (want.abs() + err * (a.abs() + b.abs())) + \
        err * (a.abs() + b.abs()) + tiny(h.dtype)
    within(h, want, bound, f"{what} h")
    want = norm(h, gamma, eps)
    within(y, want, half(y.dtype) * want.abs() * (1 + err) + err * want.abs() + tiny(y.dtype),
           f"{what} y")


def within(got, want, bound, what):
    got = got.to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN pattern"
    err = torch.where(torch.isnan(want) | (got == want), torch.zeros_like(want),
                      (got - want).abs())
    bad = ~(err <= torch.nan_to_num(bound, posinf=float("inf")))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / bound).nan_to_num().max()):.3g} of the bound")


class Pages:
    """The pages of a step, sequence by sequence: a model of KVPages on the host."""

    def __init__(self, sequences, width, num_pages, page_size, free=None):
        self.width, self.num, self.page = width, num_pages, page_size
        self.has = [[] for _ in range(sequences)]
        self.free = list(range(num_pages - 1, -1, -1)) if free is None else list(free)

    def step(self, context, new, tokens):
        """(starts, slots, positions, served, whether a sequence made no sense)."""
        starts, slots, positions, bad = [0], [], [], False
        served = len(self.has)
        plan = []
        rows = pages = 0
        for b, (c, n) in enumerate(zip(context, new)):
            need = 0
            if n != 0 and (n < 0 or c < 0 or len(self.has[b]) * self.page < c or
                           c + n > self.width * self.page):
                bad, n = True, 0
            if n:
                need = max(0, -(-(c + n) // self.page) - len(self.has[b]))
            plan.append((n, need))
            rows, pages = rows + n, pages + need
            if (rows > tokens or pages > len(self.free)) and served == len(self.has):
                served = b
        for b, (n, need) in enumerate(plan):
            if b < served:
                self.has[b] += [self.free.pop() for _ in range(need)]
                for t in range(context[b], context[b] + n):
                    page = self.has[b][t // self.page]
                    slots.append(page * self.page + t % self.page)
                    positions.append(t)
            starts.append(len(slots))
        pad = tokens - len(slots)
        return starts, slots + [-1] * pad, positions + [0] * pad, served, bad

    def trim(self, lens):
        back = []
        for b, n in enumerate(lens):
            if n < 0:
                continue
            keep = min(len(self.has[b]), -(-n // self.page))
            back += self.has[b][keep:]
            del self.has[b][keep:]
        self.free += back[::-1]

    def table(self):
        return [h + [-1] * (self.width - len(h)) for h in self.has]


def verify(probs, tokens, starts, u, v, most, draft_probs=None, parents=None):
    """(new_tokens, path, lengths) as lists, sequence by sequence in binary64: sums of
    up to 10^5 terms are off by 2^-53 of the total a term, so that a draw differs from the
    exact one where v lies that near to a border."""
    W, V = most + 1, probs.shape[1]
    new, paths, lengths = [], [], []
    for b in range(len(starts) - 1):
        lo, n = starts[b], starts[b + 1] - starts[b]
        if n == 0:
            new.append([-1] * W)
            paths.append([-1] * W)
            lengths.append(0)
            continue
        at, path = 0, [0]
        while True:
            p = probs[lo + at].to(F64)
            left, low, took = p.clone(), 0.0, None
            kids = [] if len(path) == W else \
                [r for r in range(at + 1, n) if (parents[lo + r] if parents else r - 1) == at]
            for r in kids:
                x, number = tokens[lo + r], float(u[lo + at])
                if not 0 <= x < V:
                    if draft_probs is not None:
                        left = (p - draft_probs[lo + r].to(F64)).clamp_min(0)
                    continue
                if draft_probs is not None:
                    q = draft_probs[lo + r].to(F64)
                    good = number * float(q[x]) < float(p[x])
                    left = (p - q).clamp_min(0)
                else:
                    mass = float(left[x])
                    good = low <= number < low + mass
                    low += mass
                    left[x] = 0
                if good:
                    took = r
                    break
            if took is None:
                break
            at = took
            path.append(at)
        if not kids or float(left.sum()) == 0:
            left = p
        total = left.cumsum(0)
        drawn = -1 if float(total[-1]) == 0 else \
            int(torch.searchsorted(total, total[-1] * float(v[b]), right=True))
        pad = [-1] * (W - len(path))
        new.append([tokens[lo + r] for r in path[1:]] + [drawn] + pad)
        paths.append(path + pad)
        lengths.append(len(path))
    return new, paths, lengths
