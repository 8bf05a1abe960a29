"""Binary64 definitions of the attention side, on CPU tensors, and the error
bounds its GPU tests use.

Bounds (u = 2^-24, binary32's half step; h(t) = eps(t) / 2, a storage type's):
  * norm and rotation: the sum of D <= 1024 squares by runs of <= 32 and a
    shuffle tree of <= 5 levels, the mean, rsqrtf (2 units), two products, and
    in the rotation two products and a sum: under 2^-19 of |a cos| + |b sin|;
    then one rounding, h(t) of the result (or half a subnormal step).
  * codes: u = v / s carries v's 2^-19 and three more roundings: the code is
    within half a step of the format at u, plus 2^-18 of |u|'s terms.
  * read back: one product and one rounding: h(t) + 2^-23.
  * attention: with A the largest sum |q_d K_d| * scale of a row, the scores are
    off by at most D 2^-22 A (a tensor core's binary32 sums may truncate), and by
    2^-17 max|q| sum |K_d| * scale for the queries' 8-bit pieces (the row is scaled
    to a largest magnitude in [2^7, 2^8) and the last piece's step is 2^-9: an
    element loses at most 2^-10); the weights by e^that - 1 and by binary16's
    rounding 2^-11 (their divisor too, but for that rounding), the L-term sums
    by L 2^-22: all times sum p_j |V_j|.  Weights times value scales that are
    subnormal in binary16 are off by up to 2^-25 instead: the row's largest
    weight w times 2^e, the power of two at or over a tile's largest value scale
    m (2^e < 2 m), is held at 2^3 or more, so that 2^-25 is at most 2^-27 w m, a
    key, times its code.  Then one rounding of the result.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
MAXF = {"e4m3": 448.0, "e5m2": 57344.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def half(dt):
    return torch.finfo(dt).eps / 2


def smallest(dt):
    """Half the smallest subnormal step."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def decode(codes, fmt):
    return codes.view(CODE[fmt]).float().to(F64)


def half_step(u, fmt):
    """Half the spacing of the format's values around |u|."""
    mant, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(u.abs().clamp_min(2.0 ** emin))).clamp_min(emin)
    return torch.exp2(e - mant) / 2


def norm(x, gamma, eps):
    x = x.to(F64)
    if gamma is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.to(F64)


def rotate(x, table, positions, style):
    """(rotated, the sum of the magnitudes of its terms)."""
    if table is None:
        return x, x.abs()
    r = table.shape[1]
    row = table.to(F64)[positions][:, None]
    c, s = row[..., :r // 2], row[..., r // 2:]
    ia = torch.arange(r // 2) if style == "half" else 2 * torch.arange(r // 2)
    ib = ia + (r // 2 if style == "half" else 1)
    a, b = x[..., ia], x[..., ib]
    out, mag = x.clone(), x.abs()
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return out, mag


def check_rows(got, want, mag, what=""):
    dt = got.dtype
    tol = half(dt) * want.abs() + 2.0 ** -19 * mag * (1 + half(dt)) + smallest(dt)
    err = (got.to(F64) - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err / tol).max()):.3g} tol"


def check_codes(codes, scale, want, mag, fmt, mode, what=""):
    """codes [..., D] uint8 and scale [...] (row) or a number (tensor) against
    the values they should stand for."""
    if mode == "row":
        most = want.abs().amax(-1)
        s = torch.where(most > 0, most / MAXF[fmt], torch.ones_like(most))
        rel = ((scale.to(F64) - s).abs() / s).max() if s.numel() else 0.0
        assert rel <= 4e-6, f"{what}: scale off by {float(rel):.3g}"
        s = s[..., None]
    else:
        s = float(scale)
    u = (want / s).clamp(-MAXF[fmt], MAXF[fmt])
    err = (decode(codes, fmt) - u).abs()
    tol = half_step(u, fmt) + 2.0 ** -18 * (mag / s)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, {float((err / tol).max()):.3g} tol"


def attention(q, k, v, visible, scale, codes=None):
    """One sequence: q [n, Hq, D], k, v [L, Hk, D] binary64, visible [n, L];
    codes [L, Hk, D]: magnitudes of the values' codes times the largest value
    scale of their head.  (out, its bound without the last rounding)."""
    n, Hq, D = q.shape
    L, Hk = k.shape[0], k.shape[1]
    G = Hq // Hk
    out, tol = torch.zeros(n, Hq, D, dtype=F64), torch.zeros(n, Hq, D, dtype=F64)
    q = q.to(F64)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        for i in range(n):
            w = visible[i].nonzero()[:, 0]
            if not len(w):
                continue
            s = (kh[w] @ q[i, h]) * scale
            p = torch.softmax(s, 0)
            A = float(((kh[w].abs() @ q[i, h].abs()) * scale).max())
            cut = float(kh[w].abs().sum(-1).max() * q[i, h].abs().max()) * scale * 2.0 ** -17
            rel = (2.0 ** -11 + 2 * math.expm1(D * 2.0 ** -22 * A + cut) + L * 2.0 ** -22 +
                   2.0 ** -20)
            out[i, h] = p @ vh[w]
            tol[i, h] = rel * (p @ vh[w].abs())
            if codes is not None:
                tol[i, h] += 2.0 ** -27 * p.max() * codes[w, h // G].sum(0)
    return out, tol


def check_attention(got, want, tol, what=""):
    dt = got.dtype
    bound = half(dt) * want.abs() + tol * (1 + half(dt)) + smallest(dt)
    got = got.to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN pattern"
    err = torch.where(torch.isnan(want), torch.zeros_like(want), (got - want).abs())
    bad = err > torch.nan_to_num(bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float((err / bound.clamp_min(1e-300)).nan_to_num().max()):.3g} tol")
