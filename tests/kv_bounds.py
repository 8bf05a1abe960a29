"""An error bound of the attention over the 8-bit cache, key by key, for caches
whose scales differ so much that one bound for all keys says nothing.

One row: scores s_j, weights p_j = softmax, o = sum p_j V_j.
  * Scores are off by d_j <= D 2^-22 sum |q_d K_jd| (a tensor core's binary32
    sums) + sum |r_d K_jd|, times the softmax scale and the key's.  r_d is what the
    queries' 8-bit pieces lose: with the row scaled by a power of two to a largest
    magnitude in [2^7, 2^8), an element's 8 or 11 bits are held but for what lies
    under the last piece's step, 2^-9: its distance from a multiple of that.
    With t the key of the largest weight, and sum p_j (V_j - o) = 0,
      o' - o = sum p_j (e^d_j - e^d_t) (V_j - o) / sum p_j e^d_j,
    at most the sum over j != t of (p_j / p_t) (e^(|d_j| + |d_t|) - 1) |V_j - o|.
  * A weight times its value scale is rounded to binary16: by 2^-11 of it, or by
    2^-25 where it is subnormal; the row's largest weight w times the largest
    value scale m that it sees is held at 2^1 w m / 2^e or more, e the exponent
    over m and up to two more: 2^-25 w m, but never more than the term itself.
  * Sums of L binary32 terms: L 2^-22 of their magnitudes; the divisor 2^-20.
"""
import torch

from kv_ref import F64


def attention(q, kc, ks, vc, vs, visible, scale):
    """One sequence: q [n, Hq, D]; codes' values kc, vc [L, Hk, D] and scales ks,
    vs [L, Hk] in binary64; visible [n, L].  (out, bound, sum p_j |V_j|)."""
    n, Hq, D = q.shape
    L, Hk = ks.shape
    G = Hq // Hk
    q = q.to(F64)
    out, tol, mag = (torch.zeros(n, Hq, D, dtype=F64) for _ in range(3))
    for h in range(Hq):
        hk = h // G
        K, V = kc[:, hk] * ks[:, hk, None], vc[:, hk] * vs[:, hk, None]
        for i in range(n):
            w = visible[i].nonzero()[:, 0]
            if not len(w):
                continue
            k, v = K[w], V[w]
            s = (k @ q[i, h]) * scale
            p = torch.softmax(s, 0)
            unit = torch.exp2(torch.floor(torch.log2(q[i, h].abs().max())) - 7 - 9)
            r = (q[i, h] - torch.round(q[i, h] / unit) * unit).abs()
            d = (D * 2.0 ** -22 * (k.abs() @ q[i, h].abs()) + k.abs() @ r) * scale
            t = int(p.argmax())
            o = p @ v
            far = (p / p[t]) * torch.expm1((d + d[t]).clamp_max(700.0))
            far[t] = 0
            size = p @ v.abs()
            term = p[:, None] * v.abs()
            small = 2.0 ** -25 * p[t] * vs[w, hk].abs().max() * vc[w, hk].abs()
            out[i, h], mag[i, h] = o, size
            tol[i, h] = (far @ (v - o).abs() + torch.minimum(term, small).sum(0) +
                         (2.0 ** -11 + 2.0 ** -20 + L * 2.0 ** -22) * size)
    return out, tol, mag
