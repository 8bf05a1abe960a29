"""A run of a step's operators together: a small model decoded token by token, and
with drafted trees that are verified, must say the same and leave the same cache.

The model's next token is a hash of the histogram of all tokens seen and of the
last one.  Queries of zeros weigh all visible keys alike and values are one-hot, so
that the attention's output times the number of tokens is the histogram; with 2^-10
of error on at most 130 tokens it rounds to whole numbers, and nothing hangs on
rounding.  A single row too many or too few seen, or one in a wrong slot, changes
what is said from there on."""
import random

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
import step_ref as R

pytestmark = pytest.mark.gpu

V, H, HQ, HK, D, PAGE, WIDTH = 64, 256, 8, 2, 64, 16, 12
EPS = 1e-6


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


class Model:
    """Keys: projected, normalised, turned by three axes; values: one-hot tokens."""

    def __init__(self, sequences, seed=0):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return torch.randn(*shape, generator=g).to(torch.bfloat16).cuda()

        self.embed, self.keys = w(V, H), w(V, HK, D)
        self.values = torch.eye(V, dtype=torch.bfloat16, device="cuda")[:, None].repeat(1, HK, 1)
        self.gamma, self.gate = w(H).abs() + 0.5, w(H)
        self.qg = torch.zeros(D, dtype=torch.bfloat16, device="cuda")
        self.kg = w(D).abs() + 0.5
        self.primes = ints([r for r in torch.randint(1, 10 ** 6, (V,), generator=g).tolist()],
                           torch.int64)
        f = 100.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
        a = torch.arange(256, dtype=torch.float64)[:, None] * f
        self.table = torch.cat([a.cos(), a.sin()], 1).float().cuda()
        self.cache = rarn.KVCache.empty(sequences * WIDTH, PAGE, HK, D)
        self.pages = rarn.KVPages.empty(sequences, WIDTH, sequences * WIDTH, PAGE)

    def write(self, tokens, positions, slots):
        axes = torch.stack([positions, positions // 8, positions % 8])
        q = torch.ones(len(tokens), HQ, D, dtype=torch.bfloat16, device="cuda")
        return rarn.qk_norm_rope_kv_write(q, self.keys[tokens], self.values[tokens], self.qg,
                                          self.kg, EPS, self.table, axes, self.cache, slots,
                                          sections=(8, 12, 12), section_order="cyclic")

    def probs(self, tokens, positions, slots, context, starts, mask):
        """The target's distributions behind tokens: all weight on one."""
        q = self.write(tokens, positions, slots)
        att = rarn.tree_attention(q, self.cache, self.pages.page_table, context, starts, mask)
        seen = att[:, 0].float() * (positions + 1)[:, None]
        count = seen.round()
        live = slots >= 0
        assert float((seen - count).abs()[live].max()) < 0.25
        # the norms around the block, in passing
        x, stream = self.embed[tokens], att.reshape(len(tokens), -1)[:, :H].float()
        y = rarn.gated_add_rms_norm(x, stream, self.gamma, self.gamma, EPS, gate=self.gate,
                                    scale=2.0)
        n = int(live.sum())
        R.check_block(y.cpu()[:n], stream.cpu()[:n], x.cpu()[:n],
                      att.reshape(len(tokens), -1)[:n, :H].float().cpu(), self.gamma.cpu(),
                      self.gamma.cpu(), EPS, self.gate.cpu().expand(n, H), 2.0)
        following = ((count.long() * self.primes).sum(-1) + 31 * tokens) % V
        return torch.nn.functional.one_hot(following, V).float()


def decode(model, prompts, count, drafter=None):
    """At least `count` tokens behind each prompt; drafter(b, said) -> drafted (token,
    parent) pairs below the last token."""
    B = len(prompts)
    said = [[] for _ in prompts]
    last = [p[-1] for p in prompts]
    context = [0] * B
    # the prompts but for their last tokens, as one chain each
    new = [len(p) - 1 for p in prompts]
    starts, slots, positions, _ = rarn.kv_step(model.pages, ints(context), ints(new), sum(new))
    flat = ints([t for p in prompts for t in p[:-1]], torch.int64)
    model.probs(flat, positions, slots, ints(context), starts, None)
    context = new
    while min(len(s) for s in said) < count:
        trees = [[(last[b], -1)] + (drafter(b, said[b]) if drafter else []) for b in range(B)]
        new = [len(t) for t in trees]
        N = sum(new) + 5            # padded, as a captured step is
        starts, slots, _, served = rarn.kv_step(model.pages, ints(context), ints(new), N)
        assert int(served) == B
        tokens, parents, positions, mask = [], [], [], []
        for b, t in enumerate(trees):
            seen, deep = [], []
            for i, (token, up) in enumerate(t):
                seen.append((seen[up] if up >= 0 else 0) | 1 << i)
                deep.append(deep[up] + 1 if up >= 0 else context[b])
                tokens.append(token)
                parents.append(up)
            mask += seen
            positions += deep
        pad = [0] * 5
        tokens = ints(tokens + pad, torch.int64)
        p = model.probs(tokens, ints(positions + pad, torch.int64), slots, ints(context), starts,
                        ints(mask + pad)[:, None])
        out, path, lengths = rarn.verify_drafts(p, tokens, starts, torch.rand(N, device="cuda"),
                                                torch.rand(B, device="cuda"), 4,
                                                parents=ints(parents + pad))
        rarn.kv_cache_compact(model.cache, model.pages.page_table, ints(context), path, lengths)
        got = out.tolist()
        for b, n in enumerate(lengths.tolist()):
            said[b] += got[b][:n]
            last[b] = got[b][n - 1]
            context[b] += n
        rarn.kv_trim(model.pages, ints(context))
        assert model.pages.held.tolist() == [-(-n // PAGE) for n in context]
    return said, context


def read(model, context):
    total = sum(context)
    k, v = (torch.empty(total, HK, D, device="cuda") for _ in range(2))
    starts = [0]
    for n in context:
        starts.append(starts[-1] + n)
    rarn.kv_cache_read(model.cache, model.pages.page_table, ints(starts), k, v)
    return k, v


@pytest.mark.parametrize("seed", [0, 1, 2])
def test_drafts_change_nothing_that_is_said(seed):
    rarn.watchdog(clear=True)
    r = random.Random(seed)
    B, count = 5, 40
    prompts = [[r.randrange(V) for _ in range(r.randint(2, 50))] for _ in range(B)]
    plain, _ = decode(Model(B, seed), prompts, count + 6)
    assert len({t for s in plain for t in s}) > V // 2      # a varied text
    # the same on the host
    m = Model(B, seed)
    primes = m.primes.tolist()
    for p, s in zip(prompts, plain):
        text = list(p)
        for t in s:
            assert t == (sum(primes[x] for x in text) + 31 * text[-1]) % V
            text.append(t)
    steps = [0]

    def drafter(b, said):
        """A tree with the right continuation somewhere, as far as it is drawn."""
        steps[0] += 1
        tree, at, n = [], 0, len(said)
        for i in range(r.randint(0, 5)):
            right = plain[b][n + i] if n + i < count and r.random() < 0.8 else r.randrange(V)
            row = [r.randrange(V) for _ in range(r.randint(0, 3))] + [right]
            r.shuffle(row)
            first = len(tree) + 1
            tree += [(t, at) for t in row]
            at = first + row.index(right)
        return tree

    said, context = decode(m, prompts, count, drafter)
    for got, want in zip(said, plain):
        n = min(len(got), len(want))
        assert n >= count and got[:n] == want[:n]
    assert steps[0] < B * count * 0.7       # drafts were accepted
    # the cache is that of the text written at once
    k, v = read(m, context)
    whole = Model(B, seed)
    texts = [(p + s)[:n] for p, s, n in zip(prompts, said, context)]
    flat = ints([t for x in texts for t in x], torch.int64)
    _, slots, positions, _ = rarn.kv_step(whole.pages, ints([0] * B), ints(context), len(flat))
    whole.write(flat, positions, slots)
    k2, v2 = read(whole, context)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    # everything is given back
    rarn.kv_trim(m.pages, ints([0] * B))
    assert int(m.pages.free_count) == B * WIDTH
    assert sorted(m.pages.free_pages.tolist()) == list(range(B * WIDTH))
    assert rarn.watchdog() == 0
