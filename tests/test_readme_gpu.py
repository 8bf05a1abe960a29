"""The README's step of drafted tokens, run as it stands there: a tree's accepted tokens must
leave the cache of their text written at once."""
import os
import re

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn

pytestmark = pytest.mark.gpu

V, H, HQ, HK, D = 64, 128, 4, 2, 64
LAYERS = ("q = rarn.qk_norm_rope_kv_write(q, k, v_rows, g, g, 1e-6, cos_sin, positions, cache, "
          "slots)\n")


def step_of_the_readme():
    here = os.path.dirname(os.path.abspath(__file__))
    text = open(os.path.join(os.path.dirname(here), "README.md")).read()
    code = re.search(r"# a step of drafted tokens around it.*?\n\n", text, re.S).group(0)
    return re.sub(r"(?m)^\.\.\. .*\n", LAYERS, code)


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def test_a_tree_leaves_the_cache_of_its_text():
    rarn.watchdog(clear=True)
    gen = torch.Generator().manual_seed(3)

    def rand(*shape):
        return torch.randn(*shape, generator=gen).to(torch.bfloat16).cuda()

    keys, values, g = rand(V, HK, D), rand(V, HK, D), rand(D).abs() + 0.5
    angle = torch.arange(64, dtype=torch.float64)[:, None] * 0.7 ** torch.arange(D // 2)
    table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    # two trees and two rows of padding; the tokens that the target accepts stand on
    # branches that lie apart
    parents = [-1, 0, 0, 2, 2, 4] + [-1, 0, 1, 1, 0] + [0, 0]
    drafts = ints([5, 6, 7, 8, 9, 10] + [11, 12, 13, 14, 15] + [0, 0], torch.int64)
    text = [[5, 7, 9, 10], [11, 12, 14]]
    follow = {5: 7, 7: 9, 9: 10, 10: 1, 11: 12, 12: 14, 14: 2}
    probs = torch.zeros(13, V)
    for r, t in enumerate(drafts.tolist()):
        probs[r, follow.get(t, 3)] = 1
    x = rand(13, H)
    space = dict(rarn=rarn, torch=torch, B=2, width=2, num_pages=4, T=13, context_lens=ints([0, 0]),
                 new_lens=ints([6, 5]), drafts=drafts, parents=ints(parents), probs=probs.cuda(),
                 depths=ints([0, 1, 1, 2, 2, 3] + [0, 1, 2, 2, 1] + [0, 0], torch.int64),
                 rows=ints([*range(6), *range(5), 0, 0], torch.int64), most=4,
                 u=torch.full((13,), 0.5, device="cuda"), v=torch.full((2,), 0.5, device="cuda"),
                 block_out=x, residual=x.clone(), gate=x[0], post_gamma=x[1], pre_gamma=x[2],
                 cache=rarn.KVCache.empty(4, 16, HK, D), cos_sin=table, g=g, q=rand(13, HQ, D),
                 k=keys[drafts], v_rows=values[drafts])
    exec(step_of_the_readme(), space)
    assert space["context_lens"].tolist() == [4, 3]
    assert [t[:n] for t, n in zip(space["tokens"].tolist(), (4, 3))] == [[7, 9, 10, 1], [12, 14, 2]]

    def read(cache, page_table):
        k, v = (torch.empty(7, HK, D, device="cuda") for _ in range(2))
        rarn.kv_cache_read(cache, page_table, ints([0, 4, 7]), k, v)
        return k, v

    flat = ints([t for s in text for t in s], torch.int64)
    once = rarn.KVCache.empty(4, 16, HK, D)
    pages = rarn.KVPages.empty(2, 2, 4, 16)
    _, slots, positions, _ = rarn.kv_step(pages, ints([0, 0]), ints([4, 3]), 7)
    rarn.qk_norm_rope_kv_write(rand(7, HQ, D), keys[flat], values[flat], g, g, 1e-6, table,
                               positions, once, slots)
    for got, want in zip(read(space["cache"], space["pages"].page_table),
                         read(once, pages.page_table)):
        assert torch.equal(got, want)
    assert rarn.watchdog() == 0
