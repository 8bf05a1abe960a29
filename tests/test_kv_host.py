"""Host-side checks of the attention side of the C ABI (per-head norm and
rotation, the 8-bit cache, attention of drafted tokens): argument errors come
before anything touches a GPU.  CPU only: no call here launches anything; the
addresses are fake and never dereferenced."""
import ctypes
import dataclasses

import pytest

import residual_add_rmsnorm_gb300 as rarn
from residual_add_rmsnorm_gb300 import build as rbuild

OK, INVALID, UNSUPPORTED, ALIAS, CUDA = 0, 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 2
BASE = 1 << 44


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rarn.library()


def at(i):
    """The i-th fake allocation, 16 TiB apart."""
    return (i + 1) * BASE


@dataclasses.dataclass
class Call:
    """A sound call's parts, to be spoilt one at a time."""
    T: int = 8
    D: int = 64
    Hq: int = 8
    Hk: int = 2
    dt: int = BF16
    eps: float = 1e-6

    def heads(self, i, n, **kw):
        d = dict(data=at(i), token_stride=n * self.D, head_stride=self.D, heads=n, dtype=self.dt)
        d.update(kw)
        return rarn.Heads(d["data"], d["token_stride"], d["head_stride"], d["heads"], d["dtype"])

    def rotation(self, **kw):
        d = dict(cos_sin=at(10), positions=at(11), table_rows=100, rot_dim=64, style=0)
        d.update(kw)
        return ctypes.byref(rarn.Rotation(d["cos_sin"], d["positions"], d["table_rows"],
                                          d["rot_dim"], d["style"]))

    def cache(self, **kw):
        D, H, ps = self.D, self.Hk, 16
        d = dict(k=at(12), v=at(13), k_scale=at(14), v_scale=at(15), page_stride=H * ps * D,
                 head_stride=ps * D, slot_stride=D, scale_page_stride=H * ps,
                 scale_head_stride=ps, scale_slot_stride=1, num_pages=20, page_size=ps, heads=H,
                 head_dim=D, format=0, scale_mode=1)
        d.update(kw)
        return ctypes.byref(rarn.KvCacheDesc(*[d[f] for f, _ in rarn.KvCacheDesc._fields_]))


def rope(lib, c, **kw):
    d = dict(q_out=c.heads(0, c.Hq), k_out=c.heads(1, c.Hk), q=c.heads(2, c.Hq),
             k=c.heads(3, c.Hk), q_gamma=at(4), k_gamma=at(5), rot=c.rotation(), T=c.T, D=c.D,
             eps=c.eps)
    d.update(kw)
    return lib.rarn_qk_norm_rope(d["q_out"], d["k_out"], d["q"], d["k"], d["q_gamma"],
                                 d["k_gamma"], d["rot"], d["T"], d["D"], d["eps"], None)


def write(lib, c, **kw):
    d = dict(cache=c.cache(), k=c.heads(3, c.Hk), v=c.heads(6, c.Hk), slots=at(7), T=c.T)
    d.update(kw)
    return lib.rarn_kv_cache_write(d["cache"], d["k"], d["v"], d["slots"], d["T"], None)


def fused(lib, c, **kw):
    d = dict(q_out=c.heads(0, c.Hq), cache=c.cache(), q=c.heads(2, c.Hq), k=c.heads(3, c.Hk),
             v=c.heads(6, c.Hk), q_gamma=at(4), k_gamma=at(5), rot=c.rotation(), slots=at(7),
             T=c.T, eps=c.eps)
    d.update(kw)
    return lib.rarn_qk_norm_rope_kv_write(d["q_out"], d["cache"], d["q"], d["k"], d["v"],
                                          d["q_gamma"], d["k_gamma"], d["rot"], d["slots"],
                                          d["T"], d["eps"], None)


def read(lib, c, **kw):
    d = dict(k_out=c.heads(0, c.Hk), v_out=c.heads(1, c.Hk), cache=c.cache(), table=at(7),
             stride=4, width=4, starts=at(8), B=3, rows=c.T)
    d.update(kw)
    return lib.rarn_kv_cache_read(d["k_out"], d["v_out"], d["cache"], d["table"], d["stride"],
                                  d["width"], d["starts"], d["B"], d["rows"], None)


def tree(lib, c, **kw):
    d = dict(out=c.heads(0, c.Hq), q=c.heads(2, c.Hq), cache=c.cache(), table=at(7), stride=4,
             width=4, ctx=at(8), starts=at(9), mask=at(16), words=1, B=3, tokens=c.T, scale=0.1,
             ws=at(17), bytes=1 << 30)
    d.update(kw)
    return lib.rarn_tree_attention(d["out"], d["q"], d["cache"], d["table"], d["stride"],
                                   d["width"], d["ctx"], d["starts"], d["mask"], d["words"],
                                   d["B"], d["tokens"], d["scale"], d["ws"], d["bytes"], None)


C = Call()

# a sound call gets as far as asking for a device
SOUND = [rope, write, fused, read, tree]


def _no_device():
    import torch
    return not torch.cuda.is_available()


@pytest.mark.parametrize("call", SOUND)
def test_sound_calls_pass_the_checks(lib, call):
    if not _no_device():
        pytest.skip("fake addresses: only without a device")
    assert call(lib, C) == CUDA


@pytest.mark.parametrize("kw", [
    dict(T=0), dict(T=0, q=C.heads(2, 8, data=None), q_gamma=None),
])
def test_no_rows_is_a_no_op(lib, kw):
    assert rope(lib, C, **kw) == OK
    assert write(lib, C, T=0) == OK
    assert fused(lib, C, T=0) == OK
    assert read(lib, C, rows=0) == OK and read(lib, C, B=0) == OK
    assert tree(lib, C, tokens=0) == OK and tree(lib, C, B=0) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID),
    (dict(D=0), INVALID),
    (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID),
    (dict(q=C.heads(2, 8, data=None)), INVALID),
    (dict(k_out=C.heads(1, 2, data=None)), INVALID),
    (dict(q=C.heads(2, 0)), INVALID),
    (dict(q=C.heads(2, 8, dtype=9)), INVALID),
    (dict(q=C.heads(2, 8, token_stride=-512)), INVALID),
    (dict(q_out=C.heads(0, 4)), INVALID),                       # other heads than q
    (dict(q_out=C.heads(0, 8, token_stride=100)), INVALID),     # rows of the output overlap
    (dict(q_out=C.heads(0, 8, head_stride=32)), INVALID),
    (dict(q=C.heads(2, 8, dtype=F16)), UNSUPPORTED),            # mixed types
    (dict(q=C.heads(2, 8, data=at(2) + 1)), INVALID),           # not element aligned
    (dict(q=C.heads(2, 5000), q_out=C.heads(0, 5000)), UNSUPPORTED),
    (dict(T=1 << 40), UNSUPPORTED),
    (dict(D=2048, q_out=C.heads(0, 8, token_stride=1 << 20, head_stride=2048),
          k_out=C.heads(1, 2, token_stride=1 << 20, head_stride=2048)), UNSUPPORTED),
    (dict(rot=C.rotation(rot_dim=63)), INVALID),
    (dict(rot=C.rotation(rot_dim=66)), INVALID),                # more than D
    (dict(rot=C.rotation(rot_dim=0)), INVALID),
    (dict(rot=C.rotation(style=2)), INVALID),
    (dict(rot=C.rotation(cos_sin=None)), INVALID),
    (dict(rot=C.rotation(positions=None)), INVALID),
    (dict(rot=C.rotation(table_rows=0)), INVALID),
    (dict(q_out=C.heads(2, 8, data=at(2) + 128)), ALIAS),       # shifted in place
    (dict(q_out=C.heads(3, 8)), ALIAS),                         # onto k
    (dict(k_out=C.heads(0, 2)), ALIAS),                         # onto q_out
    (dict(q_gamma=at(0) + 128), ALIAS),
    (dict(rot=C.rotation(cos_sin=at(1))), ALIAS),
    (dict(rot=C.rotation(positions=at(0))), ALIAS),
])
def test_norm_rope_refusals(lib, kw, want):
    assert rope(lib, C, **kw) == want


def test_in_place_inside_a_packed_projection(lib):
    """q, k and v side by side in one allocation: in place is no overlap, one
    element further is."""
    if not _no_device():
        pytest.skip("fake addresses: only without a device")
    row = (8 + 2 + 2) * 64
    q = C.heads(2, 8, token_stride=row)
    k = C.heads(2, 2, data=at(2) + 8 * 64 * 2, token_stride=row)
    assert rope(lib, C, q=q, k=k, q_out=q, k_out=k) == CUDA
    bad = C.heads(2, 2, data=at(2) + 7 * 64 * 2, token_stride=row)
    assert rope(lib, C, q=q, k=k, q_out=q, k_out=bad) == ALIAS
    # a head-major output
    hm = C.heads(0, 8, token_stride=64, head_stride=8 * 64)
    assert rope(lib, C, q_out=hm) == CUDA


CACHE_BAD = [
    (dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(format=5), INVALID), (dict(scale_mode=3), INVALID),
    (dict(head_stride=-16), INVALID),
    (dict(slot_stride=32), INVALID),                # slots overlap
    (dict(page_stride=16 * 64), INVALID),           # pages overlap
    (dict(scale_slot_stride=0), INVALID),
    (dict(head_dim=40, slot_stride=64), UNSUPPORTED),
    (dict(head_dim=272, slot_stride=272, head_stride=16 * 272, page_stride=32 * 272),
     UNSUPPORTED),
    (dict(k=at(12) + 8), UNSUPPORTED), (dict(slot_stride=72, head_stride=2048, page_stride=8192),
                                        UNSUPPORTED),
    (dict(page_size=(1 << 20) + 1), UNSUPPORTED),
    (dict(num_pages=1 << 31), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", CACHE_BAD)
def test_cache_refusals(lib, kw, want):
    for call in (write, fused, read, tree):
        assert call(lib, C, cache=C.cache(**kw)) == want


@pytest.mark.parametrize("call", [write, fused])
def test_write_refusals(lib, call):
    assert call(lib, C, cache=None) == INVALID
    assert call(lib, C, slots=None) == INVALID
    assert call(lib, C, slots=at(7) + 4) == INVALID
    assert call(lib, C, k=C.heads(3, 4)) == INVALID             # other heads than the cache
    assert call(lib, C, v=C.heads(6, 4)) == INVALID
    assert call(lib, C, v=C.heads(6, 2, dtype=F32)) == UNSUPPORTED
    assert call(lib, C, v=C.heads(12, 2)) == ALIAS              # v inside the cache's keys
    assert call(lib, C, slots=at(13)) == ALIAS
    assert call(lib, C, cache=C.cache(v=at(12) + 64)) == ALIAS  # keys over values
    assert call(lib, C, cache=C.cache(v_scale=at(14))) == ALIAS
    assert call(lib, C, cache=C.cache(k_scale=at(12))) == ALIAS
    # one scale per tensor is read: it may not lie inside the codes
    assert call(lib, C, cache=C.cache(scale_mode=0, k_scale=at(13) + 64)) == ALIAS


def test_pools_with_keys_and_values_interleaved_by_pages(lib):
    if not _no_device():
        pytest.skip("fake addresses: only without a device")
    half = 2 * 16 * 64
    assert write(lib, C, cache=C.cache(v=at(12) + half, page_stride=2 * half)) == CUDA
    assert write(lib, C, cache=C.cache(v=at(12) + half - 64, page_stride=2 * half)) == ALIAS


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(B=-1), INVALID), (dict(width=-1), INVALID),
    (dict(stride=-1), INVALID), (dict(table=None), INVALID), (dict(starts=None), INVALID),
    (dict(starts=at(8) + 2), INVALID), (dict(B=(1 << 20) + 1), UNSUPPORTED),
    (dict(k_out=C.heads(0, 3)), INVALID),
    (dict(v_out=C.heads(1, 2, dtype=F16)), UNSUPPORTED),
    (dict(v_out=C.heads(0, 2)), ALIAS), (dict(k_out=C.heads(12, 2)), ALIAS),
    (dict(k_out=C.heads(7, 2)), ALIAS), (dict(v_out=C.heads(14, 2)), ALIAS),
    (dict(rows=1 << 33), UNSUPPORTED),
])
def test_read_refusals(lib, kw, want):
    assert read(lib, C, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(words=-1), INVALID), (dict(words=0), INVALID),
    (dict(mask=at(16) + 1), INVALID), (dict(words=(1 << 16) + 1), UNSUPPORTED),
    (dict(ctx=None), INVALID), (dict(starts=None), INVALID), (dict(table=None), INVALID),
    (dict(q=C.heads(2, 7), out=C.heads(0, 7)), INVALID),        # heads not in groups
    (dict(out=C.heads(0, 4)), INVALID),
    (dict(q=C.heads(2, 8, dtype=F32), out=C.heads(0, 8, dtype=F32)), UNSUPPORTED),
    (dict(q=C.heads(2, 8, dtype=F16)), UNSUPPORTED),
    (dict(q=C.heads(2, 8, data=at(2) + 2)), UNSUPPORTED),       # q not 16-byte aligned
    (dict(q=C.heads(2, 8, token_stride=516)), UNSUPPORTED),
    (dict(ws=None), INVALID), (dict(ws=at(17) + 8), INVALID), (dict(bytes=1000), INVALID),
    (dict(out=C.heads(2, 8)), ALIAS), (dict(ws=at(0)), ALIAS), (dict(ws=at(12)), ALIAS),
    (dict(out=C.heads(16, 8)), ALIAS), (dict(ws=at(8)), ALIAS),
])
def test_tree_refusals(lib, kw, want):
    assert tree(lib, C, **kw) == want


def test_tree_needs_a_supported_head_size(lib):
    for D in (16, 32, 48, 80, 112, 160):
        c = Call(D=D)
        assert tree(lib, c) == UNSUPPORTED
        assert lib.rarn_tree_attention_workspace_bytes(8, 3, 8, 2, D) == -1


@pytest.mark.parametrize("args", [(-1, 1, 8, 2, 64), (1, -1, 8, 2, 64), (1, 1, 0, 2, 64),
                                  (1, 1, 8, 3, 64), (1, 1, 8, 2, 65), (1 << 40, 1, 8, 2, 64)])
def test_workspace_query_refusals(lib, args):
    assert lib.rarn_tree_attention_workspace_bytes(*args) == -1


def test_workspace_query(lib):
    assert lib.rarn_tree_attention_workspace_bytes(0, 4, 8, 2, 64) == 0
    for D in (64, 96, 128, 192, 256):
        n = lib.rarn_tree_attention_workspace_bytes(32, 4, 8, 2, D)
        c = Call(D=D, T=32)
        assert n > 0 and n % 16 == 0
        assert tree(lib, c, B=4, bytes=n - 1) == INVALID
        if _no_device():
            assert tree(lib, c, B=4, bytes=n) == CUDA


@pytest.mark.parametrize("call", SOUND)
def test_sizes_whose_offsets_would_overflow(lib, call):
    """Steps times strides beyond 2^40 are refused before they are multiplied."""
    c = Call(T=1 << 20)
    heads = {rope: ("q", 2, 8), write: ("k", 3, 2), fused: ("q", 2, 8), read: ("k_out", 0, 2),
             tree: ("q", 2, 8)}[call]
    far = {heads[0]: c.heads(heads[1], heads[2], token_stride=1 << 38)}
    assert call(lib, c, **far) == UNSUPPORTED
    if call is not rope:
        assert call(lib, C, cache=C.cache(num_pages=1 << 20, page_stride=1 << 36)) == UNSUPPORTED
        assert call(lib, C, cache=C.cache(scale_page_stride=1 << 39)) == UNSUPPORTED
    if call in (rope, fused):
        assert call(lib, C, rot=C.rotation(table_rows=1 << 60)) == UNSUPPORTED
    if call is tree:
        assert call(lib, C, width=1 << 27) == UNSUPPORTED   # 2^31 keys of a sequence
        if _no_device():
            assert call(lib, C, width=(1 << 27) - 256) == CUDA


def test_strides_of_dimensions_of_one_do_not_matter(lib):
    if not _no_device():
        pytest.skip("fake addresses: only without a device")
    c = Call(T=1)
    assert tree(lib, c, q=c.heads(2, 8, token_stride=3)) == CUDA
    c = Call(Hq=2, Hk=1)
    assert tree(lib, c, q=c.heads(2, 2, head_stride=65)) == UNSUPPORTED
    c = Call(Hq=1, Hk=1)
    assert tree(lib, c, q=c.heads(2, 1, head_stride=65)) == CUDA


@pytest.mark.parametrize("args,want", [
    ((1, 1, 32, 8, 128, 16), "tree.rows rows=8"), ((64, 64, 32, 8, 128, 16), "tree.rows rows=8"),
    ((4, 1, 32, 8, 128, 16), "tree.rows rows=16"), ((5, 1, 32, 8, 128, 16), "tree.tiles rows=128"),
    ((5, 1, 32, 8, 128, 12), "tree.rows rows=16"), ((50, 1, 32, 8, 256, 16), "tree.rows rows=8"),
    ((64 * 8, 64, 32, 8, 128, 16), "tree.rows rows=16"),
    ((64 * 9, 64, 32, 8, 128, 16), "tree.tiles rows=128"),
    ((16 * 32, 16, 64, 8, 64, 8), "tree.tiles rows=256"),
    ((8, 1, 32, 8, 192, 16), "tree.rows rows=8"), ((9, 1, 32, 8, 192, 16), "tree.rows rows=16"),
    ((0, 4, 8, 2, 64, 16), "none: no rows"),
    ((4, 4, 8, 2, 80, 16), "none: unsupported sizes"),
])
def test_plan_tree_attention(lib, args, want):
    assert rarn.plan_tree_attention(*args) == want


def test_plan_tree_attention_refusals(lib):
    buf = ctypes.create_string_buffer(64)
    assert lib.rarn_plan_tree_attention(-1, 1, 8, 2, 64, 16, buf, 64) == INVALID
    assert lib.rarn_plan_tree_attention(1, 1, 8, 2, 64, 0, buf, 64) == INVALID
    assert lib.rarn_plan_tree_attention(1, 1, 8, 2, 64, 16, None, 64) == INVALID
    assert lib.rarn_plan_tree_attention(1, 1, 8, 2, 64, 16, buf, 0) == INVALID
