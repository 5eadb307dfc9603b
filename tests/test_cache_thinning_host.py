"""Host side of the rotation over several axes, the attention's log-sum-exp, the cached tokens' scores and the eviction
(CPU only): refusals before any launch, the binding's checks; and pins of the fp64 statements that the GPU tests
compare with."""
import ctypes
import math
import pathlib
import re

import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_linear_conv1d_gb300 import build as gdn_build  # noqa: E402
from tests import attnref as R  # noqa: E402
from tests import thinref as T  # noqa: E402
from tests.test_attention_host import BAD_CACHES, ODD, P, cache  # noqa: E402


@pytest.fixture(scope="module")
def b():
    gdn_build.build()
    from gated_deltanet_linear_conv1d_gb300 import binding
    return binding


def mrope_call(b, axes, q=P, k=P, qo=P, ko=P, rot=64, pos=P, f=P, v=None, cc=None, slot=None, n=4, hq=24, hkv=4, d=256,
               eps=1e-6, qg=P):
    return b._lib.gdn_qk_norm_mrope(q, 6144, 256, k, 1024, 256, qg, P, eps, pos, f, rot, axes, 0, qo, ko, v, 1024, 256, cc,
                                    slot, n, hq, hkv, d, None, None)


def score_call(b, c, q=P, lse=P, table=P, mp=2, ctx=P, mask=None, scale=0.1, decay=1.0, score=P, slot=P, init=None, slots=4,
               room=128, N=2, nodes=8, hq=24):
    return b._lib.gdn_kv_score(ctypes.byref(c), q, lse, table, mp, ctx, mask, scale, decay, score, slot, init, slots, room, N,
                               nodes, hq, None, None)


def evict_call(b, c, table=P, mp=2, length=P, budget=P, sinks=0, recent=0, dst=None, dmp=0, score=P, slot=P, dst_slot=None,
               slots=4, room=128, kept=P, most=10, new_len=512, N=2):
    return b._lib.gdn_kv_evict(ctypes.byref(c), table, mp, length, budget, sinks, recent, dst, dmp, score, slot, dst_slot, slots,
                               room, kept, most, new_len, N, None, None)


@pytest.mark.parametrize("kw,why", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry_point(b, kw, why):
    c, want = cache(b, **kw), getattr(b, "GDN_ERR_" + why)
    p, axes = ctypes.byref(c), ctypes.byref(b.make_rope_axes((12, 10, 10)))
    assert mrope_call(b, axes, v=P, cc=p, slot=P, hkv=c.num_kv_heads, d=c.head_dim) == want
    assert b._lib.gdn_tree_attention_lse(p, P, P, 2, P, None, None, 0.1, P, P, 2, 1, 24, P, 1 << 30, None, None) == want
    assert score_call(b, c) == want
    assert evict_call(b, c) == want


def test_mrope_arguments(b):
    axes = b.make_rope_axes((12, 10, 10))
    ref = ctypes.byref(axes)
    for kw in (dict(k=None), dict(q=None), dict(qo=None), dict(ko=None), dict(qg=None), dict(eps=-1.0), dict(pos=None),
               dict(f=None), dict(rot=72), dict(rot=272), dict(k=ODD), dict(n=-1), dict(hq=0), dict(v=P), dict(slot=P)):
        assert mrope_call(b, ref, **kw) == b.GDN_ERR_INVALID_ARG, kw
    assert mrope_call(b, None) == b.GDN_ERR_INVALID_ARG
    for num, at, axis in ((0, 0, 0), (5, 0, 0), (-1, 0, 0), (3, 31, 3), (1, 12, 1), (4, 0, 255)):
        bad = b.GdnRopeAxes(num, axes.axis)
        bad.axis[at] = axis
        assert mrope_call(b, ctypes.byref(bad)) == b.GDN_ERR_INVALID_ARG, (num, at, axis)
    assert mrope_call(b, ref, d=64) == b.GDN_ERR_UNSUPPORTED
    assert mrope_call(b, ref, n=0) == b.GDN_OK
    behind = b.make_rope_axes((12, 10, 10))
    behind.axis[32] = 9  # not one of the 32 frequencies
    assert mrope_call(b, ctypes.byref(behind), n=0) == b.GDN_OK


def test_axes_of_the_frequencies(b):
    def axis(*a, **kw):
        x = b.make_rope_axes(*a, **kw)
        return list(x.axis)[:sum(a[0])]

    assert axis((2, 1, 1)) == [0, 0, 1, 2]
    assert axis((4, 2, 1), mixed=True) == [0, 1, 2, 0, 1, 0, 0]
    assert axis((2, 2, 2, 2), mixed=True) == [0, 1, 2, 3] * 2
    assert axis((12, 10, 10), mixed=True).count(1) == 10
    assert axis((3,), mixed=True) == [0] * 3
    for bad in ((), (1, 2, 3, 4, 5), (-1, 5), (100, 29)):
        with pytest.raises(ValueError):
            b.make_rope_axes(bad)
    with pytest.raises(ValueError, match="turns"):
        b.make_rope_axes((1, 5, 5), mixed=True)


@pytest.mark.parametrize("sections", [(6, 5, 5), (24, 20, 20), (32, 1)])
def test_axes_of_more_or_fewer_frequencies_are_refused(b, sections):
    """The frequencies without a section would all turn by axis 0."""
    x, gamma = torch.zeros(2, 4, 256, dtype=torch.bfloat16), torch.ones(256)
    pos, freq = torch.zeros(len(sections), 2, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="frequencies"):
        b.gdn_qk_norm_mrope(x, x, gamma, gamma, 1e-6, pos, freq, b.make_rope_axes(sections), x.clone(), x.clone())


def test_lse_arguments(b):
    c = cache(b)
    ref = ctypes.byref(c)
    need = b.gdn_tree_attention_workspace_bytes(c, 2, 8, 24)

    def attn(lse=P, q=P, N=2, size=need):
        return b._lib.gdn_tree_attention_lse(ref, q, P, 2, P, None, None, 0.1, P, lse, N, 8, 24, P, size, None, None)

    for kw in (dict(lse=None), dict(lse=258), dict(q=None), dict(size=need - 1), dict(N=-1)):
        assert attn(**kw) == b.GDN_ERR_INVALID_ARG, kw
    assert attn(N=0) == b.GDN_OK and attn(N=0, lse=None) == b.GDN_OK


def test_score_arguments(b):
    c = cache(b)
    for kw in (dict(q=None), dict(lse=None), dict(table=None), dict(mp=0), dict(mp=-1), dict(ctx=None), dict(score=None),
               dict(slot=None), dict(q=ODD), dict(lse=257), dict(mask=257), dict(score=258), dict(scale=math.inf),
               dict(decay=math.nan), dict(decay=math.inf), dict(slots=0), dict(room=0), dict(room=-1), dict(N=-1),
               dict(N=65536), dict(nodes=0), dict(nodes=65), dict(hq=0)):
        assert score_call(b, c, **kw) == b.GDN_ERR_INVALID_ARG, kw
    for kw in (dict(hq=25), dict(hq=260), dict(room=(1 << 30) + 1)):
        assert score_call(b, c, **kw) == b.GDN_ERR_UNSUPPORTED, kw
    assert score_call(b, c, N=0) == b.GDN_OK


def test_evict_arguments(b):
    c = cache(b)
    for kw in (dict(table=None), dict(mp=0), dict(mp=-1), dict(length=None), dict(budget=None), dict(sinks=-1),
               dict(recent=-1), dict(dst=512, dmp=-1, dst_slot=512), dict(dmp=3), dict(dst=512, dmp=2), dict(dst_slot=512),
               dict(dst=P, dmp=2, dst_slot=512), dict(dst=512, dmp=2, dst_slot=P), dict(score=None), dict(score=258), dict(slot=None),
               dict(slots=0), dict(room=0), dict(kept=None), dict(most=-1), dict(new_len=None), dict(new_len=P), dict(N=-1),
               dict(budget=P, new_len=P), dict(slot=512), dict(table=512), dict(dst=P + 64, dmp=2, dst_slot=512)):
        assert evict_call(b, c, **kw) == b.GDN_ERR_INVALID_ARG, kw
    assert evict_call(b, c, room=(1 << 30) + 1) == b.GDN_ERR_UNSUPPORTED
    assert evict_call(b, c, N=(1 << 26) + 1) == b.GDN_ERR_UNSUPPORTED  # 2^28 heads
    assert evict_call(b, c, N=0) == b.GDN_OK


def test_evict_of_more_heads_than_a_grid_has_blocks_is_refused(b):
    """2^28 (request, head) pairs of eight blocks each are 2^31, one more than a grid may have."""
    assert evict_call(b, cache(b), N=1 << 26) == b.GDN_ERR_UNSUPPORTED


def test_binding_checks(b):
    c = cache(b)
    x = torch.zeros(2, 24, 256, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    score = torch.zeros(4, 4, 128)
    with pytest.raises(ValueError, match="CUDA"):
        b.gdn_kv_score(c, x, torch.zeros(2, 24), torch.zeros(2, 2, dtype=torch.int32), i, 0.1, score, i)
    with pytest.raises(ValueError, match="CUDA"):
        b.gdn_kv_evict(c, torch.zeros(2, 2, dtype=torch.int32), i, i, score, i, torch.zeros(2, 4, 9, dtype=torch.int32),
                       i.clone())
    with pytest.raises(ValueError, match="new_len"):
        b.gdn_kv_evict(c, torch.zeros(2, 2, dtype=torch.int32), i, i, score, i, torch.zeros(2, 4, 9, dtype=torch.int32), i)


def test_what_the_kernel_in_front_writes_is_read_by_plain_loads():
    """These kernels may begin before the one in front of them ends. A read-only load (__ldg) is for memory that nobody writes
    while a kernel is there: not for the weights, the log-sum-exps, the kept indices and the new lengths."""
    csrc = pathlib.Path(gdn_build.CSRC)
    for name in ("kv_evict.cu", "kv_score.cu", "kv_score.cuh", "kv_score_pair.cu"):
        text = (csrc / name).read_text()
        assert "griddepcontrol.wait" in text or name.endswith("h")
        found = re.findall(r"__ldg\(\s*(?:w|kept|lse_g|p\.(?:score|lse|kept|new_len))\b[^;]*;", text)
        assert not found, (name, found)


# ---------------------------------------------------------------- pins of the fp64 statements

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_weights_by_hand(fmt):
    """Every row hands out a weight of one over the tokens that it sees; equal keys share it alike; a row that is left out
    hands out nothing; what was there fades by the decay; new tokens start from zero."""
    pool = R.Pool(6, 2, 16, 128, fmt, "cpu", seed=3)
    table = R.tables([19, 3], 16, 6, "cpu")
    ctx = torch.tensor([16, 0])
    q = torch.randn(6, 4, 128).to(torch.bfloat16)
    lse = T.lse(pool, q, table, ctx, 0.1, 3)[0]
    w = torch.ones(2, 2, 25)
    slot = torch.tensor([1, 0])
    got = T.score(pool, q, lse, table, ctx, 0.1, 3, w, slot, decay=0.5)[0]
    assert torch.allclose(got[1, :, :19].sum(-1), torch.tensor(6 + 16 * 0.5, dtype=torch.float64))
    assert torch.allclose(got[0, :, :3].sum(-1), torch.tensor(6.0, dtype=torch.float64))
    assert torch.equal(got[:, :, 19:], torch.ones(2, 2, 6, dtype=torch.float64))
    zero = q * 0
    lse = T.lse(pool, zero, table, ctx, 0.1, 3)[0]
    assert torch.allclose(lse[2], torch.full((4,), math.log(19), dtype=torch.float64))
    lse[0] = math.inf
    got = T.score(pool, zero, lse, table, ctx, 0.1, 3, w, slot, init=[False, True])[0]
    # rows 1 and 2 of two heads: 18 and 19 tokens each
    assert torch.allclose(got[1, 0, :18], torch.full((18,), 2 / 18 + 2 / 19, dtype=torch.float64) -
                          torch.tensor([0.0] * 18, dtype=torch.float64))
    assert torch.allclose(got[1, 0, 18], torch.tensor(2 / 19, dtype=torch.float64))
    mask = torch.tensor([[1, 2, 6], [0, 0, 0]])
    lse = T.lse(pool, q, table, ctx, 0.1, 3, mask)[0]
    assert bool(lse[:3].isfinite().all()) and bool((lse[3:] == -math.inf).all())


def test_eviction_by_hand():
    pool = R.Pool(4, 1, 16, 128, "bf16", "cpu", seed=3)
    table = torch.tensor([[2, 0]], dtype=torch.int32)
    w = torch.tensor([[[1, 5, 5, math.nan, -0.0, 0.0, 7, 5, 2, 1] + [0] * 7]])
    slot = torch.tensor([0])
    kept, new_len, now, w_now = T.evict(pool, table, [10], [4], w, slot)
    assert kept == [[[1, 2, 6, 7]]] and new_len == [4]
    assert torch.equal(now["k"][2, 0, :4], pool.k[2, 0, [1, 2, 6, 7]]) and torch.equal(now["k"][2, 0, 4:], pool.k[2, 0, 4:])
    assert w_now[0, 0, :5].tolist() == [5, 5, 7, 5, 0]
    assert T.evict(pool, table, [10], [4], w, slot, 1, 1)[0] == [[[0, 1, 6, 9]]]
    assert T.evict(pool, table, [10], [4], w, slot, 3, 9)[0] == [[[0, 1, 2, 3]]]
    assert T.evict(pool, table, [10], [9], w, slot)[0] == [[[0, 1, 2, 4, 5, 6, 7, 8, 9]]]
    assert T.evict(pool, table, [10], [8], w, slot)[0] == [[[0, 1, 2, 4, 6, 7, 8, 9]]]  # -0 and 0 alike: the first
    assert T.evict(pool, table, [0], [8], w, slot)[1] == [0]
