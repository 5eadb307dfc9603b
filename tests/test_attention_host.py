"""The attention-side entry points' host side (CPU only): refusals before any launch, workspace sizes, the
binding's checks; and pins of the fp64 statements that the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gated_deltanet_linear_conv1d_gb300 import build as gdn_build  # noqa: E402
from gated_deltanet_linear_conv1d_gb300 import synth  # noqa: E402
from tests import attnref as R  # noqa: E402


@pytest.fixture(scope="module")
def b():
    gdn_build.build()
    from gated_deltanet_linear_conv1d_gb300 import binding
    return binding


P, ODD = 256, 264  # never dereferenced; 264 is not 16-byte aligned


def cache(b, **kw):
    c = dict(k=P, v=P, k_scale=None, v_scale=None, num_pages=10, page_tokens=64, num_kv_heads=4, head_dim=256,
             format=b.GDN_KV_BF16)
    c.update(kw)
    return b.GdnKvCache(*(c[f] for f, _ in b.GdnKvCache._fields_))


BAD_CACHES = [
    (dict(k=None), "INVALID_ARG"), (dict(v=ODD), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(page_tokens=-64), "INVALID_ARG"), (dict(format=2), "INVALID_ARG"), (dict(format=1), "INVALID_ARG"),
    (dict(k_scale=P, v_scale=P), "INVALID_ARG"), (dict(head_dim=64), "UNSUPPORTED"), (dict(head_dim=192), "UNSUPPORTED"),
    (dict(page_tokens=24), "UNSUPPORTED"), (dict(page_tokens=8), "UNSUPPORTED"),
    (dict(num_pages=1 << 24, page_tokens=128), "UNSUPPORTED"),            # 2^31 slots
    (dict(num_pages=1 << 24, page_tokens=64, num_kv_heads=4), "UNSUPPORTED"),  # 2^32 rows
    (dict(format=1, k_scale=P, v_scale=ODD), "INVALID_ARG"),
]


@pytest.mark.parametrize("kw,why", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry_point(b, kw, why):
    lib, c, want = b._lib, cache(b, **kw), getattr(b, "GDN_ERR_" + why)
    p = ctypes.byref(c)
    assert lib.gdn_kv_cache_write(p, P, 1024, 256, P, 1024, 256, P, 4, None, None) == want
    assert lib.gdn_kv_cache_read(p, P, 2, P, 2, 100, P, P, None, None) == want
    assert lib.gdn_qk_norm_rope(P, 6144, 256, P, 1024, 256, P, P, 1e-6, P, P, 64, 0, P, None, P, 1024, 256, p, P, 4, 24,
                                c.num_kv_heads, c.head_dim, None, None) == want
    assert lib.gdn_tree_attention(p, P, P, 2, P, None, None, 0.1, P, 2, 1, 24, P, 1 << 30, None, None) == want
    assert lib.gdn_tree_attention_workspace_bytes(p, 2, 1, 24) == 0


def test_cache_write_and_read_arguments(b):
    lib, c = b._lib, cache(b)
    p = ctypes.byref(c)

    def write(k=P, kt=1024, kh=256, v=P, vt=1024, vh=256, slot=P, T=4):
        return lib.gdn_kv_cache_write(p, k, kt, kh, v, vt, vh, slot, T, None, None)

    for kw in (dict(k=None), dict(v=None), dict(slot=None), dict(k=ODD), dict(kt=1020), dict(vh=252), dict(T=-1)):
        assert write(**kw) == b.GDN_ERR_INVALID_ARG, kw
    assert write(k=None, v=None, slot=None, T=0) == b.GDN_OK

    def read(table=P, mp=2, start=P, N=2, T=100, k=P, v=P):
        return lib.gdn_kv_cache_read(p, table, mp, start, N, T, k, v, None, None)

    for kw in (dict(table=None), dict(mp=0), dict(mp=-1), dict(start=None), dict(N=-1), dict(N=0), dict(T=-1), dict(k=None),
               dict(v=ODD)):
        assert read(**kw) == b.GDN_ERR_INVALID_ARG, kw
    assert read(T=0) == b.GDN_OK and read(N=0, T=0) == b.GDN_OK


def test_norm_rope_arguments(b):
    lib, c = b._lib, cache(b)
    ref = ctypes.byref(c)

    def rope(q=P, qt=6144, qh=256, k=P, kt=1024, kh=256, qg=P, kg=P, eps=1e-6, pos=P, f=P, rot=64, qo=P, ko=P, v=None,
             cc=None, slot=None, T=4, hq=24, hkv=4, d=256):
        return lib.gdn_qk_norm_rope(q, qt, qh, k, kt, kh, qg, kg, eps, pos, f, rot, 0, qo, ko, v, 1024, 256, cc, slot, T,
                                    hq, hkv, d, None, None)

    for kw in (dict(k=None), dict(q=None), dict(qo=None), dict(ko=None), dict(qg=None), dict(kg=ODD), dict(eps=-1.0),
               dict(eps=math.nan), dict(pos=None), dict(f=None), dict(rot=72), dict(rot=-16), dict(rot=272), dict(qt=6140),
               dict(kh=4), dict(q=ODD), dict(ko=ODD), dict(T=-1), dict(hq=0), dict(hkv=-1), dict(v=P), dict(slot=P),
               dict(cc=ref), dict(cc=ref, v=P), dict(cc=ref, slot=P), dict(cc=ref, v=P, slot=P, hkv=2),
               dict(cc=ref, v=P, slot=P, d=128, rot=64), dict(cc=ref, v=ODD, slot=P)):
        assert rope(**kw) == b.GDN_ERR_INVALID_ARG, kw
    assert rope(d=64) == b.GDN_ERR_UNSUPPORTED
    assert rope(rot=96) == b.GDN_ERR_UNSUPPORTED  # no power of two
    assert rope(T=0) == b.GDN_OK


def test_tree_attention_arguments(b):
    lib, c = b._lib, cache(b)
    ref = ctypes.byref(c)
    need = b.gdn_tree_attention_workspace_bytes(c, 2, 8, 24)
    assert 0 < need < 1 << 28

    def attn(q=P, table=P, mp=2, ctx=P, mask=None, gate=None, scale=0.1, out=P, N=2, nodes=8, hq=24, ws=P, size=need):
        return lib.gdn_tree_attention(ref, q, table, mp, ctx, mask, gate, scale, out, N, nodes, hq, ws, size, None, None)

    for kw in (dict(q=None), dict(table=None), dict(mp=0), dict(ctx=None), dict(out=None), dict(q=ODD), dict(out=ODD),
               dict(gate=ODD), dict(mask=257), dict(scale=math.inf), dict(scale=math.nan), dict(N=-1), dict(N=65536),
               dict(nodes=0), dict(nodes=65), dict(hq=0), dict(ws=None), dict(ws=ODD), dict(size=need - 1)):
        assert attn(**kw) == b.GDN_ERR_INVALID_ARG, kw
    assert attn(hq=25) == b.GDN_ERR_UNSUPPORTED and attn(hq=260) == b.GDN_ERR_UNSUPPORTED
    assert attn(N=0) == b.GDN_OK
    # whatever the lengths: the workspace goes by the sizes alone, and a larger batch fits a larger one's
    assert b.gdn_tree_attention_workspace_bytes(c, 0, 8, 24) == 0
    assert b.gdn_tree_attention_workspace_bytes(c, 65535, 64, 24) >= b.gdn_tree_attention_workspace_bytes(c, 1, 64, 24)


def test_verify_tree_arguments(b):
    lib = b._lib
    d = b.make_dims(synth.RANK_HEADS, 8)

    def verify(parent=P, nodes=4, N=2, qkv0=P):
        return lib.gdn_spec_verify_tree(ctypes.byref(d), qkv0, P, P, P, P, P, parent, P, P, P, P, 1e-6, None, P, N, nodes,
                                        None, None)

    assert verify(parent=None) == b.GDN_ERR_INVALID_ARG
    assert verify(nodes=0) == b.GDN_ERR_INVALID_ARG and verify(nodes=9) == b.GDN_ERR_INVALID_ARG
    assert verify(qkv0=ODD) == b.GDN_ERR_INVALID_ARG
    assert verify(N=0) == b.GDN_OK


def test_binding_checks(b):
    k = torch.zeros((2, 1, 16, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        b.make_kv_cache(k, k)
    with pytest.raises(ValueError, match="num_pages"):
        b.make_kv_cache(k[0], k[0])


# ---------------------------------------------------------------- pins of the fp64 statements

def test_rotation_keeps_lengths_and_goes_by_differences():
    """A rotation keeps each pair's length, and the product of a rotated query and key depends on their
    distance alone."""
    torch.manual_seed(0)
    f = 1e4 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    q, k, one = torch.randn(1, 1, 128), torch.randn(1, 1, 128), torch.ones(128)
    for inter in (False, True):
        def at(x, pos):
            return R.norm_rope(x, one, 1e-6, torch.tensor([pos]), f, inter)[0][0, 0]
        assert torch.allclose(at(q, 5) @ at(k, 2), at(q, 1003) @ at(k, 1000), rtol=1e-9)
        assert torch.allclose(at(q, 7).norm(), at(q, 0).norm(), rtol=1e-12)
        assert torch.allclose(at(q, 9)[32:], at(q, 0)[32:])


def test_rotation_by_a_quarter_turn():
    x = torch.zeros(1, 1, 128)
    x[0, 0, 0], x[0, 0, 8] = 3.0, 4.0
    f = torch.full((8,), math.pi / 2, dtype=torch.float64)
    scale = math.sqrt(25 / 128)
    y, _ = R.norm_rope(x, torch.ones(128), 0.0, torch.tensor([1]), f)
    assert torch.allclose(y[0, 0, [0, 8]] * scale, torch.tensor([-4.0, 3.0], dtype=torch.float64))
    x[0, 0, 1], x[0, 0, 8] = 4.0, 0.0
    y, _ = R.norm_rope(x, torch.ones(128), 0.0, torch.tensor([1]), f, True)
    assert torch.allclose(y[0, 0, [0, 1]] * scale, torch.tensor([-4.0, 3.0], dtype=torch.float64))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_attention_statement_by_hand(fmt):
    """A chain equals its mask; one visible token is returned as it is; equal keys give the mean; an empty row gives
    zeros; a planted mistake in the mask shows."""
    pool = R.Pool(6, 2, 16, 128, fmt, "cpu", seed=3)
    table = R.tables([19, 3], 16, 6, "cpu")
    ctx = torch.tensor([16, 0])
    q = torch.randn(6, 4, 128).to(torch.bfloat16)
    chain = R.tree_attention(pool, q, table, ctx, 0.1, 3)[0]
    mask = torch.tensor([[1, 3, 7], [1, 3, 7]])
    assert torch.equal(chain, R.tree_attention(pool, q, table, ctx, 0.1, 3, mask)[0])
    first = pool.values("v", table[1, :1].long())[:, 0]
    assert torch.allclose(chain[3], first.repeat_interleave(2, 0))
    wrong = mask.clone()
    wrong[0, 2] = 5
    assert not torch.allclose(chain[2], R.tree_attention(pool, q, table, ctx, 0.1, 3, wrong)[0][2])
    none = R.tree_attention(pool, q, table, ctx, 0.1, 3, torch.zeros(2, 3, dtype=torch.int64))[0]
    assert torch.equal(none[3:], torch.zeros_like(none[3:]))
    assert torch.equal(none[0], none[0]) and none[0].abs().sum() > 0
    zero = R.tree_attention(pool, q * 0, table, ctx, 0.1, 3)[0]
    v = pool.values("v", table[0, :2].long())[:, :18].mean(1)
    assert torch.allclose(zero[1], v.repeat_interleave(2, 0))


def test_trees_and_masks_agree():
    par, mask = R.tree(4, 64, seed=1)
    for n in range(4):
        for p in range(64):
            at, want = p, 0
            while at >= 0:
                want |= 1 << at
                at = int(par[n, at])
            assert int(np.int64(mask[n, p]).view(np.uint64)) == want
