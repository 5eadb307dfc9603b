"""The attention-side operators on the GPU against their fp64 statements: head norms and rotation, the paged
cache, tree attention, the linear layers' verify of a tree, and a speculative step through all of them.
Tolerances count the roundings (attnref)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gated_deltanet_linear_conv1d_gb300 import synth  # noqa: E402
from oracle import oracle  # noqa: E402
from tests import attnref as R  # noqa: E402
from tests import gdnutil as U  # noqa: E402

HEADS = {"24x4x256": (24, 4, 256), "6x1x256": (6, 1, 256), "32x8x128": (32, 8, 128), "5x5x128": (5, 5, 128)}


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_conv1d_gb300 import build
    build.build()
    from gated_deltanet_linear_conv1d_gb300 import binding
    return binding


@pytest.fixture
def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8)


def inside(got, ref, bound, what):
    got = got.double()
    off = (got - ref).abs()
    bad = ~(off <= bound) & ~(got.isnan() & ref.isnan()) & ~(got == ref)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound)[bad].max())}" \
                                f" times its bound at {torch.nonzero(bad)[0].tolist()}"


# ---------------------------------------------------------------- head norms and rotation

ROPE = [("24x4x256", 1, 64, False), ("24x4x256", 333, 64, False), ("24x4x256", 5000, 64, True), ("6x1x256", 3, 256, False),
        ("32x8x128", 17, 128, True), ("32x8x128", 700, 32, False), ("5x5x128", 2, 16, False), ("6x1x256", 9, 0, False)]


@pytest.mark.parametrize("heads,T,rotary,inter", ROPE)
def test_norm_rope(b, err, heads, T, rotary, inter):
    hq, hkv, d = HEADS[heads]
    packed = (randn(T, hq + 2 * hkv, d, seed=T) * 2).to(torch.bfloat16)
    q, k = packed[:, :hq], packed[:, hq:hq + hkv]
    qg, kg = randn(d, seed=1).abs() + 0.1, randn(d, seed=2)
    pos = torch.randint(0, 2 ** 31 - 1, (T,), device="cuda", dtype=torch.int32) >> torch.randint(0, 31, (T,), device="cuda")
    pos = pos.to(torch.int32)
    f = 1e7 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / max(rotary, 1)) if rotary else None
    qo, ko = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hkv, d, dtype=torch.bfloat16,
                                                                                     device="cuda")
    b.gdn_qk_norm_rope(q, k, qg, kg, 1e-6, pos, f, qo, ko, interleaved=inter, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    for x, g, out, what in ((q, qg, qo, "q"), (k, kg, ko, "k")):
        ref, mag = R.norm_rope(x, g, 1e-6, pos, f, inter)
        # the fp64 angle itself is exact to 2^-52 of up to 2^31 radians
        inside(out, ref, R.rope_bound(ref, mag), what)
    # in place, and the keys alone: the same bits
    dense_q, dense_k = (t.clone(memory_format=torch.contiguous_format) for t in (q, k))
    b.gdn_qk_norm_rope(dense_q, dense_k, qg, kg, 1e-6, pos, f, dense_q, dense_k, interleaved=inter)
    assert torch.equal(bits(dense_q), bits(qo)) and torch.equal(bits(dense_k), bits(ko))
    alone = torch.empty_like(ko)
    b.gdn_qk_norm_rope(None, k, None, kg, 1e-6, pos, f, None, alone, interleaved=inter)
    assert torch.equal(bits(alone), bits(ko))


def test_norm_rope_of_extreme_rows(b):
    """A zero row stays zero; the largest bf16 values overflow no sum that fp32 holds; a NaN stays in its row."""
    T, hq, hkv, d = 4, 2, 1, 128
    x = torch.zeros(T, hq, d, device="cuda", dtype=torch.bfloat16)
    x[1] = 1e18
    x[2, 0] = float("nan")
    x[3] = 1e-20
    k = x[:, :1].contiguous()
    g = torch.ones(d, device="cuda")
    out, ko = torch.empty_like(x), torch.empty_like(k)
    f = torch.ones(8, dtype=torch.float64, device="cuda")
    b.gdn_qk_norm_rope(x, k, g, g, 1e-6, torch.zeros(T, dtype=torch.int32, device="cuda"), f, out, ko)
    assert torch.equal(out[0], torch.zeros_like(out[0]))
    assert torch.allclose(out[1].float(), torch.ones(hq, d, device="cuda"))
    assert bool(out[2, 0].isnan().all()) and torch.equal(out[2, 1], torch.zeros(d, device="cuda", dtype=torch.bfloat16))
    assert bool(out[3].isfinite().all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,T,page", [("24x4x256", 1, 16), ("24x4x256", 300, 64), ("6x1x256", 41, 48),
                                          ("32x8x128", 77, 128), ("5x5x128", 1300, 16)])
def test_norm_rope_into_the_cache(b, err, fmt, heads, T, page):
    hq, hkv, d = HEADS[heads]
    pool = R.Pool(-(-T // page) + 3, hkv, page, d, fmt, seed=T)
    was = [t.clone() if t is not None else None for t in (pool.k, pool.v, pool.k_scale, pool.v_scale)]
    packed = (randn(T, hq + 2 * hkv, d, seed=T) * 2).to(torch.bfloat16)
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    g = randn(d, seed=2).abs() + 0.5
    pos = torch.randint(0, 1 << 20, (T,), device="cuda", dtype=torch.int32)
    f = 1e7 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device="cuda") / 64)
    slots = torch.randperm(pool.k.shape[0] * page, device="cuda")[:T].to(torch.int32)
    if T > 10:
        slots[3] = -1
        slots[7] = -(2 ** 31)
    qo, ko = (torch.empty(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    c = pool.handle(b)
    b.gdn_qk_norm_rope(q, k, g, g, 1e-6, pos, f, qo, ko, v=v, cache=c, kv_slot=slots, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ref, mag = R.norm_rope(k, g, 1e-6, pos, f)
    inside(ko, ref, R.rope_bound(ref, mag), "k_out")
    kept = slots >= 0
    at = slots[kept].long()
    pg, row = at // page, at % page
    if fmt == "bf16":
        assert torch.equal(bits(pool.k[pg, :, row]), bits(ko[kept]))
        assert torch.equal(bits(pool.v[pg, :, row]), bits(v[kept]))
    else:
        for name, x, m in (("k", ref, mag), ("v", v.double(), None)):
            x = x[kept]
            s = pool.k_scale[pg, :, row] if name == "k" else pool.v_scale[pg, :, row]
            amax = x.abs().amax(-1)
            slack = 0 if m is None else (2.0 ** -16 + 2.0 ** -20) * m[kept]
            # the scale: the largest value's error and a division; then half a step of its code
            assert bool(((s.double() - amax / 448).abs() <= (2.0 ** -14 if m is not None else 2.0 ** -23) * amax / 448).all())
            code = (pool.k if name == "k" else pool.v)[pg, :, row]
            val = R._TABLE.cuda()[code.long()] * s.double()[..., None]
            assert bool(((val - x).abs() <= R.E4M3 * x.abs() * (1 + 2.0 ** -12) + 2.0 ** -10 * s.double()[..., None]
                         + 2 * slack).all()), name
        codes, s = R.quantise(v[kept].float())
        assert torch.equal(pool.v[pg, :, row].cpu(), codes) and torch.equal(pool.v_scale[pg, :, row].cpu(), s)
    # nothing else moved
    touched = torch.zeros(pool.k.shape[0], page, dtype=torch.bool, device="cuda")
    touched[pg, row] = True
    for t, w in zip((pool.k, pool.v, pool.k_scale, pool.v_scale), was):
        if t is not None:
            keep = ~touched[:, None].expand(-1, hkv, -1)
            assert torch.equal(bits(t[keep]), bits(w[keep]))
    # the same rows once more, alone, at other slots: the same bits there
    other = R.Pool(pool.k.shape[0], hkv, page, d, fmt, seed=5)
    moved = torch.where(kept, (slots + 1) % (pool.k.shape[0] * page), slots)
    b.gdn_qk_norm_rope(None, k, None, g, 1e-6, pos, f, None, v=v, cache=other.handle(b), kv_slot=moved)
    to = moved[kept].long()
    assert torch.equal(bits(other.k[to // page, :, to % page]), bits(pool.k[pg, :, row]))


# ---------------------------------------------------------------- the cache

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page,lens", [("24x4x256", 64, [1]), ("24x4x256", 16, [0, 300, 1, 0, 17, 16]),
                                             ("6x1x256", 48, [47, 48, 49]), ("32x8x128", 128, [129, 5, 0]),
                                             ("5x5x128", 256, [700, 0, 0, 1])])
def test_cache_write_then_read(b, err, fmt, heads, page, lens):
    _, hkv, d = HEADS[heads]
    T = sum(lens)
    pages = sum(-(-n // page) for n in lens) + 2
    pool = R.Pool(pages, hkv, page, d, fmt, seed=1)
    table = R.tables(lens, page, pages)
    slots = torch.cat([table[i, torch.arange(n) // page] * page + torch.arange(n, device="cuda").to(torch.int32) % page
                       for i, n in enumerate(lens)]).to(torch.int32)
    wide = randn(T, 2, hkv, d + 8, seed=3).to(torch.bfloat16)  # strided tokens and heads
    wide[0, 0, 0, :d] = 0
    k, v = wide[:, 0, :, :d], wide[:, 1, :, 8:]
    c = pool.handle(b)
    b.gdn_kv_cache_write(c, k, v, slots, dev_err=err)
    ko, vo = (torch.full((T, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    start = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    b.gdn_kv_cache_read(c, table, start, ko, vo, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    for x, out in ((k, ko), (v, vo)):
        if fmt == "bf16":
            assert torch.equal(bits(out), bits(x))
        else:
            codes, s = R.quantise(x.float())
            val = R._TABLE[codes.long()] * s.double()[..., None]
            # the exact product, rounded to fp32 and to bf16: the nearest bf16, or its neighbour at a tie
            assert torch.equal(bits(out.cpu()), bits(val.float().to(torch.bfloat16)))


def test_cache_write_codes_of_special_rows(b):
    """Zero rows, the largest values, subnormal codes, NaN and infinities, as the header states them."""
    pool = R.Pool(1, 1, 16, 128, "e4m3", seed=1)
    x = torch.zeros(5, 1, 128, device="cuda")
    x[1, 0] = 3.3895e38
    x[2, 0, 0], x[2, 0, 1:] = 448.0, torch.linspace(-0.02, 0.02, 127)
    x[3, 0, 5], x[3, 0, 6] = float("nan"), 7.0
    x[4, 0, 5], x[4, 0, 6] = float("inf"), 7.0
    x = x.to(torch.bfloat16)
    b.gdn_kv_cache_write(pool.handle(b), x, x, torch.arange(5, dtype=torch.int32, device="cuda"))
    k, s = pool.k[0, 0, :5].cpu(), pool.k_scale[0, 0, :5].cpu()
    assert torch.equal(k[0], torch.zeros(128, dtype=torch.uint8)) and float(s[0]) == np.float32(1e-12) / np.float32(448)
    assert bool((k[1] == 0x7E).all())
    codes, scale = R.quantise(x[2].float())
    assert torch.equal(k[2], codes[0]) and float(s[2]) == float(scale[0]) == 1.0
    assert int(k[3, 5]) & 0x7F == 0x7F and int(k[3, 6]) == 0x7E and float(s[3]) == 7.0 / 448
    assert int(k[4, 5]) & 0x7F == 0x7F and int(k[4, 6]) == 0 and float(s[4]) == float("inf")
    assert torch.equal(pool.v[0, 0, :5].cpu(), k)


def test_cache_write_codes_are_those_of_the_division(b):
    """Every pair of bf16 significands (value, row's largest) at sixteen distances of their exponents: the codes of the
    quotients rounded to fp32, ties among them."""
    top, j = torch.arange(128, device="cuda"), torch.arange(128, device="cuda")
    row = torch.cat([torch.stack([(1 + j / 128) * 2.0 ** -off * (-1) ** (j + m) for m in range(128)]) for off in
                     range(1, 17)])
    x = torch.zeros(16 * 128, 1, 256, device="cuda")
    x[:, 0, :128] = row
    x[:, 0, 200] = (1 + top / 128).repeat(16)
    x = x.to(torch.bfloat16)
    pool = R.Pool(x.shape[0] // 16, 1, 16, 256, "e4m3", seed=1)
    b.gdn_kv_cache_write(pool.handle(b), x, x, torch.arange(x.shape[0], dtype=torch.int32, device="cuda"))
    codes, scale = R.quantise(x.float())
    got = pool.k.reshape(-1, 1, 256).cpu()
    assert torch.equal(pool.k_scale.reshape(-1, 1).cpu(), scale)
    assert torch.equal(got, codes), torch.nonzero(got != codes)[:5].tolist()


def test_cache_flags_bad_slots_pages_and_offsets(b, err):
    pool = R.Pool(4, 2, 16, 128, "e4m3", seed=1)
    c = pool.handle(b)
    was = pool.k.clone()
    x = randn(3, 2, 128).to(torch.bfloat16)
    slots = torch.tensor([64, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    b.gdn_kv_cache_write(c, x, x, slots, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT
    was[0, :, 5] = pool.k[0, :, 5]
    assert torch.equal(pool.k, was) and not torch.equal(pool.k[0, :, 5], R.Pool(4, 2, 16, 128, "e4m3", seed=1).k[0, :, 5])

    def read(table, start, T):
        ko, vo = (torch.full((T, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        b.gdn_kv_cache_read(c, torch.tensor(table, dtype=torch.int32, device="cuda"),
                            torch.tensor(start, dtype=torch.int32, device="cuda"), ko, vo, dev_err=err)
        return b.gdn_read_device_error(err), (ko != 7.0).any(-1).any(-1).cpu().tolist()

    assert read([[0, 4], [1, 2]], [0, 20, 40], 40) == (b.GDN_DEVERR_SLOT, [True] * 16 + [False] * 4 + [True] * 20)
    assert read([[0, -1], [1, 2]], [0, 17, 18], 18) == (b.GDN_DEVERR_SLOT, [True] * 16 + [False] + [True])
    assert read([[0, 1]], [0, 33], 33) == (b.GDN_DEVERR_OFFSETS, [False] * 33)        # three pages
    assert read([[0, 1], [2, 3]], [0, 8, 5], 5)[0] == b.GDN_DEVERR_OFFSETS           # not monotone
    assert read([[0, 1]], [0, 9], 5)[0] == b.GDN_DEVERR_OFFSETS                       # past the output
    assert read([[0, 1]], [0, 3], 5) == (b.GDN_DEVERR_OFFSETS, [True] * 3 + [False] * 2)
    assert read([[0, 1]], [2, 5], 5)[0] == b.GDN_DEVERR_OFFSETS


# ---------------------------------------------------------------- tree attention

def attend(b, pool, q, table, ctx, scale, nodes, mask=None, gate=None, out=None, **kw):
    out = torch.full_like(q, float("nan")) if out is None else out
    b.gdn_tree_attention(pool.handle(b), q, table, ctx, scale, out, nodes, tree_mask=mask, gate=gate, **kw)
    return out


def case(heads, fmt, page, lens, nodes, seed=0, strong=1.0):
    hq, hkv, d = HEADS[heads] if isinstance(heads, str) else heads
    held = [n + nodes if n >= 0 else 0 for n in lens]
    pages = sum(-(-n // page) for n in held) + 2
    pool = R.Pool(pages, hkv, page, d, fmt, seed=seed)
    table = R.tables(held, page, pages, seed=seed)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = (randn(len(lens) * nodes, hq, d, seed=seed + 9) * strong).to(torch.bfloat16)
    return pool, table, ctx, q, d ** -0.5


ATTN = [  # heads, page, context lengths, nodes, tree, gate, strength of the scores
    ("24x4x256", 64, [0], 1, False, False, 1), ("24x4x256", 64, [1], 1, False, True, 1),
    ("24x4x256", 64, [127], 1, False, False, 1), ("24x4x256", 64, [128], 1, False, False, 3),
    ("24x4x256", 16, [509, 3, 0, 1000], 1, False, False, 1), ("24x4x256", 64, [5000], 4, False, False, 2),
    ("24x4x256", 128, [0, 100, 126, 127, 128], 8, True, True, 1), ("24x4x256", 48, [700, 2, 333], 5, True, False, 3),
    ("24x4x256", 256, [1023, 77], 64, True, True, 1), ("6x1x256", 16, [40, 260], 64, True, False, 2),
    ("6x1x256", 64, [20000], 3, False, False, 4), ("32x8x128", 64, [900, 0, 31], 7, True, False, 1),
    ("32x8x128", 16, [2047], 16, False, True, 2), ("5x5x128", 64, [130, 64, 1], 9, True, False, 1),
    ("32x8x128", 128, list(range(0, 1200, 37)), 2, True, False, 1), ((64, 1, 128), 16, [300, 12], 5, True, False, 1),
    ((3, 1, 256), 16, [17] * 40, 1, False, False, 1),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page,lens,nodes,tree,gated,strong", ATTN)
def test_tree_attention(b, err, fmt, heads, page, lens, nodes, tree, gated, strong):
    pool, table, ctx, q, scale = case(heads, fmt, page, lens, nodes, strong=strong)
    mask = R.tree(len(lens), nodes)[1].cuda() if tree else None
    gate = randn(*q.shape, seed=4).to(torch.bfloat16) if gated else None
    out = attend(b, pool, q, table, ctx, scale, nodes, mask, gate, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, nodes, mask, gate)
    inside(out, ref, bound, "out")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(6))
def test_tree_attention_of_random_sizes(b, err, fmt, seed):
    rng = np.random.default_rng(100 + seed)
    hkv, group, d = int(rng.integers(1, 6)), int(rng.integers(1, 13)), int(rng.choice([128, 256]))
    nodes = int(np.exp(rng.uniform(0, np.log(64.99))))
    n = int(rng.integers(1, 9))
    page = int(rng.choice([16, 32, 48, 64, 96, 128, 192]))
    lens = [int(np.exp(rng.uniform(0, np.log(3000)))) - 1 for _ in range(n)]
    pool, table, ctx, q, scale = case((hkv * group, hkv, d), fmt, page, lens, nodes, seed=seed, strong=2)
    mask = torch.from_numpy(rng.integers(-2 ** 63, 2 ** 63 - 1, (n, nodes))).cuda()  # any mask, empty rows among them
    mask[:, ::3] = 0
    out = attend(b, pool, q, table, ctx, scale, nodes, mask, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, nodes, mask)
    inside(out, ref, bound, "out")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_what_is_not_seen_contributes_nothing(b, err, fmt):
    """NaN and infinities behind the last token, in unused pages and in nodes of other branches leave a row as it was;
    a node that sees nothing gives zeros; where such a node is seen, it shows."""
    lens, nodes = [130, 0, 200], 6
    pool, table, ctx, q, scale = case("24x4x256", fmt, 64, lens, nodes)
    par = torch.tensor([[-1, 0, 0, 1, 2, 2]] * 3)
    mask = torch.tensor([[0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100101]] * 3, device="cuda")
    mask[1, 4] = 0
    clean = attend(b, pool, q, table, ctx, scale, nodes, mask, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, nodes, mask)
    inside(clean, ref, bound, "clean")
    assert torch.equal(clean[nodes + 4], torch.zeros_like(clean[0]))
    bad_code = [0x7F, 0xFF]
    used = torch.zeros(pool.k.shape[0], pool.page, dtype=torch.bool, device="cuda")
    for n, c in enumerate(lens):
        t = torch.arange(c + nodes, device="cuda")
        used[table[n, t // 64].long(), t % 64] = True
    for t, s in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
        dead = ~used[:, None].expand(-1, t.shape[1], -1)
        if fmt == "e4m3":
            t[dead] = bad_code[0]
            s[dead] = float("nan")
        else:
            t[dead] = float("nan")
    same = attend(b, pool, q, table, ctx, scale, nodes, mask, dev_err=err)
    assert torch.equal(bits(same), bits(clean))
    # node 1 of every request holds no numbers: nodes 1 and 3 see it, the others do not
    for n, c in enumerate(lens):
        t = c + 1
        pg, row = int(table[n, t // 64]), t % 64
        for x, s in ((pool.k, pool.k_scale), (pool.v, pool.v_scale)):
            if fmt == "e4m3":
                x[pg, :, row, 3] = bad_code[1]
            else:
                x[pg, :, row, 3] = float("nan") if n < 2 else float("inf")
    out = attend(b, pool, q, table, ctx, scale, nodes, mask, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    for n in range(3):
        for j in range(nodes):
            r = n * nodes + j
            if int(mask[n, j]) >> 1 & 1:
                assert not bool(out[r].isfinite().all()), (n, j)
            else:
                inside(out[r], ref[r], bound[r], f"node {j} of request {n}")
    assert par.shape == mask.shape


def test_infinite_keys_take_the_whole_weight_or_none(b, err):
    """A key of -inf score has no weight, one of +inf makes the row NaN, as the formula says; the values of the
    unweighted one still count as 0 times theirs."""
    pool, table, ctx, q, scale = case("6x1x256", "bf16", 64, [10], 1)
    q = q.abs() + 0.1
    pool.k[int(table[0, 0]), :, 4] = -float("inf")
    out = attend(b, pool, q, table, ctx, scale, 1, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, 1)
    assert bool(ref.isfinite().all())
    inside(out, ref, bound.nan_to_num(1e-2, 1e-2), "one key of -inf")
    pool.k[int(table[0, 0]), :, 4] = float("inf")
    assert bool(attend(b, pool, q, table, ctx, scale, 1).isnan().all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_values_far_apart(b, err, fmt):
    """Scores of hundreds (all weight on one token), of one value (equal weights) and a cache whose rows differ by
    many orders of magnitude keep their accuracy."""
    for strong, rows in ((60.0, None), (0.0, None), (1.0, "rows")):
        pool, table, ctx, q, scale = case("24x4x256", fmt, 64, [777, 12], 3, strong=strong)
        if rows:
            f = torch.exp2(torch.randint(-20, 21, pool.k.shape[:3], device="cuda").float())
            if fmt == "e4m3":
                pool.v_scale.mul_(f)
            else:
                pool.v.mul_(f[..., None].to(torch.bfloat16))
        out = attend(b, pool, q, table, ctx, scale, 3, dev_err=err)
        assert b.gdn_read_device_error(err) == 0
        ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, 3)
        inside(out, ref, bound, f"strength {strong}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_padding_bad_pages_and_lengths(b, err, fmt):
    lens, nodes = [200, -1, 90, 3, 150, -5], 3
    pool, table, ctx, q, scale = case("24x4x256", fmt, 64, lens, nodes)
    pages = pool.k.shape[0]
    table[2, 1] = pages            # out of the pool
    ctx[3] = 64 * table.shape[1] - 1  # more than the table holds
    out = torch.full_like(q, 7.0)
    attend(b, pool, q, table, ctx, scale, nodes, out=out, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT | b.GDN_DEVERR_OFFSETS
    for n in (1, 2, 3, 5):
        assert bool((out[n * nodes:(n + 1) * nodes] == 7.0).all()), n
    ok = [0, 4]
    ref, bound, _ = R.tree_attention(pool, q.reshape(6, nodes, 24, 256)[ok].reshape(-1, 24, 256), table[ok], ctx[ok], scale,
                                     nodes)
    inside(out.reshape(6, nodes, 24, 256)[ok].reshape(-1, 24, 256), ref, bound, "the others")
    table[2, 1] = -1
    out2 = torch.full_like(q, 7.0)
    ctx[3] = 2 ** 31 - 1
    attend(b, pool, q, table, ctx, scale, nodes, out=out2, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT | b.GDN_DEVERR_OFFSETS
    assert torch.equal(bits(out2), bits(out))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [[40000], [3000, 100, 64000, 0]])
def test_split_contexts_repeat_bit_for_bit_and_leave_the_workspace_reusable(b, err, fmt, lens):
    nodes = 4
    pool, table, ctx, q, scale = case("24x4x256", fmt, 64, lens, nodes)
    c = pool.handle(b)
    ws = torch.zeros(b.gdn_tree_attention_workspace_bytes(c, len(lens), nodes, 24), dtype=torch.uint8, device="cuda")
    first = attend(b, pool, q, table, ctx, scale, nodes, workspace=ws, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, nodes)
    inside(first, ref, bound, "out")
    for _ in range(4):
        assert torch.equal(bits(attend(b, pool, q, table, ctx, scale, nodes, workspace=ws, dev_err=err)), bits(first))
    # other sizes through the same workspace
    p2, t2, c2, q2, s2 = case("24x4x256", fmt, 16, [999], 1, seed=3)
    out = attend(b, p2, q2, t2, c2, s2, 1, workspace=ws, dev_err=err)
    ref, bound, _ = R.tree_attention(p2, q2, t2, c2, s2, 1)
    inside(out, ref, bound, "after another call")
    # out may be q or the gate itself
    g = randn(*q.shape, seed=2).to(torch.bfloat16)
    want = attend(b, pool, q, table, ctx, scale, nodes, gate=g, workspace=ws)
    for alias in ("q", "gate"):
        qq, gg = q.clone(), g.clone()
        got = attend(b, pool, qq, table, ctx, scale, nodes, gate=gg, out=qq if alias == "q" else gg, workspace=ws)
        assert torch.equal(bits(got), bits(want)), alias
    assert b.gdn_read_device_error(err) == 0


def test_captured_with_lengths_that_change_between_replays(b, err):
    pool, table, ctx, q, scale = case("24x4x256", "e4m3", 64, [5000, 300, 64], 4)
    ws = torch.zeros(b.gdn_tree_attention_workspace_bytes(pool.handle(b), 3, 4, 24), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    attend(b, pool, q, table, ctx, scale, 4, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attend(b, pool, q, table, ctx, scale, 4, out=out, workspace=ws, dev_err=err)
    for lens in ([5000, 300, 64], [17, -1, 0], [4999, 1, 63]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        ref, bound, live = R.tree_attention(pool, q, table, ctx, scale, 4)
        inside(out[live], ref[live], bound[live], str(lens))
        assert bool((out[~live] == 7.0).all())
    assert b.gdn_read_device_error(err) == 0


def test_two_streams_with_a_workspace_each(b, err):
    cases = [case("24x4x256", fmt, 64, [30000, 40], 2, seed=i) for i, fmt in enumerate(("bf16", "e4m3"))]
    want = [attend(b, *c[:1], c[3], c[1], c[2], c[4], 2) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [torch.zeros(b.gdn_tree_attention_workspace_bytes(c[0].handle(b), 2, 2, 24), dtype=torch.uint8, device="cuda")
              for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s, ws in zip(cases, streams, spaces):
            out = torch.empty_like(c[3])
            s.wait_stream(torch.cuda.current_stream())
            attend(b, c[0], c[3], c[1], c[2], c[4], 2, out=out, workspace=ws, dev_err=err, stream=s)
            got.append(out)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(bits(x), bits(y))
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_pool_beyond_32_bit_offsets(b, err, fmt):
    """Pages at the far end of a pool of more than 2^32 elements."""
    pages, hkv, page, d = (1 << 32) // (4 * 64 * 256) + 40, 4, 64, 256
    dt = torch.uint8 if fmt == "e4m3" else torch.bfloat16
    pool = R.Pool(40, hkv, page, d, fmt, seed=2)
    small = {x: getattr(pool, x) for x in ("k", "v")}
    for x in ("k", "v"):
        big = torch.zeros((pages, hkv, page, d), dtype=dt, device="cuda")
        big[-40:] = small[x]
        setattr(pool, x, big)
        if fmt == "e4m3":
            s = torch.zeros((pages, hkv, page), device="cuda")
            s[-40:] = getattr(pool, x + "_scale")
            setattr(pool, x + "_scale", s)
    table = R.tables([1500, 700], page, 40) + (pages - 40)
    ctx = torch.tensor([1490, 690], dtype=torch.int32, device="cuda")
    q = randn(20, 24, d).to(torch.bfloat16)
    out = attend(b, pool, q, table, ctx, 0.1, 10, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, 0.1, 10)
    inside(out, ref, bound, "far pages")
    ko, vo = (torch.empty(1500, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    start = torch.tensor([0, 1500], dtype=torch.int32, device="cuda")
    b.gdn_kv_cache_read(pool.handle(b), table[:1].contiguous(), start, ko, vo, dev_err=err)
    assert torch.equal(vo.cpu(), pool.values("v", table[0, :24].long())[:, :1500].transpose(0, 1).float().to(torch.bfloat16).cpu())
    b.gdn_kv_cache_write(pool.handle(b), ko, vo, torch.arange(pages * page - 1500, pages * page, dtype=torch.int32,
                                                              device="cuda"), dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    assert bool((pool.v[-1, :, -1] != small["v"][-1, :, -1]).any())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.0625, 2.0 ** -30, 1.0])
def test_scales_of_any_sign_and_size(b, err, fmt, scale):
    pool, table, ctx, q, _ = case("24x4x256", fmt, 64, [400, 0, 129], 7)
    mask = R.tree(3, 7)[1].cuda()
    out = attend(b, pool, q, table, ctx, scale, 7, mask, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, 7, mask)
    inside(out, ref, bound, "out")
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_requests_that_share_pages(b, err, fmt):
    """A common prefix, and one request's whole table twice."""
    pool, table, ctx, q, scale = case("24x4x256", fmt, 16, [600, 640, 600], 3)
    table[1, :30] = table[0, :30]
    table[2] = table[0]
    out = attend(b, pool, q, table, ctx, scale, 3, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, 3)
    inside(out, ref, bound, "out")
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,nodes", [("24x4x256", 1), ("24x4x256", 5), ("24x4x256", 9), ("5x5x128", 2)])
def test_many_short_requests(b, err, fmt, heads, nodes):
    """Pieces of many units: more segments than barriers and buffers, requests without tiles between them."""
    rng = np.random.default_rng(nodes)
    lens = [int(x) for x in rng.choice([-1, 0, 1, 100, 127, 128, 129, 300], 500)]
    pool, table, ctx, q, scale = case(heads, fmt, 16, lens, nodes)
    out = torch.full_like(q, 7.0)
    attend(b, pool, q, table, ctx, scale, nodes, out=out, dev_err=err)
    ref, bound, live = R.tree_attention(pool, q, table, ctx, scale, nodes)
    inside(out[live], ref[live], bound[live], "out")
    assert bool((out[~live] == 7.0).all()) and b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_most_rows_and_most_requests(b, err, fmt):
    pool, table, ctx, q, scale = case((64, 1, 128), fmt, 64, [1000], 64)  # 4096 rows of one kv head
    out = attend(b, pool, q, table, ctx, scale, 64, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q, table, ctx, scale, 64)
    inside(out, ref, bound, "rows")
    some, n = {0: 5, 40000: 300, 65534: 17}, 65535
    pool, few, _, _, scale = case((1, 1, 128), fmt, 16, list(some.values()), 1)
    table = torch.full((n, few.shape[1]), -1, dtype=torch.int32, device="cuda")
    ctx = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    at = torch.tensor(list(some), device="cuda")
    table[at], ctx[at] = few, torch.tensor(list(some.values()), dtype=torch.int32, device="cuda")
    q = randn(n, 1, 128, seed=1).to(torch.bfloat16)
    out = torch.full_like(q, 7.0)
    attend(b, pool, q, table, ctx, scale, 1, out=out, dev_err=err)
    ref, bound, _ = R.tree_attention(pool, q[at], few, ctx[at], scale, 1)
    inside(out[at], ref, bound, "requests")
    out[at] = 7.0
    assert bool((out == 7.0).all()) and b.gdn_read_device_error(err) == 0


def test_rows_in_place_and_rows_of_stride_zero(b, err):
    T = 300
    one, f = torch.ones(256, device="cuda"), torch.rand(32, dtype=torch.float64, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    q, k = randn(T, 24, 256).to(torch.bfloat16), randn(T, 4, 256, seed=1).to(torch.bfloat16)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    b.gdn_qk_norm_rope(q, k, one, one, 1e-6, pos, f, qo, ko, dev_err=err)
    b.gdn_qk_norm_rope(q, k, one, one, 1e-6, pos, f, q, ko, dev_err=err)
    assert torch.equal(bits(q), bits(qo))
    pools = [R.Pool(5, 4, 64, 256, "e4m3") for _ in range(2)]
    slots = torch.randperm(320, device="cuda")[:T].to(torch.int32)
    b.gdn_kv_cache_write(pools[0].handle(b), k[:1].expand(T, -1, -1), k[:, :1].expand(-1, 4, -1), slots, dev_err=err)
    b.gdn_kv_cache_write(pools[1].handle(b), k[:1].repeat(T, 1, 1), k[:, :1].repeat(1, 4, 1), slots, dev_err=err)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(bits(getattr(pools[0], name)), bits(getattr(pools[1], name))), name
    assert b.gdn_read_device_error(err) == 0


def test_guard_bands(b, err):
    """Outputs, pools and workspace between bands that every call must leave alone."""
    from tests.test_gpu_guards import Guarded
    for fmt in ("bf16", "e4m3"):
        lens, nodes = [1000, 1, 129], 5
        pool, table, ctx, q, scale = case("6x1x256", fmt, 16, lens, nodes)
        gk, gv = (Guarded(t.shape, t.dtype, t) for t in (pool.k, pool.v))
        pool.k, pool.v = gk.t, gv.t
        scales = []
        if fmt == "e4m3":
            scales = [Guarded(t.shape, t.dtype, t) for t in (pool.k_scale, pool.v_scale)]
            pool.k_scale, pool.v_scale = (g.t for g in scales)
        out = Guarded(q.shape, torch.bfloat16)
        ws = Guarded((b.gdn_tree_attention_workspace_bytes(pool.handle(b), 3, nodes, 6),), torch.uint8)
        ws.t.zero_()
        attend(b, pool, q, table, ctx, scale, nodes, out=out.t, workspace=ws.t, dev_err=err)
        T = sum(lens)
        ko, vo = (Guarded((T, 1, 256), torch.bfloat16) for _ in range(2))
        start = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        b.gdn_kv_cache_read(pool.handle(b), table, start, ko.t, vo.t, dev_err=err)
        qo, kk = Guarded((T, 6, 256), torch.bfloat16), Guarded((T, 1, 256), torch.bfloat16)
        x = randn(T, 6, 256).to(torch.bfloat16)
        slots = torch.randperm(pool.k.shape[0] * 16, device="cuda")[:T].to(torch.int32)
        one = torch.ones(256, device="cuda")
        f = torch.ones(32, dtype=torch.float64, device="cuda")
        b.gdn_qk_norm_rope(x, x[:, :1], one, one, 1e-6, slots, f, qo.t, kk.t, v=x[:, 1:2], cache=pool.handle(b), kv_slot=slots,
                           dev_err=err)
        assert b.gdn_read_device_error(err) == 0
        for g in [gk, gv, out, ws, ko, vo, qo, kk] + scales:
            g.check(fmt)


# ---------------------------------------------------------------- the linear layers' verify of a tree

def _paths(w, par):
    """The oracle's result of every node by its own path, as requests of their own from copies of the live slot."""
    N, P = par.shape
    dims = w["dims"]
    toks, lens, live = [], [], []
    for n in range(N):
        for p in range(P):
            path, at = [], p
            while at >= 0:
                path.append(n * P + at)
                at = int(par[n, at])
            toks += path[::-1]
            lens.append(len(path))
            live.append(w["slot_idx"][n])
    r = oracle.forward(dims, w["qkv0"][toks], w["conv_w"], np.ascontiguousarray(w["conv_hist"][live]),
                       np.ascontiguousarray(w["state"][live]), synth.pack_offsets(np.array(lens)),
                       np.arange(N * P, dtype=np.int32), w["alpha"][toks], w["beta"][toks], w["z"][toks], w["gamma"],
                       w["eps"], inplace=True)
    last = np.cumsum(lens) - 1
    return r["o"][last], r["ogate"][last], r["state"], r["conv_hist"]


@pytest.mark.parametrize("geom,N,P", [(synth.RANK_HEADS, 1, 1), (synth.RANK_HEADS, 3, 8), (synth.FULL_HEADS, 2, 5),
                                      (synth.Dims(8, 8, 128, 128, 4), 5, 7), (synth.Dims(2, 16, 128, 128, 4), 2, 8),
                                      (synth.RANK_HEADS, 60, 6)])
def test_verify_tree(b, err, geom, N, P):
    w = synth.spec_workload(geom, N, P, seed=17 + P)
    par = R.tree(N, P, seed=P)[0].numpy()
    d = U.to_device(w)
    D = b.make_dims(geom, w["num_slots"])
    o = torch.zeros(N * P, geom.num_v_heads, 128, dtype=torch.bfloat16, device="cuda")
    og = torch.zeros(N * P, geom.num_v_heads * 128, dtype=torch.bfloat16, device="cuda")
    b.gdn_spec_verify_tree(D, d["qkv0"], d["conv_w"], d["conv_hist"], d["state"], d["slot_idx"], d["spec_slot_idx"],
                           torch.from_numpy(par).cuda(), d["alpha"], d["beta"], d["z"], d["gamma"], w["eps"], o=o, ogate=og,
                           dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ro, rg, state, hist = _paths(w, par)
    U.check_out(U.host_f64_from_bf16(o), ro, "o")
    U.check_out(U.host_f64_from_bf16(og), rg, "ogate")
    ck = torch.from_numpy(w["spec_slot_idx"].reshape(-1).astype(np.int64)).cuda()
    U.check_state(d["state"][ck].cpu().numpy(), state, U.STATE_REL_L2_DECODE, "checkpoints")
    np.testing.assert_array_equal(U.host_bits(d["conv_hist"][ck]), hist)
    live = torch.from_numpy(w["slot_idx"].astype(np.int64)).cuda()
    assert torch.equal(d["state"][live].cpu(), torch.from_numpy(w["state"][w["slot_idx"]]))


@pytest.mark.parametrize("P", [1, 4, 8])
def test_verify_tree_of_a_chain_is_spec_verify(b, P):
    geom, N = synth.FULL_HEADS, 5
    w = synth.spec_workload(geom, N, P, seed=5)
    par = torch.arange(-1, P - 1, dtype=torch.int32, device="cuda").expand(N, P).contiguous()
    runs = []
    for tree in (False, True):
        d = U.to_device(w)
        og = torch.zeros(N * P, geom.num_v_heads * 128, dtype=torch.bfloat16, device="cuda")
        args = [b.make_dims(geom, w["num_slots"]), d["qkv0"], d["conv_w"], d["conv_hist"], d["state"], d["slot_idx"],
                d["spec_slot_idx"]] + ([par] if tree else []) + [d["alpha"], d["beta"], d["z"], d["gamma"], w["eps"]]
        (b.gdn_spec_verify_tree if tree else b.gdn_spec_verify)(*args, ogate=og)
        runs.append((og, d["state"], d["conv_hist"]))
    for x, y in zip(*runs):
        assert torch.equal(bits(x), bits(y))


def test_verify_tree_flags_bad_parents_and_skips_padding(b, err):
    geom, N, P = synth.RANK_HEADS, 5, 4
    w = synth.spec_workload(geom, N, P, seed=6)
    par = np.array([[-1, 0, 0, 1]] * N, np.int32)
    par[1, 2] = 2
    par[3, 0] = -2
    w["slot_idx"][2] = -1
    d = U.to_device(w)
    og = torch.full((N * P, geom.num_v_heads * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    b.gdn_spec_verify_tree(b.make_dims(geom, w["num_slots"]), d["qkv0"], d["conv_w"], d["conv_hist"], d["state"],
                           d["slot_idx"], d["spec_slot_idx"], torch.from_numpy(par).cuda(), d["alpha"], d["beta"], d["z"],
                           d["gamma"], w["eps"], ogate=og, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_TREE
    for n in (1, 2, 3):
        assert bool((og[n * P:(n + 1) * P] == 7.0).all())
        ck = w["spec_slot_idx"][n]
        assert torch.equal(d["state"][torch.from_numpy(ck.astype(np.int64)).cuda()].cpu(), torch.from_numpy(w["state"][ck]))
    ok = [0, 4]
    sub = {k: w[k] for k in ("dims", "conv_w", "conv_hist", "state", "gamma", "eps")}
    sub["slot_idx"] = w["slot_idx"][ok]
    rows = np.concatenate([np.arange(n * P, (n + 1) * P) for n in ok])
    for k in ("qkv0", "alpha", "beta", "z"):
        sub[k] = w[k][rows]
    U.check_out(U.host_f64_from_bf16(og[torch.from_numpy(rows).cuda()]), _paths(sub, par[ok])[1], "the others")


# ---------------------------------------------------------------- a speculative step through both layer types

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_drafted_tree_ends_where_plain_decoding_ends(b, err, fmt):
    """A tree of drafts is verified (attention layer: norms, rotation, cache, tree attention; linear layer: tree
    verify) and one path accepted: keys and values are written again at their final slots, the linear state is
    committed. Then cache, states and the next token's attention equal those of decoding the path token by token."""
    hq, hkv, d, page, ctx0, P = 6, 1, 256, 16, 75, 7
    par = [-1, 0, 0, 1, 2, 2, 4]
    path = [0, 2, 4, 6]
    mask = torch.tensor([[0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100101, 0b1010101]], device="cuda")
    f = 1e7 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device="cuda") / 64)
    g = randn(d, seed=8).abs() + 0.5
    table = R.tables([ctx0 + P], page, 12)
    drafts = randn(P + 1, hq + 2 * hkv, d, seed=7).to(torch.bfloat16)  # the last row: the token after the path
    geom = synth.RANK_HEADS
    w = synth.spec_workload(geom, 1, P, seed=3)
    D = b.make_dims(geom, w["num_slots"])

    def slots(positions):
        p = torch.tensor(positions, device="cuda")
        return (table[0, p.clamp_min(0) // page] * page + (p.clamp_min(0) % page).to(torch.int32)).where(p >= 0, -1).to(
            torch.int32)

    def layer(pool, rows, positions, at, ctx, nodes, m=None):
        """One attention layer's step over the given token rows."""
        x = drafts[rows]
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        qo, out = (torch.empty(len(rows), hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
        b.gdn_qk_norm_rope(q, k, g, g, 1e-6, pos, f, qo, v=v, cache=pool.handle(b), kv_slot=slots(at), dev_err=err)
        b.gdn_tree_attention(pool.handle(b), qo, table, torch.tensor([ctx], dtype=torch.int32, device="cuda"), d ** -0.5,
                             out, nodes, tree_mask=m, dev_err=err)
        return out

    depth = [0, 1, 1, 2, 2, 2, 3]
    spec, plain = (R.Pool(12, hkv, page, d, fmt, seed=4) for _ in range(2))
    tree_out = layer(spec, list(range(P)), [ctx0 + x for x in depth], [ctx0 + i for i in range(P)], ctx0, P, mask)
    x = drafts[path]
    final = [ctx0 + i for i in range(len(path))]
    b.gdn_qk_norm_rope(None, x[:, hq:hq + hkv], None, g, 1e-6, torch.tensor(final, dtype=torch.int32, device="cuda"), f, None,
                       v=x[:, hq + hkv:], cache=spec.handle(b), kv_slot=slots(final), dev_err=err)
    seq_out = [layer(plain, [r], [ctx0 + i], [ctx0 + i], ctx0 + i, 1) for i, r in enumerate(path)]
    for i, r in enumerate(path):  # the same sums over other tiles of the cache: fp32 orders apart, so one bf16 step
        a, c = tree_out[r].float(), seq_out[i][0].float()
        assert bool(((a - c).abs() <= 2 * R.BF16 * (a.abs() + 0.2)).all())
    at = slots(final).long()
    for name in ("k", "v") + (("k_scale", "v_scale") if fmt == "e4m3" else ()):
        assert torch.equal(bits(getattr(spec, name)[at // page, :, at % page]),
                           bits(getattr(plain, name)[at // page, :, at % page])), name
    nxt = [layer(p, [P], [ctx0 + 4], [ctx0 + 4], ctx0 + 4, 1) for p in (spec, plain)]
    assert torch.equal(bits(nxt[0]), bits(nxt[1]))

    # the linear layer: verify the tree and commit its accepted leaf; or decode the path
    t = U.to_device(w)
    og = torch.zeros(P, geom.num_v_heads * 128, dtype=torch.bfloat16, device="cuda")
    b.gdn_spec_verify_tree(D, t["qkv0"], t["conv_w"], t["conv_hist"], t["state"], t["slot_idx"], t["spec_slot_idx"],
                           torch.tensor([par], dtype=torch.int32, device="cuda"), t["alpha"], t["beta"], t["z"], t["gamma"],
                           w["eps"], ogate=og, dev_err=err)
    b.gdn_spec_commit(D, torch.tensor([path[-1]], dtype=torch.int32, device="cuda"), t["spec_slot_idx"], t["slot_idx"],
                      t["state"], t["conv_hist"], dev_err=err)
    s = U.to_device(w)
    step = torch.zeros(1, geom.num_v_heads * 128, dtype=torch.bfloat16, device="cuda")
    for r in path:
        b.gdn_decode_step(D, s["qkv0"][r:r + 1].contiguous(), s["conv_w"], s["conv_hist"], s["state"], s["slot_idx"],
                          s["alpha"][r:r + 1].contiguous(), s["beta"][r:r + 1].contiguous(), s["z"][r:r + 1].contiguous(),
                          s["gamma"], w["eps"], ogate=step, dev_err=err)
    live = int(w["slot_idx"][0])
    U.check_state(t["state"][live].cpu().numpy(), s["state"][live].cpu().numpy().astype(np.float64), U.STATE_REL_L2_DECODE,
                  "committed state")
    assert torch.equal(t["conv_hist"][live], s["conv_hist"][live])
    assert bool(((og[path[-1]].float() - step[0].float()).abs() <= 2 * R.BF16 * (step[0].float().abs() + 1e-2)).all())
    assert b.gdn_read_device_error(err) == 0
