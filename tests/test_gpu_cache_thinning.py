"""What thins out a cache, and the rotation over several axes, on the GPU against their fp64 statements: head norms with
a position per axis, the attention's log-sum-exp, the weight that cached tokens receive, eviction by it, and a
request's way through all of them. Tolerances count the roundings (attnref, thinref)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import attnref as R  # noqa: E402
from tests import thinref as T  # noqa: E402

HEADS = {"24x4x256": (24, 4, 256), "6x1x256": (6, 1, 256), "32x8x128": (32, 8, 128), "5x5x128": (5, 5, 128)}
NAN, INF = float("nan"), float("inf")


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


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8)


def inside(got, ref, bound, what):
    got = got.double()
    off = (got - ref).abs()
    bad = ~(off <= bound) & ~(got.isnan() & ref.isnan()) & ~(got == ref)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound)[bad].max())}" \
                                f" times its bound at {torch.nonzero(bad)[0].tolist()}"


# ---------------------------------------------------------------- the rotation over several axes

def grid_positions(axes, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 1 << 20, (axes, n), generator=g, device="cuda", dtype=torch.int32)


MROPE = [("24x4x256", 1, (12, 10, 10), True, False), ("24x4x256", 333, (16, 8, 8), False, False),
         ("24x4x256", 5000, (12, 10, 10), True, True), ("6x1x256", 3, (48, 40, 40), True, False),
         ("32x8x128", 700, (0, 8, 8), False, False), ("5x5x128", 2, (2, 2, 2, 2), True, False),
         ("32x8x128", 17, (64,), False, True)]


@pytest.mark.parametrize("heads,n,sections,mixed,inter", MROPE)
def test_mrope(b, err, heads, n, sections, mixed, inter):
    hq, hkv, d = HEADS[heads]
    packed = (randn(n, hq + 2 * hkv, d, seed=n) * 2).to(torch.bfloat16)
    q, k = packed[:, :hq], packed[:, hq:hq + hkv]
    qg, kg = randn(d, seed=1).abs() + 0.1, randn(d, seed=2)
    half = sum(sections)
    pos = grid_positions(len(sections), n, n)
    f = 1e7 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    axes = b.make_rope_axes(sections, mixed)
    qo, ko = (torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv))
    b.gdn_qk_norm_mrope(q, k, qg, kg, 1e-6, pos, f, axes, qo, ko, interleaved=inter, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    axis = [axes.axis[i] for i in range(half)]
    assert [axis.count(a) for a in range(len(sections))] == list(sections)
    for x, g, out, what in ((q, qg, qo, "q"), (k, kg, ko, "k")):
        # an axis at a time: its frequencies turn by its positions, the others not at all
        ref, mag = None, None
        for a in range(len(sections)):
            mine = torch.tensor([float(y == a) for y in axis], dtype=torch.float64, device="cuda")
            r, m = R.norm_rope(x, g, 1e-6, pos[a], f * mine, inter)
            i = torch.tensor([j for j, y in enumerate(axis) if y == a], dtype=torch.long, device="cuda")
            where = torch.cat((2 * i, 2 * i + 1) if inter else (i, i + half))
            if ref is None:
                ref, mag = r.clone(), m.clone()
            ref[..., where], mag[..., where] = r[..., where], m[..., where]
        inside(out, ref, R.rope_bound(ref, mag), what)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_mrope_of_equal_positions_is_the_rotation_by_one(b, err, fmt):
    """The same bits, dense and in the cache; a captured call replayed with other positions takes them."""
    hq, hkv, d, n, page = 24, 4, 256, 77, 16
    q, k, v = (randn(n, h, d, seed=h).to(torch.bfloat16) for h in (hq, hkv, hkv))
    g = randn(d, seed=2).abs() + 0.5
    pos = grid_positions(1, n, 3)
    f = 1e7 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    slots = torch.randperm(10 * page, device="cuda")[:n].to(torch.int32)
    one, many = (R.Pool(10, hkv, page, d, fmt, seed=4) for _ in range(2))
    out = [torch.empty_like(x) for x in (q, k, q, k)]
    b.gdn_qk_norm_rope(q, k, g, g, 1e-6, pos[0], f, out[0], out[1], v=v, cache=one.handle(b), kv_slot=slots)
    axes, three = b.make_rope_axes((12, 10, 10), True), pos.expand(3, n).contiguous()
    c = many.handle(b)

    def call():
        b.gdn_qk_norm_mrope(q, k, g, g, 1e-6, three, f, axes, out[2], out[3], v=v, cache=c, kv_slot=slots, dev_err=err)

    call()
    same = [(out[0], out[2]), (out[1], out[3]), (one.k, many.k), (one.v, many.v), (one.k_scale, many.k_scale)]
    for x, y in same:
        assert x is None or torch.equal(bits(x), bits(y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    three.add_(5)
    graph.replay()
    b.gdn_qk_norm_rope(q, k, g, g, 1e-6, pos[0] + 5, f, out[0], out[1], v=v, cache=one.handle(b), kv_slot=slots)
    for x, y in same:
        assert x is None or torch.equal(bits(x), bits(y))
    assert b.gdn_read_device_error(err) == 0


# ---------------------------------------------------------------- log-sum-exp and weights

def case(heads, fmt, page, lens, nodes, seed=0, strong=1.0):
    hq, hkv, d = HEADS[heads] if isinstance(heads, str) else heads
    held = [n + nodes if n >= 0 else 0 for n in lens]
    pages = sum(-(-n // page) for n in held) + 2
    pool = R.Pool(pages, hkv, page, d, fmt, seed=seed)
    table = R.tables(held, page, pages, seed=seed)
    q = (randn(len(lens) * nodes, hq, d, seed=seed + 9) * strong).to(torch.bfloat16)
    return pool, table, ints(lens), q, d ** -0.5


def attend(b, pool, q, table, ctx, scale, nodes, mask=None, **kw):
    out, lse = torch.full_like(q, NAN), torch.full(q.shape[:2], NAN, device="cuda")
    b.gdn_tree_attention_lse(pool.handle(b), q, table, ctx, scale, out, lse, nodes, tree_mask=mask, **kw)
    return out, lse


SIZES = [  # heads, page, context lengths, nodes, tree, strength of the scores
    ("24x4x256", 64, [0], 1, False, 1), ("24x4x256", 64, [1], 1, False, 1), ("24x4x256", 64, [127], 1, False, 1),
    ("24x4x256", 64, [128], 1, False, 3), ("24x4x256", 16, [509, 3, 0, 1000], 1, False, 1),
    ("24x4x256", 64, [5000], 4, False, 2), ("24x4x256", 128, [0, 100, 126, 127, 128], 8, True, 1),
    ("24x4x256", 48, [700, 2, 333], 5, True, 3), ("24x4x256", 256, [1023, 77], 64, True, 1),
    ("24x4x256", 16, [2100, 40, 0], 33, False, 2), ("6x1x256", 16, [40, 260], 64, True, 2),
    ("6x1x256", 64, [20000], 3, False, 4), ("6x1x256", 64, [9000, 1], 50, False, 1),
    ("32x8x128", 64, [900, 0, 31], 7, True, 1), ("32x8x128", 16, [2047], 16, False, 2),
    ("32x8x128", 64, [3000, 200], 64, False, 1), ("5x5x128", 64, [130, 64, 1], 9, True, 1),
    ("32x8x128", 128, list(range(0, 1200, 37)), 2, True, 1), ((64, 1, 128), 16, [300, 12], 5, True, 1),
    ((64, 1, 256), 32, [300, 1200], 64, False, 1), ((3, 1, 256), 16, [17] * 40, 1, False, 1),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page,lens,nodes,tree,strong", SIZES)
def test_lse_and_score(b, err, fmt, heads, page, lens, nodes, tree, strong):
    pool, table, ctx, q, scale = case(heads, fmt, page, lens, nodes, strong=strong)
    N, hkv = len(lens), pool.k.shape[1]
    mask = R.tree(N, nodes)[1].cuda() if tree else None
    out, lse = attend(b, pool, q, table, ctx, scale, nodes, mask, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    alone = torch.empty_like(out)
    b.gdn_tree_attention(pool.handle(b), q, table, ctx, scale, alone, nodes, tree_mask=mask)
    assert torch.equal(bits(alone), bits(out))
    ref, bound = T.lse(pool, q, table, ctx, scale, nodes, mask)
    inside(lse, ref, bound, "lse")
    room = max(lens) + nodes + 5
    weights = randn(N + 2, hkv, room, seed=3).abs()
    slot = torch.randperm(N + 2, device="cuda")[:N].to(torch.int32)
    init = torch.tensor([n % 3 != 1 for n in range(N)], device="cuda")
    ref, bound = T.score(pool, q, lse, table, ctx, scale, nodes, weights, slot, mask, 0.75, init)
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, weights, slot, nodes, tree_mask=mask, decay=0.75,
                   has_init=init, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    inside(weights, ref, bound, "score")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,nodes", [("24x4x256", 1), ("24x4x256", 7), ("32x8x128", 64)])
def test_lse_of_rows_that_see_nothing_and_of_requests_left_out(b, err, fmt, heads, nodes):
    """-inf without a context and without a node; a padding request's, a bad page's and a too long request's rows stay."""
    lens = [0, 700, -3, 0, 200, 90, 5000]
    pool, table, ctx, q, scale = case(heads, fmt, 64, lens, nodes)
    mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (len(lens), nodes), device="cuda")
    mask[0] = 0
    mask[3, ::2] = 0
    ref, bound = T.lse(pool, q, table, ctx, scale, nodes, mask)
    gone = [2, 4, 5]
    table[4, 1] = pool.k.shape[0]
    ctx[5] = 64 * table.shape[1] - nodes + 1
    _, lse = attend(b, pool, q, table, ctx, scale, nodes, mask, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT | b.GDN_DEVERR_OFFSETS
    rows = lambda n: slice(n * nodes, (n + 1) * nodes)  # noqa: E731
    for n in gone:
        assert bool(lse[rows(n)].isnan().all()), n
    keep = torch.cat([torch.arange(len(lens) * nodes, device="cuda")[rows(n)] for n in range(len(lens)) if n not in gone])
    inside(lse[keep], ref[keep], bound[keep], "lse")
    assert bool((lse[rows(0)] == -INF).all()) and bool((lse[rows(3)][::2] == -INF).all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [2, 64])
def test_captured_scores_and_evictions_replay_with_other_lengths(b, err, fmt, nodes):
    """A step's scores and its eviction as one graph: replayed with other contexts, slots and budgets it takes them, as
    eager calls do; two graphs of the same buffers in turn."""
    pool, table, ctx, q, scale = case("24x4x256", fmt, 64, [900, 300, 40], nodes)
    lse = T.lse(pool, q, table, ctx, scale, nodes)[0].float()
    slot, weights = ints([0, 1, 2]), torch.zeros(6, 4, 1000, device="cuda")
    length, budget, new_len = ints([0, 0, 0]), ints([500, 100, 60]), ints([0, 0, 0])
    kept = torch.zeros(3, 4, 1000, dtype=torch.int32, device="cuda")

    def step():
        b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, weights, slot, nodes, dev_err=err)
        torch.add(ctx, nodes, out=length)
        b.gdn_kv_evict(pool.handle(b), table, length, budget, weights, slot, kept, new_len, 2, 8, dev_err=err)
        torch.sub(new_len, nodes, out=ctx)

    state = (pool.k, pool.v, weights, ctx, new_len, kept) + ((pool.k_scale, pool.v_scale) if fmt == "e4m3" else ())
    start = [t.clone() for t in state]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g, stream=side):
            step()
    plans = [([500, 100, 60], [0, 1, 2]), ([400, 100, 66], [2, 0, 1]), ([333, -1, 0], [0, 1, 2]), ([nodes + 1] * 3, [3, 4, -1])]
    results = []
    for replayed in (False, True):
        for t, was in zip(state, start):
            t.copy_(was)
        for i, (most, where) in enumerate(plans):
            budget.copy_(ints(most))
            slot.copy_(ints(where))
            ctx.clamp_(min=0)
            graphs[i % 2].replay() if replayed else step()
        torch.cuda.synchronize()
        results.append([t.clone() for t in state])
        assert b.gdn_read_device_error(err) == b.GDN_DEVERR_OFFSETS  # the negative budget
    for x, y in zip(*results):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(8))
def test_score_of_random_sizes(b, err, fmt, seed):
    """Any mask, rows left out, padding requests and slots, shared pages; the scores of a new token start from zero whatever
    was there; the same call twice gives the same bits."""
    rng = np.random.default_rng(200 + seed)
    hkv, group, d = int(rng.integers(1, 6)), int(rng.integers(1, 13)), int(rng.choice([128, 256]))
    nodes = int(np.exp(rng.uniform(0, np.log(64.99))))
    N = int(rng.integers(1, 9))
    page = int(rng.choice([16, 32, 48, 64, 96, 128, 192]))
    lens = [int(np.exp(rng.uniform(0, np.log(3000)))) - 1 for _ in range(N)]
    if N > 2:
        lens[1] = -5
    pool, table, ctx, q, scale = case((hkv * group, hkv, d), fmt, page, lens, nodes, seed=seed, strong=2)
    if N > 3:  # two requests of the same prefix
        shared = min(table.shape[1], max(lens[0], 0) // page, max(lens[3], 0) // page)
        table[3, :shared] = table[0, :shared]
    mask = torch.from_numpy(rng.integers(-2 ** 63, 2 ** 63 - 1, (N, nodes))).cuda()
    lse = T.lse(pool, q, table, ctx, scale, nodes, mask)[0].float()
    drop = torch.from_numpy(rng.random(lse.shape) < 0.2).cuda()
    lse[drop] = torch.tensor([INF, -INF, NAN], device="cuda")[torch.arange(int(drop.sum()), device="cuda") % 3]
    room = max(max(lens), 0) + nodes + int(rng.integers(0, 100))
    weights = randn(N + 3, hkv, room, seed=seed)
    for n, c in enumerate(lens):
        if c >= 0:
            weights[n + 1, :, c:] = NAN
    slot = torch.arange(1, N + 1, dtype=torch.int32, device="cuda")
    if N > 4:
        slot[4] = -1
    again = weights.clone()
    ref, bound = T.score(pool, q, lse, table, ctx, scale, nodes, weights, slot, mask, 0.9)
    for w in (weights, again):
        b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, w, slot, nodes, tree_mask=mask, decay=0.9, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    inside(weights, ref, bound, "score")
    assert torch.equal(bits(weights), bits(again))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,nodes,lens", [("24x4x256", 1, [300]), ("24x4x256", 10, [700, 130]), ("24x4x256", 64, [1000, 3]),
                                              ("32x8x128", 20, [50, 900])])
def test_score_of_rows_far_apart(b, err, fmt, heads, nodes, lens):
    """Query rows from 2^-30 to 2^8 of each other, zeros among them, and rows left out that are large or no numbers: what a
    row's weights are off by is counted by that row's own size."""
    pool, table, ctx, q, scale = case(heads, fmt, 64, lens, nodes, seed=nodes)
    g = torch.Generator(device="cuda").manual_seed(nodes)
    power = torch.randint(-30, 9, q.shape[:2], generator=g, device="cuda").double()
    power[torch.rand(power.shape, generator=g, device="cuda") < 0.3] = 0
    q = (q.double() * 2 ** power[..., None]).to(torch.bfloat16)
    q[0, 1] = 0
    gone = torch.rand(q.shape[:2], generator=g, device="cuda") < 0.1
    for i, value in enumerate((3e38, NAN, INF)):
        q[..., 7 + i] = torch.where(gone & (torch.arange(q.shape[1], device="cuda") % 3 == i), value, q[..., 7 + i])
    finite = torch.where(gone[..., None], 0, q)
    lse = T.lse(pool, finite, table, ctx, scale, nodes)[0].float()
    lse[gone] = INF
    weights = randn(len(lens), pool.k.shape[1], max(lens) + nodes, seed=3)
    slot = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    ref, bound = T.score(pool, finite, lse, table, ctx, scale, nodes, weights, slot)
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, weights, slot, nodes, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    inside(weights, ref, bound, "score")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [1, 48])
def test_score_of_rows_that_are_no_numbers(b, err, fmt, nodes):
    """A row with an infinity or a NaN and a finite lse: no score of a token that it sees is a number, other heads' are."""
    pool, table, ctx, q, scale = case("24x4x256", fmt, 64, [300], nodes)
    lse = T.lse(pool, q, table, ctx, scale, nodes)[0].float()
    q[0, 2, 5] = NAN  # of kv head 0
    q[0, 20, 5] = NAN  # of kv head 3
    q[0, 20, 6] = INF
    weights = torch.zeros(1, 4, 300 + nodes, device="cuda")
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, weights, ints([0]), nodes, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    assert bool(weights[0, [0, 3], :301].isnan().all())
    assert bool(weights[0, [0, 3], 301:].isfinite().all()) and bool(weights[0, 1:3].isfinite().all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [6, 48])
def test_score_of_what_no_row_sees(b, err, fmt, nodes):
    """Keys that are no numbers, in nodes that no row sees, behind the last token and in unused pages, leave the others'
    scores as they were; a node that no row sees gets zero; where such a key is seen, its own token shows it alone."""
    lens = [130, 0, 200]
    pool, table, ctx, q, scale = case("24x4x256", fmt, 64, lens, nodes)
    mask = torch.tensor([[1 << j | 1 for j in range(nodes)]] * 3, device="cuda")
    mask[:, 4] = 1  # nobody sees node 4
    lse = T.lse(pool, q, table, ctx, scale, nodes, mask)[0].float()
    slot, room = ints([2, 0, 1]), 300
    clean, dirty = (torch.zeros(3, 4, room, device="cuda") for _ in range(2))
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, clean, slot, nodes, tree_mask=mask)
    for n, c in enumerate(lens):
        page, row = int(table[n, (c + 4) // 64]), (c + 4) % 64
        last_page, last = int(table[n, (c + nodes - 1) // 64]), (c + nodes - 1) % 64
        if fmt == "e4m3":
            pool.k[page, :, row] = 0x7F
            pool.k_scale[page, 0, row] = INF
            pool.k[last_page, :, last + 1:] = 0xFF
            pool.k_scale[last_page, :, last + 1:] = NAN
        else:
            pool.k[page, :, row] = NAN
            pool.k[page, 0, row] = INF
            pool.k[last_page, :, last + 1:] = NAN
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, dirty, slot, nodes, tree_mask=mask, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    assert torch.equal(bits(clean), bits(dirty))
    for n, c in enumerate(lens):
        assert not bool(clean[int(slot[n]), :, c + 4].any())
    page, row = int(table[0, 1]), 5  # token 69, of the context: every row sees it
    if fmt == "e4m3":
        pool.k_scale[page, :, row] = NAN
    else:
        pool.k[page, :, row] = NAN
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, dirty, slot, nodes, tree_mask=mask)
    assert bool(dirty[2, :, 69].isnan().all())
    dirty[2, :, 69] = 0
    assert bool(dirty.isfinite().all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale,decay", [(0.0, 1.0), (-0.1, 0.0), (1.5, -2.0)])
def test_score_of_any_scale(b, err, fmt, scale, decay):
    nodes, lens = 3, [300, 5]
    pool, table, ctx, q, _ = case("6x1x256", fmt, 16, lens, nodes)
    q *= 0.25
    _, lse = attend(b, pool, q, table, ctx, scale, nodes)
    ref, bound = T.lse(pool, q, table, ctx, scale, nodes)
    inside(lse, ref, bound, "lse")
    weights = randn(2, 1, 310)
    slot = ints([1, 0])
    ref, bound = T.score(pool, q, lse, table, ctx, scale, nodes, weights, slot, None, decay)
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, weights, slot, nodes, decay=decay, dev_err=err)
    inside(weights, ref, bound, "score")
    assert b.gdn_read_device_error(err) == 0


def test_score_flags_what_breaks_the_limits(b, err):
    """A table or a row of scores that cannot hold the tokens, a slot past the pool: the request writes nothing, the
    others are whole. A page out of the pool: its tokens' scores stay."""
    nodes, lens = 2, [40, 40, 40, 40]
    pool, table, ctx, q, scale = case("5x5x128", "bf16", 16, lens, nodes)
    lse = T.lse(pool, q, table, ctx, scale, nodes)[0].float()
    was = randn(5, 5, 42)
    slot = ints([0, 1, 2, 3])

    def run(table=table, ctx=ctx, slot=slot, room=42):
        w = was[..., :room].clone(memory_format=torch.contiguous_format)
        b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, w, slot, nodes, dev_err=err)
        return b.gdn_read_device_error(err), (w != was[..., :room]).any(1)

    flag, moved = run()
    assert flag == 0 and bool(moved[:4].all()) and not bool(moved[4].any())
    assert run(ctx=ints([40, 47, 40, 40]))[0] == b.GDN_DEVERR_OFFSETS  # a fourth page
    flag, moved = run(ctx=ints([30, 41, 30, 2 ** 31 - 1]), room=42)
    assert flag == b.GDN_DEVERR_OFFSETS and not bool(moved[[1, 3]].any()) and bool(moved[[0, 2]].any(1).all())
    flag, moved = run(slot=ints([0, 5, 2, 2 ** 31 - 1]))
    assert flag == b.GDN_DEVERR_SLOT and not bool(moved[[1, 3]].any()) and bool(moved[[0, 2]].all())
    for bad in (-1, pool.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[2, 1] = bad
        flag, moved = run(table=t)
        assert flag == b.GDN_DEVERR_SLOT
        assert bool(moved[[0, 1, 3]].all()) and moved[2].tolist() == [True] * 16 + [False] * 16 + [True] * 10


# ---------------------------------------------------------------- eviction

def evict_case(fmt, heads, d, page, lens, budgets, seed=0, spare=0, ties=True):
    pages = sum(-(-max(n, 0) // page) for n in lens) + 1
    more = sum(-(-max(n, 0) // page) for n in budgets)
    pool = R.Pool(pages + more, heads, page, d, fmt, seed=seed)
    table = R.tables(lens, page, pages, seed=seed, spare=spare)
    N = len(lens)
    w = randn(2 * N + 1, heads, max(max(lens), 1) + 7, seed=seed + 1).abs()
    if ties:
        w = torch.round(w * 8) / 8
    fresh = R.tables(budgets, page, more, seed=seed + 2) if more else torch.full((N, 1), -1, dtype=torch.int32, device="cuda")
    fresh = torch.where(fresh >= 0, fresh + pages, fresh)
    return pool, table, w, fresh


def check_evict(b, err, pool, table, lens, budgets, w, slot, sinks, recent, dst_table=None, dst_slot=None, spare=3):
    N, heads = len(lens), pool.k.shape[1]
    most = max([min(x, y) for x, y in zip(lens, budgets)] + [0]) + spare
    kept = torch.full((N, heads, most), -7, dtype=torch.int32, device="cuda")
    new_len = torch.full((N,), -9, dtype=torch.int32, device="cuda")
    want, want_len, now, w_now = T.evict(pool, table, lens, budgets, w, slot, sinks, recent, dst_table, dst_slot)
    b.gdn_kv_evict(pool.handle(b), table, ints(lens), ints(budgets), w, slot, kept, new_len, sinks, recent, dst_table,
                   dst_slot, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    assert new_len.tolist() == want_len
    for n in range(N):
        for h in range(heads):
            assert kept[n, h].tolist() == want[n][h] + [-7] * (most - len(want[n][h])), (n, h)
    for x, t in now.items():
        assert torch.equal(bits(getattr(pool, x)), bits(t)), x
    assert torch.equal(bits(w), bits(w_now))


EVICT = [  # kv heads, head_dim, page, lengths, budgets, sinks, recent
    (4, 256, 64, [1000], [500], 4, 64), (4, 256, 64, [1], [1], 0, 0), (4, 256, 64, [0, 5], [3, 0], 2, 2),
    (1, 256, 16, [17, 40, 3, 0, 129], [16, 39, 3, 9, 1], 1, 0), (8, 128, 16, [700, 20], [33, 19], 0, 5),
    (5, 128, 48, [333, 95, 96, 97], [100, 94, 48, 49], 3, 7), (2, 128, 256, [2500], [2499], 0, 0),
    (3, 256, 32, [64, 64], [10, 10], 8, 30), (4, 256, 128, [3000] * 9, list(range(100, 2800, 300)), 4, 32),
    (1, 128, 16, [9000], [4000], 16, 1000), (2, 128, 16, [300], [300], 0, 0),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("place", ["in place", "other pages"])
@pytest.mark.parametrize("heads,d,page,lens,budgets,sinks,recent", EVICT)
def test_evict(b, err, fmt, place, heads, d, page, lens, budgets, sinks, recent):
    pool, table, w, fresh = evict_case(fmt, heads, d, page, lens, [min(x, y) for x, y in zip(lens, budgets)])
    N = len(lens)
    slots = torch.randperm(2 * N + 1, device="cuda").to(torch.int32)
    check_evict(b, err, pool, table, lens, budgets, w, slots[:N].contiguous(), sinks, recent,
                *((fresh, slots[N:2 * N].contiguous()) if place != "in place" else ()))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("seed", range(6))
def test_evict_of_random_sizes(b, err, fmt, seed):
    """Weights of every kind; requests that share pages, which stay whole."""
    rng = np.random.default_rng(seed)
    heads, d = int(rng.integers(1, 6)), int(rng.choice([128, 256]))
    page = int(rng.choice([16, 32, 48, 64, 128]))
    lens = [int(np.exp(rng.uniform(0, np.log(5000)))) for _ in range(int(rng.integers(1, 7)))]
    budgets = [int(rng.integers(0, n + 2)) for n in lens]
    held = [min(x, y) for x, y in zip(lens, budgets)]
    pool, table, w, fresh = evict_case(fmt, heads, d, page, lens, held, seed=seed)
    odd = torch.tensor([NAN, -NAN, INF, -INF, 0.0, -0.0, 1e-42, -3.0, 3e38], device="cuda")
    pick = torch.randint(0, 60, w.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    w = torch.where(pick < 9, odd[pick.clamp_max(8)], w)
    sinks, recent = int(rng.integers(0, 6)), int(rng.integers(0, 40))
    slots = torch.randperm(2 * len(lens), device="cuda").to(torch.int32)
    if seed % 2:
        check_evict(b, err, pool, table, lens, budgets, w, slots[:len(lens)].contiguous(), sinks, recent)
        return
    for n in range(1, len(lens)):
        shared = min(lens[0], lens[n]) // page
        table[n, :shared] = table[0, :shared]
    check_evict(b, err, pool, table, lens, budgets, w, slots[:len(lens)].contiguous(), sinks, recent, fresh,
                slots[len(lens):].contiguous())


@pytest.mark.parametrize("n,budget,place", [(140000, 70001, "in place"), (131072, 1000, "other pages"),
                                            (16385, 16384, "in place")])
def test_evict_of_a_long_request(b, err, n, budget, place):
    """More tokens than the selection keeps in shared memory, one head, and all weights alike from some place on."""
    pool, table, w, fresh = evict_case("bf16", 1, 128, 16, [n], [budget], ties=False)
    w[0, 0, n // 2:] = 0.25
    check_evict(b, err, pool, table, [n], [budget], w, ints([0]), 4, 100,
                *((fresh, ints([2])) if place != "in place" else ()))


@pytest.mark.parametrize("n", [2000, 8100, 16300, 32700, 65500, 131000, 139000])
@pytest.mark.parametrize("kind", ["alike", "two values", "last bits", "steps", "few at the border"])
def test_evict_of_weights_close_together(b, err, n, kind):
    """Every number of blocks a head, with weights that differ late or not at all, beside requests of a part of the length."""
    lens = [n, n // 3, 700, 33, 1]
    budgets = [n // 2, n // 3 - 1, 699, 5, 1]
    pool, table, w, fresh = evict_case("e4m3", 2, 128, 64, lens, budgets)
    g = torch.Generator(device="cuda").manual_seed(n)
    pick = torch.randint(0, 1 << 20, w.shape, generator=g, device="cuda")
    w = {"alike": torch.zeros_like(w), "two values": torch.where(pick % 2 == 0, 0.5, 0.5 + 2.0 ** -24),
         "last bits": (0x3F000000 + pick % 1024).to(torch.int32).view(torch.float32),
         "steps": 2.0 ** -(pick % 3).float() * (1 + (pick % 5).float() * 2.0 ** -12),
         "few at the border": torch.where(pick % 4096 == 0, 1.0, torch.where(pick % 2 == 0, 2.0, 0.5))}[kind].contiguous()
    slots = torch.randperm(11, device="cuda").to(torch.int32)
    check_evict(b, err, pool, table, lens, budgets, w, slots[:5].contiguous(), 2, 9, fresh, slots[5:10].contiguous())


def test_scores_behind_32_bits(b, err):
    """A pool of scores of more than 2^31 of them: the last slot's as a small pool's, scored, evicted to another slot and in
    place."""
    lens, nodes, room = [700, 90], 3, 1 << 26
    pool, table, ctx, q, scale = case("24x4x256", "bf16", 64, lens, nodes)
    lse = T.lse(pool, q, table, ctx, scale, nodes)[0].float()
    far, near = torch.empty(9, 4, room, device="cuda"), torch.zeros(4, 4, 703, device="cuda")
    far[[0, 8]], fresh = 0, torch.zeros(2, dtype=torch.bool, device="cuda")
    kept = [torch.zeros(2, 4, 703, dtype=torch.int32, device="cuda") for _ in range(2)]
    new_len, dst = ints([0, 0]), torch.arange(20, dtype=torch.int32, device="cuda").reshape(2, 10)
    big = R.Pool(20 + pool.k.shape[0], 4, 64, 256, "bf16", seed=3)
    for w, slot, to, k in ((far, ints([8, 7]), ints([6, 0]), kept[0]), (near, ints([3, 2]), ints([1, 0]), kept[1])):
        b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, w, slot, nodes, has_init=fresh, dev_err=err)
        b.gdn_kv_evict(big.handle(b), table + 20, ctx + nodes, ints([300, 50]), w, slot, k, new_len, 1, 2, dst, to, dev_err=err)
    assert b.gdn_read_device_error(err) == 0 and new_len.tolist() == [300, 50]
    assert torch.equal(kept[0], kept[1])
    for x, y, n in ((8, 3, 703), (7, 2, 93), (6, 1, 300), (0, 0, 50)):
        assert torch.equal(bits(far[x, :, :n]), bits(near[y, :, :n])), x


def test_evict_of_many_short_requests(b, err):
    lens = [1 + i % 37 for i in range(300)]
    pool, table, w, _ = evict_case("bf16", 2, 128, 16, lens, [n // 2 for n in lens])
    slot = torch.randperm(300, device="cuda").to(torch.int32)
    check_evict(b, err, pool, table, lens, [n // 2 for n in lens], w, slot, 1, 1)


def test_evict_flags_what_breaks_the_limits(b, err):
    """Such a request writes nothing but a new length of -1, a padding request nothing at all; the others are whole."""
    lens, budgets = [40, 40, 40], [20, 20, 20]

    def run(length=lens, budget=budgets, slot=(0, 1, 2), dst=None, dst_slot=(3, 4, 5), bad_page=None, most=25, room=47):
        pool, table, w, fresh = evict_case("bf16", 2, 128, 16, lens, budgets, ties=False)
        w = w[:6, :, :room].contiguous()
        if bad_page:
            table[bad_page[0], bad_page[1]] = bad_page[2]
        if dst:
            fresh[dst[0], dst[1]] = dst[2]
        was, w_was = pool.k.clone(), w.clone()
        kept, new_len = torch.full((3, 2, most), -7, dtype=torch.int32, device="cuda"), ints([-9] * 3)
        b.gdn_kv_evict(pool.handle(b), table, ints(length), ints(budget), w, ints(slot), kept, new_len, 0, 0,
                       fresh if dst else None, ints(dst_slot) if dst else None, dev_err=err)
        used = [fresh[n][:2] if dst else table[n][:3] for n in range(3)]
        moved = [bool((pool.k[u.clamp(0, pool.k.shape[0] - 1).long()] != was[u.clamp(0, pool.k.shape[0] - 1).long()]).any())
                 for u in used]
        kept_moved = [bool((kept[n] != -7).any()) for n in range(3)]
        w_moved = [0 <= s < 6 and bool((w[s] != w_was[s]).any()) for s in (dst_slot if dst else slot)]
        return b.gdn_read_device_error(err), new_len.tolist(), moved, kept_moved, w_moved

    whole = [True, True, True]
    assert run() == (0, [20, 20, 20], whole, whole, whole)
    part = [True, False, True]
    SLOT, OFFSETS = b.GDN_DEVERR_SLOT, b.GDN_DEVERR_OFFSETS
    assert run(length=[40, -1, 40]) == (0, [20, -9, 20], part, part, part)
    assert run(slot=(0, -1, 2)) == (0, [20, -9, 20], part, part, part)
    for kw, flag in ((dict(length=[40, 49, 40], room=49), OFFSETS), (dict(length=[40, 45, 40], room=44), OFFSETS),
                     (dict(length=[40, 2 ** 31 - 1, 40]), OFFSETS), (dict(budget=[20, -1, 20]), OFFSETS),
                     (dict(budget=[20, 26, 20]), OFFSETS), (dict(slot=(0, 6, 2)), SLOT),
                     (dict(dst=(1, 1, 9), dst_slot=(3, 6, 5)), SLOT), (dict(dst=(1, 1, 9), dst_slot=(3, -1, 5)), SLOT),
                     (dict(bad_page=(1, 2, -1)), SLOT), (dict(bad_page=(1, 0, 1000)), SLOT),
                     (dict(bad_page=(1, 1, 2 ** 31 - 1)), SLOT), (dict(dst=(1, 1, -1)), SLOT),
                     (dict(dst=(1, 0, 2 ** 31 - 1)), SLOT)):
        got = run(**kw)
        assert got[:2] == (flag, [20, -1, 20]), (kw, got)
        assert got[3] == part and got[4] == part and (got[2] == part or "bad_page" in kw or "dst" in kw), (kw, got)
        assert got[2][0] and got[2][2], (kw, got)
    # a budget past every length is no limit broken as long as the kept tokens fit
    assert run(budget=[2 ** 31 - 1] * 3, most=40)[:2] == (0, [40, 40, 40])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_request_through_all_of_them(b, err, fmt):
    """A prompt of image and text rotated into the cache; its last rows' weights; the cache cut down; then decode steps, each
    written behind what is left, attended, scored, and cut down again: captured once as a graph on a stream of
    its own and replayed. Against the fp64 statements on the cache as it is before each call."""
    hq, hkv, d, page, prompt, window, budget = 24, 4, 256, 16, 700, 32, 300
    N, steps = 3, 4
    lens = [prompt, prompt - 123, 64]
    pages = sum(-(-(n + steps + 1) // page) for n in lens) + 2
    pool = R.Pool(pages, hkv, page, d, fmt, seed=1)
    table = R.tables([n + steps + 1 for n in lens], page, pages)
    c, scale = pool.handle(b), d ** -0.5
    g = randn(d, seed=2).abs() + 0.5
    f = 1e7 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    axes = b.make_rope_axes((12, 10, 10), True)
    slot = ints([2, 0, 1])
    weights = torch.full((3, hkv, max(lens) + steps + 8), NAN, device="cuda")

    def slots_of(n, first, count):
        t = torch.arange(first, first + count, device="cuda")
        return table[n, t // page] * page + (t % page).to(torch.int32)

    def rotated(rows, pos, kv_slot):
        packed = randn(rows, hq + 2 * hkv, d, seed=rows).to(torch.bfloat16)
        q = torch.empty(rows, hq, d, dtype=torch.bfloat16, device="cuda")
        b.gdn_qk_norm_mrope(packed[:, :hq], packed[:, hq:hq + hkv], g, g, 1e-6, pos, f, axes, q, v=packed[:, hq + hkv:],
                            cache=c, kv_slot=kv_slot, dev_err=err)
        return q

    # the prompts, packed; an image of 16 x 16 patches in each of the first two
    pos = []
    for n in lens:
        t = torch.arange(n, device="cuda", dtype=torch.int32)
        image = (t >= 50) & (t < 50 + 256) & (n > 400)
        i = t - 50
        pos.append(torch.stack((torch.where(image, 50, t), torch.where(image, 50 + i // 16, t),
                                torch.where(image, 50 + i % 16, t))))
    q = rotated(sum(lens), torch.cat(pos, 1).to(torch.int32).contiguous(), torch.cat([slots_of(n, 0, x) for n, x in enumerate(lens)]))
    start = np.cumsum([0] + lens)
    last = torch.cat([q[start[n + 1] - window:start[n + 1]] for n in range(N)])
    ctx = ints([n - window for n in lens])
    _, lse = attend(b, pool, last, table, ctx, scale, window, dev_err=err)
    init = torch.zeros(N, dtype=torch.uint8, device="cuda")
    ref, bound = T.score(pool, last, lse, table, ctx, scale, window, weights, slot, init=init)
    b.gdn_kv_score(c, last, lse, table, ctx, scale, weights, slot, window, has_init=init, dev_err=err)
    inside(weights, ref, bound, "prompt's weights")
    # every row's weights add up to one: what all tokens of a head receive is the number of its rows
    for n in range(N):
        total = weights[int(slot[n]), :, :lens[n]].double().sum(-1)
        assert bool(((total - window * hq / hkv).abs() <= 1e-4 * window * hq / hkv).all())
    length, budgets = ints(lens), ints([budget] * N)
    kept = torch.zeros(N, hkv, budget, dtype=torch.int32, device="cuda")
    new_len = torch.zeros(N, dtype=torch.int32, device="cuda")
    want, want_len, now, w_now = T.evict(pool, table, lens, [budget] * N, weights, slot, 4, window)
    b.gdn_kv_evict(c, table, length, budgets, weights, slot, kept, new_len, 4, window, dev_err=err)
    assert new_len.tolist() == want_len == [budget, budget, 64]
    assert torch.equal(bits(pool.k), bits(now["k"])) and torch.equal(bits(pool.v), bits(now["v"]))
    assert torch.equal(bits(weights), bits(w_now))

    # decode: everything that changes lies in device memory, so one captured step serves all of them
    step_pos = torch.stack([ints(lens)] * 3).contiguous()
    packed = torch.empty(N, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    kv_slot, cur = torch.zeros(N, dtype=torch.int32, device="cuda"), new_len.clone()
    q1, out = torch.empty(N, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(N, hq, d, dtype=torch.bfloat16, device="cuda")
    lse1 = torch.empty(N, hq, device="cuda")
    ws = torch.empty(b.gdn_tree_attention_workspace_bytes(c, N, 1, hq), dtype=torch.uint8, device="cuda")
    grown, left = torch.zeros_like(cur), torch.zeros_like(cur)

    def step(stream):
        b.gdn_qk_norm_mrope(packed[:, :hq], packed[:, hq:hq + hkv], g, g, 1e-6, step_pos, f, axes, q1,
                            v=packed[:, hq + hkv:], cache=c, kv_slot=kv_slot, dev_err=err, stream=stream)
        b.gdn_tree_attention_lse(c, q1, table, cur, scale, out, lse1, workspace=ws, dev_err=err, stream=stream)
        b.gdn_kv_score(c, q1, lse1, table, cur, scale, weights, slot, decay=0.95, dev_err=err, stream=stream)
        b.gdn_kv_evict(c, table, grown, budgets, weights, slot, kept, left, 4, window, dev_err=err, stream=stream)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    saved = [x.clone() for x in (pool.k, pool.v, weights)]
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        step(side)  # the first call outside the capture, on garbage; what it did is taken back
        for x, y in zip((pool.k, pool.v, weights), saved):
            x.copy_(y)
        with torch.cuda.graph(graph, stream=side):
            step(side)
    torch.cuda.synchronize()
    for i in range(steps):
        packed.copy_(randn(N, hq + 2 * hkv, d, seed=50 + i))
        at = cur.tolist()
        kv_slot.copy_(torch.cat([slots_of(n, at[n], 1) for n in range(N)]))
        grown.copy_(cur + 1)
        before = R.Pool(pages, hkv, page, d, fmt, seed=1)
        for x in ("k", "v", "k_scale", "v_scale"):
            if getattr(pool, x) is not None:
                getattr(before, x).copy_(getattr(pool, x))
        w_before = weights.clone()
        graph.replay()
        torch.cuda.synchronize()
        # the row written, by the same call into the copy
        qq = torch.empty_like(q1)
        b.gdn_qk_norm_mrope(packed[:, :hq], packed[:, hq:hq + hkv], g, g, 1e-6, step_pos, f, axes, qq,
                            v=packed[:, hq + hkv:], cache=before.handle(b), kv_slot=kv_slot)
        assert torch.equal(bits(qq), bits(q1))
        ref, bound, _ = R.tree_attention(before, q1, table, cur, scale, 1)
        inside(out, ref, bound, f"attention of step {i}")
        ref, bound = T.lse(before, q1, table, cur, scale, 1)
        inside(lse1, ref, bound, f"lse of step {i}")
        # the eviction moved the scores: which ones, by the kept indices it left
        scored = w_before.clone()
        b.gdn_kv_score(before.handle(b), q1, lse1, table, cur, scale, scored, slot, decay=0.95)
        ref, bound = T.score(before, q1, lse1, table, cur, scale, 1, w_before, slot, decay=0.95)
        inside(scored, ref, bound, f"weights of step {i}")
        _, want_len, now, w_now = T.evict(before, table, grown.tolist(), [budget] * N, scored, slot, 4, window)
        assert left.tolist() == want_len
        for x, t in now.items():
            assert torch.equal(bits(getattr(pool, x)), bits(t)), (i, x)
        assert torch.equal(bits(weights), bits(w_now))
        cur.copy_(left)
        step_pos.add_(1)
    assert b.gdn_read_device_error(err) == 0


def test_calls_on_two_streams_and_with_strided_rows_beside_them(b, err):
    """Two batches at once on two streams, as alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    cases = [case("24x4x256", fmt, 64, [900, 20, 3000], 4, seed=i) for i, fmt in enumerate(("bf16", "e4m3"))]
    alone, both = [], []
    for together in (False, True):
        for i, (pool, table, ctx, q, scale) in enumerate(cases):
            w = torch.zeros(3, 4, 3100, device="cuda")
            lse = T.lse(pool, q, table, ctx, scale, 4)[0].float()
            torch.cuda.synchronize()
            with torch.cuda.stream(streams[i]):
                for _ in range(3):
                    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, w, ints([0, 1, 2]), 4, dev_err=err,
                                   stream=streams[i])
            if not together:
                torch.cuda.synchronize()
            (both if together else alone).append(w)
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        assert torch.equal(bits(x), bits(y))
    assert b.gdn_read_device_error(err) == 0
    assert math.isfinite(float(alone[0].sum()))
