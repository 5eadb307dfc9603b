"""Edges of what thins out a cache: values and pages that are no good, memory that the call in front has just written, long
pieces of the line of tiles, calls on two streams, a captured step. Against the fp64 statements, whose tolerances count the
roundings (attnref, thinref)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import attnref as R  # noqa: E402
from tests import thinref as T  # noqa: E402

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
    off = (got.double() - ref).abs()
    bad = ~(off <= bound) & ~(got.isnan() & ref.isnan()) & ~(got.double() == ref)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / bound)[bad].max())}" \
                                f" times its bound at {torch.nonzero(bad)[0].tolist()}"


def case(heads, fmt, page, lens, nodes, seed=0, strong=1.0):
    hq, hkv, d = heads
    held = [n + nodes for n in lens]
    pages = sum(-(-n // page) for n in held) + 2
    pool = R.Pool(pages, hkv, page, d, fmt, seed=seed)
    table = R.tables(held, page, pages, seed=seed)
    q = (randn(len(lens) * nodes, hq, d, seed=seed + 9) * strong).to(torch.bfloat16)
    return pool, table, ints(lens), q, d ** -0.5


def attend(b, pool, q, table, ctx, scale, nodes, was=NAN, **kw):
    out, lse = torch.full_like(q, NAN), torch.full(q.shape[:2], was, device="cuda")
    b.gdn_tree_attention_lse(pool.handle(b), q, table, ctx, scale, out, lse, nodes, **kw)
    return out, lse


def parts(pool):
    return [x for x in ("k", "v", "k_scale", "v_scale") if getattr(pool, x) is not None]


def copy_of(pool):
    """A pool with the same contents."""
    other = R.Pool(1, 1, pool.page, pool.k.shape[-1], pool.fmt)
    for x in parts(pool):
        setattr(other, x, getattr(pool, x).clone())
    return other


# ---------------------------------------------------------------- the log-sum-exp over an E4M3 cache

# heads, nodes: a row tile of up to 16, of up to 32 and of up to 64 rows, and several of them
ROWS = [((24, 4, 256), 1), ((24, 4, 256), 5), ((32, 8, 128), 7), ((24, 4, 256), 20)]


def spread_bound(ref, bound):
    """The attention's maxima are of scores with the exponents of the values' scales, of up to 128, in them: the score with
    the exponent, that less the maximum, the maximum with the sum's logarithm (the sum is 2^-190 of the largest weight at
    least) and its product with ln 2 are each rounded to fp32, 2^-24 of numbers of up to twice the log-sum-exp and 400."""
    return bound + 4 * (2 * ref.abs().nan_to_num(0, 0, 0) + 400) * 2.0 ** -24


@pytest.mark.parametrize("odd", [NAN, INF, -INF])
@pytest.mark.parametrize("heads,nodes", ROWS)
def test_lse_of_values_that_are_no_numbers(b, err, heads, nodes, odd):
    """The log-sum-exp is of queries and keys: a token whose values, or their scale, are no numbers counts in it like any
    other, while the request's output shows it."""
    lens = [300, 20000, 40]
    pool, table, ctx, q, scale = case(heads, "e4m3", 64, lens, nodes)
    ref, bound = T.lse(pool, q, table, ctx, scale, nodes)
    weight = torch.exp(T.logits(pool, q, table, 2, lens[2], scale, nodes)[0][..., 7].reshape(nodes, -1) - ref[2 * nodes:])
    assert float(weight.max()) > 1e-2  # what would be missing
    for n, t in ((1, 0), (1, 19999), (2, 7)):
        pool.v_scale[int(table[n, t // 64]), :, t % 64] = odd
    pool.v[int(table[2, 0]), :, 9] = 0x7F
    out, lse = attend(b, pool, q, table, ctx, scale, nodes, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    inside(lse, ref, spread_bound(ref, bound), "lse")
    assert not bool(out[nodes:].isfinite().any()) and bool(out[:nodes].isfinite().all())


@pytest.mark.parametrize("heads,nodes", ROWS)
@pytest.mark.parametrize("strong", [0.0, 1.0, 12.0])
@pytest.mark.parametrize("kind", ["0", "5", "60", "one large", "one small"])
def test_lse_over_value_scales_far_apart(b, err, heads, nodes, strong, kind):
    """Every token's values with a scale of their own, of either sign, or one token's at the other end of the format."""
    lens = [777, 12, 127, 9000]
    pool, table, ctx, q, scale = case(heads, "e4m3", 16, lens, nodes, seed=3, strong=strong)
    if kind in ("one large", "one small"):
        few, most = (2.0 ** 111, 1e-12 / 448) if kind == "one large" else (1e-12 / 448, 2.0 ** 111)
        pool.v_scale.fill_(most)
        for n, c in enumerate(lens):
            pool.v_scale[int(table[n, c // 2 // 16]), :, c // 2 % 16] = few
    else:
        g = torch.Generator(device="cuda").manual_seed(7)
        up = torch.randint(-int(kind), int(kind) + 1, pool.v_scale.shape, generator=g, device="cuda").float() / 2
        sign = torch.randint(0, 2, pool.v_scale.shape, generator=g, device="cuda") * 2 - 1
        pool.v_scale.mul_(torch.exp2(up) * sign)
        if kind == "0":
            pool.v_scale[:, :, ::3] = 0.0
    _, lse = attend(b, pool, q, table, ctx, scale, nodes, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ref, bound = T.lse(pool, q, table, ctx, scale, nodes)
    inside(lse, ref, spread_bound(ref, bound), "lse")


# ---------------------------------------------------------------- a page out of the pool

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,nodes", [((24, 4, 256), 1), ((24, 4, 256), 7), ((32, 8, 128), 30), ((24, 4, 256), 64)])
def test_a_bad_page_leaves_no_weights_of_an_older_lse(b, err, fmt, heads, nodes):
    """The attention leaves a request out that has a page outside the pool, and its log-sum-exp too: the buffer's older
    contents, here the sums of much smaller scores, must not become weights. Scores of the other pages fade, new tokens' are
    zero, the bad page's stay; the other requests are whole."""
    lens = [300, 700, 20000, 20000, 90]
    pool, table, ctx, q, scale = case(heads, fmt, 64, lens, nodes)
    ref, bound = T.lse(pool, q, table, ctx, scale, nodes)
    good = table.clone()
    gone = {1: 3, 2: 0, 3: 20000 // 64}
    for n, page in gone.items():
        table[n, page] = pool.k.shape[0] if n % 2 else -1
    _, lse = attend(b, pool, q, table, ctx, scale, nodes, was=-50.0, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT
    live = torch.tensor([n not in gone for n in range(5)], device="cuda").repeat_interleave(nodes)
    assert bool(lse[~live].isnan().all())
    inside(lse[live], ref[live], bound[live], "lse")
    weights = randn(5, heads[1], 20100, seed=3).abs()
    was, slot = weights.clone(), torch.arange(5, dtype=torch.int32, device="cuda")
    want, lim = T.score(pool, q, lse, good, ctx, scale, nodes, weights, slot, None, 0.5)
    b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, weights, slot, nodes, decay=0.5, dev_err=err)
    assert b.gdn_read_device_error(err) == b.GDN_DEVERR_SLOT
    for n, page in gone.items():
        rows = slice(page * 64, page * 64 + 64)
        want[n, :, rows], lim[n, :, rows] = was[n, :, rows].double(), 0
    inside(weights, want, lim, "score")


# ---------------------------------------------------------------- memory that the call in front has written

def test_evictions_read_what_their_selection_left(b, err):
    """Calls one behind the other without a wait, with the lengths, the budgets, the new lengths and the kept indices in one
    line of memory: the move takes this call's, whatever lay there."""
    lens, rounds = [40, 25], 60
    pool = R.Pool(40, 2, 16, 128, "bf16", seed=1)
    table, fresh = R.tables([64, 64], 16, 10), R.tables([64, 64], 16, 10) + 20
    weights = randn(4, 2, 64, seed=2)
    line = torch.zeros(2 + 2 + 2 + 2 * 2 * 40, dtype=torch.int32, device="cuda")
    new_len, length, budget, kept = line[:2], line[2:4], line[4:6], line[6:].reshape(2, 2, 40)
    slot, dst = ints([0, 1]), ints([2, 3])
    plans = [ints([1 + (7 * i) % x for x in lens]) for i in range(rounds)]
    length.copy_(ints(lens))
    got = []
    c = pool.handle(b)
    torch.cuda.synchronize()
    for i in range(rounds):
        pool.k[20:].zero_()
        budget.copy_(plans[i])
        b.gdn_kv_evict(c, table, length, budget, weights, slot, kept, new_len, 1, 2, fresh, dst, dev_err=err)
        got.append((new_len.clone(), kept.clone(), pool.k.clone(), weights[2:].clone()))
    assert b.gdn_read_device_error(err) == 0
    for i, (n, k, keys, w) in enumerate(got):
        m = plans[i].tolist()
        assert n.tolist() == m
        want = T.evict(pool, table, lens, m, weights, slot, 1, 2)[0]
        for r in range(2):
            dst_page, row = fresh[r, torch.arange(m[r], device="cuda") // 16].long(), torch.arange(m[r], device="cuda") % 16
            for h in range(2):
                assert k[r, h, :m[r]].tolist() == want[r][h], (i, r, h)
                src = torch.tensor(want[r][h], device="cuda")
                assert torch.equal(keys[dst_page, h, row], pool.k[table[r, src // 16].long(), h, src % 16]), (i, r, h)
                assert torch.equal(w[r, h, :m[r]], weights[r, h, src]), (i, r, h)


@pytest.mark.parametrize("nodes", [1, 20])
def test_selections_read_what_the_scores_in_front_left(b, err, nodes):
    """Attention, scores and eviction one behind the other without a wait, a head's scores beginning anywhere in a line of
    memory: as with a wait between the calls."""
    lens, room, rounds = [1500, 700, 90], 1531, 12
    pool, table, ctx, q, scale = case((24, 4, 256), "bf16", 64, lens, nodes)
    fresh = R.Pool(pool.k.shape[0] + 60, 4, 64, 256, "bf16", seed=4)
    fresh.k[:pool.k.shape[0]], fresh.v[:pool.k.shape[0]] = pool.k, pool.v
    dst = torch.arange(pool.k.shape[0], pool.k.shape[0] + 60, dtype=torch.int32, device="cuda").reshape(3, 20)
    slot, to, length, budget = ints([0, 1, 2]), ints([3, 4, 5]), ctx + nodes, ints([600, 300, 40])
    out, c = torch.empty_like(q), fresh.handle(b)
    ws = torch.empty(b.gdn_tree_attention_workspace_bytes(c, 3, nodes, 24), dtype=torch.uint8, device="cuda")
    results = []
    for wait in (True, False):
        weights, lse = torch.zeros(6, 4, room, device="cuda"), torch.full(q.shape[:2], NAN, device="cuda")
        kept, new_len = torch.zeros(3, 4, 600, dtype=torch.int32, device="cuda"), ints([0, 0, 0])
        scales = [scale * (1 + 0.1 * i) for i in range(rounds)]
        here = []
        for s in scales:
            for call in (lambda: b.gdn_tree_attention_lse(c, q, table, ctx, s, out, lse, nodes, workspace=ws, dev_err=err),
                         lambda: b.gdn_kv_score(c, q, lse, table, ctx, s, weights, slot, nodes, decay=0.5, dev_err=err),
                         lambda: b.gdn_kv_evict(c, table, length, budget, weights, slot, kept, new_len, 0, 0, dst, to, dev_err=err)):
                call()
                if wait:
                    torch.cuda.synchronize()
            here.append([x.clone() for x in (lse, weights, kept, new_len, fresh.k[dst.flatten().long()])])
        results.append(here)
    assert b.gdn_read_device_error(err) == 0
    for i, (x, y) in enumerate(zip(*results)):
        for u, v in zip(x, y):
            assert torch.equal(bits(u), bits(v)), i


# ---------------------------------------------------------------- long pieces of the line of tiles

LONG = [  # heads, context lengths, nodes, strength: tiles a CTA, or pair tiles a pair, with 152 SMs
    ((24, 4, 256), [30000] * 8, 1, 1), ((32, 8, 128), [20000, 33, 47000, 9000], 6, 2),  # 49 and 31 tiles
    ((24, 4, 256), [131000], 8, 1),                      # 27 tiles
    ((24, 4, 256), [131071], 64, 1),                     # 27 pair tiles, two steps of 192 rows
    ((24, 4, 256), [40000, 30000, 50, 20001, 9000], 32, 2),  # 21, one step, pieces over several requests and heads
    ((6, 1, 256), [99999, 77777], 50, 1),                # 9, two steps of 160 rows
    ((128, 8, 256), [60000], 64, 1),                     # 1024 rows in three chunks, 25 places a pair: several runs of tiles
    ((64, 4, 128), [50001, 70000, 200], 40, 1),          # 640 rows in two chunks
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,lens,nodes,strong", LONG)
def test_scores_of_long_pieces(b, err, fmt, heads, lens, nodes, strong):
    """Many tiles a CTA, over several requests and heads, rings and buffers gone round many times; with more rows than a pair
    keeps, several chunks in turn over runs of tiles. What was there fades once."""
    pool, table, ctx, q, scale = case(heads, fmt, 64, lens, nodes, strong=strong)
    _, lse = attend(b, pool, q, table, ctx, scale, nodes, dev_err=err)
    room = max(lens) + nodes + 3
    weights = randn(len(lens) + 1, heads[1], room, seed=3).abs()
    weights *= 0.01
    slot = torch.randperm(len(lens) + 1, device="cuda")[:len(lens)].to(torch.int32)
    ref, bound = T.score(pool, q, lse, table, ctx, scale, nodes, weights, slot, None, 0.75)
    again = weights.clone()
    for w in (weights, again):
        b.gdn_kv_score(pool.handle(b), q, lse, table, ctx, scale, w, slot, nodes, decay=0.75, dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    inside(weights, ref, bound, "score")
    assert torch.equal(bits(weights), bits(again))
    for n, c in enumerate(lens):  # what a kv head's rows hand out is one each
        total = weights[int(slot[n]), :, :c + nodes].double().sum(-1)
        assert bool((total >= nodes * heads[0] / heads[1] * 0.999).all())
    for n, c in enumerate(lens):
        ref, bound = T.lse(pool, q[n * nodes:(n + 1) * nodes], table[n:n + 1], ctx[n:n + 1], scale, nodes)
        inside(lse[n * nodes:(n + 1) * nodes], ref, bound, f"lse of request {n}")


# ---------------------------------------------------------------- two streams, a captured step

def test_batches_on_two_streams_at_once(b, err):
    """A batch on each of two streams, their calls enqueued in turn behind a pause and without a wait between them: rotation
    of rows strided inside a packed projection, attention, scores of few rows and of many, evictions in place and to other
    pages. Each batch's results are those of a run alone."""
    hq, hkv, d, page, few, many = 24, 4, 256, 64, 4, 40
    lens = [[2100, 70, 900], [1300, 3000]]
    f = 1e7 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    axes, g = b.make_rope_axes((12, 10, 10), True), randn(d, seed=2).abs() + 0.5

    class Batch:
        def __init__(self, i, stream):
            N, fmt, self.stream = len(lens[i]), ("bf16", "e4m3")[i], stream
            self.N, need = N, [n + many for n in lens[i]]
            pages = sum(-(-n // page) for n in need)
            self.pool = R.Pool(pages + 20 * N, hkv, page, d, fmt, seed=i)
            self.c = self.pool.handle(b)
            self.table = R.tables(need, page, pages, seed=i)
            self.dst = torch.arange(pages, pages + 20 * N, dtype=torch.int32, device="cuda").reshape(N, 20)
            self.ctx, self.length = ints(lens[i]), ints(need)
            self.packed = randn(N * many, hq + 2 * hkv, d, seed=9 + i).to(torch.bfloat16)
            self.pos = torch.randint(0, 9999, (3, N * many), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda",
                                     dtype=torch.int32)
            t = torch.cat([torch.arange(n, n + many) for n in lens[i]]).cuda()
            rows = torch.arange(N, device="cuda").repeat_interleave(many)
            self.kv_slot = (self.table[rows, t // page] * page + t % page).to(torch.int32)
            self.q = torch.zeros(N * many, hq, d, dtype=torch.bfloat16, device="cuda")
            self.q_few = randn(N * few, hq, d, seed=20 + i).to(torch.bfloat16)
            self.out, self.out_few = torch.zeros_like(self.q), torch.zeros_like(self.q_few)
            self.lse, self.lse_few = (torch.zeros(x.shape[:2], device="cuda") for x in (self.q, self.q_few))
            self.ws = [torch.empty(b.gdn_tree_attention_workspace_bytes(self.c, N, n, hq), dtype=torch.uint8, device="cuda")
                       for n in (few, many)]
            self.weights = torch.zeros(2 * N, hkv, 3100, device="cuda")
            self.slot, self.to = ints(list(range(N))), ints(list(range(N, 2 * N)))
            self.budget, self.half = ints([900] * N), ints([1100] * N)
            self.kept = [torch.zeros(N, hkv, 1100, dtype=torch.int32, device="cuda") for _ in range(2)]
            self.new_len = [torch.zeros(N, dtype=torch.int32, device="cuda") for _ in range(2)]

        def calls(self):
            kw = dict(dev_err=err, stream=self.stream)
            p, s = self.packed, d ** -0.5
            yield lambda: b.gdn_qk_norm_mrope(p[:, :hq], p[:, hq:hq + hkv], g, g, 1e-6, self.pos, f, axes, self.q,
                                              v=p[:, hq + hkv:], cache=self.c, kv_slot=self.kv_slot, **kw)
            yield lambda: b.gdn_tree_attention_lse(self.c, self.q, self.table, self.ctx, s, self.out, self.lse, many,
                                                   workspace=self.ws[1], **kw)
            yield lambda: b.gdn_tree_attention_lse(self.c, self.q_few, self.table, self.ctx, s, self.out_few, self.lse_few, few,
                                                   workspace=self.ws[0], **kw)
            yield lambda: b.gdn_kv_score(self.c, self.q, self.lse, self.table, self.ctx, s, self.weights, self.slot, many,
                                         decay=0.9, **kw)
            yield lambda: b.gdn_kv_score(self.c, self.q_few, self.lse_few, self.table, self.ctx, s, self.weights, self.slot, few,
                                         decay=0.9, **kw)
            yield lambda: b.gdn_kv_evict(self.c, self.table, self.length, self.budget, self.weights, self.slot, self.kept[0],
                                         self.new_len[0], 2, 30, self.dst, self.to, **kw)
            yield lambda: b.gdn_kv_evict(self.c, self.table, self.length, self.half, self.weights, self.slot, self.kept[1],
                                         self.new_len[1], 2, 30, **kw)

        def results(self):
            return [getattr(self.pool, x) for x in parts(self.pool)] + [self.q, self.out, self.out_few, self.lse, self.lse_few,
                                                                      self.weights, *self.kept, *self.new_len]

    streams = [torch.cuda.Stream() for _ in range(2)]
    alone, both = ([Batch(i, streams[i]) for i in range(2)] for _ in range(2))
    torch.cuda.synchronize()
    for x in alone:
        for _ in range(3):
            for call in x.calls():
                call()
        torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(4_000_000)  # some milliseconds: the calls below wait for each other on the host only
    for _ in range(3):
        for pair in zip(*(x.calls() for x in both)):
            for call in pair:
                call()
    torch.cuda.synchronize()
    assert b.gdn_read_device_error(err) == 0
    for x, y in zip(alone, both):
        for i, (u, v) in enumerate(zip(x.results(), y.results())):
            assert torch.equal(bits(u), bits(v)), i


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [2, 33, 64])
def test_a_captured_step_against_the_statements(b, err, fmt, nodes):
    """Scores and eviction in place captured on a stream that waits for what made its inputs; every replay, with contexts,
    slots and budgets of its own, is the fp64 statements' step on the state in front of it."""
    lens = [900, 300, 40]
    pool, table, ctx, q, scale = case((24, 4, 256), fmt, 64, lens, nodes)
    c = pool.handle(b)
    lse = T.lse(pool, q, table, ctx, scale, nodes)[0].float()
    slot, length, budget, new_len = ints([0, 1, 2]), ints([0, 0, 0]), ints([1, 1, 1]), ints([0, 0, 0])
    weights, kept = randn(5, 4, 1000, seed=5).abs(), torch.zeros(3, 4, 1000, dtype=torch.int32, device="cuda")

    def step(stream):
        b.gdn_kv_score(c, q, lse, table, ctx, scale, weights, slot, nodes, decay=0.5, dev_err=err, stream=stream)
        torch.add(ctx, nodes, out=length)
        b.gdn_kv_evict(c, table, length, budget, weights, slot, kept, new_len, 2, 8, dev_err=err, stream=stream)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    step(torch.cuda.current_stream())  # the first call outside the capture
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(side)
    for held, most, where in ((lens, [500, 100, 60], [0, 1, 2]), ([500, 100, 20], [400, 90, 10], [2, 4, 1]),
                              ([0, 300, 1], [1, 0, 2000], [3, 0, 4])):
        ctx.copy_(ints(held))
        budget.copy_(ints([min(m, 1000) for m in most]))
        slot.copy_(ints(where))
        before, w = copy_of(pool), weights.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert b.gdn_read_device_error(err) == 0
        scored = w.clone()
        b.gdn_kv_score(before.handle(b), q, lse, table, ctx, scale, scored, slot, nodes, decay=0.5)
        ref, bound = T.score(before, q, lse, table, ctx, scale, nodes, w, slot, None, 0.5)
        inside(scored, ref, bound, "score")
        full = [n + nodes for n in held]
        want, want_len, now, w_now = T.evict(before, table, full, most, scored, slot, 2, 8)
        assert new_len.tolist() == want_len
        for n in range(3):
            for h in range(4):
                assert kept[n, h, :want_len[n]].tolist() == want[n][h], (n, h)
        for x, t in now.items():
            assert torch.equal(bits(getattr(pool, x)), bits(t)), x
        assert torch.equal(bits(weights), bits(w_now))


# ---------------------------------------------------------------- the rotation over several axes, into the cache

@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,n,sections,mixed,inter,page", [
    ((24, 4, 256), 256, (12, 10, 10), True, False, 64), ((24, 4, 256), 3001, (16, 8, 8), False, False, 48),
    ((6, 1, 256), 41, (48, 40, 40), True, True, 16), ((32, 8, 128), 700, (2, 2, 2, 2), True, False, 128)])
def test_rotation_by_other_positions_an_axis_into_the_cache(b, err, fmt, heads, n, sections, mixed, inter, page):
    """Positions that differ between the axes: the cached keys against the statement, an axis at a time; the values' codes
    and scales are the oracle's, bit by bit; nothing else moves."""
    hq, hkv, d = heads
    pool = R.Pool(-(-n // page) + 2, hkv, page, d, fmt, seed=n)
    was = copy_of(pool)
    packed = (randn(n, hq + 2 * hkv, d, seed=n) * 2).to(torch.bfloat16)
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    gain, half = randn(d, seed=2).abs() + 0.5, sum(sections)
    g = torch.Generator(device="cuda").manual_seed(n)
    pos = torch.randint(0, 1 << 20, (len(sections), n), generator=g, device="cuda", dtype=torch.int32)
    f = 1e7 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    axes = b.make_rope_axes(sections, mixed)
    slots = torch.randperm(pool.k.shape[0] * page, generator=g, device="cuda")[:n].to(torch.int32)
    slots[n // 2] = -1
    qo = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    b.gdn_qk_norm_mrope(q, k, gain, gain, 1e-6, pos, f, axes, qo, v=v, cache=pool.handle(b), kv_slot=slots, interleaved=inter,
                        dev_err=err)
    assert b.gdn_read_device_error(err) == 0
    ref, mag = R.norm_rope(k, gain, 1e-6, pos[0], f * 0, inter)
    for a in range(len(sections)):
        i = torch.tensor([j for j in range(half) if axes.axis[j] == a], dtype=torch.long, device="cuda")
        mine = torch.zeros(half, dtype=torch.float64, device="cuda")
        mine[i] = 1
        where = torch.cat((2 * i, 2 * i + 1) if inter else (i, i + half))
        r, m = R.norm_rope(k, gain, 1e-6, pos[a], f * mine, inter)
        ref[..., where], mag[..., where] = r[..., where], m[..., where]
    kept = slots >= 0
    pg, row = slots[kept].long() // page, slots[kept].long() % page
    ref, mag = ref[kept], mag[kept]
    if fmt == "bf16":
        inside(pool.k[pg, :, row], ref, R.rope_bound(ref, mag), "keys")
        assert torch.equal(bits(pool.v[pg, :, row]), bits(v[kept]))
    else:
        s, amax = pool.k_scale[pg, :, row].double(), ref.abs().amax(-1)
        # the largest value: what rope_bound counts beside the rounding to bf16, of the largest pair; then a division
        slack = (2.0 ** -16 + 2.0 ** -20) * mag
        assert bool(((s - amax / 448).abs() <= slack.amax(-1) / 448 + 2.0 ** -23 * amax / 448).all())
        val = R._TABLE.cuda()[pool.k[pg, :, row].long()] * s[..., None]
        # half a step of the code, relative (2^-4) or E4M3's smallest (2^-10 of the scale), of a value that is off by slack
        inside(val, ref, R.E4M3 * (ref.abs() + slack) * (1 + 2.0 ** -20) + 2.0 ** -10 * s[..., None] + slack, "keys")
        codes, scale = R.quantise(v[kept].float())
        assert torch.equal(pool.v[pg, :, row].cpu(), codes) and torch.equal(pool.v_scale[pg, :, row].cpu(), scale)
    touched = torch.zeros(pool.k.shape[0], page, dtype=torch.bool, device="cuda")
    touched[pg, row] = True
    keep = ~touched[:, None].expand(-1, hkv, -1)
    for x in parts(pool):
        assert torch.equal(bits(getattr(pool, x)[keep]), bits(getattr(was, x)[keep])), x
