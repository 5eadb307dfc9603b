"""gdn_tree_attention over an E4M3 cache whose value scales lie far apart: what a row's weights lose goes by the tokens
that this row sees and by what they weigh."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests import attnref as R  # noqa: E402


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


def inside(got, ref, bound, what):
    off = (got.double() - ref).abs()
    bad = ~(off <= bound) & ~(got.isnan() & ref.isnan())
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
                                f"{float((off / bound)[bad].max())} times its bound at {torch.nonzero(bad)[0].tolist()}"


def statement(pool, q, table, ctx, scale, nodes, mask=None):
    """(out, bound) in fp64. A score is an fp32 sum of D products (D + 8 roundings of 2^-24) of a query that is held to
    2^-17 of its largest value, brought to base 2 and taken to a power: relative to a weight, that is the weight's error.
    The power is of the score with the exponent of the value's scale, less the row's largest such sum: three roundings of
    numbers of up to 190 more than the score. A weight times its value's scale, rounded to fp16 (2^-11) and held as two
    E4M3 terms of 4 + 4 bits, is off by 2^-8 + 2^-11 of itself, or by half of E4M3's smallest step, 2^-10, where 224 at
    least stands for the row's largest such product of a tile of 128 tokens: by 2^-17 of that product. The output is
    rounded once to bf16, 2^-8."""
    N, P, D = table.shape[0], nodes, q.shape[-1]
    Hq, Hkv = q.shape[1], pool.k.shape[1]
    outs, bounds = [], []
    for n in range(N):
        c = int(ctx[n])
        pages = table[n, :-(-(c + P) // pool.page)].long()
        k = pool.values("k", pages)[:, :c + P]
        code = R._TABLE.to(q.device)[pool.v[pages].long()].transpose(0, 1).reshape(Hkv, -1, D)[:, :c + P]
        sv = pool.v_scale[pages].double().transpose(0, 1).reshape(Hkv, -1)[:, :c + P]
        seen = torch.ones((P, c + P), dtype=torch.bool, device=q.device)
        words = [(2 << j) - 1 for j in range(P)] if mask is None else [int(w) for w in mask[n]]
        seen[:, c:] = torch.tensor([[bool(w >> i & 1) for i in range(P)] for w in words], device=q.device)
        x = q[n * P:(n + 1) * P].double().reshape(P, Hkv, Hq // Hkv, D)
        s = torch.einsum("phgd,htd->phgt", x, k) * scale
        here = seen[:, None, None, :].expand_as(s)
        reach = torch.einsum("phgd,htd->phgt", x.abs(), k.abs()) * abs(scale)
        coarse = x.abs().amax(-1, keepdim=True) * k.abs().sum(-1)[None, :, None, :] * abs(scale) * 2.0 ** -17
        ds = torch.where(here, reach * (D + 8) * 2.0 ** -24 + coarse + (c + P + 400) * 2.0 ** -24, 0).amax(-1)[..., None]
        p = torch.softmax(s.masked_fill(~here, float("-inf")), -1).nan_to_num(0)
        u = p * sv[None, :, None, :]
        o = torch.einsum("phgt,htd->phgd", u, code)
        lim = R.BF16 * o.abs() + (R.BF16 + 2.0 ** -11 + 2 * ds) * torch.einsum("phgt,htd->phgd", u.abs(), code.abs())
        for t0 in range(0, c + P, 128):
            t = slice(t0, t0 + 128)
            codes = torch.einsum("phgt,htd->phgd", here[..., t].double(), code[:, t].abs())
            lim = lim + 2.0 ** -17 * u[..., t].abs().amax(-1)[..., None] * codes
        outs.append(o.reshape(P, Hq, D))
        bounds.append(lim.reshape(P, Hq, D))
    return torch.cat(outs), torch.cat(bounds)


def make(heads, lens, nodes, page=64, strong=1.0, seed=0):
    hq, hkv, d = heads
    pages = sum(-(-(n + nodes) // page) for n in lens) + 1
    pool = R.Pool(pages, hkv, page, d, "e4m3", seed=seed)
    table = R.tables([n + nodes for n in lens], page, pages, seed=seed)
    q = (randn(len(lens) * nodes, hq, d, seed=seed + 9) * strong).to(torch.bfloat16)
    return pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), q, d ** -0.5


def attend(b, pool, q, table, ctx, scale, nodes, mask=None, dev_err=None):
    out = torch.full_like(q, float("nan"))
    b.gdn_tree_attention(pool.handle(b), q, table, ctx, scale, out, nodes, tree_mask=mask, dev_err=dev_err)
    return out


def place(pool, table, n, t):
    return int(table[n, t // pool.page]), t % pool.page


# heads, nodes: a row tile of up to 16, of up to 32 and of up to 64 rows, for heads of 256 and of 128
ROWS = [((6, 1, 256), 2), ((24, 4, 256), 5), ((24, 4, 256), 9), ((32, 8, 128), 3), ((32, 8, 128), 7), ((5, 5, 128), 60)]


@pytest.mark.parametrize("heads,nodes", ROWS)
def test_a_large_value_scale_of_an_unseen_node_leaves_a_row_as_it_is(b, err, heads, nodes):
    """Node 1's values are multiplied by ever more. The nodes that do not see it stay within the bound of the run
    without, the others within their own."""
    lens = [130, 40, 3, 700]
    pool, table, ctx, q, scale = make(heads, lens, nodes)
    words = [1] + [(1 << j) | 1 | (2 if j % 2 else 0) for j in range(1, nodes)]  # the odd nodes see node 1
    mask = torch.tensor([words] * len(lens), dtype=torch.int64, device="cuda")
    ref, bound = statement(pool, q, table, ctx, scale, nodes, mask)
    inside(attend(b, pool, q, table, ctx, scale, nodes, mask, err), ref, bound, "as they are")
    was = pool.v_scale.clone()
    blind = torch.tensor([j % 2 == 0 for j in range(nodes)] * len(lens), device="cuda")
    for up in (3, 5, 10, 14, 18, 30, 80, 110):
        for n, c in enumerate(lens):
            pg, row = place(pool, table, n, c + 1)
            pool.v_scale[pg, :, row] = was[pg, :, row].clamp(max=2.0 ** -7) * 2.0 ** up
        out = attend(b, pool, q, table, ctx, scale, nodes, mask, err)
        inside(out[blind], ref[blind], bound[blind], f"2^{up}, not seen")
        r2, b2 = statement(pool, q, table, ctx, scale, nodes, mask)
        inside(out[~blind], r2[~blind], b2[~blind], f"2^{up}, seen")
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("heads,nodes", ROWS)
def test_a_large_value_scale_of_a_token_that_hardly_weighs(b, err, heads, nodes):
    """A context token with the keys turned against every query, so that it weighs next to nothing, and a scale that
    would take the others' weights below E4M3's smallest step."""
    lens = [200, 64, 1500]
    pool, table, ctx, q, scale = make(heads, lens, nodes)
    q = q.abs()
    for n in range(len(lens)):
        pg, row = place(pool, table, n, 33)
        pool.k[pg, :, row] = 0xF8  # -256
        pool.k_scale[pg, :, row] = 0.02
        for up in (12, 20, 40):
            pool.v_scale[pg, :, row] = 2.0 ** (up - 8)
            out = attend(b, pool, q, table, ctx, scale, nodes, None, err)
            ref, bound = statement(pool, q, table, ctx, scale, nodes)
            assert float(ref[n * nodes:(n + 1) * nodes].abs().max()) < 8  # the token's part is none
            inside(out, ref, bound, f"request {n}, 2^{up}")
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("heads,nodes", ROWS + [((24, 4, 256), 1)])
@pytest.mark.parametrize("strong", [0.0, 1.0, 12.0])
@pytest.mark.parametrize("spread", [3, 4, 5, 9, 20, 60])
def test_scales_spread_over_many_powers(b, err, heads, nodes, strong, spread):
    """Every token with a scale of its own, of either sign; two pieces of a long request among them."""
    lens = [777, 12, 127, 9000]
    pool, table, ctx, q, scale = make(heads, lens, nodes, 16, strong, seed=spread)
    g = torch.Generator(device="cuda").manual_seed(spread)
    up = torch.randint(-spread, spread + 1, pool.v_scale.shape, generator=g, device="cuda").float() / 2
    sign = torch.randint(0, 2, pool.v_scale.shape, generator=g, device="cuda") * 2 - 1
    pool.v_scale.mul_(torch.exp2(up) * sign)
    out = attend(b, pool, q, table, ctx, scale, nodes, None, err)
    ref, bound = statement(pool, q, table, ctx, scale, nodes)
    inside(out, ref, bound, "out")
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("heads,nodes", ROWS)
def test_scales_of_zero_and_of_everything(b, err, heads, nodes):
    """Tokens without values: their weight counts in the sum. A tile, a request without any gives zeros. A scale that
    is no number shows in every row, as does an infinite one."""
    lens = [300, 20, 128]
    pool, table, ctx, q, scale = make(heads, lens, nodes, strong=4.0)
    pool.v_scale[:, :, ::3] = 0.0
    for t in range(lens[1] + nodes):
        pg, row = place(pool, table, 1, t)
        pool.v_scale[pg, :, row] = 0.0
    for t in range(128):
        pg, row = place(pool, table, 0, t)
        pool.v_scale[pg, :, row] = 0.0
    out = attend(b, pool, q, table, ctx, scale, nodes, None, err)
    ref, bound = statement(pool, q, table, ctx, scale, nodes)
    inside(out, ref, bound, "zeros")
    rows = slice(nodes, 2 * nodes)
    assert torch.equal(out[rows], torch.zeros_like(out[rows]))
    for odd in (float("nan"), float("inf")):
        pg, row = place(pool, table, 2, 5)
        pool.v_scale[pg, :, row] = odd
        pool.v[pg, :, row] = 0x30
        pool.v[pg, :, row, :7] = 0
        out = attend(b, pool, q, table, ctx, scale, nodes, None, err)
        assert not bool(out[2 * nodes:].isfinite().any())
        inside(out[:2 * nodes], ref[:2 * nodes], bound[:2 * nodes], "the other requests")
    assert b.gdn_read_device_error(err) == 0


@pytest.mark.parametrize("heads,nodes", ROWS + [((24, 4, 256), 1)])
@pytest.mark.parametrize("lens", [[40000], [300, 5]])
def test_scales_at_both_ends_of_the_format(b, err, heads, nodes, lens):
    """Equal weights, so that each token counts in the sum. All scales the smallest that a write leaves (rows of zeros
    have it); one token's near the largest beside them, 2^160 times as large; and the smallest among large ones."""
    pool, table, ctx, q, scale = make(heads, lens, nodes, strong=0.0)
    small, large = 1e-12 / 448, 2.0 ** 111
    for most, few in ((small, small), (small, large), (large, small), (large, large)):
        pool.v_scale.fill_(most)
        for n, c in enumerate(lens):
            pg, row = place(pool, table, n, c // 2)
            pool.v_scale[pg, :, row] = few
        out = attend(b, pool, q, table, ctx, scale, nodes, None, err)
        ref, bound = statement(pool, q, table, ctx, scale, nodes)
        inside(out, ref, bound, f"{most}, one of {few}")
        assert float(out.abs().max()) > 0
    assert b.gdn_read_device_error(err) == 0
