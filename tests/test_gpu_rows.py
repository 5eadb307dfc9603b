"""The rows of gdn_qk_norm_rope and gdn_kv_cache_write where a block's copies run ahead: many tokens a block against
few, bit for bit."""
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


FEW = 152  # tokens of a call whose blocks have one token each: no buffer is used twice within a head's rows


@pytest.mark.parametrize("fmt", [None, "bf16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,rotary,inter", [
    (24, 4, 256, 256, False), (24, 4, 256, 64, True), (6, 1, 256, 0, False), (32, 8, 128, 128, True),
    (5, 5, 128, 128, False), (70, 35, 128, 64, True), (40, 20, 256, 64, False)])
def test_many_tokens_a_block_give_the_bits_of_few(b, fmt, hq, hkv, d, rotary, inter):
    """A batch of rows is copied into the buffer that the batch before it was read from, sixteen tokens a block. A row's
    arithmetic is the same whatever stands around it, so its bits are those of a call with one token a block."""
    T = 16 * FEW - 3
    g = torch.Generator(device="cuda").manual_seed(T + d + rotary)
    packed = torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    gamma = torch.rand(d, generator=g, device="cuda") + 0.5
    pos = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = 1e7 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / max(rotary, 1)) if rotary else None
    slots = torch.randperm(-(-T // 64) * 64, generator=g, device="cuda")[:T].to(torch.int32)
    runs = []
    for step in (T, FEW):
        qo, ko = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(
            k, memory_format=torch.contiguous_format)
        pools = [] if fmt is None else [R.Pool(-(-T // 64), hkv, 64, d, fmt) for _ in range(2)]
        caches = [p.handle(b) for p in pools]
        for t in range(0, T, step):
            at = slice(t, t + step)
            kw = {} if fmt is None else dict(v=v[at], cache=caches[0], kv_slot=slots[at])
            b.gdn_qk_norm_rope(q[at], k[at], gamma, gamma, 1e-6, pos[at], f, qo[at], ko[at], interleaved=inter, **kw)
            if fmt is not None:
                b.gdn_kv_cache_write(caches[1], k[at], v[at], slots[at])
        runs.append([qo, ko] + [x for p in pools for x in (p.k, p.v, p.k_scale, p.v_scale) if x is not None])
    for x, y in zip(*runs):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("T,heads", [(5, 1), (1, 3), (1, 1)])
def test_strides_of_dimensions_with_one_entry_do_not_count(b, T, heads):
    """One head or one token: whatever stride the tensor names for it, here one element, the rows are the same."""
    d = 128
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, heads, d, generator=g, device="cuda").to(torch.bfloat16)
    odd = x.as_strided(x.shape, (d * heads if T > 1 else 1, d if heads > 1 else 1, 1))
    assert torch.equal(odd, x)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    pos, f = slots.clone(), torch.ones(8, dtype=torch.float64, device="cuda")
    gamma = torch.ones(d, device="cuda")
    runs = []
    for t in (x, odd):
        pools = [R.Pool(1, heads, 16, d, "e4m3") for _ in range(2)]
        out = torch.empty_like(x)
        b.gdn_kv_cache_write(pools[0].handle(b), t, t, slots)
        b.gdn_qk_norm_rope(t, t, gamma, gamma, 1e-6, pos, f, out, v=t, cache=pools[1].handle(b), kv_slot=slots)
        runs.append([out] + [y for p in pools for y in (p.k, p.v, p.k_scale, p.v_scale)])
    for a, c in zip(*runs):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))
