"""Plain fp64 statements of the attention-side operators (head norm and rotation, the paged key/value
cache, tree attention) for the tests, in torch on any device, straight from the formulas; and the error
bounds that a kernel with fp32 sums and one rounding to bf16 keeps.

A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24, to E4M3 by 2^-4 (or half of
the smallest step, 2^-10 of the scale)."""
import math

import numpy as np
import torch

from oracle import oracle

BF16, E4M3 = 2.0 ** -8, 2.0 ** -4


def norm_rope(x, gamma, eps, positions, inv_freq, interleaved=False):
    """x [T, H, D] -> (rotated fp64 values, the largest magnitude of each value's pair)."""
    x = x.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
    mag = y.abs()
    half = 0 if inv_freq is None else inv_freq.numel()
    if half:
        angle = (positions.double()[:, None] * inv_freq.double())[:, None]
        c, s = torch.cos(angle), torch.sin(angle)
        i = torch.arange(half, device=x.device)
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[..., ia].clone(), y[..., ib].clone()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        pair = torch.hypot(a, b)
        mag[..., ia], mag[..., ib] = pair, pair
    return y, mag


def rope_bound(ref, mag):
    """One rounding to bf16, and fp32 arithmetic: the sum of squares and the root (2^-16 of the value holds
    (D + 4) 2^-24), the angle and its sine and cosine (under 2^-20 of the pair)."""
    return BF16 * ref.abs() + (2.0 ** -16 + 2.0 ** -20) * mag


def quantise(x):
    """x [..., D] fp32 tensor -> (codes uint8, scales fp32), by the oracle's E4M3."""
    a = x.detach().float().cpu().numpy()
    s = oracle._fp8_block_scale(np.abs(a).max(-1))
    codes = oracle.e4m3_from_f32((a / s[..., None]).astype(np.float32))
    return torch.from_numpy(codes), torch.from_numpy(s)


_TABLE = torch.from_numpy(oracle.e4m3_to_f64(np.arange(256, dtype=np.uint8)))


class Pool:
    """A cache on the device: k, v and (quantised) their scales."""

    def __init__(self, pages, heads, page, d, fmt, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        shape = (pages, heads, page, d)
        self.fmt, self.page = fmt, page
        x = [torch.randn(shape, generator=g, device=device) for _ in range(2)]
        if fmt == "e4m3":
            self.k_scale, self.v_scale = (t.abs().amax(-1) / 448 for t in x)
            self.k, self.v = ((t / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                              for t, s in zip(x, (self.k_scale, self.v_scale)))
        else:
            self.k, self.v = (t.to(torch.bfloat16) for t in x)
            self.k_scale = self.v_scale = None

    def handle(self, b):
        return b.make_kv_cache(self.k, self.v, self.k_scale, self.v_scale)

    def values(self, name, pages):
        """fp64 values [H, pages * page, D] of the listed pages."""
        x = getattr(self, name)[pages]
        if self.fmt == "e4m3":
            x = _TABLE.to(x.device)[x.long()] * getattr(self, name + "_scale")[pages].double()[..., None]
        x = x.double().transpose(0, 1)
        return x.reshape(x.shape[0], -1, x.shape[-1])


def tree_attention(pool, q, table, ctx, scale, nodes, mask=None, gate=None):
    """-> (out [N * P, Hq, D] fp64, bound, live [N * P] bool). A node with nothing to see gives zeros."""
    N, P, D = table.shape[0], nodes, q.shape[-1]
    Hq, Hkv = q.shape[1], pool.k.shape[1]
    G, dev = Hq // Hkv, q.device
    out = torch.zeros((N * P, Hq, D), dtype=torch.float64, device=dev)
    bound = torch.zeros_like(out)
    live = torch.zeros(N * P, dtype=torch.bool, device=dev)
    for n in range(N):
        c = int(ctx[n])
        if c < 0:
            continue
        rows = slice(n * P, (n + 1) * P)
        live[rows] = True
        pages = table[n, :-(-(c + P) // pool.page)].long()
        k, v = (pool.values(x, pages)[:, :c + P] for x in ("k", "v"))
        seen = torch.ones((P, c + P), dtype=torch.bool, device=dev)
        words = [(2 << j) - 1 for j in range(P)] if mask is None else [int(w) & (2 ** 64 - 1) for w in mask[n]]
        seen[:, c:] = torch.tensor([[bool(w >> i & 1) for i in range(P)] for w in words], device=dev)
        x = q[rows].double().reshape(P, Hkv, G, D)
        s = torch.einsum("phgd,htd->phgt", x, k) * scale
        reach = torch.einsum("phgd,htd->phgt", x.abs(), k.abs()) * abs(scale)
        here = seen[:, None, None, :].expand_as(s)
        s, reach = s.masked_fill(~here, -math.inf), torch.where(here, reach, 0)
        m = s.amax(-1, keepdim=True)
        p = torch.where(here, torch.exp(s - torch.where(torch.isinf(m), 0, m)), 0)
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0)
        # what no node sees has no part in the sums, whatever its values
        v = torch.where(seen.any(0)[None, :, None], v, 0)
        o = torch.einsum("phgt,htd->phgd", p, v)
        if not bool(torch.isfinite(v).all()):  # a masked value is no part of a node's sum: node by node
            o = torch.stack([torch.einsum("hgt,htd->hgd", p[j][..., seen[j]], v[:, seen[j]]) for j in range(P)])
        mass = torch.einsum("phgt,htd->phgd", p, torch.nan_to_num(v, 0, 0, 0).abs())
        # a score is a fp32 sum of D products, scaled and taken to base 2; each weight and its sum once more
        ds = (reach.amax(-1) * (D + 8) * 2.0 ** -24 + (c + P + 16) * 2.0 ** -24)[..., None]
        lim = BF16 * o.abs() + (BF16 + 2 * ds) * mass
        if pool.fmt == "e4m3":
            # A weight times its value's scale is held as two E4M3 terms, 256 standing for the largest weight times
            # the largest scale of its tile of 128 tokens: below 2^-6 a term's step is 2^-9, so what is left is off
            # by up to 2^-10 of 256, 2^-18 of that product, whatever the weight itself.
            sv = torch.nan_to_num(pool.v_scale[pages].double().transpose(0, 1).reshape(Hkv, -1)[:, :c + P], 0, 0, 0)
            code = torch.nan_to_num(v / sv[..., None], 0, 0, 0).abs()
            for t0 in range(0, c + P, 128):
                t = slice(t0, t0 + 128)
                top = p[..., t].amax(-1) * sv[:, t].amax(-1)[None, :, None]
                lim = lim + 2.0 ** -18 * top[..., None] * code[:, t].sum(1)[None, :, None]
        o, lim = o.reshape(P, Hq, D), lim.reshape(P, Hq, D)
        if gate is not None:
            w = torch.sigmoid(gate[rows].double())
            o, lim = o * w, lim * w + 2.0 ** -16 * (o * w).abs()
        out[rows], bound[rows] = o, lim
    return out, bound, live


def tables(lens, page, pages, device="cuda", seed=0, spare=0):
    """Distinct random pages for requests of the given token counts; -1 behind them."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(t, 0) // page) for t in lens]
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + spare), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = perm[at:at + k]
        at += k
    assert at <= pages
    return table.to(device)


def tree(n, nodes, seed=0):
    """Random parents [n, nodes] (-1: the committed token) and the ancestor masks as int64 words."""
    rng = np.random.default_rng(seed)
    par = np.full((n, nodes), -1, np.int32)
    mask = np.zeros((n, nodes), np.uint64)
    for r in range(n):
        for p in range(nodes):
            par[r, p] = rng.integers(-1, p) if p else -1
            up = mask[r, par[r, p]] if par[r, p] >= 0 else np.uint64(0)
            mask[r, p] = up | np.uint64(1 << p)
    return torch.from_numpy(par), torch.from_numpy(mask.view(np.int64))
