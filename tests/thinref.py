"""Plain fp64 statements of what thins out a cache (a row's log-sum-exp, the attention weight that cached tokens receive,
eviction by it), for the tests, in torch on any device, straight from the formulas; and the error bounds that a kernel
with fp32 sums keeps.

A sum of n fp32 terms in any order is off by at most n 2^-23 of the terms' magnitudes, each addition cut or rounded."""
import math

import torch

from tests import attnref as R

F32 = 2.0 ** -23


def logits(pool, q, table, n, ctx, scale, nodes, mask=None, together=False):
    """Request n's scale (q . k) [P, Hkv, G, tokens], -inf where a row does not see the token, and their error bounds;
    `together`: of rows that an E4M3 cache's products take by one power of two."""
    P, D, Hkv = nodes, q.shape[-1], pool.k.shape[1]
    G = q.shape[1] // Hkv
    pages = table[n, :-(-(ctx + P) // pool.page)].long()
    k = pool.values("k", pages)[:, :ctx + P]
    x = q[n * P:(n + 1) * P].double().reshape(P, Hkv, G, D)
    seen = torch.ones((P, ctx + P), dtype=torch.bool, device=q.device)
    words = [(2 << j) - 1 for j in range(P)] if mask is None else [int(w) & (2 ** 64 - 1) for w in mask[n]]
    seen[:, ctx:] = torch.tensor([[bool(w >> i & 1) for i in range(P)] for w in words], device=q.device)
    seen = seen[:, None, None, :]
    s = (torch.einsum("phgd,htd->phgt", x, k) * scale).masked_fill(~seen, -math.inf)
    # D products and additions, the key's scale, the factor and its rounding
    off = torch.einsum("phgd,htd->phgt", x.abs(), k.abs()) * abs(scale) * (D + 8) * F32
    if pool.fmt == "e4m3":
        # q as two E4M3 terms. The largest value is taken into [128, 256). A bf16 value has 8 bits: the first term takes at
        # least 4 of them, and the second holds the rest where the last of them counts 2^-9, E4M3's smallest step, or more;
        # else it is off by half of that step, 2^-10: 2^-17 of the head row's largest value.
        most = x.abs().nan_to_num(0, 0, 0).amax(-1, keepdim=True)
        by = 2.0 ** -17 * most
        if together:  # The largest of all the kv head's rows goes there, or a smaller one: 2^-17 of it. A row whose largest
            # value is two powers below goes into [32, 64) at least, so that 2^-10 is 2^-15 of it; smaller ones have their own.
            by = torch.minimum(2.0 ** -17 * most.amax((0, 2), keepdim=True), 4 * by)
        off = off + by * k.abs().sum(-1)[None, :, None, :] * abs(scale)
    return s, torch.where(seen, off, 0)


def lse(pool, q, table, ctx, scale, nodes, mask=None):
    """-> (lse [N * P, Hq] fp64, bound)."""
    N, P, Hq = table.shape[0], nodes, q.shape[1]
    out = torch.full((N * P, Hq), -math.inf, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for n in range(N):
        c = int(ctx[n])
        if c < 0:
            continue
        s, off = logits(pool, q, table, n, c, scale, P, mask)
        rows = slice(n * P, (n + 1) * P)
        out[rows] = torch.logsumexp(s, -1).reshape(P, Hq)
        # each weight's exponential (2^-21), their sum (parts of 128 and then one by one), the logarithms
        bound[rows] = (off.amax(-1).reshape(P, Hq) * 1.01 + 2.0 ** -21 + (160 + (c + P) / 64) * F32
                       + (torch.nan_to_num(out[rows], 0, 0, 0).abs() + 64) * 4 * F32)
    return out, bound


def score(pool, q, lses, table, ctx, scale, nodes, weights, slot, mask=None, decay=1.0, init=None):
    """-> (weights after the call fp64, bound)."""
    out, bound = weights.double(), torch.zeros_like(weights, dtype=torch.float64)
    P, Hkv = nodes, pool.k.shape[1]
    G = q.shape[1] // Hkv
    for n in range(table.shape[0]):
        c, at = int(ctx[n]), int(slot[n])
        if c < 0 or at < 0 or at >= weights.shape[0]:
            continue
        s, off = logits(pool, q, table, n, c, scale, P, mask, together=True)
        z = lses[n * P:(n + 1) * P].double().reshape(P, Hkv, G, 1)
        live = z.isfinite()
        p = torch.where(live & (s > -math.inf), torch.exp(s - torch.where(live, z, 0)), 0)
        add = p.sum((0, 2))  # [Hkv, tokens]
        # a weight: its score's error, the two logarithms' roundings, the exponential; then the sum over the rows
        rel = torch.expm1(off + (z.abs().nan_to_num(0, 0, 0) + s.abs().nan_to_num(0, 0, 0) + 4) * 4 * F32 + 2.0 ** -21)
        lim = (p * rel).sum((0, 2)) + add * (P * G + 4) * F32
        old = out[at, :, :c + P] * decay
        old[:, c:] = 0
        if init is not None and not bool(init[n]):
            old = torch.zeros_like(old)
        out[at, :, :c + P] = old + add
        bound[at, :, :c + P] = lim + 3 * F32 * (old.abs() + add)
    return out, bound


def ranks(w, sinks, recent):
    """The order of a head's tokens: a list of sort keys, the largest kept first."""
    n = len(w)

    def key(t):
        if t < sinks or t >= n - recent:
            return (0, 0.0, t)
        return (2, 0.0, t) if math.isnan(w[t]) else (1, -w[t], t)
    return sorted(range(n), key=key)


def evict(pool, table, length, budget, weights, slot, sinks=0, recent=0, dst_table=None, dst_slot=None, max_kept=None):
    """-> (kept lists [N][Hkv], new_len, and copies of k, v, k_scale, v_scale, weights after the call)."""
    dst_table = table if dst_table is None else dst_table
    dst_slot = slot if dst_slot is None else dst_slot
    was = {x: getattr(pool, x) for x in ("k", "v", "k_scale", "v_scale") if getattr(pool, x) is not None}
    now = {x: t.clone() for x, t in was.items()}
    w_now = weights.clone()
    kept_all, new_len = [], []
    for n in range(table.shape[0]):
        L, m = int(length[n]), min(int(length[n]), int(budget[n]))
        new_len.append(m)
        kept_all.append([])
        for h in range(pool.k.shape[1]):
            w = weights[int(slot[n]), h, :max(L, 0)].tolist()
            kept = sorted(ranks(w, sinks, recent)[:max(m, 0)])
            kept_all[-1].append(kept)
            if not kept:
                continue
            src = torch.tensor(kept, device=table.device)
            dst = torch.arange(m, device=table.device)
            sp, dp = table[n].long()[src // pool.page], dst_table[n].long()[dst // pool.page]
            for x in now:
                now[x][dp, h, dst % pool.page] = was[x][sp, h, src % pool.page]
            w_now[int(dst_slot[n]), h, :m] = weights[int(slot[n]), h, src]
    return kept_all, new_len, now, w_now


__all__ = ["F32", "R", "evict", "logits", "lse", "ranks", "score"]
