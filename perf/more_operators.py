"""Measured cases of the operators that thin out a long cache and of the rotation that image and video prompts need: query/key
head norms with a rotation over several position axes (time, height, width), straight into the paged key/value cache;
the attention weight that every cached token receives, accumulated per request; and the eviction of a cache down to a
budget of tokens by that weight.

``run`` computes an operator in its plain form (elementary torch operations in fp32, fp64 for the angles), or, where
``own`` is true, makes the library call a serving program makes. ``exact`` is the same result from the definitions in
64 bits. The head layouts are those of the decoder whose linear-attention layers the library serves (24 query and 4
key/value heads of 256 with 64 rotated dimensions) and of one of its four tensor-parallel ranks (6 and 1), plus one
generic layout (32 and 8 heads of 128).
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e7  # rotation base
FP8_MAX = 448.0  # largest finite E4M3 value
MIN_AMAX = 1e-12


# ------------------------------------------------------------------------------------------------ cases

def _mrope(name, tokens, grid, far, q_heads=24, kv_heads=4, head_dim=256, rotary=64, mixed=True, cache="e4m3",
           keep_k=False, page=64):
    """`grid`: height and width, in merged patches, of the prompt's frames; 0: text alone. `mixed`: the axes take
    turns along the frequencies, otherwise each has a run of them."""
    return {"name": name, "op": "qk_norm_mrope", "tokens": tokens, "grid": grid, "far": far, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "rotary": rotary, "mixed": mixed, "cache": cache,
            "keep_k": keep_k, "page": page}


def _score(name, seqs, nodes, tree, lo, hi, cache, q_heads=24, kv_heads=4, head_dim=256, page=64, decay=1.0, fresh=False):
    """`tree`: "chain" (the new tokens in order) or "tree" (a drafted tree, about half of its nodes rejected).
    `fresh`: the requests have no weights yet."""
    return {"name": name, "op": "kv_score", "seqs": seqs, "nodes": nodes, "tree": tree, "lo": lo, "hi": hi,
            "cache": cache, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "decay": decay, "fresh": fresh}


def _evict(name, seqs, lo, hi, share, cache, kv_heads=4, head_dim=256, page=64, sinks=4, recent=64):
    """`share`: the part of a request's tokens that its budget keeps."""
    return {"name": name, "op": "kv_evict", "seqs": seqs, "lo": lo, "hi": hi, "share": share, "cache": cache,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "sinks": sinks, "recent": recent}


def listed():
    return [
        # a decode step of 256 requests in multimodal conversations: every token has a position per axis
        _mrope("mrope decode 256 to e4m3", 256, 0, 131072),
        # a video prompt of 16384 merged patches, 24 x 24 a frame, the keys kept for the prompt's own attention too
        _mrope("mrope video 16384 to bf16", 16384, 24, 4096, cache="bf16", keep_k=True),
        # one request's decode step at a short context: latency
        _score("score decode 1 x 509 bf16", 1, 1, "chain", 509, 509, "bf16"),
        # a decode batch of 256 requests over the quantised cache, older weight fading
        _score("score decode 256 x 1k..8k e4m3", 256, 1, "chain", 1024, 8192, "e4m3", decay=0.98),
        # verified draft trees of 32 requests, the rejected nodes' rows empty
        _score("score tree 32 x 8 nodes e4m3", 32, 8, "tree", 129, 16384, "e4m3", page=16),
        # the last 32 tokens of 8 prompts look back over them: the first weights of a new request
        _score("score prompts 8 x 32 bf16", 8, 32, "chain", 1500, 32768, "bf16", fresh=True),
        # the last 64 tokens of one long prompt
        _score("score prompt 1 x 64 131071 bf16", 1, 64, "chain", 131071, 131071, "bf16", fresh=True),
        # the same over the quantised cache, in one rank's heads
        _score("score prompt 2 x 64 rank e4m3", 2, 64, "chain", 40001, 70000, "e4m3", 6, 1, fresh=True),
        # one short conversation cut to half
        _evict("evict 1 x 1000 bf16", 1, 1000, 1000, 0.5, "bf16"),
        # 32 conversations cut to half
        _evict("evict 32 x 2k..32k e4m3", 32, 2048, 32768, 0.5, "e4m3"),
        # one long prompt cut to a quarter
        _evict("evict 1 x 131071 bf16", 1, 131071, 131071, 0.25, "bf16"),
        # a batch of 128 in the generic layout, small pages
        _evict("evict 128 x 300..8k, 8 x 128", 128, 300, 8192, 0.4, "bf16", 8, 128, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_mrope", "kv_score", "kv_score", "kv_evict", "kv_evict"])
    cache = rng.choice(["bf16", "e4m3"])
    hq, hkv, d = rng.choice([(24, 4, 256), (6, 1, 256), (32, 8, 128)])
    page = rng.choice([16, 64, 128])
    if op == "qk_norm_mrope":
        c = _mrope("", _log(rng, 1, 16384), rng.choice([0, 7, 24, 40]), rng.choice([4096, 131072]), hq, hkv, d,
                   rng.choice([32, 64, d]), rng.random() < 0.5, cache, rng.random() < 0.5, page)
    elif op == "kv_score":
        nodes = _log(rng, 1, 64)
        seqs = _log(rng, 1, max(1, 256 // nodes))
        most = min(131072, max(64, 860000 // seqs // (1 if cache == "e4m3" else 2)), (1 << 23) // (seqs * nodes))
        lo = _log(rng, 1, most)
        c = _score("", seqs, nodes, rng.choice(["chain", "chain", "tree"]), lo, _log(rng, lo, most), cache, hq, hkv, d,
                   page, rng.choice([1.0, 0.9]), rng.random() < 0.3)
    else:
        seqs = _log(rng, 1, 128)
        most = min(131072, 380000 // seqs)
        lo = _log(rng, 1, most)
        c = _evict("", seqs, lo, _log(rng, lo, most), rng.choice([0.1, 0.25, 0.5, 0.8, 1.0]), cache, hkv, d, page,
                   rng.choice([0, 1, 4, 16]), rng.choice([0, 1, 32, 128]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _lengths(case):
    """Lengths spread evenly over the logarithm of the case's range."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (i + 0.5) / n)) for i in range(n)]


def _budgets(case):
    return [round(n * case["share"]) for n in _lengths(case)]


def _sections(case):
    """Frequencies of the time, height and width axes: about 3 : 2.5 : 2.5 of the rotated pairs."""
    half = case["rotary"] // 2
    side = half * 5 // 16
    return half - 2 * side, side, side


def _axis(case):
    """The axis of each frequency."""
    t, h, w = _sections(case)
    if not case["mixed"]:
        return [0] * t + [1] * h + [2] * w
    return [1 if i % 3 == 1 and i < 3 * h else 2 if i % 3 == 2 and i < 3 * w else 0 for i in range(t + h + w)]


def _grid_positions(g, case):
    """Positions [3, T]: of text all three alike, of frames the frame's time with the patch's row and column."""
    T, side, far = case["tokens"], case["grid"], case["far"]
    if side == 0:
        return torch.randint(0, far, (1, T), generator=g, device="cuda", dtype=torch.int32).expand(3, T).contiguous()
    i = torch.arange(T, device="cuda")
    start = torch.randint(0, far, (1,), generator=g, device="cuda")
    return torch.stack((start + i // (side * side), start + i // side % side, start + i % side)).to(torch.int32)


def _encode(x):
    """fp32 values of the last axis to E4M3 codes and one scale."""
    s = x.abs().amax(-1).clamp_min(MIN_AMAX) / FP8_MAX
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def _pool(g, case, pages, filled):
    """A key/value cache of `pages` pages, the first `filled` of them written: k, v and, quantised, their scales."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    e4m3 = case["cache"] == "e4m3"
    gain = _rand(g, shape[3]) * 1.5 + 0.5  # what a head norm leaves in the keys: unit rows times a gain
    pool = {}
    for name in ("k", "v"):
        x = torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
        scale = torch.zeros(shape[:3], device="cuda") if e4m3 else None
        step = max(1, (1 << 28) // (shape[1] * shape[2] * shape[3]))
        for at in range(0, filled, step):  # in pieces: fp32 values take four times the pool's room
            y = _randn(g, min(step, filled - at), *shape[1:])
            if name == "k":
                y *= gain
            if e4m3:
                y, scale[at:at + step][:y.shape[0]] = _encode(y)
                y = y.view(torch.uint8)
            x[at:at + y.shape[0]] = y
        pool[name], pool[name + "_scale"] = x, scale
    return pool


def _table(case, tokens, pages):
    """Block tables of requests with `tokens` cached tokens each, out of the page numbers `pages`."""
    need = [-(-t // case["page"]) for t in tokens]
    table = torch.full((len(tokens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = pages[at:at + n]
        at += n
    return table


def _pages(case, tokens):
    return sum(-(-t // case["page"]) for t in tokens)


def _parents(g, seqs, nodes):
    """Random draft trees, parents before children: parent -1 is the last committed token."""
    par = torch.empty((seqs, nodes), dtype=torch.int32, device="cuda")
    par[:, 0] = -1
    for p in range(1, nodes):
        par[:, p] = torch.randint(max(-1, p - 6), p, (seqs,), generator=g, device="cuda")
    return par


def _tree_mask(par):
    """Bit i of word [n, p]: node p descends from node i, or is it."""
    n, nodes = par.shape
    mask = torch.zeros((n, nodes + 1), dtype=torch.int64, device="cuda")  # column 0: the committed token
    rows = torch.arange(n, device="cuda")
    for p in range(nodes):
        mask[:, p + 1] = mask[rows, par[:, p].long() + 1] | (1 << p if p < 63 else -(1 << 63))
    return mask[:, 1:].contiguous()


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    {"qk_norm_mrope": _prepare_mrope, "kv_score": _prepare_score, "kv_evict": _prepare_evict}[case["op"]](s, g, case)
    if own:
        _own_handles(s)
    return s


def _prepare_mrope(s, g, case):
    T, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    packed = _randn(g, T, hq + 2 * hkv, d).mul_(1.5).to(torch.bfloat16)  # one projection's output
    s["q"], s["k"], s["v"] = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
    s["q_gamma"], s["k_gamma"] = _rand(g, d) + 0.5, _rand(g, d) + 0.5
    s["positions"] = _grid_positions(g, case)
    i = torch.arange(0, case["rotary"], 2, dtype=torch.float64, device="cuda")
    s["inv_freq"] = torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"), -i / case["rotary"])
    s["axis"] = torch.tensor(_axis(case), device="cuda")
    pages = -(-2 * T // case["page"])
    s["slots"] = torch.randperm(pages * case["page"], generator=g, device="cuda")[:T].to(torch.int32)
    s["pool"] = _pool(g, case, pages, 0)
    s["q_out"] = torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
    s["k_out"] = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device="cuda") if case["keep_k"] else None


def _prepare_score(s, g, case):
    N, P, hq, hkv, d = case["seqs"], case["nodes"], case["q_heads"], case["kv_heads"], case["head_dim"]
    lens = _lengths(case)
    order = torch.randperm(N, generator=g, device="cuda").tolist()
    lens = [lens[i] for i in order]
    tokens = [t + P for t in lens]
    pages = _pages(case, tokens) + 3
    s["table"] = _table(case, tokens, torch.randperm(pages, generator=g, device="cuda").to(torch.int32))
    s["pool"] = _pool(g, case, pages, pages)
    s["longest"] = max(lens)
    s["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = (_randn(g, N * P, hq, d) * (_rand(g, d) * 1.5 + 0.5)).to(torch.bfloat16)
    s["scale"] = d ** -0.5
    s["mask"] = _tree_mask(_parents(g, N, P)) if case["tree"] == "tree" else None
    # what the attention over the same rows leaves: the logarithm of each row's sum of weights
    lse = torch.logsumexp(_plain_logits(s).reshape(N, hkv, P, hq // hkv, -1), -1)
    s["lse"] = lse.permute(0, 2, 1, 3).reshape(N * P, hq).contiguous()
    if case["tree"] == "tree":  # the rows of rejected nodes are left out
        s["lse"][_rand(g, N * P) < 0.5] = float("-inf")
    slots = 2 * N
    s["slot"] = torch.randperm(slots, generator=g, device="cuda")[:N].to(torch.int32)
    s["init"] = None
    if case["fresh"]:
        s["init"] = torch.zeros(N, dtype=torch.uint8, device="cuda")
    # [slots][kv heads][room for tokens]: what some steps before left, a few tokens having most of it
    w = torch.exp(_randn(g, slots, hkv, -(-(max(tokens) + 100) // 128) * 128) * 1.5 - 1)
    s["weights"] = w.mul_(P * hq / hkv * N / sum(tokens))


def _prepare_evict(s, g, case):
    N, hkv = case["seqs"], case["kv_heads"]
    order = torch.randperm(N, generator=g, device="cuda").tolist()
    lens, budgets = _lengths(case), _budgets(case)
    lens, budgets = [lens[i] for i in order], [budgets[i] for i in order]
    here, there = _pages(case, lens), _pages(case, budgets)
    perm = torch.randperm(here, generator=g, device="cuda").to(torch.int32)
    s["table"] = _table(case, lens, perm)
    # the kept tokens go to pages of their own: the old ones may be shared with other requests' prefixes
    s["dst"] = _table(case, budgets, here + torch.randperm(there, generator=g, device="cuda").to(torch.int32))
    s["pool"] = _pool(g, case, here + there, here)
    s["len"], s["budget"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (lens, budgets))
    s["longest"], s["most"] = max(lens), max(max(budgets), 1)
    slots = torch.randperm(2 * N, generator=g, device="cuda").to(torch.int32)
    s["slot"], s["dst_slot"] = slots[:N].contiguous(), slots[N:].contiguous()
    # accumulated weights: a few tokens have most of it, some have none
    w = torch.exp(_randn(g, 2 * N, hkv, -(-max(lens) // 128) * 128) * 2 - 4)
    s["weights"] = w.masked_fill_(_rand(g, *w.shape) < 0.05, 0.0)
    s["kept"] = torch.full((N, hkv, s["most"]), -1, dtype=torch.int32, device="cuda")
    s["new_len"] = torch.zeros(N, dtype=torch.int32, device="cuda")


def _own_handles(s):
    """What a serving program makes once and keeps: the cache handle, the axes of the frequencies."""
    from gated_deltanet_linear_conv1d_gb300 import binding as b
    s["b"] = b
    p = s["pool"]
    s["cache_handle"] = b.make_kv_cache(p["k"], p["v"], p["k_scale"], p["v_scale"])
    if s["op"] == "qk_norm_mrope":
        s["axes"] = b.make_rope_axes(_sections(s), mixed=s["mixed"])


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _pool_values(pool):
    """The cache's contents: bf16 values, or E4M3 values and their scales."""
    if pool["k_scale"] is None:
        return {"k": pool["k"], "v": pool["v"]}
    e = torch.float8_e4m3fn
    return {"k": pool["k"].view(e), "v": pool["v"].view(e), "k_scale": pool["k_scale"], "v_scale": pool["v_scale"]}


def _own_mrope(s):
    s["b"].gdn_qk_norm_mrope(s["q"], s["k"], s["q_gamma"], s["k_gamma"], EPS, s["positions"], s["inv_freq"], s["axes"],
                             s["q_out"], k_out=s["k_out"], v=s["v"], cache=s["cache_handle"], kv_slot=s["slots"])
    return {"q": s["q_out"], "k": s["k_out"], "cache": _pool_values(s["pool"])}


def _own_score(s):
    s["b"].gdn_kv_score(s["cache_handle"], s["q"], s["lse"], s["table"], s["ctx"], s["scale"], s["weights"], s["slot"],
                        num_pos=s["nodes"], tree_mask=s["mask"], decay=s["decay"], has_init=s["init"])
    return s["weights"]


def _own_evict(s):
    s["b"].gdn_kv_evict(s["cache_handle"], s["table"], s["len"], s["budget"], s["weights"], s["slot"], s["kept"],
                        s["new_len"], sink_tokens=s["sinks"], recent_tokens=s["recent"], dst_table=s["dst"],
                        dst_slot=s["dst_slot"])
    return {"kept": s["kept"], "new_len": s["new_len"], "weights": s["weights"], "cache": _pool_values(s["pool"])}


def _plain_norm(x, gamma):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma


def _plain_rotate(x, angle):
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = angle.shape[1]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]), -1)


def _plain_mrope(s):
    angle = s["positions"].double()[s["axis"]].T * s["inv_freq"]
    q = _plain_rotate(_plain_norm(s["q"], s["q_gamma"]), angle)
    k = _plain_rotate(_plain_norm(s["k"], s["k_gamma"]), angle)
    pool, at = s["pool"], s["slots"].long()
    page, row = at // s["page"], at % s["page"]
    for name, x in (("k", k), ("v", s["v"].float())):
        if pool["k_scale"] is None:
            pool[name][page, :, row] = x.to(torch.bfloat16)
        else:
            x, scale = _encode(x)
            pool[name][page, :, row] = x.view(torch.uint8)
            pool[name + "_scale"][page, :, row] = scale
    s["q_out"] = q.to(torch.bfloat16)
    return {"q": s["q_out"], "k": k.to(torch.bfloat16) if s["keep_k"] else None, "cache": _pool_values(pool)}


def _plain_logits(s):
    """scale (q . k) of every row and token [N, Hkv, P x group, tokens], -inf where the row does not see the token."""
    N, P, hq, hkv, d = s["seqs"], s["nodes"], s["q_heads"], s["kv_heads"], s["head_dim"]
    pool = s["pool"]
    t = torch.arange(s["longest"] + P, device="cuda")
    page = s["table"][:, t // s["page"]].long().clamp_min(0)
    row = (t % s["page"]).expand(N, -1)
    k = pool["k"][page, :, row]
    if pool["k_scale"] is None:
        k = k.float()
    else:
        k = k.view(torch.float8_e4m3fn).float().mul_(pool["k_scale"][page, :, row][..., None])
    q = s["q"].float().reshape(N, P, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(N, hkv, -1, d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"])
    del k
    draft = t - s["ctx"][:, None]  # [N, L]: the node a token is, negative: of the context
    node = torch.arange(P, device="cuda")
    if s["mask"] is None:
        seen = draft[:, None] <= node[:, None]
    else:
        seen = (draft < 0)[:, None] | ((s["mask"][..., None] >> draft.clamp(0, 63)[:, None]) & 1 == 1)
        seen &= (draft < P)[:, None]
    seen = seen[:, None, :, None].expand(N, hkv, P, hq // hkv, -1).reshape(score.shape)
    return score.masked_fill_(~seen, float("-inf"))


def _plain_score(s):
    N, P, hq, hkv = s["seqs"], s["nodes"], s["q_heads"], s["kv_heads"]
    lse = s["lse"].reshape(N, P, hkv, hq // hkv).permute(0, 2, 1, 3).reshape(N, hkv, -1, 1)
    lse = torch.where(lse.isfinite(), lse, float("inf"))  # a row that is left out: exp(-inf)
    p = _plain_logits(s).sub_(lse).exp_()
    add = p.sum(2)
    t = torch.arange(add.shape[-1], device="cuda")
    ctx = s["ctx"][:, None, None]
    slot = s["slot"].long()
    rows = s["weights"][slot]
    old = torch.where(t < ctx, rows[..., :t.numel()] * s["decay"], 0.0) if s["init"] is None else torch.zeros_like(add)
    rows[..., :t.numel()] = torch.where(t < ctx + P, old + add, rows[..., :t.numel()])
    s["weights"][slot] = rows
    return s["weights"]


def _plain_evict(s):
    N, hkv, L, K = s["seqs"], s["kv_heads"], s["longest"], s["most"]
    page, pool, slot = s["page"], s["pool"], s["slot"].long()
    t = torch.arange(L, device="cuda")
    n = s["len"][:, None, None]
    w = s["weights"][slot][..., :L]
    rank = torch.where((t < s["sinks"]) | (t >= n - s["recent"]), float("inf"), w).masked_fill(t >= n, float("-inf"))
    best = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :K]
    new_len = torch.minimum(s["len"], s["budget"])
    i = torch.arange(K, device="cuda")
    live = (i < new_len[:, None, None]).expand(N, hkv, K)  # [N, Hkv, K]
    kept = torch.sort(torch.where(live, best, L), dim=-1).values
    s["kept"] = torch.where(live, kept, s["kept"].long()).to(torch.int32)
    s["new_len"] = new_len
    row = torch.arange(N, device="cuda")[:, None, None].expand_as(live)[live]
    head = torch.arange(hkv, device="cuda")[:, None].expand_as(live)[live]
    src, dst = kept[live], i.expand_as(live)[live]
    src_page, dst_page = s["table"][row, src // page].long(), s["dst"][row, dst // page].long()
    for name in pool:
        if pool[name] is not None:
            pool[name][dst_page, head, dst % page] = pool[name][src_page, head, src % page]
    s["weights"][s["dst_slot"].long()[row], head, dst] = s["weights"][slot[row], head, src]
    return {"kept": s["kept"], "new_len": new_len, "weights": s["weights"], "cache": _pool_values(pool)}


_run_plain = {"qk_norm_mrope": _plain_mrope, "kv_score": _plain_score, "kv_evict": _plain_evict}
_run_own = {"qk_norm_mrope": _own_mrope, "kv_score": _own_score, "kv_evict": _own_evict}


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op, hkv, d = case["op"], case["kv_heads"], case["head_dim"]
    half = hkv * (d + 4 if case["cache"] == "e4m3" else 2 * d)  # bytes of one token's keys, or values, in the cache
    if op == "qk_norm_mrope":
        T, hq = case["tokens"], case["q_heads"]
        kept = hkv * d * 2 if case["keep_k"] else 0
        return {"bytes": T * ((2 * hq + 2 * hkv) * d * 2 + kept + 2 * half + 16) + 8 * d,
                "flops": T * ((hq + hkv) * (4 * d + 3 * case["rotary"]) + 2 * hkv * d)}
    lens = _lengths(case)
    if op == "kv_score":
        N, P, hq = case["seqs"], case["nodes"], case["q_heads"]
        tokens = sum(lens) + N * P
        return {"bytes": tokens * (half + hkv * (4 if case["fresh"] else 8)) + N * P * hq * (d * 2 + 4),
                "flops": P * hq * tokens * (2 * d + 4)}
    moved = sum(_budgets(case))
    return {"bytes": sum(lens) * hkv * 4 + moved * (4 * half + 12 * hkv), "flops": sum(lens) * hkv * 4}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_e4m3(x):
    """The nearest E4M3 value of each fp64 x, ties to the even code."""
    mag = x.abs().clamp_max(FP8_MAX)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(mag / step) * step


def _exact_decode(codes):
    """E4M3 codes as fp64."""
    code = codes.long()
    e, m = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(code >= 128, -mag, mag)


def _exact_mrope(s):
    half = s["inv_freq"].numel()
    where = torch.stack([s["positions"][a] for a in _axis(s)], 1).double()  # [T, half]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), where * s["inv_freq"])[:, None]
    done = []
    for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
        x = x.double()
        x = gamma.double() * x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS)
        pair = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        x[..., :half], x[..., half:2 * half] = pair.real, pair.imag
        done.append(x)
    pool, at, cache = s["pool"], s["slots"].long(), {}
    for name, x in (("k", done[1]), ("v", s["v"].double())):
        n, h, page, d = pool[name].shape
        flat = torch.zeros((n * page, h, d), dtype=torch.float64, device="cuda")
        if pool["k_scale"] is None:
            flat[at] = x
        else:
            scale = torch.clamp(x.abs().amax(-1), min=MIN_AMAX) / FP8_MAX
            flat[at] = _exact_e4m3(x / scale[..., None])
            whole = torch.zeros((n * page, h), dtype=torch.float64, device="cuda")
            whole[at] = scale
            cache[name + "_scale"] = whole.reshape(n, page, h).transpose(1, 2).contiguous()
        cache[name] = flat.reshape(n, page, h, d).transpose(1, 2).contiguous()
    return {"q": done[0], "k": done[1] if s["keep_k"] else None, "cache": cache}


def _exact_score(s):
    """Request by request and head by head: the softmax weights' column sums."""
    P, hkv, page = s["nodes"], s["kv_heads"], s["page"]
    group = s["q_heads"] // hkv
    weights = s["weights"].double()
    pool = s["pool"]
    for n, ctx in enumerate(s["ctx"].tolist()):
        seen = torch.ones((P, ctx + P), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            seen[:, ctx:] = torch.ones((P, P), device="cuda").tril() > 0
        else:
            bits = [w & ((1 << 64) - 1) for w in s["mask"][n].tolist()]
            seen[:, ctx:] = torch.tensor([[w >> i & 1 for i in range(P)] for w in bits], device="cuda") > 0
        used = s["table"][n, :-(-(ctx + P) // page)].long()
        for h in range(hkv):
            k = pool["k"][used, h]
            k = k.double() if pool["k_scale"] is None else _exact_decode(k) * pool["k_scale"][used, h, :, None].double()
            k = k.reshape(-1, k.shape[-1])[:ctx + P]
            total = torch.zeros(ctx + P, dtype=torch.float64, device="cuda")
            for j in range(group):
                at = h * group + j
                logit = s["q"][n * P:(n + 1) * P, at].double() @ k.T * s["scale"]
                lse = s["lse"][n * P:(n + 1) * P, at, None].double()
                total += torch.where(seen & lse.isfinite(), torch.exp(logit - lse), 0.0).sum(0)
            row = weights[s["slot"][n].long(), h]
            if s["init"] is None:
                total[:ctx] += row[:ctx] * s["decay"]
            row[:ctx + P] = total
    return weights


def _exact_evict(s):
    """Request by request and head by head: everything above the smallest kept weight, then the first of those equal to it."""
    page, pool = s["page"], s["pool"]
    weights = s["weights"].double()
    kept_all, cache = s["kept"].clone(), {}
    for name in pool:
        if pool[name] is not None:
            values = _exact_decode(pool[name]) if pool[name].dtype == torch.uint8 else pool[name].double()
            cache[name] = values
    slots, dst_slots = s["slot"].tolist(), s["dst_slot"].tolist()
    for n, (length, budget) in enumerate(zip(s["len"].tolist(), s["budget"].tolist())):
        m = min(length, budget)
        if m == 0:
            continue
        for h in range(s["kv_heads"]):
            rank = weights[slots[n], h, :length].clone()
            rank[:s["sinks"]] = math.inf
            rank[max(0, length - s["recent"]):] = math.inf
            least = torch.topk(rank, m).values[-1]
            above, equal = rank > least, rank == least
            keep = above | (equal & (torch.cumsum(equal, 0) <= m - above.sum()))
            src = torch.nonzero(keep)[:, 0]
            dst = torch.arange(m, device="cuda")
            kept_all[n, h, :m] = src.to(torch.int32)
            src_page, dst_page = s["table"][n].long()[src // page], s["dst"][n].long()[dst // page]
            for x in cache.values():
                x[dst_page, h, dst % page] = x[src_page, h, src % page]
            weights[dst_slots[n], h, :m] = weights[slots[n], h, src]
    return {"kept": kept_all, "new_len": torch.minimum(s["len"], s["budget"]), "weights": weights, "cache": cache}


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm_mrope": _exact_mrope, "kv_score": _exact_score, "kv_evict": _exact_evict}[case["op"]](s)
