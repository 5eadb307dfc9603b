"""Measured cases of the attention-side operators: query/key head norms with the position rotation, the paged key/value
cache (written in bf16 or quantised to E4M3, and read back), attention of a tree of drafted tokens over that cache, and
the Gated DeltaNet verify of a drafted tree.

``run`` computes an operator in its plain form (elementary torch operations in fp32, fp64 for the angles), or, where
``own`` is true, makes the library call a serving program makes. ``exact`` is the same result from the definitions in
64 bits. The head layouts are those of the decoder whose linear-attention layers the library serves (24 query and 4
key/value heads of 256 with 64 rotated dimensions; 16 key and 48 value heads of 128 in the linear layers) and of one
of its four tensor-parallel ranks (6 and 1; 4 and 12), plus one generic layout (32 and 8 heads of 128).
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 1e7  # rotation base
FP8_MAX = 448.0  # largest finite E4M3 value
MIN_AMAX = 1e-12


# ------------------------------------------------------------------------------------------------ cases

def _rope(name, tokens, far, q_heads=24, kv_heads=4, head_dim=256, rotary=64, cache="e4m3", keep_k=False):
    return {"name": name, "op": "qk_norm_rope", "tokens": tokens, "far": far, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rotary": rotary, "cache": cache, "keep_k": keep_k, "page": 64}


def _write(name, tokens, cache, kv_heads=4, head_dim=256, skip=0):
    return {"name": name, "op": "kv_cache_write", "tokens": tokens, "cache": cache, "kv_heads": kv_heads,
            "head_dim": head_dim, "skip": skip, "page": 64}


def _read(name, seqs, lo, hi, cache, kv_heads=4, head_dim=256, page=64):
    return {"name": name, "op": "kv_cache_read", "seqs": seqs, "lo": lo, "hi": hi, "cache": cache, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page}


def _attn(name, seqs, nodes, tree, lo, hi, cache, q_heads=24, kv_heads=4, head_dim=256, page=64, gate=False):
    return {"name": name, "op": "tree_attention", "seqs": seqs, "nodes": nodes, "tree": tree, "lo": lo, "hi": hi,
            "cache": cache, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "gate": gate}


def _verify(name, seqs, nodes, k_heads=16, v_heads=48):
    return {"name": name, "op": "spec_verify_tree", "seqs": seqs, "nodes": nodes, "k_heads": k_heads,
            "v_heads": v_heads}


def listed():
    return [
        # a decode step of 256 requests: queries and keys straight from the projection, keys and values into the cache
        _rope("rope decode 256 to e4m3", 256, 131072),
        # eight prompt chunks of 2048 tokens, the keys kept for the prompt's own attention too
        _rope("rope prompt 16384 to bf16", 16384, 32768, cache="bf16", keep_k=True),
        # accepted drafts of 256 requests x 4 positions, the rejected half skipped
        _write("write 1024 half skipped", 1024, "bf16", skip=512),
        # a prompt batch into the quantised cache
        _write("write 16384 to e4m3", 16384, "e4m3"),
        # one cached prefix of 2047 tokens read back
        _read("read 1 prefix of 2047", 1, 2047, 2047, "bf16"),
        # 64 cached prompts, lengths log-spread over 16 .. 8192
        _read("read 64 prefixes e4m3", 64, 16, 8192, "e4m3"),
        # one request's decode step at a short context: latency
        _attn("decode 1 x 509 bf16", 1, 1, "none", 509, 509, "bf16"),
        # a decode batch of 256 requests over the quantised cache
        _attn("decode 256 x 1k..8k e4m3", 256, 1, "none", 1024, 8192, "e4m3"),
        # the verify of 8-node draft trees of 32 requests, ragged contexts, the output gate in the same pass
        _attn("tree 32 x 8 nodes bf16", 32, 8, "tree", 129, 16384, "bf16", gate=True, page=16),
        # one request's wide tree over a long context
        _attn("tree 1 x 64 nodes 131071 e4m3", 1, 64, "tree", 131071, 131071, "e4m3"),
        # the linear layers' verify of one request's tree on one tensor-parallel rank, and of 64 requests' trees
        _verify("gdn tree 1 x 5, rank heads", 1, 5, 4, 12),
        _verify("gdn tree 64 x 8", 64, 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_cache_write", "kv_cache_read", "tree_attention", "tree_attention",
                     "spec_verify_tree"])
    cache = rng.choice(["bf16", "e4m3"])
    hq, hkv, d = rng.choice([(24, 4, 256), (6, 1, 256), (32, 8, 128)])
    page = rng.choice([16, 64, 128])
    if op == "qk_norm_rope":
        c = _rope("", _log(rng, 1, 16384), rng.choice([4096, 131072, 1 << 20]), hq, hkv, d,
                  rng.choice([32, 64, d]), cache, rng.random() < 0.5)
        c["page"] = page
    elif op == "kv_cache_write":
        t = _log(rng, 1, 16384)
        c = _write("", t, cache, hkv, d, rng.randrange(t // 2 + 1))
        c["page"] = page
    elif op == "kv_cache_read":
        lo = _log(rng, 1, 512)
        c = _read("", _log(rng, 1, 64), lo, _log(rng, lo, 8192), cache, hkv, d, page)
    elif op == "tree_attention":
        nodes = _log(rng, 1, 64)
        seqs = _log(rng, 1, max(1, 256 // nodes))
        most = min(131072, max(64, 860000 // seqs // (1 if cache == "e4m3" else 2)), (1 << 23) // (seqs * nodes))
        lo = _log(rng, 1, most)
        c = _attn("", seqs, nodes, "none" if nodes == 1 else rng.choice(["chain", "tree"]), lo, _log(rng, lo, most),
                  cache, hq, hkv, d, page, rng.random() < 0.5)
    else:
        k, v = rng.choice([(16, 48), (4, 12), (8, 8)])
        c = _verify("", _log(rng, 1, 64), rng.randint(1, 8), k, v)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _lengths(case):
    """Lengths spread evenly over the logarithm of the case's range."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * (i + 0.5) / n)) for i in range(n)]


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _inv_freq(case):
    r = case["rotary"]
    i = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    return torch.pow(torch.tensor(THETA, dtype=torch.float64, device="cuda"), -i / r)


def _encode(x):
    """fp32 values of the last axis to E4M3 codes and one scale."""
    s = x.abs().amax(-1).clamp_min(MIN_AMAX) / FP8_MAX
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def _pool(g, case, pages, filled):
    """A key/value cache of `pages` pages: k, v and, quantised, their scales."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    e4m3 = case["cache"] == "e4m3"
    pool = {}
    for name in ("k", "v"):
        if not filled:
            pool[name] = torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
            pool[name + "_scale"] = torch.zeros(shape[:3], device="cuda") if e4m3 else None
            continue
        x = _randn(g, *shape)
        if name == "k":  # what a head norm leaves: unit rows times a gain, some channels stronger than others
            x *= torch.rand(shape[3], generator=g, device="cuda") * 1.5 + 0.5
        if e4m3:
            x, pool[name + "_scale"] = _encode(x)
            pool[name] = x.view(torch.uint8)
        else:
            pool[name], pool[name + "_scale"] = x.to(torch.bfloat16), None
    return pool


def _tables(g, case, tokens):
    """Block tables of requests with `tokens` cached tokens each, and the number of pages of the pool."""
    page = case["page"]
    need = [-(-t // page) for t in tokens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(tokens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, pages


def _slots(g, case, tokens, skip):
    """Distinct cache slots for `tokens` tokens, `skip` of them none (-1), and the number of pages of the pool."""
    pages = -(-2 * tokens // case["page"])
    slots = torch.randperm(pages * case["page"], generator=g, device="cuda")[:tokens].to(torch.int32)
    if skip:
        slots[torch.randperm(tokens, generator=g, device="cuda")[:skip]] = -1
    return slots, pages


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
    op = case["op"]
    if op == "qk_norm_rope":
        T, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        packed = _randn(g, T, hq + 2 * hkv, d).mul_(1.5).to(torch.bfloat16)  # one projection's output
        s["q"], s["k"], s["v"] = packed[:, :hq], packed[:, hq:hq + hkv], packed[:, hq + hkv:]
        s["q_gamma"], s["k_gamma"] = (torch.rand(d, generator=g, device="cuda") + 0.5 for _ in range(2))
        s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case)
        s["slots"], pages = _slots(g, case, T, 0)
        s["pool"] = _pool(g, case, pages, False)
        s["q_out"] = torch.zeros((T, hq, d), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros((T, hkv, d), dtype=torch.bfloat16, device="cuda") if case["keep_k"] else None
    elif op == "kv_cache_write":
        T, hkv, d = case["tokens"], case["kv_heads"], case["head_dim"]
        s["k"], s["v"] = (_randn(g, T, hkv, d).to(torch.bfloat16) for _ in range(2))
        s["slots"], pages = _slots(g, case, T, case["skip"])
        s["pool"] = _pool(g, case, pages, False)
    elif op == "kv_cache_read":
        lens = _lengths(case)
        order = torch.randperm(len(lens), generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["table"], pages = _tables(g, case, lens)
        s["pool"] = _pool(g, case, pages, True)
        s["starts"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        shape = (sum(lens), case["kv_heads"], case["head_dim"])
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif op == "tree_attention":
        P, hq, d = case["nodes"], case["q_heads"], case["head_dim"]
        lens = _lengths(case)
        order = torch.randperm(len(lens), generator=g, device="cuda").tolist()
        lens = [lens[i] for i in order]
        s["table"], pages = _tables(g, case, [t + P for t in lens])
        s["pool"] = _pool(g, case, pages, True)
        s["longest"] = max(lens)
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = (_randn(g, len(lens) * P, hq, d) * (torch.rand(d, generator=g, device="cuda") * 1.5 + 0.5)).to(
            torch.bfloat16)
        s["mask"] = _tree_mask(_parents(g, len(lens), P)) if case["tree"] == "tree" else None
        s["gate"] = _randn(g, len(lens) * P, hq, d).to(torch.bfloat16) if case["gate"] else None
        s["scale"] = d ** -0.5
        s["out"] = torch.zeros((len(lens) * P, hq, d), dtype=torch.bfloat16, device="cuda")
    else:
        n, P, hk, hv = case["seqs"], case["nodes"], case["k_heads"], case["v_heads"]
        ch, slots = (2 * hk + hv) * 128, n * (P + 1)
        s["qkv0"] = _randn(g, n * P, ch).to(torch.bfloat16)
        s["conv_w"] = _randn(g, ch, 4) * 0.25
        s["conv_hist"] = _randn(g, slots, ch, 3).to(torch.bfloat16)
        s["state"] = _randn(g, slots, hv, 128, 128).mul_(0.02)
        s["alpha"] = torch.exp(-(torch.rand((n * P, hv), generator=g, device="cuda") * 0.099 + 0.001))
        s["beta"] = torch.rand((n * P, hv), generator=g, device="cuda")
        s["z"] = _randn(g, n * P, hv, 128).to(torch.bfloat16)
        s["gamma"] = torch.ones(128, device="cuda")
        perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
        s["live"], s["spec"] = perm[:n].contiguous(), perm[n:].reshape(n, P).contiguous()
        s["parent"] = _parents(g, n, P)
        s["ogate"] = torch.zeros((n * P, hv * 128), dtype=torch.bfloat16, device="cuda")
    if own:
        _own_handles(s)
    return s


def _own_handles(s):
    """What a serving program makes once and keeps: the cache handle, the workspace, the geometry."""
    from gated_deltanet_linear_conv1d_gb300 import binding as b
    s["b"] = b
    if "pool" in s:
        p = s["pool"]
        s["cache_handle"] = b.make_kv_cache(p["k"], p["v"], p["k_scale"], p["v_scale"])
    if s["op"] == "tree_attention":
        need = b.gdn_tree_attention_workspace_bytes(s["cache_handle"], s["seqs"], s["nodes"], s["q_heads"])
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    elif s["op"] == "spec_verify_tree":
        s["dims"] = b.GdnDims(s["k_heads"], s["v_heads"], 128, 128, 4, s["state"].shape[0])


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)[s["op"]](s)


def _pool_values(pool):
    """The cache's contents: bf16 values, or E4M3 values and their scales."""
    if pool["k_scale"] is None:
        return {"k": pool["k"], "v": pool["v"]}
    e = torch.float8_e4m3fn
    return {"k": pool["k"].view(e), "v": pool["v"].view(e), "k_scale": pool["k_scale"], "v_scale": pool["v_scale"]}


def _own_rope(s):
    s["b"].gdn_qk_norm_rope(s["q"], s["k"], s["q_gamma"], s["k_gamma"], EPS, s["positions"], s["inv_freq"],
                            s["q_out"], k_out=s["k_out"], v=s["v"], cache=s["cache_handle"], kv_slot=s["slots"])
    return {"q": s["q_out"], "k": s["k_out"], "cache": _pool_values(s["pool"])}


def _own_write(s):
    s["b"].gdn_kv_cache_write(s["cache_handle"], s["k"], s["v"], s["slots"])
    return _pool_values(s["pool"])


def _own_read(s):
    s["b"].gdn_kv_cache_read(s["cache_handle"], s["table"], s["starts"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attention(s):
    s["b"].gdn_tree_attention(s["cache_handle"], s["q"], s["table"], s["ctx"], s["scale"], s["out"], s["nodes"],
                              tree_mask=s["mask"], gate=s["gate"], workspace=s["workspace"])
    return s["out"]


def _own_verify(s):
    s["b"].gdn_spec_verify_tree(s["dims"], s["qkv0"], s["conv_w"], s["conv_hist"], s["state"], s["live"], s["spec"],
                                s["parent"], s["alpha"], s["beta"], s["z"], s["gamma"], EPS, ogate=s["ogate"])
    return {"ogate": s["ogate"], "state": s["state"], "conv_hist": s["conv_hist"]}


def _plain_norm(x, gamma):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma


def _plain_rotate(x, positions, inv_freq):
    angle = positions.double()[:, None] * inv_freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    half = inv_freq.numel()
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., 2 * half:]), -1)


def _plain_store(pool, slots, k, v):
    kept = slots >= 0
    at = slots[kept].long()
    page, row = at // pool["k"].shape[2], at % pool["k"].shape[2]
    for name, x in (("k", k), ("v", v)):
        x = x[kept].float()
        if pool["k_scale"] is None:
            pool[name][page, :, row] = x.to(torch.bfloat16)
        else:
            x, scale = _encode(x)
            pool[name][page, :, row] = x.view(torch.uint8)
            pool[name + "_scale"][page, :, row] = scale


def _plain_rope(s):
    q = _plain_rotate(_plain_norm(s["q"], s["q_gamma"]), s["positions"], s["inv_freq"])
    k = _plain_rotate(_plain_norm(s["k"], s["k_gamma"]), s["positions"], s["inv_freq"])
    _plain_store(s["pool"], s["slots"], k, s["v"])
    return {"q": q.to(torch.bfloat16), "k": k.to(torch.bfloat16) if s["keep_k"] else None,
            "cache": _pool_values(s["pool"])}


def _plain_write(s):
    _plain_store(s["pool"], s["slots"], s["k"], s["v"])
    return _pool_values(s["pool"])


def _plain_gather(pool, name, page, row):
    x = pool[name][page, :, row]
    if pool["k_scale"] is None:
        return x.float()
    return x.view(torch.float8_e4m3fn).float() * pool[name + "_scale"][page, :, row][..., None]


def _plain_read(s):
    starts = s["starts"].long()
    t = torch.arange(s["k_out"].shape[0], device="cuda")
    n = torch.searchsorted(starts, t, right=True) - 1
    t = t - starts[n]
    page = s["table"][n, t // s["page"]].long()
    return {x: _plain_gather(s["pool"], x, page, t % s["page"]).to(torch.bfloat16) for x in ("k", "v")}


def _plain_attention(s):
    N, P, hq, hkv, d = s["seqs"], s["nodes"], s["q_heads"], s["kv_heads"], s["head_dim"]
    t = torch.arange(s["longest"] + P, device="cuda")
    page = s["table"][:, t // s["page"]].long().clamp_min(0)
    row = (t % s["page"]).expand(N, -1)
    draft = t - s["ctx"][:, None]  # [N, L]: the node a token is, negative: of the context
    k = _plain_gather(s["pool"], "k", page, row).permute(0, 2, 3, 1)  # [N, Hkv, D, L]
    q = s["q"].float().reshape(N, P, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(N, hkv, -1, d)
    score = torch.matmul(q, k).mul_(s["scale"]).reshape(N, hkv, P, hq // hkv, -1)
    del k
    node = torch.arange(P, device="cuda")
    if s["mask"] is None:
        seen = draft[:, None] <= node[:, None]
    else:
        seen = (draft < 0)[:, None] | ((s["mask"][..., None] >> draft.clamp(0, 63)[:, None]) & 1 == 1)
        seen &= (draft < P)[:, None]
    score = score.masked_fill_(~seen[:, None, :, None], float("-inf"))
    score = torch.exp(score - score.amax(-1, keepdim=True))
    total = score.sum(-1)
    v = _plain_gather(s["pool"], "v", page, row).permute(0, 2, 1, 3)
    out = torch.matmul(score.reshape(N, hkv, -1, t.numel()), v).reshape(N, hkv, P, hq // hkv, d) / total[..., None]
    out = out.permute(0, 2, 1, 3, 4).reshape(N * P, hq, d)
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].float()))
    return out.to(torch.bfloat16)


def _plain_silu(x):
    return x / (1 + torch.exp(-x))


def _plain_verify(s):
    n, P, hk, hv = s["seqs"], s["nodes"], s["k_heads"], s["v_heads"]
    rows, live, spec = torch.arange(n, device="cuda"), s["live"].long(), s["spec"].long()
    x = s["qkv0"].reshape(n, P, -1)
    state = torch.empty((n, P + 1, hv, 128, 128), device="cuda")
    hist = torch.empty((n, P + 1) + s["conv_hist"].shape[1:], dtype=torch.bfloat16, device="cuda")
    state[:, 0], hist[:, 0] = s["state"][live], s["conv_hist"][live]
    out = []
    for p in range(P):  # a node's state comes from its parent's
        at = s["parent"][:, p].long() + 1
        window = torch.cat((hist[rows, at], x[:, p, :, None]), -1)  # time-ascending
        hist[:, p + 1] = window[..., 1:]
        y = _plain_silu((window.float() * s["conv_w"].flip(-1)).sum(-1))
        q, k, v = y[:, :hk * 128].reshape(n, hk, 128), y[:, hk * 128:2 * hk * 128].reshape(n, hk, 128), y[:, 2 * hk * 128:]
        q, k = (u * torch.rsqrt(u.square().sum(-1, keepdim=True) + 1e-12) for u in (q, k))
        q, k = (u.repeat_interleave(hv // hk, 1) for u in (q, k))
        a, b = (s[w].reshape(n, P, hv)[:, p, :, None] for w in ("alpha", "beta"))
        prev = state[rows, at] * a[..., None]
        e = v.reshape(n, hv, 128) - (prev * k[:, :, None]).sum(-1)
        state[:, p + 1] = prev + (b * e)[..., None] * k[:, :, None]
        out.append((state[:, p + 1] * q[:, :, None]).sum(-1) * 128 ** -0.5)
    o = torch.stack(out, 1).reshape(n * P, hv, 128)
    gated = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["gamma"] * _plain_silu(s["z"].float())
    s["state"][spec], s["conv_hist"][spec] = state[:, 1:], hist[:, 1:]
    return {"ogate": gated.to(torch.bfloat16).reshape(n * P, -1), "state": s["state"], "conv_hist": s["conv_hist"]}


_run_plain = {"qk_norm_rope": _plain_rope, "kv_cache_write": _plain_write, "kv_cache_read": _plain_read,
              "tree_attention": _plain_attention, "spec_verify_tree": _plain_verify}
_run_own = {"qk_norm_rope": _own_rope, "kv_cache_write": _own_write, "kv_cache_read": _own_read,
            "tree_attention": _own_attention, "spec_verify_tree": _own_verify}


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    if op == "spec_verify_tree":
        n, P, hk, hv = case["seqs"], case["nodes"], case["k_heads"], case["v_heads"]
        ch = (2 * hk + hv) * 128
        state = n * (P + 1) * (hv * 65536 + ch * 6)  # the live slot in, every node's out
        token = n * P * (ch * 2 + hv * (8 + 128 * 4))  # qkv0, alpha, beta, z in, ogate out
        return {"bytes": state + token + ch * 16, "flops": n * P * hv * (128 * 128 * 8 + 128 * 12)}
    hkv, d = case["kv_heads"], case["head_dim"]
    held = 2 * hkv * (d + 4 if case["cache"] == "e4m3" else 2 * d)  # bytes of one token in the cache
    if op == "qk_norm_rope":
        T, hq = case["tokens"], case["q_heads"]
        kept = hkv * d * 2 if case["keep_k"] else 0
        return {"bytes": T * ((2 * hq + 2 * hkv) * d * 2 + kept + held + 8) + 8 * d,
                "flops": T * ((hq + hkv) * (4 * d + 3 * case["rotary"]) + 2 * hkv * d)}
    if op == "kv_cache_write":
        T = case["tokens"] - case["skip"]
        return {"bytes": T * (2 * hkv * d * 2 + held) + 4 * case["tokens"], "flops": T * 4 * hkv * d}
    tokens = sum(_lengths(case))
    if op == "kv_cache_read":
        return {"bytes": tokens * (held + 2 * hkv * d * 2), "flops": tokens * 2 * hkv * d}
    N, P, hq = case["seqs"], case["nodes"], case["q_heads"]
    tokens += N * P
    rows = N * P * hq * d * 2
    return {"bytes": tokens * held + rows * (3 if case["gate"] else 2), "flops": 4 * P * hq * d * tokens}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_e4m3(x):
    """The nearest E4M3 value of each fp64 x, ties to the even code."""
    mag = x.abs().clamp_max(FP8_MAX)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(mag / step) * step


def _exact_decode(pool, name, page, rows):
    """fp64 rows [rows, Hkv, D] of one page."""
    x = pool[name][page, :, :rows]
    if pool["k_scale"] is None:
        return x.double().transpose(0, 1)
    code = x.long()
    e, m = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).double()))
    mag = torch.where(code >= 128, -mag, mag) * pool[name + "_scale"][page, :, :rows, None].double()
    return mag.transpose(0, 1)


def _exact_sequence(s, n, name, tokens):
    page = s["page"]
    table = s["table"][n].tolist()
    return torch.cat([_exact_decode(s["pool"], name, table[i], min(page, tokens - i * page))
                      for i in range(-(-tokens // page))])


def _exact_cache(pool, slots, k, v):
    """The pool after rows k, v went to their slots."""
    page = pool["k"].shape[2]
    out = {}
    kept = torch.nonzero(slots >= 0)[:, 0]
    at = slots[kept].long()
    for name, x in (("k", k), ("v", v)):
        n, h, _, d = pool[name].shape
        flat = torch.zeros((n * page, h, d), dtype=torch.float64, device="cuda")
        if pool["k_scale"] is None:
            flat[at] = x[kept]
        else:
            scale = torch.clamp(x[kept].abs().amax(-1), min=MIN_AMAX) / FP8_MAX
            flat[at] = _exact_e4m3(x[kept] / scale[..., None])
            whole = torch.zeros((n * page, h), dtype=torch.float64, device="cuda")
            whole[at] = scale
            out[name + "_scale"] = whole.reshape(n, page, h).transpose(1, 2).contiguous()
        out[name] = flat.reshape(n, page, h, d).transpose(1, 2).contiguous()
    return out


def _exact_rope(s):
    half = s["inv_freq"].numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.outer(s["positions"].double(), s["inv_freq"]))[:, None]
    done = []
    for x, gamma in ((s["q"], s["q_gamma"]), (s["k"], s["k_gamma"])):
        x = x.double()
        x = gamma.double() * x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS)
        pair = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
        x[..., :half], x[..., half:2 * half] = pair.real, pair.imag
        done.append(x)
    return {"q": done[0], "k": done[1] if s["keep_k"] else None,
            "cache": _exact_cache(s["pool"], s["slots"], done[1], s["v"].double())}


def _exact_read(s):
    lens = s["starts"].diff().tolist()
    return {x: torch.cat([_exact_sequence(s, n, x, t) for n, t in enumerate(lens)]) for x in ("k", "v")}


def _exact_attention(s):
    P, hkv, d, group = s["nodes"], s["kv_heads"], s["head_dim"], s["q_heads"] // s["kv_heads"]
    out = []
    for n, ctx in enumerate(s["ctx"].tolist()):
        seen = torch.ones((P, ctx + P), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            seen[:, ctx:] = torch.ones((P, P), device="cuda").tril() > 0
        else:
            bits = [w & ((1 << 64) - 1) for w in s["mask"][n].tolist()]
            seen[:, ctx:] = torch.tensor([[w >> i & 1 for i in range(P)] for w in bits], device="cuda") > 0
        k, v = (_exact_sequence(s, n, x, ctx + P) for x in ("k", "v"))
        q = s["q"][n * P:(n + 1) * P].double()
        rows = torch.empty((P, hkv * group, d), dtype=torch.float64, device="cuda")
        for h in range(hkv):
            for j in range(group):
                score = q[:, h * group + j] @ k[:, h].T * s["scale"]
                p = torch.softmax(score.masked_fill(~seen, -math.inf), -1)
                rows[:, h * group + j] = p @ v[:, h]
        out.append(rows)
    out = torch.cat(out)
    return out if s["gate"] is None else out * torch.sigmoid(s["gate"].double())


def _exact_verify(s):
    """Every node from the live state along its own path."""
    n, P, hk, hv = s["seqs"], s["nodes"], s["k_heads"], s["v_heads"]
    x, w = s["qkv0"].double().reshape(n, P, -1), s["conv_w"].double()
    alpha, beta = (s[name].double().reshape(n, P, hv) for name in ("alpha", "beta"))
    state, hist = s["state"].double(), s["conv_hist"].double()
    live, spec, parents = s["live"].long(), s["spec"].long(), s["parent"].tolist()
    ogate = torch.empty((n, P, hv, 128), dtype=torch.float64, device="cuda")
    for r in range(n):
        for p in range(P):
            path, at = [], p
            while at >= 0:
                path.append(at)
                at = parents[r][at]
            path.reverse()
            inputs = torch.cat((hist[live[r]].T, x[r, path]))  # [3 + steps, CH]
            S = state[live[r]].clone()
            for i, node in enumerate(path):
                pre = inputs[i + 3] * w[:, 0] + inputs[i + 2] * w[:, 1] + inputs[i + 1] * w[:, 2] + inputs[i] * w[:, 3]
                y = pre * torch.sigmoid(pre)
                q, k, v = torch.split(y, [hk * 128, hk * 128, hv * 128])
                q, k = (torch.nn.functional.normalize(u.reshape(hk, 128), dim=-1).repeat_interleave(hv // hk, 0)
                        for u in (q, k))
                S *= alpha[r, node][:, None, None]
                e = v.reshape(hv, 128) - torch.einsum("hij,hj->hi", S, k)
                S += torch.einsum("h,hi,hj->hij", beta[r, node], e, k)
            o = torch.einsum("hij,hj->hi", S, q) / math.sqrt(128)
            z = s["z"][r * P + p].double()
            ogate[r, p] = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["gamma"] * z * torch.sigmoid(z)
            state[spec[r, p]], hist[spec[r, p]] = S, inputs[-3:].T
    return {"ogate": ogate.reshape(n * P, -1), "state": state, "conv_hist": hist}


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm_rope": _exact_rope, "kv_cache_read": _exact_read, "tree_attention": _exact_attention,
            "spec_verify_tree": _exact_verify,
            "kv_cache_write": lambda s: _exact_cache(s["pool"], s["slots"], s["k"].double(), s["v"].double()),
            }[case["op"]](s)
