"""Runs one libgdn entry point a few times on a synthetic workload, for profilers.

    python -m gated_deltanet_linear_conv1d_gb300.profile_case decode  --requests 64 --slots 128 --launches 3
    python -m gated_deltanet_linear_conv1d_gb300.profile_case prefill --lengths 2048x8 --launches 2
    python -m gated_deltanet_linear_conv1d_gb300.profile_case spec    --requests 64 --launches 2
    python -m gated_deltanet_linear_conv1d_gb300.profile_case commit  --requests 256 --launches 3
    python -m gated_deltanet_linear_conv1d_gb300.profile_case fp8     --requests 4096 --k 6144 --n 5120
    python -m gated_deltanet_linear_conv1d_gb300.profile_case gemm    --requests 256 --k 6144 --n 5120
    python -m gated_deltanet_linear_conv1d_gb300.profile_case attn    --lengths 4096x64 --cache e4m3 --nodes 1
    python -m gated_deltanet_linear_conv1d_gb300.profile_case rope    --requests 16384 --cache bf16
    python -m gated_deltanet_linear_conv1d_gb300.profile_case kvread  --lengths 4096x64 --cache e4m3
    python -m gated_deltanet_linear_conv1d_gb300.profile_case spectree --requests 64 --nodes 8

Each launch is preceded by the same warm-up launches (--warmup) and followed
by a device synchronisation; nothing else runs on the GPU besides the input
upload, so a profiler can select the kernel by name and skip the warm-ups.
"""
from __future__ import annotations

import argparse

import numpy as np
import torch

from . import synth


def _dev(w, dev):
    out = {}
    for k, v in w.items():
        if not isinstance(v, np.ndarray):
            continue
        if k in ("qkv0", "z", "conv_hist"):
            out[k] = torch.from_numpy(np.ascontiguousarray(v).view(np.int16)).view(torch.bfloat16).to(dev)
        else:
            out[k] = torch.from_numpy(np.ascontiguousarray(v)).to(dev)
    return out


def _lengths(spec: str) -> list[int]:
    out = []
    for part in spec.split(","):
        if "x" in part:
            n, c = part.split("x")
            out += [int(n)] * int(c)
        else:
            out.append(int(part))
    return out


def _cache(gen, tokens, page, heads, fmt, dev):
    """A filled key/value cache for requests of `tokens` tokens, and their block table (pages in random order)."""
    from . import binding as b
    need = [-(-t // page) for t in tokens]
    pages = sum(need)
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(tokens), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    pool, scale = [], [None, None]
    for i in range(2):
        x = torch.randn((pages, heads, page, 256), generator=gen, device=dev)
        if fmt == "e4m3":
            scale[i] = x.abs().amax(-1) / 448
            pool.append((x / scale[i][..., None]).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            pool.append(x.to(torch.bfloat16))
    return b.make_kv_cache(pool[0], pool[1], *scale), table


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("case", choices=["decode", "prefill", "spec", "commit", "conv", "rmsnorm", "fp8", "gemm", "attn",
                                     "rope", "kvread", "spectree"])
    ap.add_argument("--heads", choices=["full", "rank"], default="full")
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--slots", type=int, default=0)
    ap.add_argument("--lengths", default="2048x8",
                    help="prefill lengths or cached contexts, e.g. 2048x8 or 16,300,8192")
    ap.add_argument("--nodes", type=int, default=1, help="attn, spectree: drafted tokens per request")
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="e4m3", help="attn, rope, kvread: the cache's format")
    ap.add_argument("--page", type=int, default=64, help="attn, rope, kvread: tokens per page")
    ap.add_argument("--loguniform", type=int, default=0, help="prefill: N log-uniform lengths in [16, 8192]")
    ap.add_argument("--k", type=int, default=6144, help="fp8, gemm: input features")
    ap.add_argument("--n", type=int, default=5120, help="fp8, gemm: output features")
    ap.add_argument("--launches", type=int, default=3)
    ap.add_argument("--warmup", type=int, default=2)
    args = ap.parse_args(argv)

    from . import binding as b
    geom = synth.FULL_HEADS if args.heads == "full" else synth.RANK_HEADS
    dev = torch.device("cuda", 0)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    if args.case == "decode":
        w = synth.decode_workload(geom, args.requests, args.slots or 2 * args.requests, seed=1)
        d = _dev(w, dev)
        D = b.make_dims(geom, w["num_slots"])
        og = torch.empty((args.requests, geom.num_v_heads * 128), dtype=torch.bfloat16, device=dev)

        def run():
            b.gdn_decode_step(D, d["qkv0"], d["conv_w"], d["conv_hist"], d["state"], d["slot_idx"], d["alpha"],
                              d["beta"], d["z"], d["gamma"], w["eps"], ogate=og, dev_err=err)
    elif args.case in ("prefill", "conv"):
        lengths = (synth.loguniform_lengths(np.random.default_rng(3), args.loguniform, 16, 8192)
                   if args.loguniform else _lengths(args.lengths))
        w = synth.prefill_workload(geom, lengths, seed=3)
        d = _dev(w, dev)
        D = b.make_dims(geom, w["num_slots"])
        T = int(np.sum(lengths))
        og = torch.empty((T, geom.num_v_heads * 128), dtype=torch.bfloat16, device=dev)
        y = torch.empty((T, geom.channels), dtype=torch.bfloat16, device=dev) if args.case == "conv" else None
        ws = torch.empty(b.gdn_prefill_workspace_bytes(D, len(lengths), T), dtype=torch.uint8, device=dev)

        def run():
            if args.case == "conv":
                b.gdn_conv_update(D, d["qkv0"], d["conv_w"], d["conv_hist"], d["query_start_loc"], d["slot_idx"],
                                  y, has_init=d["has_init"], dev_err=err)
            else:
                b.gdn_chunk_prefill(D, d["qkv0"], d["conv_w"], d["conv_hist"], d["state"], d["query_start_loc"],
                                    d["slot_idx"], d["alpha"], d["beta"], d["z"], d["gamma"], w["eps"], ogate=og,
                                    has_init=d["has_init"], workspace=ws, dev_err=err)
    elif args.case in ("spec", "commit"):
        w = synth.spec_workload(geom, args.requests, num_pos=4, seed=4)
        d = _dev(w, dev)
        D = b.make_dims(geom, w["num_slots"])
        og = torch.empty((args.requests * 4, geom.num_v_heads * 128), dtype=torch.bfloat16, device=dev)
        acc = torch.from_numpy(w["accepted"]).to(dev)

        def run():
            if args.case == "commit":  # copy the accepted position's checkpoint into the live slot
                b.gdn_spec_commit(D, acc, d["spec_slot_idx"], d["slot_idx"], d["state"], d["conv_hist"],
                                  mode=b.GDN_COMMIT_COPY, dev_err=err)
            else:
                b.gdn_spec_verify(D, d["qkv0"], d["conv_w"], d["conv_hist"], d["state"], d["slot_idx"],
                                  d["spec_slot_idx"], d["alpha"], d["beta"], d["z"], d["gamma"], w["eps"], ogate=og,
                                  dev_err=err)
    elif args.case == "fp8":
        # out [T, N] = dequant(x8) dequant(w8)^T with block scales: random E4M3 codes and scales
        rng = np.random.default_rng(6)
        T, K, N = args.requests, args.k, args.n
        x8 = torch.from_numpy(synth.fp8_codes(rng, (T, K))).to(dev)
        w8 = torch.from_numpy(synth.fp8_codes(rng, (N, K))).to(dev)
        xs = torch.from_numpy(rng.uniform(0.002, 0.02, size=(T, K // 128)).astype(np.float32)).to(dev)
        ws = torch.from_numpy(rng.uniform(1e-4, 1e-3, size=((N + 127) // 128, K // 128)).astype(np.float32)).to(dev)
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
        wsp = torch.zeros(max(256, b.gdn_fp8_linear_workspace_bytes(T, K, N)), dtype=torch.uint8, device=dev)

        def run():
            b.gdn_fp8_linear(x8, xs, w8, ws, out, workspace=wsp, dev_err=err)
    elif args.case == "gemm":
        # out [T, N] = x [T, K] w[N, K]^T + out (gdn_out_proj, the residual in place)
        g = torch.Generator(device=dev)
        g.manual_seed(7)
        T, K, N = args.requests, args.k, args.n
        x = torch.randn((T, K), generator=g, device=dev).to(torch.bfloat16)
        wt = (torch.randn((N, K), generator=g, device=dev) / K ** 0.5).to(torch.bfloat16)
        out = torch.randn((T, N), generator=g, device=dev).to(torch.bfloat16)

        def run():
            b.gdn_out_proj(x, wt, out, residual=out, dev_err=err)
    elif args.case in ("attn", "rope", "kvread"):
        gen = torch.Generator(device=dev)
        gen.manual_seed(8)
        hq, hkv = (24, 4) if args.heads == "full" else (6, 1)
        if args.case == "rope":
            T = args.requests
            cache, _ = _cache(gen, [T], args.page, hkv, args.cache, dev)
            x = torch.randn((T, hq + 2 * hkv, 256), generator=gen, device=dev).to(torch.bfloat16)
            gain = torch.ones(256, device=dev)
            pos = torch.arange(T, dtype=torch.int32, device=dev)
            freq = 1e7 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device=dev) / 64)
            out = torch.empty((T, hq, 256), dtype=torch.bfloat16, device=dev)

            def run():
                b.gdn_qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], gain, gain, 1e-6, pos, freq, out, v=x[:, hq + hkv:],
                                   cache=cache, kv_slot=pos, dev_err=err)
        else:
            lengths, P = _lengths(args.lengths), args.nodes
            cache, table = _cache(gen, [n + P for n in lengths], args.page, hkv, args.cache, dev)
            N, T = len(lengths), sum(lengths) if args.case == "kvread" else len(lengths) * P
            if args.case == "kvread":
                start = torch.tensor([0] + lengths, device=dev).cumsum(0).to(torch.int32)
                ko, vo = (torch.empty((T, hkv, 256), dtype=torch.bfloat16, device=dev) for _ in range(2))
            else:
                ctx = torch.tensor(lengths, dtype=torch.int32, device=dev)
                q = torch.randn((T, hq, 256), generator=gen, device=dev).to(torch.bfloat16)
                out = torch.empty_like(q)
                ws = torch.empty(b.gdn_tree_attention_workspace_bytes(cache, N, P, hq), dtype=torch.uint8, device=dev)

            def run():
                if args.case == "kvread":
                    b.gdn_kv_cache_read(cache, table, start, ko, vo, dev_err=err)
                else:
                    b.gdn_tree_attention(cache, q, table, ctx, 256 ** -0.5, out, P, workspace=ws, dev_err=err)
    elif args.case == "spectree":
        w = synth.spec_workload(geom, args.requests, num_pos=args.nodes, seed=4)
        d = _dev(w, dev)
        D = b.make_dims(geom, w["num_slots"])
        rng = np.random.default_rng(9)
        parent = torch.from_numpy(np.array([[rng.integers(-1, p) for p in range(args.nodes)]
                                            for _ in range(args.requests)], dtype=np.int32)).to(dev)
        T = args.requests * args.nodes
        og = torch.empty((T, geom.num_v_heads * 128), dtype=torch.bfloat16, device=dev)

        def run():
            b.gdn_spec_verify_tree(D, d["qkv0"], d["conv_w"], d["conv_hist"], d["state"], d["slot_idx"],
                                   d["spec_slot_idx"], parent, d["alpha"], d["beta"], d["z"], d["gamma"], w["eps"],
                                   ogate=og, dev_err=err)
    else:
        rng = np.random.default_rng(5)
        T = args.requests
        o = torch.from_numpy(synth.bf16_bits(rng.standard_normal((T, 48, 128)).astype(np.float32)).view(np.int16))
        z = torch.from_numpy(synth.bf16_bits(rng.standard_normal((T, 48, 128)).astype(np.float32)).view(np.int16))
        o, z = o.view(torch.bfloat16).to(dev), z.view(torch.bfloat16).to(dev)
        gamma = torch.ones(128, dtype=torch.float32, device=dev)
        out = torch.empty((T, 48 * 128), dtype=torch.bfloat16, device=dev)

        def run():
            b.gdn_gated_rmsnorm(o, z, gamma, 1e-6, out)

    times = []
    for it in range(args.warmup + args.launches):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        run()
        e1.record()
        torch.cuda.synchronize()
        if it >= args.warmup:
            times.append(e0.elapsed_time(e1))
    flag = b.gdn_read_device_error(err)
    tokens = {"decode": args.requests, "spec": args.requests * 4, "commit": args.requests,
              "fp8": args.requests, "gemm": args.requests}.get(args.case)
    if args.case in ("prefill", "conv", "attn", "rope", "kvread", "spectree"):
        tokens = T
    ms = sum(times) / max(1, len(times))
    rate = f", {tokens / (ms / 1e3):.4g} tokens/s" if tokens else ""
    print(f"profile_case {args.case}: {args.launches} launches after {args.warmup} warm-up, "
          f"mean {ms:.4f} ms{rate}, device error word {flag}")
    if flag:
        raise SystemExit(1)


if __name__ == "__main__":
    main()
