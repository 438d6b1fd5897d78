"""Run the finalize on one synthetic configuration a few times (no checks).

For profilers: one process, a handful of launches, a known input size.

  python -m moe_deferred_finalize_gb300.run_case --workload decode_bs256 --iters 3
  python -m moe_deferred_finalize_gb300.run_case --prefill-tokens 4096 --iters 3
  python -m moe_deferred_finalize_gb300.run_case --workload decode_bs1_packed --unfused
  python -m moe_deferred_finalize_gb300.run_case --gate-tokens 16384 --iters 3
  python -m moe_deferred_finalize_gb300.run_case --tp 8 16 --form one_shot --iters 3
  python -m moe_deferred_finalize_gb300.run_case --tp-procs 16 --iters 300
  python -m moe_deferred_finalize_gb300.run_case --layer 256 --iters 20
  python -m moe_deferred_finalize_gb300.run_case --train 4096 --iters 3

--tp-procs times the orchestration of the all-reduce-fused finalize across
processes (moe_deferred_finalize_gb300.tp, two-phase form): two processes on
GPU 0, a gloo group for set-up and the per-step host barrier; it prints the
wall time per step and of the barrier alone.

--layer runs a whole MoE layer on that many tokens (router product, gate, row
map, expert products, shared expert, finalize with RMSNorm; 256 experts, top-8,
H = 7168, I = 2048, random weights made on the device, 23 GB) as one captured
graph, and prints its time and that of each step.

--train runs a training step of such a layer with 64 experts on that many tokens:
forward with what the backward pass needs kept, the gradients of all inputs and
weights, and an AdamW step with fp32 master weights and states of --state-bits
(28 GB with 8); also as one captured graph, with the time of each part.
"""
import argparse
import time

import numpy as np
import torch

import moe_deferred_finalize_gb300 as mf
from moe_deferred_finalize_gb300 import workloads as W


def _dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(a).cuda()


def _tp_procs_worker(rank, port, T, steps, q):
    import torch.distributed as dist
    from moe_deferred_finalize_gb300 import tp
    torch.cuda.set_device(0)
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{port}", rank=rank,
                            world_size=2)
    try:
        g = W.tp_decode(2, T, seed=7)
        wl = g.ranks[rank]
        x = {"permuted_out": _dev(wl.permuted_out), "idx_map": _dev(wl.idx),
             "weights": _dev(wl.weights), "shared_out": _dev(wl.shared)}
        outs = {k: torch.empty((T, g.H), dtype=torch.bfloat16, device="cuda")
                for k in ("out", "residual_out", "norm_out")}
        ep = dict(residual=_dev(g.residual), gamma=_dev(g.gamma), eps=g.eps)
        group = tp.TPFinalize(dist.group.WORLD, T, g.H)
        res = {}
        for n, key in ((20, None), (steps, "us_per_step")):
            torch.cuda.synchronize()
            dist.barrier()
            t0 = time.perf_counter()
            for _ in range(n):
                group.step(x, g.wkind, g.routed_scale, T, outs=outs, **ep)
            torch.cuda.synchronize()
            if key:
                res[key] = (time.perf_counter() - t0) / n * 1e6
        t0 = time.perf_counter()
        for _ in range(steps):
            dist.barrier()
        res["us_per_barrier"] = (time.perf_counter() - t0) / steps * 1e6
        group.close()
        q.put((rank, res))
    finally:
        dist.destroy_process_group()


def _tp_procs(T, steps):
    import multiprocessing as mp
    import socket
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        port = sk.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_tp_procs_worker, args=(r, port, T, steps, q)) for r in range(2)]
    for pr in procs:
        pr.start()
    got = dict(q.get(timeout=600) for _ in procs)
    for pr in procs:
        pr.join(120)
        if pr.exitcode != 0:
            raise RuntimeError(f"rank process exited with {pr.exitcode}")
    for rank in sorted(got):
        r = got[rank]
        print(f"tp-procs: rank {rank} T={T} steps={steps}: {r['us_per_step']:.1f} us per "
              f"two-phase step, {r['us_per_barrier']:.1f} us per host barrier")


def _layer(T, iters):
    E, K, H, I, tile = 256, 8, 7168, 2048, 16
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(
            0.0, scale, generator=g)

    x, residual, gamma = rand(T, H), rand(T, H, scale=2.0), rand(H)
    router = rand(E, H, scale=H ** -0.5)
    w13, w2 = rand(E, 2 * I, H, scale=H ** -0.5), rand(E, H, I, scale=I ** -0.5)
    s13, s2 = rand(2 * I, H, scale=H ** -0.5), rand(H, I, scale=I ** -0.5)
    t = {}

    def step(name, fn):
        t[name] = fn
        return fn()

    def layer():
        logits = step("router", lambda: mf.linear(x, router, out_dtype=torch.float32)["out"])
        route = step("gate", lambda: mf.topk_route(logits, K, "sigmoid"))
        m = step("row map", lambda: mf.permute_tokens(route["expert_ids"], E, tile))
        h = step("experts up", lambda: mf.expert_gated_ffn(x, m["row_token"], m["offsets"],
                                                           m["counts"], w13))
        rows = step("experts down", lambda: mf.expert_linear(h, m["offsets"], m["counts"], w2))
        hs = step("shared up", lambda: mf.gated_ffn(x, s13)["out"])
        shared = step("shared down", lambda: mf.linear(hs, s2)["out"])
        return step("finalize", lambda: mf.moe_finalize(
            rows, m["idx_map"], route["weights"], "fp32", shared, routed_scale=2.5,
            residual=residual, gamma=gamma, write_out=False))

    _report("layer", T, layer, t, iters)


def _report(what, T, whole, parts, iters):
    """The time of `whole` and of each of the parts that it filled in."""
    def timed(fn, n):
        fn()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = [fn() for _ in range(n)]
        graph.replay()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        del kept
        return a.elapsed_time(b) * 1e3 / n

    total = timed(whole, iters)
    # each step by itself, on the layer's own operands (small ones run from L2)
    each = {name: timed(fn, iters) for name, fn in list(parts.items())}
    print(f"{what}: T={T} {total:.1f} us; " +
          ", ".join(f"{name} {us:.1f}" for name, us in each.items()))


def _train(T, iters, bits):
    E, K, H, I, tile = 64, 8, 7168, 2048, 16
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, scale=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(
            0.0, scale, generator=g)

    x, residual = rand(T, H), rand(T, H, scale=2.0)
    dnorm, dres = rand(T, H, scale=0.01), rand(T, H, scale=0.01)
    w = {"router": rand(E, H, scale=H ** -0.5), "w13": rand(E, 2 * I, H, scale=H ** -0.5),
         "w2": rand(E, H, I, scale=I ** -0.5), "s13": rand(2 * I, H, scale=H ** -0.5),
         "s2": rand(H, I, scale=I ** -0.5), "gamma": rand(H)}
    d = {k: torch.zeros_like(v) for k, v in w.items()}
    update = mf.bind_adamw(list(w.values()), list(d.values()),
                           **mf.adamw_state(list(w.values()), bits, master=True))
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    P = mf.permute_rows(T, K, E, tile)
    preact = torch.empty((P, 2 * I), dtype=torch.bfloat16, device="cuda")
    drows, dh, dxr = (torch.empty((P, n), dtype=torch.bfloat16, device="cuda") for n in (H, I, H))
    t = {}

    def part(name, fn):
        t[name] = fn
        return fn()

    def step():
        logits = part("router", lambda: mf.linear(x, w["router"], out_dtype=torch.float32)["out"])
        route = part("gate", lambda: mf.topk_route(logits, K, "sigmoid"))
        m = part("row map", lambda: mf.permute_tokens(route["expert_ids"], E, tile))
        offsets, counts = m["offsets"], m["counts"]
        h = part("experts up", lambda: mf.expert_gated_ffn(
            x, m["row_token"], offsets, counts, w["w13"], preact=preact))
        rows = part("experts down", lambda: mf.expert_linear(h, offsets, counts, w["w2"]))
        up = part("shared up", lambda: mf.gated_ffn(x, w["s13"], save_preact=True))
        shared = part("shared down", lambda: mf.linear(up["out"], w["s2"])["out"])
        out = part("finalize", lambda: mf.moe_finalize(
            rows, m["idx_map"], route["weights"], "fp32", shared, routed_scale=2.5,
            residual=residual, gamma=w["gamma"], write_out=False))
        f = part("finalize backward", lambda: mf.moe_finalize_backward(
            rows, m["idx_map"], route["weights"], "fp32", routed_scale=2.5, dresidual_out=dres,
            dnorm_out=dnorm, residual_out=out["residual_out"], gamma=w["gamma"], drows=drows,
            dgamma=d["gamma"]))
        part("experts down backward", lambda: mf.expert_linear_backward(
            drows, h, offsets, counts, w["w2"], dx=dh, dweight=d["w2"]))
        part("experts up backward", lambda: mf.expert_gated_ffn_backward(
            dh, x, m["row_token"], offsets, counts, w["w13"], preact, dx=dxr, dweight=d["w13"]))
        s2 = part("shared down backward", lambda: mf.linear_backward(
            f["dshared"], up["out"], w["s2"], dweight=d["s2"]))
        s13 = part("shared up backward", lambda: mf.gated_ffn_backward(
            s2["dx"], x, w["s13"], up["preact"], dweight=d["s13"]))
        dlogits = part("gate backward", lambda: mf.topk_route_backward(
            f["dweights"], route["weights"], route["expert_ids"], E, "sigmoid", logits=logits))
        r = part("router backward", lambda: mf.linear_backward(dlogits, x, w["router"],
                                                               dweight=d["router"]))
        dx = part("unpermute", lambda: mf.unpermute_tokens(dxr, m["idx_map"],
                                                           add=(s13["dx"], r["dx"])))

        def adamw():
            count.add_(1)
            update(step=count, lr=1e-4)
            return dx

        return part("adamw", adamw)

    _report(f"train, {bits}-bit states", T, step, t, iters)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    g = ap.add_mutually_exclusive_group(required=True)
    g.add_argument("--workload", choices=W.CONFIG_NAMES)
    g.add_argument("--prefill-tokens", type=int)
    g.add_argument("--gate-tokens", type=int,
                   help="run the top-K gate (E=256, K=8, sigmoid, packed) on this many tokens")
    g.add_argument("--tp", type=int, nargs=2, metavar=("R", "T"),
                   help="the all-reduce-fused finalize over R ranks at decode batch T "
                        "(1, 16 or 256), H=7168, residual + RMSNorm")
    g.add_argument("--tp-procs", type=int, metavar="T",
                   help="time the two-process orchestration (two-phase form, R=2) at batch T "
                        "(1, 16 or 256) on GPU 0 for --iters steps")
    g.add_argument("--layer", type=int, metavar="T", help="run a whole MoE layer on T tokens")
    g.add_argument("--train", type=int, metavar="T",
                   help="run a training step of an MoE layer on T tokens")
    ap.add_argument("--state-bits", type=int, choices=[8, 32], default=8,
                    help="with --train: bits of the AdamW states")
    ap.add_argument("--form", choices=["one_shot", "two_phase", "plain"], default="one_shot",
                    help="with --tp: one-shot, two-phase (phase 1 per rank, then phase 2), "
                         "or the plain finalize of rank 0's operands")
    ap.add_argument("--iters", type=int, default=3)
    ap.add_argument("--write-out", action="store_true",
                    help="with a residual, also write out (default: residual_out + norm_out only)")
    ap.add_argument("--unfused", action="store_true", help="run the unfused A/B path")
    ap.add_argument("--splits", type=int, default=0)
    ap.add_argument("--threads", type=int, default=0)
    args = ap.parse_args(argv)
    if args.layer:
        _layer(args.layer, args.iters)
        return
    if args.train:
        _train(args.train, args.iters, args.state_bits)
        return
    if args.tp_procs:
        _tp_procs(args.tp_procs, args.iters)
        return
    if args.gate_tokens:
        g_ = torch.Generator(device="cuda").manual_seed(0)
        z = torch.randn((args.gate_tokens, 256), generator=g_, device="cuda")
        for _ in range(args.iters):
            mf.topk_route(z, 8, "sigmoid", want_packed=True)
        torch.cuda.synchronize()
        print(f"gate: T={args.gate_tokens} E=256 K=8 iters={args.iters} ok")
        return
    if args.tp:
        R, T = args.tp
        g = W.tp_decode(R, T)
        ranks = [{"permuted_out": _dev(wl.permuted_out), "idx_map": _dev(wl.idx),
                  "weights": _dev(wl.weights), "shared_out": _dev(wl.shared)} for wl in g.ranks]
        ep = dict(residual=_dev(g.residual), gamma=_dev(g.gamma), eps=g.eps, write_out=False)
        for _ in range(args.iters):
            if args.form == "one_shot":
                mf.moe_finalize_allreduce(ranks, g.wkind, routed_scale=g.routed_scale, **ep)
            elif args.form == "two_phase":
                parts = [mf.moe_finalize_partial(r["permuted_out"], r["idx_map"], r["weights"],
                                                 g.wkind, r["shared_out"],
                                                 routed_scale=g.routed_scale) for r in ranks]
                mf.moe_finalize_allreduce_reduce(parts, **ep)
            else:
                r0 = ranks[0]
                mf.moe_finalize(r0["permuted_out"], r0["idx_map"], r0["weights"], g.wkind,
                                r0["shared_out"], routed_scale=g.routed_scale, **ep)
        torch.cuda.synchronize()
        print(f"tp: R={R} T={T} form={args.form} iters={args.iters} ok")
        return
    wl = W.make(args.workload) if args.workload else W.prefill(args.prefill_tokens)
    x, idx, w, sh = _dev(wl.permuted_out), _dev(wl.idx), _dev(wl.weights), _dev(wl.shared)
    res = _dev(wl.residual) if wl.with_norm else None
    gam = _dev(wl.gamma) if wl.with_norm else None
    for _ in range(args.iters):
        if args.unfused:
            mf.moe_finalize_unfused(x, idx, w, wl.wkind, sh, routed_scale=wl.routed_scale,
                                    residual=res, gamma=gam, eps=wl.eps)
        else:
            mf.moe_finalize(x, idx, w, wl.wkind, sh, routed_scale=wl.routed_scale, residual=res,
                            gamma=gam, eps=wl.eps, write_out=args.write_out or not wl.with_norm,
                            splits=args.splits, threads=args.threads)
    torch.cuda.synchronize()
    print(f"{wl.name}: T={wl.T} K={wl.K} H={wl.H} P={wl.P} iters={args.iters} ok")


if __name__ == "__main__":
    main()
