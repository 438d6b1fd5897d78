"""The training side of the MoE layer, as it is measured.

The layer runs forward as router product -> top-K gate -> row map -> expert products -> finalize.  Measured here is
the way back through it, and the update of its weights:

  finalize_bwd   gradients of the finalize: of the expert rows, the routing weights, the shared output, the residual
                 and gamma
  unpermute      rows grouped by expert back to their tokens, summed over the slots: the gradient of the row gather
  gate_bwd       gradients of the top-K gate's weights, into its logits
  experts_bwd    gradients of the two products over rows grouped by expert (up: gated, x gathered; down: linear)
  adamw          one AdamW step over all tensors of some layers, states in 32 bits or in 8
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BLOCK = 256         # values of an 8-bit state that share a scale
F8_MAX = 448.0


def listed():
    return [
        # the finalize of 16 tokens with residual and RMSNorm, packed routing words: a small step, latency counts
        {"name": "finalize backward T=16", "op": "finalize_bwd", "T": 16, "topk": 8, "E": 384, "H": 7168, "tile": 64, "wkind": "packed", "norm": True, "dout": False, "scale": 1.0, "pad": 0},
        # the same over a training batch; the finalized output is used beside the norm
        {"name": "finalize backward T=4096", "op": "finalize_bwd", "T": 4096, "topk": 8, "E": 256, "H": 7168, "tile": 128, "wkind": "fp32", "norm": True, "dout": True, "scale": 2.5, "pad": 0},
        # token gradients of a small batch, its last tokens padding; the shared expert's gradient is added
        {"name": "unpermute T=256", "op": "unpermute", "T": 256, "topk": 8, "E": 256, "H": 7168, "tile": 16, "adds": 1, "pad": 19},
        # token gradients of a long batch, the router's and the shared expert's added
        {"name": "unpermute T=16384", "op": "unpermute", "T": 16384, "topk": 8, "E": 256, "H": 7168, "tile": 128, "adds": 2, "pad": 0},
        # the gate of a small batch
        {"name": "gate backward T=256", "op": "gate_bwd", "T": 256, "topk": 8, "E": 256, "kind": "softmax", "f32": False, "pad": 0},
        # the gate of a long batch
        {"name": "gate backward T=16384", "op": "gate_bwd", "T": 16384, "topk": 8, "E": 256, "kind": "sigmoid", "f32": False, "pad": 100},
        # a small biased layer, no row of padding between its ragged experts
        {"name": "experts backward T=100", "op": "experts_bwd", "gated": True, "T": 100, "topk": 2, "E": 8, "H": 1536, "I": 520, "act": "gelu", "bias": True, "tile": 1, "pad": 3},
        # the down projections of a training batch on 64 experts
        {"name": "experts down backward T=4096", "op": "experts_bwd", "gated": False, "T": 4096, "topk": 8, "E": 64, "H": 7168, "I": 2048, "act": "none", "bias": False, "tile": 128, "pad": 0},
        # the gated up projections of the same batch, x gathered by the row map
        {"name": "experts up backward T=4096", "op": "experts_bwd", "gated": True, "T": 4096, "topk": 8, "E": 64, "H": 7168, "I": 2048, "act": "silu", "bias": False, "tile": 128, "pad": 0},
        # the update of a few small layers, fp32 states without master weights: many tensors, little in each
        {"name": "adamw 32 bits, 4 small layers", "op": "adamw", "layers": 4, "E": 8, "H": 256, "I": 128, "bits": 32, "master": False, "f32": False},
        # the update of a layer of 8 experts, fp32 states and master weights
        {"name": "adamw 32 bits, 8 experts", "op": "adamw", "layers": 1, "E": 8, "H": 7168, "I": 2048, "bits": 32, "master": True, "f32": False},
        # the same with 8-bit states
        {"name": "adamw 8 bits, 8 experts", "op": "adamw", "layers": 1, "E": 8, "H": 7168, "I": 2048, "bits": 8, "master": True, "f32": False},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["finalize_bwd", "finalize_bwd", "unpermute", "gate_bwd", "experts_bwd", "experts_bwd", "experts_bwd", "adamw", "adamw"])
    E = rng.choice([8, 60, 64, 128, 256, 384])
    c = {"op": op}
    if op == "adamw":
        bits = rng.choice([8, 32])
        return dict(c, layers=rng.choice([1, 2, 5, 12]), E=rng.choice([4, 8, 16]), H=_log_int(rng, 64, 2048), I=_log_int(rng, 32, 768), bits=bits,
                    master=rng.random() < 0.5, f32=rng.random() < 0.3)
    if op == "experts_bwd":
        return dict(c, gated=rng.random() < 0.5, T=_log_int(rng, 1, 2000), topk=rng.choice([1, 2, 4, 8]), E=rng.choice([8, 16, 60, 64]), H=_log_int(rng, 256, 4096, 8),
                    I=_log_int(rng, 64, 2048, 8), act=rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]), bias=rng.random() < 0.3,
                    tile=rng.choice([1, 16, 64, 128]), pad=rng.choice([0, 0, 1]))
    T, topk = _log_int(rng, 1, 4096), rng.choice([1, 2, 4, 6, 8])
    if op == "gate_bwd":
        return dict(c, T=_log_int(rng, 1, 16384), topk=topk, E=E, kind=rng.choice(["softmax", "sigmoid"]), f32=rng.random() < 0.5, pad=rng.choice([0, T // 16]))
    H = _log_int(rng, 64, 7168, rng.choice([1, 8, 8, 8]))
    tile = rng.choice([1, 16, 64, 128])
    if op == "unpermute":
        return dict(c, T=T, topk=topk, E=E, H=H, tile=tile, adds=rng.choice([0, 1, 2]), pad=rng.choice([0, T // 10]))
    norm = rng.random() < 0.6
    return dict(c, T=T, topk=topk, E=E, H=H, tile=tile, wkind=rng.choice(["fp32", "bf16", "packed"]), norm=norm, dout=not norm or rng.random() < 0.5,
                scale=rng.choice([1.0, 2.5]), pad=rng.choice([0, T // 10]))


# ------------------------------------------------------------------ inputs


def _rows_bound(T, K, E, tile):
    """Rows that hold every padded layout of T*K slots over E experts."""
    n = T * K
    return (n + min(E, n) * (tile - 1)) // tile * tile


def _layout(ids, E, tile):
    """The padded layout of expert ids [T, K]: row map [T, K] (-1: no row), row -> token [P] (-1 on padding), first
    rows [E + 1] and row counts [E]; an expert's rows in (token, slot) order."""
    T, K = ids.shape
    P = _rows_bound(T, K, E, tile)
    flat = ids.reshape(-1).long()
    ok = flat >= 0
    key = torch.where(ok, flat, torch.full_like(flat, E))
    counts = torch.zeros(E + 1, dtype=torch.long, device=DEV).index_add_(0, key, torch.ones_like(key))
    before = torch.cumsum(counts, 0) - counts
    offsets = torch.zeros(E + 1, dtype=torch.long, device=DEV)
    offsets[1:] = torch.cumsum((counts[:E] + tile - 1) // tile * tile, 0)
    order = torch.argsort(key, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(flat.numel(), device=DEV)
    row = torch.where(ok, offsets[key] + rank - before[key], torch.full_like(rank, -1))
    token = torch.full((P + 1,), -1, dtype=torch.int32, device=DEV)
    token[torch.where(ok, row, torch.full_like(row, P))] = (torch.arange(flat.numel(), device=DEV) // K).int()
    return {"idx_map": row.int().reshape(T, K), "row_token": token[:P].contiguous(), "offsets": offsets.int(), "counts": counts[:E].int()}


def _logits(c, g):
    """Logits of a router with popular and rare experts."""
    return torch.randn(c["T"], c["E"], generator=g, device=DEV) + 0.5 * torch.randn(1, c["E"], generator=g, device=DEV)


def _ids(c, logits):
    """Its top-k expert ids; the last `pad` tokens are padding (-1)."""
    ids = logits.topk(min(c["topk"], c["E"]), dim=1).indices.int()
    pad = min(c["pad"], c["T"] - 1)
    if pad:
        ids[c["T"] - pad:] = -1
    return ids.contiguous()


def _normal(g, shape, scale=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, scale, generator=g)


def _sizes(c):
    """The tensors of the layers: router, expert and shared projections, gamma, router bias."""
    E, H, I = c["E"], c["H"], c["I"]
    return [E * H, E * 2 * I * H, E * H * I, 2 * I * H, H * I, H, E] * c["layers"]


def _f8(x, floor):
    """Values [blocks, BLOCK] as e4m3 codes and their scales; floor: values above 0 keep the least code above 0."""
    scale = x.abs().amax(1) / F8_MAX
    y = x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    if floor:
        y = torch.where(y > 0, torch.clamp(y, min=2.0 ** -9), y)
    return y.to(F8), scale


def _adamw_state(c, g):
    """Weights, gradients and states from earlier steps, each kind in one flat buffer that the tensors are views of;
    every tensor begins at a multiple of BLOCK, and what lies between two is zero."""
    sizes = _sizes(c)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    inside = torch.zeros(total + 1, dtype=torch.int8, device=DEV)
    inside[torch.tensor(starts, device=DEV)] += 1
    ends = torch.tensor([a + n for a, n in zip(starts, sizes)], device=DEV)
    inside.index_add_(0, ends, torch.full((len(sizes),), -1, dtype=torch.int8, device=DEV))
    inside = torch.cumsum(inside[:total], 0, dtype=torch.int8).to(BF16)

    def flat(scale, dtype=F32):
        return _normal(g, (total,), scale, dtype).mul_(inside)

    dtype = F32 if c["f32"] and not c["master"] else BF16
    master = flat(0.02)
    s = {"param": master.to(dtype), "grad": flat(1e-3, F32 if c["f32"] else BF16), "master": master if c["master"] else None}
    m, v = flat(3e-4), flat(1e-3).square_()
    if c["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        for key, x, floor in (("m", m, False), ("v", v.sqrt_(), True)):
            code, scale = _f8(x.view(-1, BLOCK), floor)
            s[key], s[key + "_scale"] = code.view(-1), scale
    s["sizes"], s["starts"] = sizes, starts
    return s


HYPER = {"lr": 1e-3, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1, "step": 20}


def _bind_adamw(s):
    """The framework's handle over a state's tensors, as a training program keeps it."""
    import moe_deferred_finalize_gb300 as mf

    def views(key, step=1):
        if s.get(key) is None:
            return None
        return [s[key][a // step:a // step + -(-n // step)] for a, n in zip(s["starts"], s["sizes"])]

    return mf.bind_adamw(views("param"), views("grad"), views("m"), views("v"), masters=views("master"),
                         exp_avg_scale=views("m_scale", BLOCK), exp_avg_sq_scale=views("v_scale", BLOCK))


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c, "op": c["op"]}
    if c["op"] == "adamw":
        s.update(_adamw_state(c, g))
        return s
    T, E = c["T"], c["E"]
    logits = _logits(c, g)
    ids = _ids(c, logits)
    if c["op"] == "gate_bwd":
        z = torch.where(ids >= 0, logits.gather(1, ids.clamp(min=0).long()), torch.zeros((), device=DEV))
        w = torch.softmax(z, 1) if c["kind"] == "softmax" else torch.sigmoid(z) / torch.sigmoid(z).sum(1, keepdim=True)
        s.update(logits=logits, ids=ids, weights=w.contiguous(), dweights=_normal(g, ids.shape, 0.1, F32))
        return s
    s.update(_layout(ids, E, c["tile"]))
    P, H = s["row_token"].numel(), c["H"]
    if c["op"] == "unpermute":
        s["rows"] = _normal(g, (P, H), 0.01)
        s["rows"][s["row_token"] < 0] = 1e4         # padding is never read
        s["add"] = [_normal(g, (T, H), 0.01) for _ in range(c["adds"])]
        return s
    if c["op"] == "finalize_bwd":
        K = ids.shape[1]
        w = torch.softmax(torch.randn(T, K, generator=g, device=DEV), 1)
        if c["wkind"] == "bf16":
            w = w.to(BF16)
        elif c["wkind"] == "packed":
            w = (ids.clamp(min=0) << 16) | (w.to(BF16).view(torch.int16).int() & 0xFFFF)
        s["weights"] = w.contiguous()
        s["rows"] = _normal(g, (P, H))
        s["rows"][s["row_token"] < 0] = 1e4
        s["drows"] = torch.zeros((P, H), dtype=BF16, device=DEV)
        s["dout"] = _normal(g, (T, H), 0.01) if c["dout"] else None
        if c["norm"]:
            s["dresidual_out"], s["dnorm_out"] = _normal(g, (T, H), 0.01), _normal(g, (T, H), 0.01)
            s["residual_out"] = _normal(g, (T, H), 2.0)
            s["gamma"] = (torch.rand(H, generator=g, device=DEV) + 0.5).to(BF16)
        return s
    I, gated = c["I"], c["gated"]
    x_rows, k, n = (T, H, I) if gated else (P, I, H)        # inputs of the product, width of its output
    s["cap"] = max(1, int(s["counts"].max()))
    s["x"] = _normal(g, (x_rows, k), 1.0 if gated else 0.4)
    s["w"] = _normal(g, (E, 2 * n if gated else n, k), k ** -0.5)
    s["dout"] = _normal(g, (P, n), 0.01)
    s["preact"] = _normal(g, (P, s["w"].shape[1])) if gated or c["act"] != "none" else None
    s["dx"] = torch.zeros((P, k), dtype=BF16, device=DEV)
    return s


# --------------------------------------------------------------- plain forms


def _act(z, name):
    """The activation and its derivative in 32 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.clamp(z, min=0), (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _weights(s):
    """Routing weights in 32 bits."""
    w = s["weights"]
    return (w << 16).view(F32) if s["case"]["wkind"] == "packed" else w.float()


def _plain_finalize_bwd(s):
    c, r = s["case"], {}
    dm = 0 if s["dout"] is None else s["dout"].float()
    if c["norm"]:
        x, dn, gamma = s["residual_out"].float(), s["dnorm_out"].float(), s["gamma"].float()
        inv = torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6)
        dy = dn * gamma
        dr = s["dresidual_out"].float() + inv * (dy - x * (inv * inv * (dy * x).mean(1, keepdim=True)))
        dm = dm + dr
        r["dresidual"] = dr.to(BF16)
        r["dgamma"] = (dn * x * inv).sum(0).to(BF16)
        r["dshared"] = dm.to(BF16) if c["dout"] else r["dresidual"]
    have = s["idx_map"] >= 0
    at = torch.where(have, s["idx_map"], torch.zeros_like(s["idx_map"])).long()
    dw = (s["rows"][at].float() * dm[:, None, :]).sum(2) * c["scale"]
    r["dweights"] = torch.where(have, dw, torch.zeros_like(dw))
    w = _weights(s) * c["scale"]
    P = s["rows"].shape[0]
    drows = torch.zeros((P + 1, c["H"]), dtype=BF16, device=DEV)
    drows[torch.where(have, at, torch.full_like(at, P)).reshape(-1)] = (w[:, :, None] * dm[:, None, :]).to(BF16).reshape(-1, c["H"])
    r["drows"] = drows[:P]
    return r


def _plain_unpermute(s):
    have = s["idx_map"] >= 0
    at = torch.where(have, s["idx_map"], torch.zeros_like(s["idx_map"])).long()
    rows = torch.where(have[:, :, None], s["rows"][at].float(), torch.zeros((), device=DEV))
    return {"out": sum([a.float() for a in s["add"]], rows.sum(1)).to(BF16)}


def _plain_gate_bwd(s):
    c = s["case"]
    have = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    w = torch.where(have, s["weights"], torch.zeros_like(s["weights"]))
    d = w * (s["dweights"] - (w * s["dweights"]).sum(1, keepdim=True))
    if c["kind"] == "sigmoid":
        d = d / (1 + torch.exp(s["logits"].gather(1, at)))
    d = torch.zeros((c["T"], c["E"]), device=DEV).scatter_add_(1, at, d)
    return {"dlogits": d if c["f32"] else d.to(BF16)}


def _plain_experts_bwd(s):
    """All experts' rows side by side in [E, capacity, :], batched products, back into the padded layout."""
    c, P = s["case"], s["dout"].shape[0]
    d = s["dout"].float()
    if c["gated"]:
        z = s["preact"].float()
        I = d.shape[1]
        a, da = _act(z[:, :I], c["act"])
        dz = torch.cat([d * z[:, I:] * da, d * a], dim=1)
    else:
        dz = d if s["preact"] is None else d * _act(s["preact"].float(), c["act"])[1]
    j = torch.arange(s["cap"], device=DEV)
    row = s["offsets"][:-1, None].long() + j
    valid = j < s["counts"][:, None]
    row = torch.where(valid, row, torch.zeros_like(row))
    src = torch.where(valid, s["row_token"][row].long(), torch.zeros_like(row)) if c["gated"] else row
    dz = torch.where(valid[:, :, None], dz[row], torch.zeros((), device=DEV))
    r = {"dweight": torch.matmul(dz.transpose(1, 2), s["x"][src].float()).to(BF16)}
    dx = torch.zeros((P + 1, s["x"].shape[1]), dtype=BF16, device=DEV)
    dx[torch.where(valid, row, torch.full_like(row, P))] = torch.matmul(dz, s["w"].float()).to(BF16)
    r["dx"] = dx[:P]
    if c["bias"]:
        r["dbias"] = dz.sum(1).to(BF16)
    return r


def _plain_adamw(s):
    h, bits = HYPER, s["case"]["bits"]
    b1, b2 = h["betas"]
    g = s["grad"].float()
    if bits == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square_()
    m = m.mul_(b1).add_(g, alpha=1 - b1)
    v = v.mul_(b2).add_(g * g, alpha=1 - b2)
    p = s["master"] if s["master"] is not None else s["param"].float()
    root = torch.sqrt(v)
    p = p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] / (1 - b1 ** h["step"]) * m / (root / math.sqrt(1 - b2 ** h["step"]) + h["eps"])
    if s["master"] is not None:
        s["master"].copy_(p)
    s["param"].copy_(p)
    if bits == 8:
        for key, x, floor in (("m", m, False), ("v", root, True)):
            code, scale = _f8(x.view(-1, BLOCK), floor)
            s[key].copy_(code.view(-1))
            s[key + "_scale"].copy_(scale)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


def run(state):
    s, op, c = state, state["op"], state["case"]
    if own:
        import moe_deferred_finalize_gb300 as mf
        if op == "finalize_bwd":
            norm = {k: s[k] for k in ("dresidual_out", "dnorm_out", "residual_out", "gamma")} if c["norm"] else {}
            return mf.moe_finalize_backward(s["rows"], s["idx_map"], s["weights"], c["wkind"], s["dout"], routed_scale=c["scale"], eps=1e-6, drows=s["drows"], **norm)
        if op == "unpermute":
            return {"out": mf.unpermute_tokens(s["rows"], s["idx_map"], add=s["add"])}
        if op == "gate_bwd":
            return {"dlogits": mf.topk_route_backward(s["dweights"], s["weights"], s["ids"], c["E"], c["kind"], logits=s["logits"], out_dtype=F32 if c["f32"] else BF16)}
        if op == "experts_bwd":
            if c["gated"]:
                return mf.expert_gated_ffn_backward(s["dout"], s["x"], s["row_token"], s["offsets"], s["counts"], s["w"], s["preact"], activation=c["act"],
                                                    want_dbias=c["bias"], dx=s["dx"])
            return mf.expert_linear_backward(s["dout"], s["x"], s["offsets"], s["counts"], s["w"], activation=c["act"], preact=s["preact"], want_dbias=c["bias"], dx=s["dx"])
        if "handle" not in s:
            s["handle"] = _bind_adamw(s)
        s["handle"](**HYPER)
        return _adamw_outputs(s)
    return {"finalize_bwd": _plain_finalize_bwd, "unpermute": _plain_unpermute, "gate_bwd": _plain_gate_bwd, "experts_bwd": _plain_experts_bwd,
            "adamw": _plain_adamw}[op](s)


# ------------------------------------------------------------------- floors


def work(case):
    c, op = case, case["op"]
    if op == "adamw":
        n = sum(_sizes(c))
        grad = 4 if c["f32"] else 2
        param = 2 + 8 if c["master"] else 2 * (4 if c["f32"] else 2)        # written, beside the master read and written; or both itself
        state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (grad + param + state), "flops": 0}
    T, E = c["T"], c["E"]
    k = min(c["topk"], E)
    t = T - min(c["pad"], T - 1)
    slots = t * k
    if op == "gate_bwd":
        return {"bytes": 4 * T * k * 3 + 4 * slots * (c["kind"] == "sigmoid") + T * E * (4 if c["f32"] else 2), "flops": 0}
    H = c["H"]
    if op == "unpermute":
        return {"bytes": 2 * H * (slots + T * (1 + c["adds"])) + 4 * T * k, "flops": 0}
    if op == "finalize_bwd":
        dense = c["dout"] + c["norm"] * (4 + c["dout"])     # dout; dnorm_out, dresidual_out, residual_out, dresidual and dshared
        words = 4 * T * k * 2 + (2 if c["wkind"] == "bf16" else 4) * T * k
        return {"bytes": 2 * H * (2 * slots + dense * T + 2 * c["norm"]) + words, "flops": 0}
    I, gated = c["I"], c["gated"]
    touched = E * (1 - (1 - k / E) ** t)
    weight = (2 if gated else 1) * I * H
    rows = slots * ((I + H + (2 * I if gated else 0)) if gated else (H + 2 * I + (H if c["act"] != "none" else 0)))
    return {"bytes": 2 * (touched * weight + E * weight + rows + (t * H if gated else 0) + E * c["bias"] * (2 * I if gated else H)), "flops": 4 * slots * weight}


# ------------------------------------------------- the definitions in 64 bits


def _act64(z, name):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z * (z > 0), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    b = 2 * math.sqrt(2 / math.pi)      # 0.5 (1 + tanh q) = sigmoid(2 q)
    s = torch.sigmoid(b * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * b * (1 + 0.134145 * z ** 2)


def _exact_finalize_bwd(s, c):
    T, H = s["idx_map"].shape[0], c["H"]
    out, dm = {}, torch.zeros((T, H), dtype=torch.float64, device=DEV)
    if s["dout"] is not None:
        dm += s["dout"]
    if c["norm"]:
        # norm = gamma r / q with q = sqrt(mean r^2 + eps); dq/dr_h = r_h / (H q)
        r, dn = s["residual_out"].double(), s["dnorm_out"].double()
        q = torch.sqrt(r.square().sum(1) / H + 1e-6)
        gr = torch.einsum("th,h,th->t", dn, s["gamma"].double(), r)
        dr = s["dresidual_out"].double() + dn * s["gamma"].double() / q[:, None] - r * (gr / (H * q ** 3))[:, None]
        dm += dr
        out = {"dresidual": dr, "dshared": dm, "dgamma": torch.einsum("th,th,t->h", dn, r, 1 / q)}
    w = s["weights"]
    if c["wkind"] == "packed":
        w = (w & 0xFFFF).to(torch.int16).view(BF16)
    out["drows"], out["dweights"] = torch.zeros(s["rows"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["idx_map"].shape, dtype=torch.float64, device=DEV)
    for k in range(w.shape[1]):
        t = (s["idx_map"][:, k] >= 0).nonzero()[:, 0]
        rows = s["idx_map"][t, k].long()
        out["drows"][rows] = c["scale"] * w[t, k].double()[:, None] * dm[t]
        out["dweights"][t, k] = c["scale"] * torch.linalg.vecdot(dm[t], s["rows"][rows].double())
    return out


def _exact_experts_bwd(s, c):
    P, n = s["dout"].shape
    out = {"dweight": torch.zeros(s["w"].shape, dtype=torch.float64, device=DEV), "dx": torch.zeros((P, s["x"].shape[1]), dtype=torch.float64, device=DEV)}
    if c["bias"]:
        out["dbias"] = torch.zeros(s["w"].shape[:2], dtype=torch.float64, device=DEV)
    for e, (first, count) in enumerate(zip(s["offsets"].tolist(), s["counts"].tolist())):
        if not count:
            continue
        rows = slice(first, first + count)
        d = s["dout"][rows].double()
        if c["gated"]:
            g, u = s["preact"][rows].double().split(n, dim=1)
            a, da = _act64(g, c["act"])
            d = torch.cat([d * da * u, d * a], dim=1)
        elif s["preact"] is not None:
            d = d * _act64(s["preact"][rows].double(), c["act"])[1]
        x = s["x"][s["row_token"][rows].long()] if c["gated"] else s["x"][rows]
        out["dx"][rows] = torch.einsum("rn,nk->rk", d, s["w"][e].double())
        out["dweight"][e] = torch.einsum("rn,rk->nk", d, x.double())
        if c["bias"]:
            out["dbias"][e] = d.sum(dim=0)
    return out


def _exact_adamw(s, c):
    b1, b2 = HYPER["betas"]
    t, lr = HYPER["step"], HYPER["lr"]
    g = s["grad"].double()
    if c["bits"] == 32:
        m, v = s["m"].double(), s["v"].double()
    else:
        m = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = (s["param"] if s["master"] is None else s["master"]).double()
    p = p - lr * (m / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + HYPER["eps"]) + HYPER["weight_decay"] * p)
    out = {"param": p}
    if s["master"] is not None:
        out["master"] = p
    if c["bits"] == 32:
        return dict(out, m=m, v=v)
    for key, x in (("m", m), ("v", v.sqrt())):
        top = x.view(-1, BLOCK).abs().max(dim=1).values / F8_MAX
        out[key + "_scale"] = top
        out[key] = (x.view(-1, BLOCK) / top.clamp(min=1e-300)[:, None]).view(-1)
    return out


def exact(case, seed):
    c, op = case, case["op"]
    s = prepare(case, seed)
    if op == "finalize_bwd":
        return _exact_finalize_bwd(s, c)
    if op == "experts_bwd":
        return _exact_experts_bwd(s, c)
    if op == "adamw":
        return _exact_adamw(s, c)
    if op == "unpermute":
        out = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
        for a in s["add"]:
            out += a
        token = s["row_token"].long()
        return {"out": out.index_add_(0, token[token >= 0], s["rows"][token >= 0].double())}
    out = torch.zeros((c["T"], c["E"]), dtype=torch.float64, device=DEV)
    for t, k in (((s["ids"][:, k] >= 0).nonzero()[:, 0], k) for k in range(s["ids"].shape[1])):
        w, dw = s["weights"][t].double(), s["dweights"][t].double()
        d = (w[:, k] * dw[:, k] - w[:, k] * torch.linalg.vecdot(w, dw))
        e = s["ids"][t, k].long()
        out[t, e] = d * torch.sigmoid(-s["logits"][t, e].double()) if c["kind"] == "sigmoid" else d
    return {"dlogits": out}
