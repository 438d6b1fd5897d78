"""The operators around the deferred MoE finalize, as they are measured.

An MoE layer of this framework runs: router product -> top-K gate -> row map -> expert products over the
permuted rows -> shared expert -> finalize.  Measured here are the pieces besides the gate and the finalize:

  linear      out = act(x W^T + b) + residual; bf16, or fp32 for router logits; its backward pass
  gated       h = act(x Wg^T) * (x Wu^T); its backward pass
  experts     the two products over rows grouped by expert (up: gated, gathers the token rows; down: linear)
  permute     expert ids [T, K] -> row map, row -> token map, expert offsets and counts
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


def listed():
    return [
        # router logits of one decoded token: 256 experts, fp32 out; the smallest call, latency counts
        {"name": "linear router T=1", "op": "linear", "T": 1, "K": 7168, "N": 256, "act": "none", "bias": False, "res": False, "f32": True},
        # a biased GELU layer with a residual on a ragged batch and sizes off every tile
        {"name": "linear gelu T=777", "op": "linear", "T": 777, "K": 1000, "N": 1048, "act": "gelu_tanh", "bias": True, "res": True, "f32": False},
        # the shared expert's down projection over a prefill chunk, residual added
        {"name": "linear down T=4096", "op": "linear", "T": 4096, "K": 2048, "N": 7168, "act": "none", "bias": False, "res": True, "f32": False},
        # training step of a biased GELU projection: dx, dW and db
        {"name": "linear backward T=2040", "op": "linear_bwd", "T": 2040, "K": 4096, "N": 4096, "act": "gelu_tanh", "bias": True},
        # the shared expert of one decoded token
        {"name": "gated T=1", "op": "gated", "T": 1, "H": 7168, "I": 2048, "act": "silu", "bias": False, "save": False},
        # the same over a mid-size ragged batch
        {"name": "gated T=300", "op": "gated", "T": 300, "H": 7168, "I": 2048, "act": "silu", "bias": False, "save": False},
        # a training forward over a long chunk, preactivations kept for the backward pass
        {"name": "gated T=4096", "op": "gated", "T": 4096, "H": 7168, "I": 2048, "act": "silu", "bias": True, "save": True},
        # its backward pass
        {"name": "gated backward T=4096", "op": "gated_bwd", "T": 4096, "H": 7168, "I": 2048, "act": "silu", "bias": True},
        # expert up projections of 16 decoded tokens, top-8 of 256: bound by the weights of the experts touched
        {"name": "experts up T=16", "op": "experts_up", "T": 16, "topk": 8, "E": 256, "H": 7168, "I": 2048, "act": "silu", "tile": 64, "pad": 0},
        # expert down projections of a prefill chunk, some of its rows padding of the batch
        {"name": "experts down T=4096", "op": "experts_down", "T": 4096, "topk": 8, "E": 256, "H": 7168, "I": 2048, "act": "silu", "tile": 128, "pad": 37},
        # the row map of a decode batch
        {"name": "permute T=256", "op": "permute", "T": 256, "topk": 8, "E": 256, "tile": 128, "pad": 0},
        # the row map of a long prefill
        {"name": "permute T=16384", "op": "permute", "T": 16384, "topk": 8, "E": 256, "tile": 128, "pad": 100},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "linear_bwd", "gated_bwd", "experts_up", "experts_down", "permute"])
    act = rng.choice(["silu", "gelu_tanh", "gelu", "relu"])
    if op == "permute":
        E = rng.choice([8, 60, 64, 128, 256, 384])
        T = _log_int(rng, 1, 16384)
        return {"op": op, "T": T, "topk": rng.choice([1, 2, 4, 6, 8]), "E": E, "tile": rng.choice([1, 8, 16, 64, 128]),
                "pad": rng.choice([0, 0, T // 10])}
    if op in ("experts_up", "experts_down"):
        E = rng.choice([8, 16, 60, 64, 128])
        T = _log_int(rng, 1, 2000)
        return {"op": op, "T": T, "topk": rng.choice([1, 2, 4, 8]), "E": E, "H": _log_int(rng, 256, 7168, 8),
                "I": _log_int(rng, 64, 2048, 8), "act": act, "tile": rng.choice([1, 16, 64, 128]), "pad": rng.choice([0, T // 10])}
    T = _log_int(rng, 1, 4096)
    bias = rng.random() < 0.5
    if op in ("gated", "gated_bwd"):
        c = {"op": op, "T": T, "H": _log_int(rng, 256, 7168, 8), "I": _log_int(rng, 64, 2048, 8), "act": act, "bias": bias}
        return dict(c, save=rng.random() < 0.5) if op == "gated" else c
    c = {"op": op, "T": T, "K": _log_int(rng, 128, 7168, 8), "N": _log_int(rng, 64, 7168, 8), "act": rng.choice(["none", act]), "bias": bias}
    return dict(c, res=rng.random() < 0.5, f32=rng.random() < 0.2) if op == "linear" else c


# ------------------------------------------------------------------ inputs


def _rows_bound(T, K, E, tile):
    """Rows that hold every padded layout of T*K slots over E experts."""
    n = T * K
    return (n + min(E, n) * (tile - 1)) // tile * tile


def _layout(ids, E, tile):
    """The padded layout of expert ids [T, K] (ids outside [0, E) get no row): row map [T, K], row -> token [P]
    (-1 on padding), first rows [E + 1] and row counts [E].  Rows of one expert stand in (token, slot) order."""
    T, K = ids.shape
    P = _rows_bound(T, K, E, tile)
    flat = ids.reshape(-1).long()
    ok = (flat >= 0) & (flat < E)
    key = torch.where(ok, flat, torch.full_like(flat, E))
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).index_add_(0, key, torch.ones_like(key))
    before = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + tile - 1) // tile * tile
    offsets = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offsets[1:] = torch.cumsum(padded, 0)
    order = torch.argsort(key, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(flat.numel(), device=ids.device)
    row = torch.where(ok, offsets[key] + rank - before[key], torch.full_like(rank, -1))
    token = torch.full((P + 1,), -1, dtype=torch.int32, device=ids.device)
    token[torch.where(ok, row, torch.full_like(row, P))] = (torch.arange(flat.numel(), device=ids.device) // K).int()
    token[P] = -1
    return {"idx_map": row.int().reshape(T, K), "row_token": token[:P].contiguous(), "offsets": offsets.int(),
            "counts": counts[:E].int()}


def _ids(c, g):
    """Top-k expert ids of a router with popular and rare experts; the last `pad` tokens are padding (-1)."""
    score = torch.randn(c["T"], c["E"], generator=g, device=DEV) + 0.5 * torch.randn(1, c["E"], generator=g, device=DEV)
    ids = score.topk(min(c["topk"], c["E"]), dim=1).indices.int()
    if c["pad"]:
        ids[c["T"] - c["pad"]:] = -1
    return ids.contiguous()


def _normal(g, shape, scale=1.0):
    return torch.empty(shape, dtype=BF16, device=DEV).normal_(0.0, scale, generator=g)


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": c, "op": c["op"]}
    if c["op"] == "permute":
        s["ids"] = _ids(c, g)
        return s
    T = c["T"]
    if c["op"] in ("linear", "linear_bwd"):
        K, N = c["K"], c["N"]
        s["x"], s["w"] = _normal(g, (T, K)), _normal(g, (N, K), K ** -0.5)
        s["bias"] = _normal(g, (N,), 0.5) if c["bias"] else None
        if c["op"] == "linear":
            s["res"] = _normal(g, (T, N), 2.0) if c["res"] else None
        else:
            s["dout"] = _normal(g, (T, N), 0.01)
            z = torch.mm(s["x"], s["w"].t())
            s["preact"] = (z + s["bias"]) if c["bias"] else z
        return s
    H, I = c["H"], c["I"]
    if c["op"] in ("gated", "gated_bwd"):
        s["x"], s["w"] = _normal(g, (T, H)), _normal(g, (2 * I, H), H ** -0.5)
        s["bias"] = _normal(g, (2 * I,), 0.5) if c["bias"] else None
        if c["op"] == "gated_bwd":
            s["dout"] = _normal(g, (T, I), 0.01)
            z = torch.mm(s["x"], s["w"].t())
            s["preact"] = (z + s["bias"]) if c["bias"] else z
        return s
    E = c["E"]
    s.update(_layout(_ids(c, g), E, c["tile"]))
    P = s["row_token"].numel()
    s["cap"] = max(1, int(s["counts"].max()))
    if c["op"] == "experts_up":
        s["x"], s["w"] = _normal(g, (T, H)), _normal(g, (E, 2 * I, H), H ** -0.5)
        s["out"] = torch.zeros((P, I), dtype=BF16, device=DEV)
    else:
        s["x"], s["w"] = _normal(g, (P, I), 0.4), _normal(g, (E, H, I), I ** -0.5)
        s["out"] = torch.zeros((P, H), dtype=BF16, device=DEV)
    return s


# --------------------------------------------------------------- plain forms


def _act(z, name):
    if name == "none":
        return z
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _plain_linear(s):
    c = s["case"]
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"out": y if c["f32"] else y.to(BF16)}


def _plain_backward(s, dz):
    """dx, dW and db of z = x W^T + b from dz [T, N] in 32 bits."""
    r = {"dx": torch.matmul(dz, s["w"].float()).to(BF16), "dweight": torch.matmul(dz.t(), s["x"].float()).to(BF16)}
    if s["bias"] is not None:
        r["dbias"] = dz.sum(0).to(BF16)
    return r


def _plain_gate(z, act, save):
    I = z.shape[-1] // 2
    r = {"out": (_act(z[..., :I], act) * z[..., I:]).to(BF16)}
    if save:
        r["preact"] = z.to(BF16)
    return r


def _plain_gated(s):
    c = s["case"]
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        z = z + s["bias"].float()
    return _plain_gate(z, c["act"], c["save"])


def _plain_gated_dz(s):
    z, dh = s["preact"].float(), s["dout"].float()
    I = dh.shape[1]
    g, u = z[:, :I], z[:, I:]
    return torch.cat([dh * u * _act_grad(g, s["case"]["act"]), dh * _act(g, s["case"]["act"])], dim=1)


def _plain_experts(s):
    """All experts' rows side by side in [E, capacity, :], one batched product, back into the padded layout."""
    c, P = s["case"], s["row_token"].numel()
    j = torch.arange(s["cap"], device=DEV)
    row = s["offsets"][:-1, None].long() + j
    valid = j < s["counts"][:, None]
    row = torch.where(valid, row, torch.zeros_like(row))
    src = s["row_token"][row].long() if c["op"] == "experts_up" else row
    src = torch.where(valid, src, torch.zeros_like(src))
    z = torch.matmul(s["x"][src].float(), s["w"].float().transpose(1, 2))
    y = _plain_gate(z, c["act"], False)["out"] if c["op"] == "experts_up" else z.to(BF16)
    out = torch.zeros((P + 1, y.shape[-1]), dtype=BF16, device=DEV)
    out[torch.where(valid, row, torch.full_like(row, P))] = y
    return {"out": out[:P]}


def run(state):
    s, op, c = state, state["op"], state["case"]
    if own:
        import moe_deferred_finalize_gb300 as mf
        if op == "linear":
            return {"out": mf.linear(s["x"], s["w"], bias=s["bias"], residual=s["res"], activation=c["act"],
                                     out_dtype=torch.float32 if c["f32"] else BF16)["out"]}
        if op == "gated":
            return mf.gated_ffn(s["x"], s["w"], bias=s["bias"], activation=c["act"], save_preact=c["save"])
        if op == "linear_bwd":
            return mf.linear_backward(s["dout"], s["x"], s["w"], activation=c["act"], preact=s["preact"], want_dbias=c["bias"])
        if op == "gated_bwd":
            return mf.gated_ffn_backward(s["dout"], s["x"], s["w"], s["preact"], activation=c["act"], want_dbias=c["bias"])
        if op == "experts_up":
            return {"out": mf.expert_gated_ffn(s["x"], s["row_token"], s["offsets"], s["counts"], s["w"], activation=c["act"], out=s["out"])}
        if op == "experts_down":
            return {"out": mf.expert_linear(s["x"], s["offsets"], s["counts"], s["w"], out=s["out"])}
        return mf.permute_tokens(s["ids"], c["E"], c["tile"])
    if op == "linear":
        return _plain_linear(s)
    if op == "gated":
        return _plain_gated(s)
    if op == "linear_bwd":
        return _plain_backward(s, s["dout"].float() * _act_grad(s["preact"].float(), c["act"]))
    if op == "gated_bwd":
        return _plain_backward(s, _plain_gated_dz(s))
    if op in ("experts_up", "experts_down"):
        return _plain_experts(s)
    return _layout(s["ids"], c["E"], c["tile"])


# ------------------------------------------------------------------- floors


def work(case):
    c, op = case, case["op"]
    T = c["T"]
    if op == "permute":
        n, E = T * min(c["topk"], c["E"]), c["E"]
        return {"bytes": 4 * (2 * n + _rows_bound(T, n // T, E, c["tile"]) + 2 * E + 1), "flops": 0}
    if op == "linear":
        K, N = c["K"], c["N"]
        return {"bytes": 2 * (T * K + N * K + N * c["bias"] + T * N * c["res"]) + (4 if c["f32"] else 2) * T * N, "flops": 2 * T * K * N}
    if op == "linear_bwd":
        K, N = c["K"], c["N"]
        dz = T * N * (1 + (c["act"] != "none"))
        return {"bytes": 2 * (dz + 2 * T * K + 2 * N * K + N * c["bias"]), "flops": 4 * T * K * N}
    H, I = c["H"], c["I"]
    if op == "gated":
        return {"bytes": 2 * (T * H + 2 * I * H + 2 * I * c["bias"] + T * I * (3 if c["save"] else 1)), "flops": 4 * T * H * I}
    if op == "gated_bwd":
        return {"bytes": 2 * (3 * T * I + 2 * T * H + 4 * I * H + 2 * I * c["bias"]), "flops": 8 * T * H * I}
    E, k, t = c["E"], min(c["topk"], c["E"]), T - c["pad"]
    touched, rows = E * (1 - (1 - k / E) ** t), t * k
    up = op == "experts_up"
    weights = touched * (2 * I * H if up else I * H)
    data = (t * H + rows * I) if up else rows * (I + H)
    return {"bytes": 2 * (weights + data) + 4 * (rows * up + 2 * E + 1), "flops": (4 if up else 2) * rows * H * I}


# ------------------------------------------------- the definitions in 64 bits


def _phi(z):
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


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
        return z * _phi(z), _phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # 0.5 (1 + tanh q) = sigmoid(2 q)
    b = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(b * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * b * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    c, op = case, case["op"]
    if op == "permute":     # whole numbers: nothing is rounded
        return None
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.dtype == BF16 and k != "w"}
    if op in ("experts_up", "experts_down"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        for e, (first, count) in enumerate(zip(s["offsets"].tolist(), s["counts"].tolist())):
            if count:
                rows = slice(first, first + count)
                x = d["x"][s["row_token"][rows].long()] if op == "experts_up" else d["x"][rows]
                z = x @ s["w"][e].double().mT
                if op == "experts_up":
                    g, u = z.chunk(2, dim=1)
                    z = _act64(g, c["act"])[0] * u
                out[rows] = z
        return {"out": out}
    w, b = s["w"].double(), d.get("bias")
    if op in ("linear", "gated"):
        z = torch.einsum("tk,nk->tn", d["x"], w)
        z = z if b is None else z + b
        if op == "gated":
            g, u = z.chunk(2, dim=1)
            r = {"out": _act64(g, c["act"])[0] * u}
            return dict(r, preact=z) if c["save"] else r
        y = _act64(z, c["act"])[0]
        return {"out": y if s["res"] is None else y + d["res"]}
    if op == "linear_bwd":
        dz = d["dout"] * _act64(d["preact"], c["act"])[1]
    else:
        g, u = d["preact"].chunk(2, dim=1)
        a, da = _act64(g, c["act"])
        dz = torch.cat([d["dout"] * da * u, d["dout"] * a], dim=1)
    r = {"dx": torch.einsum("tn,nk->tk", dz, w), "dweight": torch.einsum("tn,tk->nk", dz, d["x"])}
    return r if b is None else dict(r, dbias=dz.sum(dim=0))
