"""The MoE layer's training side on the GPU, against 64-bit references: the
gradients of the finalize, the row gather, the gate and the expert products,
the AdamW step, and a training step of all of them together."""
import pytest
import torch

import ffn_ref as R
import train_ref as T_

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NAN = float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def misaligned(t):
    """The same values two bytes (one element) off a 16-byte boundary."""
    n = t.numel()
    buf = torch.empty(n + 1, dtype=t.dtype, device=t.device)
    view = buf[1:].view(t.shape)
    view.copy_(t)
    return view


def routing(mf, g, T, K, E, tile, pad=0, absent=0.0):
    """ids of a router with popular experts, the last `pad` tokens without any, and
    the share `absent` of the slots; and their layout."""
    score = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g,
                                                                        device="cuda")
    ids = score.topk(K, dim=1).indices.int()
    if pad:
        ids[T - pad:] = -1
    if absent:
        ids[torch.rand(T, K, generator=g, device="cuda") < absent] = -1
    ids = ids.contiguous()
    return ids, mf.permute_tokens(ids, E, tile)


def poisoned(g, m, P, H, scale=1.0):
    """Rows of the layout, NaN where no slot has one."""
    rows = normal(g, P, H, scale=scale)
    rows[m["row_token"] < 0] = NAN
    return rows


# ------------------------------------------------------------- finalize


FINALIZE = [
    # T, K, E, H, tile, wkind, norm, dout, dres, absent
    (1, 1, 1, 8, 1, "fp32", False, True, False, 0.0),
    (1, 8, 16, 7168, 32, "packed", True, False, True, 0.0),
    (5, 2, 4, 40, 1, "bf16", True, True, False, 0.3),
    (13, 3, 8, 1001, 16, "fp32", True, True, True, 0.2),
    (16, 8, 384, 7168, 64, "fp32", True, False, True, 0.0),
    (40, 9, 16, 264, 8, "packed", False, True, True, 0.5),
    (77, 32, 40, 520, 1, "fp32", True, True, True, 0.1),
    (300, 4, 8, 4104, 16, "bf16", True, True, True, 0.0),
    (700, 2, 8, 33000, 1, "fp32", False, True, False, 0.0),
    (3, 2, 4, 20001, 1, "fp32", True, True, True, 0.0),
    (1300, 6, 60, 2048, 16, "packed", True, False, False, 1.0),
    # rows of several vectors a thread, over a cluster that goes round the tokens
    (3, 2, 4, 240000, 1, "fp32", True, True, True, 0.0),
    (90, 2, 4, 70000, 1, "fp32", True, True, True, 0.1),
    (60, 3, 4, 12008, 1, "bf16", True, False, True, 0.1),
    # both sides of the number of tokens whose dgamma is taken directly
    (32, 2, 4, 7168, 1, "fp32", True, True, True, 0.1),
    (33, 2, 4, 7168, 1, "fp32", True, True, True, 0.1),
    (32, 2, 4, 24, 1, "fp32", True, True, True, 0.1),
    (16, 2, 4, 2049, 1, "fp32", True, True, True, 0.1),
    (17, 2, 4, 2049, 1, "fp32", True, True, True, 0.1),
    (1, 2, 4, 7168, 1, "fp32", True, True, True, 0.5),
]


def finalize_inputs(mf, case, seed=0):
    T, K, E, H, tile, wkind, norm, dout, dres, absent = case
    g = gen(seed)
    ids, m = routing(mf, g, T, K, E, tile, absent=absent)
    P = m["row_token"].numel()
    w = torch.rand(T, K, generator=g, device="cuda") - 0.2
    if wkind == "bf16":
        w = w.to(BF16)
    elif wkind == "packed":
        w = mf.pack_topk_ids(ids, w)
    kw = {}
    if dres:
        kw["dresidual_out"] = normal(g, T, H, scale=0.1)
    if norm:
        kw.update(dnorm_out=normal(g, T, H, scale=0.1), residual_out=normal(g, T, H, scale=2.0),
                  gamma=normal(g, H))
    return poisoned(g, m, P, H), m, w.contiguous(), normal(g, T, H, scale=0.1) if dout else None, kw


def check_finalize(case, rows, m, w, dout, kw, res, drows0, scale, eps):
    wkind = case[5]
    idx = m["idx_map"]
    ref = T_.finalize_backward(rows, idx, T_.decoded(w, wkind), scale, dout,
                               kw.get("dresidual_out"), kw.get("dnorm_out"),
                               kw.get("residual_out"), kw.get("gamma"), eps)
    for name in ("dweights", "dresidual", "dshared", "dgamma"):
        assert (name in res) == (name in ref), name
        if name in ref:
            T_.check(res[name], ref[name], f"{case} {name}")
    have = idx >= 0
    at = idx[have].long()
    T_.check(res["drows"][at], tuple(v[have] for v in ref["drows"]), f"{case} drows")
    untouched = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    untouched[at] = False
    assert torch.equal(res["drows"][untouched], drows0[untouched])


@pytest.mark.parametrize("case", FINALIZE, ids=str)
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "misaligned"])
def test_finalize_backward(cuda_lib, case, off):
    mf = cuda_lib
    rows, m, w, dout, kw = finalize_inputs(mf, case)
    if off:
        rows, dout = misaligned(rows), None if dout is None else misaligned(dout)
        kw = {k: misaligned(v) for k, v in kw.items()}
        if case[3] > 32768 and case[6]:      # too long for single values
            with pytest.raises(mf.MoefError, match="SHAPE"):
                mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, **kw)
            return
    drows0 = torch.full_like(rows, 7.0)
    drows = drows0.clone()
    res = mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, routed_scale=2.5,
                                   eps=1e-5, drows=drows, **kw)
    check_finalize(case, rows, m, w, dout, kw, res, drows0, 2.5, 1e-5)
    again = mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, routed_scale=2.5,
                                     eps=1e-5, drows=drows0.clone(), **kw)
    for k in res:       # equal calls give equal bits
        assert torch.equal(res[k], again[k]), k


def test_finalize_backward_of_forward(cuda_lib):
    """Against differences of the 64-bit forward formula, through the GPU forward's
    own residual_out."""
    mf, g = cuda_lib, gen(3)
    T, K, E, H = 3, 2, 4, 16
    ids, m = routing(mf, g, T, K, E, 1)
    P = m["row_token"].numel()
    rows, w = normal(g, P, H), torch.rand(T, K, generator=g, device="cuda")
    shared, residual, gamma = normal(g, T, H), normal(g, T, H), normal(g, H)
    fwd = mf.moe_finalize(rows, m["idx_map"], w, "fp32", shared, routed_scale=1.5,
                          residual=residual, gamma=gamma, eps=1e-3)
    d = {k: normal(g, T, H) for k in ("out", "residual_out", "norm_out")}
    res = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", d["out"], routed_scale=1.5,
                                   dresidual_out=d["residual_out"], dnorm_out=d["norm_out"],
                                   residual_out=fwd["residual_out"], gamma=gamma, eps=1e-3)
    x = {"drows": rows, "dweights": w, "dshared": shared, "dresidual": residual, "dgamma": gamma}
    x = {k: v.double() for k, v in x.items()}

    def loss(x):
        mm = 1.5 * (x["dweights"][:, :, None] * x["drows"][m["idx_map"].long()]).sum(1) + \
            x["dshared"]
        # the forward's rounding of residual_out counts as the identity
        base = 1.5 * (w.double()[:, :, None] * rows.double()[m["idx_map"].long()]).sum(1) + \
            shared.double() + residual.double()
        r = mm + x["dresidual"] + (fwd["residual_out"].double() - base)
        n = r * (r.square().mean(1, keepdim=True) + 1e-3) ** -0.5 * x["dgamma"]
        return (mm * d["out"].double() + r * d["residual_out"].double() +
                n * d["norm_out"].double()).sum()

    for name, v in x.items():
        h = 1e-5
        for i in range(0, v.numel(), max(1, v.numel() // 12)):
            up, down = v.clone(), v.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            diff = (loss({**x, name: up}) - loss({**x, name: down})) / (2 * h)
            got = res[name].double().view(-1)[i]
            # the rounding of the gradient and h^2 times a third derivative of order 10
            assert abs(got - diff) <= 2 ** -8 * abs(diff) + 1e-4, (name, i, got, diff)


def test_finalize_backward_wants_and_in_place(cuda_lib):
    mf = cuda_lib
    case = (20, 4, 8, 256, 8, "fp32", True, True, True, 0.1)
    rows, m, w, dout, kw = finalize_inputs(mf, case)
    full = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, **kw)
    one = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, want_drows=False,
                                   want_dgamma=False, **kw)
    assert set(one) == {"dweights", "dshared", "dresidual"}
    assert torch.equal(one["dweights"], full["dweights"])
    one = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, want_dweights=False, **kw)
    assert torch.equal(one["drows"][m["idx_map"][m["idx_map"] >= 0].long()],
                       full["drows"][m["idx_map"][m["idx_map"] >= 0].long()])
    a, b = dout.clone(), kw["dresidual_out"].clone()
    one = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", a,
                                   **{**kw, "dresidual_out": b}, dshared=a, dresidual=b)
    for k in ("dshared", "dresidual", "dweights", "dgamma"):
        assert torch.equal(one[k], full[k]), k
    same = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", **kw)
    assert same["dshared"] is same["dresidual"]


def test_finalize_backward_special_values(cuda_lib):
    """Zero rows under the norm, infinities and NaN stay in their own tokens."""
    mf = cuda_lib
    case = (12, 2, 4, 64, 1, "fp32", True, True, True, 0.0)
    rows, m, w, dout, kw = finalize_inputs(mf, case)
    kw["residual_out"][0] = 0
    clean = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, **kw)
    assert torch.isfinite(clean["dresidual"]).all()
    dout[3, 5], kw["dnorm_out"][4, 7] = float("inf"), NAN
    res = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, **kw)
    keep = [t for t in range(12) if t not in (3, 4)]
    for k in ("dweights", "dresidual", "dshared"):
        assert torch.equal(res[k][keep], clean[k][keep]), k
    assert torch.isnan(res["dresidual"][4]).all() and torch.isinf(res["dshared"][3, 5])


def test_finalize_backward_without_tokens(cuda_lib):
    mf = cuda_lib
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    res = mf.moe_finalize_backward(torch.ones((4, 64), dtype=BF16, device="cuda"),
                                   torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                   torch.empty((0, 2), device="cuda"), "fp32", e, dnorm_out=e,
                                   residual_out=e,
                                   gamma=torch.ones(64, dtype=BF16, device="cuda"))
    assert not res["dgamma"].any() and res["dweights"].shape == (0, 2)


# ------------------------------------------------------------ unpermute


@pytest.mark.parametrize("T,K,E,H,tile,adds,absent",
                         [(1, 1, 1, 1, 1, 0, 0.0), (7, 3, 8, 33, 4, 1, 0.3),
                          (16, 8, 256, 7168, 16, 2, 0.0), (50, 32, 64, 200, 1, 2, 0.5),
                          (513, 9, 16, 1032, 8, 0, 0.0), (40, 4, 8, 64, 1, 1, 1.0)])
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "misaligned"])
def test_unpermute(cuda_lib, T, K, E, H, tile, adds, absent, off):
    mf, g = cuda_lib, gen(T + H)
    _, m = routing(mf, g, T, K, E, tile, absent=absent)
    rows = poisoned(g, m, m["row_token"].numel(), H)
    add = [normal(g, T, H) for _ in range(adds)]
    if off:
        rows, add = misaligned(rows), [misaligned(a) for a in add]
    ref = T_.unpermute(rows, m["idx_map"], add)
    T_.check(mf.unpermute_tokens(rows, m["idx_map"], add=add), ref, "out")
    if adds:
        got = mf.unpermute_tokens(rows, m["idx_map"], add=add, out=add[-1])
        assert got is add[-1]
        T_.check(got, ref, "in place")


@pytest.mark.parametrize("H", [64, 33])
def test_unpermute_second_addend_alone(cuda_lib, H):
    """Either addend may be missing."""
    mf, g = cuda_lib, gen(H)
    _, m = routing(mf, g, 20, 3, 8, 4, absent=0.2)
    rows, add = poisoned(g, m, m["row_token"].numel(), H), normal(g, 20, H)
    ref = T_.unpermute(rows, m["idx_map"], [add])
    for adds in ((None, add), (add, None)):
        T_.check(mf.unpermute_tokens(rows, m["idx_map"], add=adds), ref, "out")


def test_unpermute_indices_outside(cuda_lib):
    """Row numbers outside [0, P), the extremes among them, add nothing."""
    mf = cuda_lib
    rows = torch.ones((4, 16), dtype=BF16, device="cuda")
    idx = torch.tensor([[0, 4], [-1, 3], [2 ** 31 - 1, -2 ** 31], [3, 3]], dtype=torch.int32,
                       device="cuda")
    out = mf.unpermute_tokens(rows, idx)
    assert out[:, 0].tolist() == [1, 1, 0, 2]
    assert not mf.unpermute_tokens(rows[:0], idx).any()


def test_unpermute_is_the_gradient_of_the_gather(cuda_lib):
    """<rows, x[row_token]> and <unpermute(rows), x> are the same number."""
    mf, g = cuda_lib, gen(5)
    T, K, E, H = 30, 4, 8, 64
    _, m = routing(mf, g, T, K, E, 8, pad=3)
    token = m["row_token"]
    x, rows = normal(g, T, H), normal(g, token.numel(), H)
    a = (rows.double() * torch.where((token >= 0)[:, None], x[token.long()].double(), 0.0)).sum()
    out = mf.unpermute_tokens(rows, m["idx_map"])
    b = (out.double() * x.double()).sum()
    assert abs(a - b) <= 2 ** -8 * (out.double() * x.double()).abs().sum()


# ----------------------------------------------------------------- gate


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (3, 7, 7), (33, 256, 8), (50, 60, 6), (20, 1024, 32),
                                   (9, 64, 1), (5000, 8, 2)])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_gate_backward(cuda_lib, T, E, K, kind, dtype):
    mf, g = cuda_lib, gen(T + E)
    logits = torch.randn(T, E, generator=g, device="cuda") * 4
    route = mf.topk_route(logits, K, kind)
    ids = route["expert_ids"].clone()
    if T > 2:
        ids[1] = -1
        ids[2, 0] = E
    dw = torch.randn(T, K, generator=g, device="cuda")
    got = mf.topk_route_backward(dw, route["weights"], ids, E, kind, logits=logits,
                                 out_dtype=dtype)
    T_.check(got, T_.gate_backward(dw, route["weights"], ids, E, kind, logits, dtype == F32),
             "dlogits")


def test_gate_backward_of_forward(cuda_lib):
    """Against differences of the 64-bit gate, far logits among them."""
    mf, g = cuda_lib, gen(9)
    logits = torch.randn(6, 12, generator=g, device="cuda") * 3
    logits[2] -= 60
    logits[3] += 60
    dw = torch.randn(6, 4, generator=g, device="cuda")
    for kind in ("softmax", "sigmoid"):
        route = mf.topk_route(logits, 4, kind)
        ids = route["expert_ids"].long()
        got = mf.topk_route_backward(dw, route["weights"], route["expert_ids"], 12, kind,
                                     logits=logits, out_dtype=F32)

        def loss(z):
            z = z.gather(1, ids)
            w = torch.softmax(z, 1) if kind == "softmax" else \
                torch.softmax(torch.nn.functional.logsigmoid(z), 1)
            return (w * dw.double()).sum(1)

        z, h = logits.double(), 1e-5
        for e in range(12):
            d = torch.zeros_like(z)
            d[:, e] = h
            diff = (loss(z + d) - loss(z - d)) / (2 * h)
            assert ((got[:, e].double() - diff).abs() <= 1e-5).all(), (kind, e)


def test_gate_backward_same_expert_twice(cuda_lib):
    mf = cuda_lib
    ids = torch.tensor([[2, 2, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25]], device="cuda")
    dw = torch.tensor([[1.0, 2.0, -4.0]], device="cuda")
    # sum w dw = 0: d = w dw
    got = mf.topk_route_backward(dw, w, ids, 4, "softmax", out_dtype=F32)
    assert got.tolist() == [[-1.0, 0.0, 1.0, 0.0]]


# -------------------------------------------------------------- experts


EXPERTS = [
    # T, K, E, H (inputs), I, tile, act, bias, gated, pad
    (1, 1, 1, 8, 8, 1, "none", True, False, 0),
    (1, 2, 4, 64, 24, 1, "silu", False, True, 0),
    (5, 2, 8, 136, 40, 1, "gelu", True, True, 1),
    (33, 2, 4, 256, 128, 16, "silu", False, True, 0),
    (64, 4, 60, 512, 72, 1, "gelu_tanh", False, True, 3),
    (100, 2, 8, 1536, 520, 1, "relu", True, True, 3),
    (130, 2, 3, 264, 300, 128, "none", False, False, 0),
    (257, 3, 5, 128, 1000, 1, "gelu", True, False, 2),
    (300, 8, 64, 512, 256, 16, "silu", False, True, 10),
    (1000, 2, 4, 1024, 384, 64, "none", True, False, 0),
    (2000, 1, 2, 320, 640, 1, "silu", False, True, 0),
    # sizes the copies cannot take
    (40, 2, 4, 37, 24, 1, "silu", True, True, 1),
    (90, 2, 4, 64, 33, 8, "none", True, False, 0),
    (70, 3, 6, 131, 67, 1, "gelu", False, False, 2),
]


def expert_inputs(mf, case, seed=0):
    T, K, E, H, I, tile, act, bias, gated, pad = case
    g = gen(seed)
    _, m = routing(mf, g, T, K, E, tile, pad=pad)
    P = m["row_token"].numel()
    n = I
    x = normal(g, T, H) if gated else poisoned(g, m, P, H)
    w = normal(g, E, 2 * n if gated else n, H, scale=H ** -0.5)
    dout = poisoned(g, m, P, n, scale=0.1)
    preact = poisoned(g, m, P, w.shape[1]) if gated or act != "none" else None
    return m, x, w, dout, preact


def expert_call(mf, case, m, x, w, dout, preact, **kw):
    act, bias, gated = case[6], case[7], case[8]
    if gated:
        return mf.expert_gated_ffn_backward(dout, x, m["row_token"], m["offsets"], m["counts"], w,
                                            preact, activation=act, want_dbias=bias, **kw)
    return mf.expert_linear_backward(dout, x, m["offsets"], m["counts"], w, activation=act,
                                     preact=preact, want_dbias=bias, **kw)


def check_experts(case, m, x, w, dout, preact, res, dx0=None, what=""):
    ref = T_.expert_backward(dout, x, m["row_token"] if case[8] else None, m["offsets"],
                             m["counts"], w, preact, case[6], case[8])
    for k, v in res.items():
        T_.check(v, ref[k], f"{case} {what} {k}")
    if dx0 is not None:
        none = m["row_token"] < 0
        assert torch.equal(res["dx"][none], dx0[none])


@pytest.mark.parametrize("case", EXPERTS, ids=str)
def test_expert_backward(cuda_lib, case):
    mf = cuda_lib
    m, x, w, dout, preact = expert_inputs(mf, case)
    dx0 = torch.full((dout.shape[0], w.shape[2]), 3.0, dtype=BF16, device="cuda")
    res = expert_call(mf, case, m, x, w, dout, preact, dx=dx0.clone())
    check_experts(case, m, x, w, dout, preact, res, dx0)
    again = expert_call(mf, case, m, x, w, dout, preact, dx=dx0.clone())
    for k in res:
        assert torch.equal(res[k], again[k]), k
    assert mf.lost_waits() == 0


@pytest.mark.parametrize("which", ["x", "w", "dout", "preact", "dx", "dweight"])
@pytest.mark.parametrize("gated", [False, True])
def test_expert_backward_misaligned(cuda_lib, which, gated):
    mf = cuda_lib
    case = (60, 2, 4, 128, 72, 8, "silu", True, gated, 2)
    m, x, w, dout, preact = expert_inputs(mf, case)
    t = dict(x=x, w=w, dout=dout, preact=preact)
    kw = {}
    if which in t:
        t[which] = misaligned(t[which])
    else:
        shape = (dout.shape[0], 128) if which == "dx" else w.shape
        kw[which] = misaligned(torch.zeros(shape, dtype=BF16, device="cuda"))
    res = expert_call(mf, case, m, **t, **kw)
    check_experts(case, m, **t, res=res, what=which)


def test_expert_backward_linear_gathered(cuda_lib):
    """expert_linear with a row map, and row numbers outside [0, T): rows of zeros."""
    mf, g = cuda_lib, gen(4)
    T, K, E, H, N = 50, 2, 4, 64, 48
    _, m = routing(mf, g, T, K, E, 4)
    P = m["row_token"].numel()
    token = m["row_token"].clone()
    token[int(m["offsets"][1])] = T
    token[int(m["offsets"][2])] = -5
    x, w, dout = normal(g, T, H), normal(g, E, N, H), normal(g, P, N)
    preact = normal(g, P, N)
    for act, pre in (("none", None), ("gelu", preact)):
        res = mf.expert_linear_backward(dout, x, m["offsets"], m["counts"], w, row_token=token,
                                        activation=act, preact=pre, want_dbias=True)
        ref = T_.expert_backward(dout, x, token, m["offsets"], m["counts"], w, pre, act, False)
        for k in res:
            T_.check(res[k], ref[k], k)


def test_expert_backward_without_a_workspace(cuda_lib):
    """dout as dz: none is needed; dbias alone needs none either."""
    mf = cuda_lib
    case = (40, 2, 4, 64, 48, 16, "none", True, False, 0)
    m, x, w, dout, _ = expert_inputs(mf, case)
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    res = expert_call(mf, case, m, x, w, dout, None, workspace=none)
    check_experts(case, m, x, w, dout, None, res)
    case = (40, 2, 4, 64, 48, 16, "silu", True, True, 0)
    m, x, w, dout, preact = expert_inputs(mf, case)
    res = expert_call(mf, case, m, x, w, dout, preact, workspace=none, want_dx=False,
                      want_dweight=False)
    assert set(res) == {"dbias"}
    check_experts(case, m, x, w, dout, preact, res)
    with pytest.raises(mf.MoefError):
        expert_call(mf, case, m, x, w, dout, preact, workspace=none)


@pytest.mark.parametrize("sizes", [(40000, 200, 64), (300, 40, 1000), (5000, 2000, 2000)], ids=str)
def test_expert_backward_products_side_by_side(cuda_lib, sizes):
    """dweight begins while dx runs: both are complete for what comes next on the stream, a
    dx of many rounds beside a dweight of few tiles and the other way round, in plain calls
    and in a replayed graph."""
    mf, g = cuda_lib, gen(31)
    T, n, H = sizes
    _, m = routing(mf, g, T, 1, 4, 16)
    P = m["row_token"].numel()
    x, w = normal(g, T, H), normal(g, 4, 2 * n, H, scale=H ** -0.5)
    dout, preact = poisoned(g, m, P, n, scale=0.1), poisoned(g, m, P, 2 * n)

    def call(**kw):
        return mf.expert_gated_ffn_backward(dout, x, m["row_token"], m["offsets"], m["counts"], w,
                                            preact, **kw)

    dx0 = torch.zeros(P, H, dtype=BF16, device="cuda")
    dx = call(dx=dx0.clone(), want_dweight=False)["dx"]
    dweight = call(want_dx=False)["dweight"]
    out, dw = dx0.clone(), torch.empty_like(w)

    def step():
        out.zero_()
        dw.zero_()
        call(dx=out, dweight=dw)
        return out.clone(), dw.clone()

    for _ in range(10):
        a, b = step()
        sums = mf.unpermute_tokens(out, m["idx_map"])
        assert torch.equal(a, dx) and torch.equal(b, dweight)
        assert torch.equal(sums, mf.unpermute_tokens(dx, m["idx_map"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = step()
    for _ in range(10):
        a.zero_()
        b.zero_()
        graph.replay()
        assert torch.equal(a, dx) and torch.equal(b, dweight)
    assert mf.lost_waits() == 0


@pytest.mark.parametrize("sizes", [(40000, 200, 64), (300, 40, 1000), (5000, 1000, 2000)], ids=str)
def test_finalize_may_read_dx_early_behind_dweight(cuda_lib, sizes):
    """moe_finalize with routing_ready reads its weights before the kernel in front of it,
    dweight's, has finished: every kernel before that one must be complete by then.  dx,
    as bf16 weights, is the last of them."""
    mf, g = cuda_lib, gen(32)
    T, n, H = sizes
    _, m = routing(mf, g, T, 1, 4, 16)
    P = m["row_token"].numel()
    x, w = normal(g, T, H), normal(g, 4, 2 * n, H, scale=H ** -0.5)
    dout, preact = poisoned(g, m, P, n, scale=0.1), poisoned(g, m, P, 2 * n)
    zeros = torch.zeros(P, H, dtype=BF16, device="cuda")
    dx, dw = zeros.clone(), torch.empty_like(w)
    workspace = torch.empty(mf.expert_backward_workspace_bytes(P, 2 * n, H), dtype=torch.uint8,
                            device="cuda")
    F = P * H // 8 // 64 * 64       # the last rows of dx too, as 8 weights a token
    rows = normal(g, 64, 64)
    idx = torch.arange(F * 8, device="cuda").remainder(64).view(F, 8).int()
    weights = dx.view(-1)[-F * 8:].view(F, 8)
    out = torch.empty(F, 64, dtype=BF16, device="cuda")

    def call(ready):
        dx.copy_(zeros)
        mf.expert_gated_ffn_backward(dout, x, m["row_token"], m["offsets"], m["counts"], w, preact,
                                     dx=dx, dweight=dw, workspace=workspace)
        return mf.moe_finalize(rows, idx, weights, "bf16", shared, routing_ready=ready,
                               out=out)["out"].clone()

    shared = torch.zeros(F, 64, dtype=BF16, device="cuda")
    want = call(False)
    torch.cuda.synchronize()
    for _ in range(10):
        assert torch.equal(call(True), want)
    assert mf.lost_waits() == 0


def test_expert_backward_odd_layouts(cuda_lib):
    """Experts out of order, with gaps, without rows, past the buffer, in front of it."""
    mf, g = cuda_lib, gen(6)
    P, E, H, N = 300, 6, 64, 40
    offsets = torch.tensor([200, 0, 90, -4, 290, 50, 0], dtype=torch.int32, device="cuda")
    counts = torch.tensor([70, 33, 0, 20, 50, -3], dtype=torch.int32, device="cuda")
    x, w, dout = normal(g, P, H), normal(g, E, N, H), normal(g, P, N)
    res = mf.expert_linear_backward(dout, x, offsets, counts, w, want_dbias=True)
    ref = T_.expert_backward(dout, x, None, offsets, counts, w, None, "none", False)
    for k in res:
        T_.check(res[k], ref[k], k)


def test_expert_backward_without_rows(cuda_lib):
    mf = cuda_lib
    w = torch.ones((3, 8, 16), dtype=BF16, device="cuda")
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty((0, 16), dtype=BF16, device="cuda")
    res = mf.expert_linear_backward(e[:, :8].contiguous(), e, zero, zero[:3], w, want_dbias=True)
    assert not res["dweight"].any() and not res["dbias"].any() and res["dx"].shape == (0, 16)
    # rows of padding alone
    x = torch.full((20, 16), NAN, dtype=BF16, device="cuda")
    res = mf.expert_linear_backward(x[:, :8].contiguous(), x, zero, zero[:3], w, want_dbias=True)
    assert not res["dweight"].any() and not res["dbias"].any()


@pytest.mark.parametrize("gated", [False, True])
def test_expert_forward_keeps_preactivations(cuda_lib, gated):
    mf, g = cuda_lib, gen(8)
    for T, H, I in ((40, 64, 48), (30, 37, 21)):
        _, m = routing(mf, g, T, 2, 4, 8)
        P = m["row_token"].numel()
        x = normal(g, T, H)
        w = normal(g, 4, 2 * I if gated else I, H, scale=H ** -0.5)
        bias = normal(g, 4, w.shape[1])
        pre0 = torch.full((P, w.shape[1]), 5.0, dtype=BF16, device="cuda")
        pre = pre0.clone()
        if gated:
            out = mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w, bias=bias,
                                      preact=pre)
            plain = mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w, bias=bias)
        else:
            kw = dict(row_token=m["row_token"], bias=bias, activation="gelu")
            out = mf.expert_linear(x, m["offsets"], m["counts"], w, preact=pre, **kw)
            plain = mf.expert_linear(x, m["offsets"], m["counts"], w, **kw)
        have = m["row_token"] >= 0
        assert torch.equal(out[have], plain[have])
        assert torch.equal(pre[~have], pre0[~have])
        for e in range(4):
            rows = slice(int(m["offsets"][e]), int(m["offsets"][e]) + int(m["counts"][e]))
            z, tol = R.product(x[m["row_token"][rows].long()], w[e], bias[e])
            T_.check(pre[rows], T_.rounded(z, tol), "preact")


# ---------------------------------------------------------------- AdamW


ADAMW_SIZES = (1, 255, 256, 257, 5000, 8, 1024 * 17 + 3, 0, 700)
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def adamw_inputs(mf, sizes, bits, master, param, grad, off, seed=0):
    g = gen(seed)
    move = misaligned if off else (lambda t: t)
    params = [move(normal(g, n, dtype=F32).to(param)) for n in sizes]
    grads = [move(normal(g, n, scale=0.01, dtype=F32).to(grad)) for n in sizes]
    for t in grads:
        t[::7] = 0
    state = mf.adamw_state(params, bits, master)
    if off:
        state = {k: [misaligned(t) if t.dtype != F8 else misaligned(t.view(torch.uint8)).view(F8)
                     for t in ts] for k, ts in state.items()}
    return params, grads, state


def adamw_states(state, i):
    """m and v of tensor i as the numbers they stand for."""
    m, v = state["exp_avg"][i].double(), state["exp_avg_sq"][i].double()
    if "exp_avg_scale" in state:
        n = m.numel()
        m = m * state["exp_avg_scale"][i].double().repeat_interleave(256)[:n]
        v = (v * state["exp_avg_sq_scale"][i].double().repeat_interleave(256)[:n]) ** 2
    return m, v


def check_adamw(before, params, state, i, bits, param, master):
    ref = before
    T_.check(params[i], ref["param"], f"param {i}")
    if master:
        T_.check(state["masters"][i], ref["master"], f"master {i}")
        assert torch.equal(params[i], state["masters"][i].to(BF16))
    if bits == 32:
        T_.check(state["exp_avg"][i], ref["m"], f"m {i}")
        T_.check(state["exp_avg_sq"][i], ref["v"], f"v {i}")
        return
    for key, name in (("exp_avg", "m"), ("exp_avg_sq", "root")):
        codes, scales = T_.code(*ref[name], root=name == "root")
        T_.check(state[key + "_scale"][i], scales, f"{key} scale {i}")
        T_.check(state[key][i], codes, f"{key} {i}")
        if name == "root":
            assert (state[key][i].double()[ref["root"][0] > 1e-30] > 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [(BF16, BF16, False), (BF16, BF16, True),
                                               (BF16, F32, False), (BF16, F32, True),
                                               (F32, F32, False), (F32, BF16, False)], ids=str)
@pytest.mark.parametrize("off", [False, True], ids=["aligned", "misaligned"])
def test_adamw(cuda_lib, bits, param, grad, master, off):
    mf = cuda_lib
    params, grads, state = adamw_inputs(mf, ADAMW_SIZES, bits, master, param, grad, off)
    bound = mf.bind_adamw(params, grads, **state)
    for step in (1, 2, 3):
        refs = []
        for i in range(len(params)):
            m, v = adamw_states(state, i)
            p = (state["masters"] if master else params)[i].double()
            refs.append(T_.adamw(p, grads[i].double(), m, v, HYPER["lr"], HYPER["betas"],
                                 HYPER["eps"], HYPER["weight_decay"], step,
                                 param_bf16=param == BF16))
        bound(step=step, **HYPER)
        for i, ref in enumerate(refs):
            check_adamw(ref, params, state, i, bits, param, master)
        for t in grads:
            t.mul_(-0.5)


def test_adamw_codes_are_rounded_quotients(cuda_lib):
    """8-bit states against torch's fp32 operations, whose quotient and root are
    rounded to nearest.  The kernel's quotient is too; its root may be off by a unit
    in the last place, 2^-23 relative, which changes a code where one of the 8
    borders an octave lies within that: fewer than 2 * 2^-23 * 8 / ln 2 of the values
    = 2.8e-6, 3 in 2^20."""
    mf, g, n = cuda_lib, gen(7), 2 ** 20
    p = [normal(g, n)]
    grad = [normal(g, n, scale=0.01)]
    state = mf.adamw_state(p, 8)
    m = v = torch.zeros(n // 256, 256, device="cuda")
    for step in (1, 2, 3):
        mf.adamw_step(p, grad, step=step, betas=(0.9, 0.95), **state)
        gf = grad[0].float().view(-1, 256)
        m = (m * 0.9).add_(gf, alpha=1 - 0.9)
        v = (v * 0.95).add_(gf * gf, alpha=1 - 0.95)
        for key, x in (("exp_avg", m), ("exp_avg_sq", torch.sqrt(v))):
            scale = x.abs().amax(1) / 448
            codes = (x / scale[:, None]).to(F8)
            if key == "exp_avg_sq":
                codes = torch.where(x > 0, codes.float().clamp(min=2.0 ** -9), 0.0).to(F8)
            got = state[key][0].view(-1, 256)
            off = (got.view(torch.uint8) != codes.view(torch.uint8)).sum().item()
            assert off <= (3 if key == "exp_avg_sq" else 0) * step, (step, key, off)
        # on from the kernel's own states
        m = state["exp_avg"][0].float().view(-1, 256) * state["exp_avg_scale"][0][:, None]
        v = (state["exp_avg_sq"][0].float().view(-1, 256) *
             state["exp_avg_sq_scale"][0][:, None]).square()
        grad[0].neg_()


def test_adamw_many_tensors(cuda_lib):
    """More tensors than one launch takes, the last ones among them right."""
    mf = cuda_lib
    sizes = [1 + 37 * (i % 11) for i in range(600)]
    params, grads, state = adamw_inputs(mf, sizes, 32, False, BF16, BF16, False)
    refs = [T_.adamw(p.double(), g.double(), torch.zeros_like(g).double(),
                     torch.zeros_like(g).double(), 1e-3, (0.9, 0.999), 1e-8, 1e-2, 1)
            for p, g in zip(params, grads)]
    mf.adamw_step(params, grads, step=1, **state)
    for i, ref in enumerate(refs):
        check_adamw(ref, params, state, i, 32, BF16, False)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_device_numbers(cuda_lib, bits):
    """step, lr and the gradients' factor on the device: equal to host numbers, and
    read anew by a replayed graph."""
    mf = cuda_lib
    sizes = (1000, 257)
    a = adamw_inputs(mf, sizes, bits, True, BF16, BF16, False)
    b = adamw_inputs(mf, sizes, bits, True, BF16, BF16, False)
    step = torch.tensor([1], dtype=torch.int32, device="cuda")
    lr, scale = torch.tensor([3e-3], device="cuda"), torch.tensor([0.25], device="cuda")
    for t in b[1]:
        t.mul_(0.25)        # exact
    bound_a, bound_b = mf.bind_adamw(*a[:2], **a[2]), mf.bind_adamw(*b[:2], **b[2])
    bound_a(step=step, lr=lr, grad_scale=scale, betas=(0.9, 0.95))
    bound_b(step=1, lr=float(lr), betas=(0.9, 0.95))
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        bound_a(step=step, lr=lr, grad_scale=scale, betas=(0.9, 0.95))
    for k in (2, 3):
        step.fill_(k)
        lr.mul_(0.5)
        graph.replay()
        bound_b(step=k, lr=float(lr), betas=(0.9, 0.95))
    torch.cuda.synchronize()
    for x, y in zip(a[0] + a[2]["exp_avg"], b[0] + b[2]["exp_avg"]):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_adamw_not_finite(cuda_lib):
    """A gradient that is not finite stays with its value (8 bits: its block)."""
    mf = cuda_lib
    for bits in (32, 8):
        clean = adamw_inputs(mf, (1024,), bits, False, F32, F32, False)
        dirty = adamw_inputs(mf, (1024,), bits, False, F32, F32, False)
        dirty[1][0][300], dirty[1][0][600] = NAN, float("inf")
        mf.adamw_step(*clean[:2], step=1, **clean[2])
        mf.adamw_step(*dirty[:2], step=1, **dirty[2])
        assert torch.isnan(dirty[0][0][300])
        same = torch.ones(1024, dtype=torch.bool, device="cuda")
        same[300] = same[600] = False
        assert torch.equal(dirty[0][0][same], clean[0][0][same])
        m, _ = adamw_states(dirty[2], 0)
        assert not torch.isfinite(m[300]) and not torch.isfinite(m[600])
        assert torch.isfinite(m[:256]).all() and torch.isfinite(m[768:]).all()


@pytest.mark.parametrize("grad", [BF16, F32], ids=str)
def test_adamw_square_past_the_largest_number(cuda_lib, grad):
    """A finite gradient whose square is infinite in fp32: its value moves by its decay
    alone, the same in both widths of states; all other values as without it; nothing is
    NaN, then or later.  In 8 bits sqrt(v) is stored as 2^64 (1 - 2^-20)."""
    mf, at = cuda_lib, [300, 2000, 2047]
    ends = {}
    for bits in (32, 8):
        clean = adamw_inputs(mf, (4100,), bits, False, F32, grad, False)
        spike = adamw_inputs(mf, (4100,), bits, False, F32, grad, False)
        p0 = spike[0][0].clone()
        spike[1][0][at] = torch.tensor([1e20, -3e19, 1e38], device="cuda").to(grad)
        for inputs in (clean, spike):
            mf.adamw_step(*inputs[:2], step=1, **HYPER, **inputs[2])
        p = spike[0][0]
        keep = torch.tensor(1.0) - torch.tensor(HYPER["lr"]) * torch.tensor(HYPER["weight_decay"])
        assert torch.equal(p[at], p0[at] * keep.cuda())
        others = torch.ones(4100, dtype=torch.bool, device="cuda")
        others[at] = False
        assert torch.equal(p[others], clean[0][0][others])
        m, v = adamw_states(spike[2], 0)
        assert torch.isfinite(m).all()
        if bits == 8:
            root = v[at].sqrt()         # the largest of its 256: code 448, scale within 2^-22
            assert ((root / (2.0 ** 64 * (1 - 2.0 ** -20)) - 1).abs() <= 2.0 ** -21).all()
            for a, b in zip(clean[2].values(), spike[2].values()):      # blocks without it
                n = 1 if a[0].dtype == F32 else 256
                for i in (0, 2, 6, 8, 16):
                    block = slice(n * i, min(n * i + n, a[0].numel()))
                    assert torch.equal(a[0][block].view(torch.uint8),
                                       b[0][block].view(torch.uint8))
        ends[bits] = p[at].clone()
        for step in (2, 3, 4):          # back to ordinary gradients
            mf.adamw_step(spike[0], clean[1], step=step, **HYPER, **spike[2])
            assert torch.isfinite(spike[0][0]).all() and torch.isfinite(spike[2]["exp_avg"][0]
                                                                        .float()).all()
        if bits == 8:
            later = adamw_states(spike[2], 0)[1]
            assert (later[at] < v[at]).all()
    assert torch.equal(ends[8], ends[32])


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_squares_below_the_normal_range(cuda_lib, bits):
    """Gradients of 3e-22 to 3e-19, whose squares fp32 holds below its normal range, and
    zeros among them, with eps = 0: the step that the formula gives for v as fp32 holds it,
    |u| of the order of lr.  Roundings: of m, the step size, its product, the root, its
    factor and the reciprocal, 2^-22 each at most, 6 of them; of p 2^-24, of keep p 2^-24.
    In 8 bits a root's code is then off by 2^-4 of itself or 2^-10 of its scale, or at the
    least code; its scale by 2^-22."""
    mf, g, n = cuda_lib, gen(17), 2048
    lr, b1, b2 = 1e-2, 0.9, 0.95
    grad = normal(g, n, dtype=F32) * 10.0 ** (-21.5 + 3 * torch.rand(n, generator=g, device="cuda"))
    grad[::11] = 0
    p = [normal(g, n, dtype=F32)]
    p0, state = p[0].double(), mf.adamw_state(p, bits)
    mf.adamw_step(p, [grad], step=1, lr=lr, betas=(b1, b2), eps=0.0, weight_decay=0.0, **state)
    # as fp32 rounds them; the factors 1 - beta are rounded from 64 bits
    v = ((grad * grad).double() * torch.tensor(1 - b2).double().cuda()).float().double()
    m = grad.double() * (1 - b1)
    on = v > 0                          # a square may be 0: 0 / 0, m / 0
    assert on.sum() > n // 2 and (v[on] < 2.0 ** -126).sum() > n // 4
    u = lr / (1 - b1) * m / (v / (1 - b2)).sqrt()
    tol = 6 * 2.0 ** -22 * u.abs() + 2 * 2.0 ** -24 * (p0.abs() + u.abs())
    T_.check(p[0][on], ((p0 - u)[on], tol[on]), "param")
    assert not torch.isfinite(p[0][~on]).any()
    if bits == 8:
        scale = v.sqrt().view(-1, 256).amax(1) / 448
        T_.check(state["exp_avg_sq_scale"][0], (scale, 2.0 ** -22 * scale), "scale")
        code, want = state["exp_avg_sq"][0].double(), v.sqrt() / scale.repeat_interleave(256)
        least = torch.where(on & (want < 2.0 ** -9), 2.0 ** -9, want)
        T_.check(code, (least, 2.0 ** -4 * want * (1 + 2.0 ** -20) + 2.0 ** -10), "codes")
        assert (code[on] > 0).all() and not code[~on].any()


def test_adamw_not_finite_in_8_bits(cuda_lib):
    """All 256 values of both states beside a gradient that is not finite: NaN stays with
    its value; an infinite one takes exp_avg's block, and leaves exp_avg_sq's other roots
    the least code."""
    mf = cuda_lib
    clean = adamw_inputs(mf, (1024,), 8, True, BF16, F32, False)
    dirty = adamw_inputs(mf, (1024,), 8, True, BF16, F32, False)
    clean[1][0][[300, 600]] = 0     # the blocks' largest are others
    dirty[1][0][300], dirty[1][0][600] = NAN, -float("inf")
    for inputs in (clean, dirty):
        mf.adamw_step(*inputs[:2], step=1, **inputs[2])
    at = torch.arange(1024, device="cuda")
    nan, inf = at == 300, (at >= 512) & (at < 768)
    m0, m = clean[2]["exp_avg"][0].float(), dirty[2]["exp_avg"][0].float()
    v0, v = clean[2]["exp_avg_sq"][0].float(), dirty[2]["exp_avg_sq"][0].float()
    assert torch.isnan(m[nan | inf]).all() and torch.equal(m[~(nan | inf)], m0[~(nan | inf)])
    assert torch.isnan(v[nan]).all() and torch.equal(v[~(nan | inf)], v0[~(nan | inf)])
    assert v[600] == 448 and (v[inf & (at != 600)] == 2.0 ** -9 * (v0[inf & (at != 600)] > 0)).all()
    for key in ("exp_avg_scale", "exp_avg_sq_scale"):
        a, b = clean[2][key][0], dirty[2][key][0]
        assert torch.equal(a[[0, 1, 3]], b[[0, 1, 3]])
        assert torch.isinf(b[2]) if key == "exp_avg_scale" else torch.isfinite(b[2])
    p0, p = clean[2]["masters"][0], dirty[2]["masters"][0]
    own = nan | (at == 600)
    assert torch.isnan(p[own]).all() and torch.equal(p[~own], p0[~own])


# ---------------------------------------------------------- all together


def layer_weights(g, E, H, I):
    return {"router": normal(g, E, H, scale=H ** -0.5), "w13": normal(g, E, 2 * I, H, scale=H ** -0.5),
            "w2": normal(g, E, H, I, scale=I ** -0.5), "s13": normal(g, 2 * I, H, scale=H ** -0.5),
            "s2": normal(g, H, I, scale=I ** -0.5), "gamma": normal(g, H)}


def layer_step(mf, w, x, residual, dnorm, dres, K, E, tile, grads=None):
    """Forward and backward of a layer on the library; the gradients."""
    grads = grads or {}
    logits = mf.linear(x, w["router"], out_dtype=F32)["out"]
    route = mf.topk_route(logits, K, "sigmoid")
    m = mf.permute_tokens(route["expert_ids"], E, tile)
    P, I2 = m["row_token"].numel(), w["w13"].shape[1]
    pre = torch.empty((P, I2), dtype=BF16, device="cuda")
    h = mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w["w13"], preact=pre)
    rows = mf.expert_linear(h, m["offsets"], m["counts"], w["w2"])
    up = mf.gated_ffn(x, w["s13"], save_preact=True)
    shared = mf.linear(up["out"], w["s2"])["out"]
    out = mf.moe_finalize(rows, m["idx_map"], route["weights"], "fp32", shared, routed_scale=2.5,
                          residual=residual, gamma=w["gamma"], write_out=False)
    f = mf.moe_finalize_backward(rows, m["idx_map"], route["weights"], "fp32", routed_scale=2.5,
                                 dresidual_out=dres, dnorm_out=dnorm,
                                 residual_out=out["residual_out"], gamma=w["gamma"],
                                 dgamma=grads.get("gamma"))
    down = mf.expert_linear_backward(f["drows"], h, m["offsets"], m["counts"], w["w2"],
                                     dweight=grads.get("w2"))
    gate = mf.expert_gated_ffn_backward(down["dx"], x, m["row_token"], m["offsets"], m["counts"],
                                        w["w13"], pre, dweight=grads.get("w13"))
    s2 = mf.linear_backward(f["dshared"], up["out"], w["s2"], dweight=grads.get("s2"))
    s13 = mf.gated_ffn_backward(s2["dx"], x, w["s13"], up["preact"], dweight=grads.get("s13"))
    dlogits = mf.topk_route_backward(f["dweights"], route["weights"], route["expert_ids"], E,
                                     "sigmoid", logits=logits)
    r = mf.linear_backward(dlogits, x, w["router"], dweight=grads.get("router"))
    dx = mf.unpermute_tokens(gate["dx"], m["idx_map"], add=(s13["dx"], r["dx"]))
    return {"x": dx, "residual": f["dresidual"], "router": r["dweight"], "w13": gate["dweight"],
            "w2": down["dweight"], "s13": s13["dweight"], "s2": s2["dweight"],
            "gamma": f["dgamma"]}, route["expert_ids"]


def layer_reference(w, x, residual, dnorm, dres, ids):
    """The same through torch's autograd in 64 bits, the chosen experts given."""
    p = {k: v.double().requires_grad_() for k, v in w.items()}
    x = x.double().requires_grad_()
    residual = residual.double().requires_grad_()

    def gated(z):
        a, u = z.chunk(2, dim=-1)
        return a * torch.sigmoid(a) * u

    s = torch.sigmoid((x @ p["router"].T).gather(1, ids.long()))
    weight = 2.5 * s / s.sum(1, keepdim=True)
    m = gated(x @ p["s13"].T) @ p["s2"].T
    for e in range(p["router"].shape[0]):
        share = (weight * (ids == e)).sum(1, keepdim=True)
        m = m + share * (gated(x @ p["w13"][e].T) @ p["w2"][e].T)
    r = m + residual
    n = r * (r.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * p["gamma"]
    ((r * dres.double()).sum() + (n * dnorm.double()).sum()).backward()
    return {"x": x.grad, "residual": residual.grad, **{k: v.grad for k, v in p.items()}}


@pytest.mark.parametrize("T,K,E,H,I,tile", [(1, 1, 2, 64, 32, 1), (37, 2, 8, 256, 128, 16),
                                            (200, 4, 6, 136, 72, 1)])
def test_layer_gradients(cuda_lib, T, K, E, H, I, tile):
    """A whole layer's gradients.  About twenty bf16 roundings of 2^-9 relative (root
    mean square at most 2^-8 / sqrt(3)) lie on the longest way; norms of the gradients are
    compared, in which independent roundings add as squares: sqrt(20) 2^-8 / sqrt(3)
    = 0.010, and the norm's cancellation and the gate's difference of weights may
    magnify them threefold."""
    mf, g = cuda_lib, gen(T)
    w = layer_weights(g, E, H, I)
    x, residual = normal(g, T, H), normal(g, T, H, scale=2.0)
    dnorm, dres = normal(g, T, H, scale=0.1), normal(g, T, H, scale=0.1)
    got, ids = layer_step(mf, w, x, residual, dnorm, dres, K, E, tile)
    ref = layer_reference(w, x, residual, dnorm, dres, ids)
    for k, v in ref.items():
        if v.norm() == 0:       # one expert chosen of one: its weight is 1 whatever the logits
            assert got[k].double().norm() <= 1e-6, k
            continue
        rel = ((got[k].double() - v).norm() / v.norm()).item()
        assert rel <= 0.03, (k, rel)
    assert mf.lost_waits() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_layer_training_step_in_a_graph(cuda_lib, bits):
    """Forward, backward and the update captured as one graph: replays equal eager
    steps bit by bit."""
    mf = cuda_lib
    T, K, E, H, I = 64, 2, 8, 128, 64
    g = gen(1)
    x, residual = normal(g, T, H), normal(g, T, H)
    dnorm, dres = normal(g, T, H, scale=0.1), normal(g, T, H, scale=0.1)
    runs = []
    for captured in (False, True):
        w = layer_weights(gen(2), E, H, I)
        grads = {k: torch.zeros_like(v) for k, v in w.items()}
        state = mf.adamw_state(list(w.values()), bits, master=True)
        update = mf.bind_adamw(list(w.values()), list(grads.values()), **state)
        count = torch.zeros(1, dtype=torch.int32, device="cuda")

        def step():
            layer_step(mf, w, x, residual, dnorm, dres, K, E, 8, grads)
            count.add_(1)
            update(step=count, lr=1e-3)

        if captured:
            layer_step(mf, w, x, residual, dnorm, dres, K, E, 8, grads)     # first calls
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
        for _ in range(3):
            graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert int(count) == 3
        runs.append((w, state))
    for k in runs[0][0]:
        assert torch.equal(runs[0][0][k], runs[1][0][k]), k
    for k, ts in runs[0][1].items():
        for a, b in zip(ts, runs[1][1][k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_threads_with_streams_of_their_own(cuda_lib):
    """Four threads at once, each with other sizes, on its own stream."""
    import threading
    mf = cuda_lib
    jobs, wants, errors = [], [], []
    for i, (H, T) in enumerate(((256, 40), (4104, 20), (20008, 8), (7168, 350))):
        fcase = (T, 4, 8, H, 8, "fp32", True, True, True, 0.1)
        rows, m, w, dout, kw = finalize_inputs(mf, fcase, seed=i)
        ecase = (40 + 30 * i, 2, 4, 128, 40 + 8 * i, 8, "silu", True, True, 1)
        jobs.append(((rows, m, w, dout, kw), ecase, expert_inputs(mf, ecase, seed=i),
                     adamw_inputs(mf, (300 + i, 1000), 8, True, BF16, BF16, False, seed=i)))

    def work(job, adam):
        (rows, m, w, dout, kw), ecase, e, _ = job
        f = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, **kw)
        r = expert_call(mf, ecase, *e)
        u = mf.unpermute_tokens(f["drows"], m["idx_map"], add=f["dshared"])
        mf.adamw_step(adam[0], adam[1], step=1, **adam[2])
        return [f["dweights"], f["dgamma"], f["dresidual"], u, r["dweight"], r["dbias"]] + adam[0]

    for job in jobs:
        adam = job[3]
        copy = ([t.clone() for t in adam[0]], adam[1],
                {k: [t.clone() for t in ts] for k, ts in adam[2].items()})
        wants.append(work(job, copy))
    torch.cuda.synchronize()

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    adam = jobs[i][3]
                    copy = ([t.clone() for t in adam[0]], adam[1],
                            {k: [t.clone() for t in ts] for k, ts in adam[2].items()})
                    got = work(jobs[i], copy)
                    torch.cuda.current_stream().synchronize()
                    for a, b in zip(got, wants[i]):
                        assert torch.equal(a, b)
        except BaseException as e:      # noqa: B902
            errors.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    assert mf.lost_waits() == 0


@pytest.mark.parametrize("fast", [True, False])
def test_batches_of_nothing(cuda_lib, monkeypatch, fast):
    """No tokens and no rows: outputs of no elements, gradients of weights that are zeros."""
    mf = cuda_lib
    from moe_deferred_finalize_gb300 import _abi
    if not fast:
        monkeypatch.setattr(_abi, "_FAST", None)
    i32 = dict(dtype=torch.int32, device="cuda")
    e, wide = (torch.empty((0, n), dtype=BF16, device="cuda") for n in (64, 128))
    idx, w = torch.empty((0, 2), **i32), torch.empty((0, 2), device="cuda")
    for kw in ({}, dict(want_dweights=False), dict(dresidual_out=e)):
        res = mf.moe_finalize_backward(e, idx, w, "fp32", e, **kw)
        assert res and all(v.shape[0] == 0 for v in res.values())
    res = mf.moe_finalize_backward(e, idx, w, "fp32", dnorm_out=e, residual_out=e,
                                   gamma=torch.ones(64, dtype=BF16, device="cuda"))
    assert not res["dgamma"].any()
    assert mf.unpermute_tokens(e, idx, add=(e, e)).shape == (0, 64)
    assert mf.topk_route_backward(w, w, idx, 4, "softmax").shape == (0, 4)
    offsets, counts = torch.zeros(4, **i32), torch.zeros(3, **i32)
    weight = torch.ones((3, 128, 64), dtype=BF16, device="cuda")
    for want in ({}, dict(want_dweight=False), dict(want_dx=False, want_dbias=True)):
        for row_token in (None, torch.empty(0, **i32)):
            for res in (mf.expert_gated_ffn_backward(e, e, row_token, offsets, counts, weight,
                                                     wide, **want),
                        mf.expert_linear_backward(wide, e, offsets, counts, weight,
                                                  row_token=row_token, **want)):
                assert not any(v.any() for v in res.values())
                assert "dx" not in res or res["dx"].shape == (0, 64)


def test_two_streams_at_once(cuda_lib):
    """Calls on a given stream, beside others on the current one."""
    mf = cuda_lib
    case = (64, 2, 8, 256, 128, 16, "silu", True, True, 0)
    m, x, w, dout, preact = expert_inputs(mf, case)
    fcase = (40, 4, 8, 256, 8, "fp32", True, True, True, 0.0)
    rows, fm, fw, fdout, kw = finalize_inputs(mf, fcase)
    torch.cuda.synchronize()
    have = m["row_token"] >= 0
    want = expert_call(mf, case, m, x, w, dout, preact)
    fwant = mf.moe_finalize_backward(rows, fm["idx_map"], fw, "fp32", fdout, **kw)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((expert_call(mf, case, m, x, w, dout, preact, stream=other),
                    expert_call(mf, case, m, x, w, dout, preact),
                    mf.moe_finalize_backward(rows, fm["idx_map"], fw, "fp32", fdout, stream=other,
                                             **kw)))
    torch.cuda.synchronize()
    for a, b, f in got:
        for res in (a, b):
            assert torch.equal(res["dweight"], want["dweight"])
            assert torch.equal(res["dbias"], want["dbias"])
            assert torch.equal(res["dx"][have], want["dx"][have])
        for k in ("dweights", "dgamma", "dshared", "dresidual"):
            assert torch.equal(f[k], fwant[k])


# ------------------------------------------- other sizes, paths and callers


@pytest.mark.parametrize("T", [20, 900])       # one CTA a slice; rows through the ring
@pytest.mark.parametrize("K", [1, 8])
def test_finalize_backward_outputs_on_either_input(cuda_lib, T, K):
    """dshared and dresidual in place of dout and dresidual_out, either way round."""
    mf = cuda_lib
    case = (T, K, 16, 2048, 8, "fp32", True, True, True, 0.1)
    rows, m, w, dout, kw = finalize_inputs(mf, case)
    want = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", dout, **kw)
    for swap in (False, True):
        a, b = dout.clone(), kw["dresidual_out"].clone()
        out = dict(dshared=b, dresidual=a) if swap else dict(dshared=a, dresidual=b)
        got = mf.moe_finalize_backward(rows, m["idx_map"], w, "fp32", a,
                                       **{**kw, "dresidual_out": b}, **out)
        for k in ("dshared", "dresidual", "dweights", "dgamma"):
            assert torch.equal(got[k], want[k]), (swap, k)


RING = [
    # T, K, E, H, tile, wkind, norm, dout, dres, absent: both sides of the ring's rules
    (400, 8, 16, 7168, 8, "fp32", True, True, True, 0.1),
    (400, 8, 16, 7168, 8, "packed", True, False, False, 0.0),
    (400, 5, 16, 8192, 1, "fp32", True, True, True, 0.5),
    (500, 4, 8, 7168, 1, "bf16", False, True, False, 0.2),
    (500, 3, 8, 7168, 1, "bf16", False, True, False, 0.2),
    (2500, 32, 40, 128, 1, "fp32", True, True, False, 0.1),
    (3000, 2, 8, 8, 1, "fp32", True, True, True, 0.0),
    (700, 6, 8, 4096, 1, "fp32", False, True, True, 1.0),
    (610, 8, 16, 8200, 1, "fp32", True, True, True, 0.0),
]


@pytest.mark.parametrize("case", RING, ids=str)
def test_finalize_backward_many_tokens(cuda_lib, case):
    mf = cuda_lib
    rows, m, w, dout, kw = finalize_inputs(mf, case, seed=2)
    drows0 = torch.full_like(rows, 7.0)
    res = mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, routed_scale=0.5,
                                   drows=drows0.clone(), **kw)
    check_finalize(case, rows, m, w, dout, kw, res, drows0, 0.5, 1e-6)
    one = mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, routed_scale=0.5,
                                   want_drows=False, **kw)
    two = mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, routed_scale=0.5,
                                   want_dweights=False, drows=drows0.clone(), **kw)
    others = [one, two]
    if case[6] or case[8]:
        others.append(mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout,
                                               routed_scale=0.5, want_drows=False,
                                               want_dweights=False, **kw))
    for k in res:
        for other in others:
            if k in other:
                assert torch.equal(other[k], res[k]), k


LONG_ROWS = [
    # as RING, without the norm: rows of up to 8192 values fit a CTA's threads, longer ones
    # (one piece, one value more among them) are gone over in steps
    (400, 8, 8, 8192, 1, "fp32", False, True, False, 0.1),
    (400, 4, 8, 8200, 1, "fp32", False, True, False, 0.1),
    (400, 4, 8, 8193, 1, "bf16", False, True, True, 0.1),
    (700, 8, 8, 16384, 8, "fp32", False, True, False, 0.0),
    (320, 5, 8, 16392, 1, "packed", False, False, True, 0.2),
    (400, 8, 16, 20000, 1, "fp32", False, True, True, 0.1),
    (310, 32, 40, 9000, 1, "fp32", False, True, True, 0.5),
]


@pytest.mark.parametrize("case", LONG_ROWS, ids=str)
def test_finalize_backward_long_rows_without_norm(cuda_lib, case):
    """All columns of all outputs, which are made in place of values that no gradient has."""
    mf = cuda_lib
    T, H, dres = case[0], case[3], case[8]
    rows, m, w, dout, kw = finalize_inputs(mf, case, seed=5)
    drows0 = torch.full_like(rows, 7.0)
    outs = dict(drows=drows0.clone(), dweights=torch.full((T, case[1]), NAN, device="cuda"))
    if dres:
        outs["dresidual"] = torch.full((T, H), NAN, dtype=BF16, device="cuda")
        if dout is not None:
            outs["dshared"] = torch.full((T, H), NAN, dtype=BF16, device="cuda")
    res = mf.moe_finalize_backward(rows, m["idx_map"], w, case[5], dout, routed_scale=2.5, **outs,
                                   **kw)
    check_finalize(case, rows, m, w, dout, kw, res, drows0, 2.5, 1e-6)


def test_one_pass_calls_equal_checked_calls(cuda_lib, monkeypatch):
    """The same results with and without the call extension."""
    mf = cuda_lib
    from moe_deferred_finalize_gb300 import _abi
    if _abi._fastcall() is None:
        pytest.skip("_fastcall not built (no Python headers)")
    fcase = (30, 4, 8, 256, 8, "bf16", True, True, True, 0.1)
    rows, m, w, dout, kw = finalize_inputs(mf, fcase)
    ecase = (60, 2, 4, 128, 72, 8, "silu", True, True, 2)
    em, x, ew, edout, preact = expert_inputs(mf, ecase)
    lcase = (60, 2, 4, 128, 72, 8, "none", True, False, 2)
    lm, lx, lw, ldout, _ = expert_inputs(mf, lcase)
    logits = torch.randn(20, 16, device="cuda")
    route = mf.topk_route(logits, 4)
    dw = torch.randn(20, 4, device="cuda")
    add = normal(gen(0), 30, 256)

    def everything():
        zero = torch.zeros_like
        r = {("f", k): v for k, v in mf.moe_finalize_backward(
            rows, m["idx_map"], w, "bf16", dout, drows=zero(rows), **kw).items()}
        r.update({("e", k): v for k, v in expert_call(
            mf, ecase, em, x, ew, edout, preact,
            dx=zero(normal(gen(0), edout.shape[0], 128))).items()})
        r.update({("l", k): v for k, v in expert_call(
            mf, lcase, lm, lx, lw, ldout, None,
            dx=zero(normal(gen(0), ldout.shape[0], 128))).items()})
        r["u"] = mf.unpermute_tokens(rows, m["idx_map"], add=add)
        r["g"] = mf.topk_route_backward(dw, route["weights"], route["expert_ids"], 16,
                                        logits=logits)
        return r

    fast = everything()
    monkeypatch.setattr(_abi, "_FAST", None)
    slow = everything()
    assert fast.keys() == slow.keys()
    for k in fast:
        assert torch.equal(fast[k], slow[k]), k


def test_refusals_name_the_tensor(cuda_lib):
    """What the one-pass checks refuse, the binding names."""
    mf = cuda_lib
    fcase = (6, 2, 4, 64, 1, "fp32", True, True, True, 0.0)
    rows, m, w, dout, kw = finalize_inputs(mf, fcase)
    idx = m["idx_map"]
    bad = [(dict(dout=dout.float()), "dout"), (dict(dout=dout[:5]), "dout"),
           (dict(weights=w.to(BF16)), "weights"), (dict(residual_out=None), "residual_out"),
           (dict(gamma=kw["gamma"][:8]), "gamma"), (dict(dgamma=dout), "dgamma"),
           (dict(drows=rows[:1]), "drows"), (dict(dresidual=dout.T.contiguous().T), "dresidual"),
           (dict(idx_map=idx.long()), "idx_map")]
    for change, name in bad:
        args = dict(permuted_out=rows, idx_map=idx, weights=w, wkind="fp32", dout=dout, **kw)
        with pytest.raises((ValueError, TypeError), match=name):
            mf.moe_finalize_backward(**{**args, **change})
    with pytest.raises(ValueError, match="go with dnorm_out"):
        mf.moe_finalize_backward(rows, idx, w, "fp32", dout, gamma=kw["gamma"])
    with pytest.raises(ValueError, match="no gradient"):
        mf.moe_finalize_backward(rows, idx, w, "fp32")
    with pytest.raises(ValueError, match="at most two"):
        mf.unpermute_tokens(rows, idx, add=[dout] * 3)
    with pytest.raises(ValueError, match="add"):
        mf.unpermute_tokens(rows, idx, add=dout[:, :8].contiguous())
    ecase = (20, 2, 4, 64, 24, 1, "silu", False, True, 0)
    em, x, ew, edout, preact = expert_inputs(mf, ecase)
    args = dict(dout=edout, x=x, row_token=em["row_token"], offsets=em["offsets"],
                counts=em["counts"], weight=ew, preact=preact)
    for change, name in [(dict(preact=preact[:, :8].contiguous()), "preact"),
                         (dict(weight=ew[:, :8].contiguous()), "weight"),
                         (dict(row_token=em["row_token"][:3]), "row_token"),
                         (dict(row_token=None), "row_token"), (dict(dweight=ew[0]), "dweight"),
                         (dict(offsets=em["offsets"][:2]), "offsets")]:
        with pytest.raises((ValueError, TypeError), match=name):
            mf.expert_gated_ffn_backward(**{**args, **change})
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(mf.MoefError, match="SHAPE"):
        mf.expert_gated_ffn_backward(**args, workspace=small)
    p = [torch.zeros(8, dtype=BF16, device="cuda")]
    state = mf.adamw_state(p)
    for change in (dict(grads=[p[0][:4]]), dict(grads=p * 2), dict(masters=[p[0]]),
                   dict(exp_avg=[p[0]]), dict(exp_avg_scale=[torch.zeros(1, device="cuda")])):
        with pytest.raises(ValueError):
            mf.bind_adamw(**{**dict(params=p, grads=p, **state), **change})
    with pytest.raises(ValueError, match="lr"):
        mf.adamw_step(p, p, step=1, lr=torch.zeros(2, device="cuda"), **state)
    with pytest.raises(mf.MoefError, match="ARG"):
        mf.adamw_step(p, p, step=0, **state)


@pytest.mark.slow
def test_rows_past_31_bits(cuda_lib):
    """Row offsets past 2^31 values, in every operand that has rows."""
    mf, g = cuda_lib, gen(11)
    P, H, T, K = 300_000, 7168, 40, 4
    rows = torch.zeros((P, H), dtype=BF16, device="cuda")
    idx = torch.randint(P - 1000, P, (T, K), generator=g, device="cuda").int()
    idx = (torch.arange(P - T * K, P, device="cuda").int()).view(T, K).contiguous()
    rows[P - 1000:] = normal(g, 1000, H)
    w = torch.rand(T, K, generator=g, device="cuda")
    dout = normal(g, T, H)
    res = mf.moe_finalize_backward(rows, idx, w, "fp32", dout)
    ref = T_.finalize_backward(rows[P - 1000:], idx - (P - 1000), w.double(), 1.0, dout)
    T_.check(res["dweights"], ref["dweights"], "dweights")
    T_.check(res["drows"][idx.long()], ref["drows"], "drows")
    T_.check(mf.unpermute_tokens(rows, idx), T_.unpermute(rows[P - 1000:], idx - (P - 1000), []),
             "unpermute")
    del rows, res
    torch.cuda.empty_cache()
    # many tokens: dense rows past 2^31 values
    T, K, H = 310_000, 1, 7168
    rows = normal(g, 8, H)
    idx = torch.full((T, K), -1, dtype=torch.int32, device="cuda")
    idx[-4:, 0] = torch.arange(4, device="cuda").int()
    dout = torch.zeros((T, H), dtype=BF16, device="cuda")
    dout[-4:] = normal(g, 4, H)
    w = torch.ones((T, K), device="cuda")
    res = mf.moe_finalize_backward(rows, idx, w, "fp32", dout)
    T_.check(res["drows"][:4], T_.rounded(dout[-4:].double(), torch.zeros_like(dout[-4:]).double()),
             "drows")
    out = mf.unpermute_tokens(rows, idx, add=dout)
    T_.check(out[-4:], T_.unpermute(rows, idx[-4:], [dout[-4:]]), "unpermute")


@pytest.mark.slow
def test_expert_rows_past_31_bits(cuda_lib):
    mf, g = cuda_lib, gen(12)
    P, E, H, I = 540_000, 2, 64, 2048           # dz: 540000 x 4096
    offsets = torch.tensor([0, P - 70, P], dtype=torch.int32, device="cuda")
    counts = torch.tensor([30, 70], dtype=torch.int32, device="cuda")
    token = torch.zeros(P, dtype=torch.int32, device="cuda")
    token[-70:] = torch.arange(70, device="cuda").int()
    x, w = normal(g, 70, H), normal(g, E, 2 * I, H, scale=0.1)
    dout = torch.zeros((P, I), dtype=BF16, device="cuda")
    preact = torch.zeros((P, 2 * I), dtype=BF16, device="cuda")
    for rows in (slice(0, 30), slice(P - 70, P)):
        n = rows.stop - rows.start
        dout[rows], preact[rows] = normal(g, n, I), normal(g, n, 2 * I)
    res = mf.expert_gated_ffn_backward(dout, x, token, offsets, counts, w, preact,
                                       want_dbias=True)
    ref = T_.expert_backward(dout[-70:], x, token[-70:], offsets[1:] - (P - 70), counts[1:],
                             w[1:], preact[-70:], "silu", True)
    T_.check(res["dx"][-70:], ref["dx"], "dx")
    T_.check(res["dweight"][1:], ref["dweight"], "dweight")
    T_.check(res["dbias"][1:], ref["dbias"], "dbias")


@pytest.mark.slow
def test_expert_rows_up_to_the_last(cuda_lib):
    """2^31 - 1 rows of one feature: their dz and dx, the last one's too."""
    mf, P, K = cuda_lib, 2 ** 31 - 1, 8
    offsets = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    counts = torch.tensor([P], dtype=torch.int32, device="cuda")
    w = torch.arange(1, K + 1, device="cuda").to(BF16).view(1, 1, K)
    dout = torch.full((P, 1), 2.0, dtype=BF16, device="cuda")
    dout[-1] = 3.0
    x = torch.empty((1, K), dtype=BF16, device="cuda").expand(P, K)
    with pytest.raises(ValueError, match="contiguous"):
        mf.expert_linear_backward(dout, x, offsets, counts, w)
    token = torch.zeros(P, dtype=torch.int32, device="cuda")
    res = mf.expert_linear_backward(dout, x[:1].contiguous(), offsets, counts, w,
                                    row_token=token, want_dweight=False)
    row = w.view(K).float()
    for r, scale in ((0, 2), (2 ** 30 + 5, 2), (P - 2, 2), (P - 1, 3)):
        assert torch.equal(res["dx"][r].float(), scale * row), r
    assert mf.lost_waits() == 0


@pytest.mark.slow
def test_adamw_past_31_bits(cuda_lib):
    mf = cuda_lib
    n = 2 ** 31 + 1000
    p = [torch.ones(n, dtype=BF16, device="cuda")]
    grad = [torch.zeros(n, dtype=BF16, device="cuda")]
    grad[0][-700:] = 0.5
    state = mf.adamw_state(p, bits=8)
    mf.adamw_step(p, grad, step=1, lr=0.125, weight_decay=0.0, eps=0.0, **state)
    # m = 0.05, sqrt(v) = 0.0158: a step of lr; zero gradients with eps = 0 are 0 / 0
    assert (p[0][-700:].float() == 0.875).all()
    assert (state["exp_avg"][0][-700:].float() == 448).all()
    assert not state["exp_avg"][0][:1000].float().any()
    assert abs(float(state["exp_avg_scale"][0][-1]) * 448 - 0.05) < 1e-8
