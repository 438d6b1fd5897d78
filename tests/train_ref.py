"""Plain 64-bit implementations of the MoE layer's training side, and the error
bounds their GPU counterparts are held to, from ffn_ref's: an fp32 operation is
off by at most ADD of its result's magnitude (two roundings allowed for), a
sum of n terms by (n + 2) ADD of the sum of magnitudes, a rounding to bf16 by
BF16 of the value, one to e4m3 by 2^-4 of it and 2^-10 below the normal range.
rsqrtf, expf and the divisions are within 4 ADD.
"""
import torch

import ffn_ref as R
from ffn_ref import ADD, BF16, TINY

BLOCK, F8_MAX = 256, 448.0


def rounded(value, tol):
    return value, tol + BF16 * (value.abs() + tol) + TINY


def decoded(weights, wkind):
    """Routing weights as the numbers they stand for."""
    if wkind == "packed":
        return (weights << 16).view(torch.float32).double()
    return weights.double()


def finalize_backward(rows, idx, w, scale, dout=None, dres=None, dnorm=None, r=None, gamma=None,
                      eps=1e-6):
    """{name: (value, bound)}; drows as [T, K, H], one row a slot."""
    T, K = idx.shape
    H = rows.shape[1]
    zero = torch.zeros((T, H), dtype=torch.float64, device=rows.device)
    res = {}
    dr = zero if dres is None else dres.double()
    mag, err = dr.abs(), zero
    if dnorm is not None:
        x, dn, g = r.double(), dnorm.double(), gamma.double()
        inv = (x.square().mean(1, keepdim=True) + eps) ** -0.5
        e_inv = (0.5 * (H + 4) + 4) * ADD               # relative
        dy = dn * g
        s, s_mag = (dy * x).sum(1, keepdim=True), (dy * x).abs().sum(1, keepdim=True)
        mean = inv ** 2 * s / H
        e_mean = mean.abs() * (2 * e_inv + 4 * ADD) + inv ** 2 / H * (H + 4) * ADD * s_mag
        dr = dr + inv * (dy - x * mean)
        terms = inv * (dy.abs() + x.abs() * mean.abs())
        err = (e_inv + 6 * ADD) * terms + inv * x.abs() * e_mean + 2 * ADD * (mag + terms)
        mag = mag + terms
        dg = dn * x * inv
        res["dgamma"] = rounded(dg.sum(0), dg.abs().sum(0) * (e_inv + (T + 6) * ADD))
    dm = dr if dout is None else dr + dout.double()
    e_dm = err if dout is None else err + 2 * ADD * (mag + dout.double().abs())
    if dnorm is not None or dres is not None:
        res["dresidual"] = rounded(dr, err)
        res["dshared"] = rounded(dm, e_dm)
    have = (idx >= 0) & (idx < rows.shape[0])
    at = torch.where(have, idx, torch.zeros_like(idx)).long()
    ws = w * scale
    d = ws[:, :, None] * dm[:, None, :]
    e = ws.abs()[:, :, None] * (e_dm + 4 * ADD * dm.abs())[:, None, :]
    res["drows"] = rounded(d, e)
    x = torch.where(have[:, :, None], rows[at].double(), torch.zeros((), device=rows.device,
                                                                     dtype=torch.float64))
    v = scale * (x * dm[:, None, :]).sum(2)
    e = abs(scale) * ((x.abs() * e_dm[:, None, :]).sum(2) +
                      (H + 4) * ADD * (x * dm[:, None, :]).abs().sum(2))
    res["dweights"] = (v, e + TINY)
    return res


def unpermute(rows, idx, adds):
    have = (idx >= 0) & (idx < rows.shape[0])
    at = torch.where(have, idx, torch.zeros_like(idx)).long()
    x = torch.where(have[:, :, None], rows[at].double() if rows.shape[0] else 0.0,
                    torch.zeros((), device=idx.device, dtype=torch.float64))
    parts = [x.sum(1)] + [a.double() for a in adds]
    mags = [x.abs().sum(1)] + [a.double().abs() for a in adds]
    return rounded(sum(parts), (idx.shape[1] + 4) * ADD * sum(mags))


def gate_backward(dw, w, ids, E, kind, logits=None, fp32=True):
    have = (ids >= 0) & (ids < E)
    at = torch.where(have, ids, torch.zeros_like(ids)).long()
    zero = torch.zeros((), dtype=torch.float64, device=dw.device)
    w = torch.where(have, w.double(), zero)
    dw = torch.where(have, dw.double(), zero)
    s, mag = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    d = w * (dw - s)
    e = w.abs() * ((dw.shape[1] + 4) * ADD * (dw.abs() + mag))
    if kind == "sigmoid":
        f = torch.sigmoid(-logits.double().gather(1, at))
        d, e = d * f, e * f + (d * f).abs() * 16 * ADD
    d, e = torch.where(have, d, zero), torch.where(have, e, zero)
    out = torch.zeros((dw.shape[0], E), dtype=torch.float64, device=dw.device)
    value, tol = out.scatter_add(1, at, d), out.scatter_add(1, at, e)
    return (value, tol + TINY) if fp32 else rounded(value, tol)


def expert_backward(dout, x, row_token, offsets, counts, weight, preact, name, gated):
    """{name: (value, bound)}; dx only where an expert has the row (NaN bound
    elsewhere)."""
    P, E = dout.shape[0], weight.shape[0]
    kw = dict(dtype=torch.float64, device=dout.device)
    dx = torch.zeros((P, weight.shape[2]), **kw)
    e_dx = torch.full_like(dx, float("inf"))
    dw, e_dw = torch.zeros(weight.shape, **kw), torch.full(weight.shape, TINY, **kw)
    db, e_db = torch.zeros(weight.shape[:2], **kw), torch.full(weight.shape[:2], TINY, **kw)
    for e in range(E):
        first, count = int(offsets[e]), int(counts[e])
        count = 0 if first < 0 else max(0, min(count, P - first))
        if not count:
            continue
        rows = slice(first, first + count)
        xe = x[rows]
        if row_token is not None:
            token = row_token[rows].long()
            ok = (token >= 0) & (token < x.shape[0])
            xe = x[torch.where(ok, token, torch.zeros_like(token))] * ok[:, None]
        ref = R.backward(dout[rows], xe, weight[e], None if preact is None else preact[rows],
                         name, gated)
        dx[rows], e_dx[rows] = ref["dx"]
        dw[e], e_dw[e] = ref["dweight"]
        db[e], e_db[e] = ref["dbias"]
    return {"dx": (dx, e_dx), "dweight": (dw, e_dw), "dbias": (db, e_db)}


def adamw(p, g, m, v, lr, betas, eps, wd, step, grad_scale=1.0, param_bf16=True):
    """One step of flat fp64 tensors; {name: (value, bound)} before any state is
    rounded to 8 bits."""
    b1, b2 = betas
    g = g * grad_scale
    m1, m2 = b1 * m, (1 - b1) * g
    v1, v2 = b2 * v, (1 - b2) * g * g
    m, v = m1 + m2, v1 + v2
    e_m, e_v = 3 * ADD * (m1.abs() + m2.abs()), 5 * ADD * v + 1e-37
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    root = v.sqrt()
    e_root = 0.5 * e_v / root.clamp(min=1e-18) + 4 * ADD * root
    den = root / c2 ** 0.5 + eps
    u = lr / c1 * m / den
    e_u = lr / c1 * e_m / den + u.abs() * (e_root / c2 ** 0.5 / den + 16 * ADD)
    new = p * (1 - lr * wd) - u
    e = e_u + 4 * ADD * (p.abs() + u.abs()) + 2 * ADD * p.abs()
    return {"param": rounded(new, e) if param_bf16 else (new, e + TINY), "master": (new, e + TINY),
            "m": (m, e_m + TINY), "v": (v, e_v + TINY), "root": (root, e_root + TINY)}


def blocks(x):
    """x in rows of BLOCK values, zeros behind its end."""
    n = -(-x.numel() // BLOCK) * BLOCK
    return torch.cat([x, torch.zeros(n - x.numel(), dtype=x.dtype, device=x.device)]) \
        .view(-1, BLOCK)


def code(x, tol, root):
    """The 8-bit state of x, in units of its scale: (values, bounds), (scales,
    bounds)."""
    n = x.numel()
    xb, tb = blocks(x), blocks(tol)
    top = xb.abs().amax(1)
    e_top = tb.amax(1)
    scale = top / F8_MAX
    unit = torch.where(top > 0, scale, torch.ones_like(scale))[:, None]
    y = xb / unit
    # a value and its scale are off; then half a step
    e = tb / unit + y.abs() * (e_top[:, None] / unit / F8_MAX + 8 * ADD)
    e = e + 2.0 ** -4 * (y.abs() + e) + 2.0 ** -10
    if root:        # values above 0 keep the least code
        e = e + 2.0 ** -9 * (y < 2.0 ** -9)
    return (y.view(-1)[:n], e.view(-1)[:n]), (scale, e_top / F8_MAX + 4 * ADD * scale + TINY)


def check(got, ref, what=""):
    """Every element within its bound; bounds of infinity say nothing."""
    value, tol = ref
    g = got.double()
    assert g.shape == value.shape, (what, g.shape, value.shape)
    bad = ~((g - value).abs() <= tol) & ~torch.isinf(tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                             f"{g[i].item()!r}, expected {value[i].item()!r} +- {tol[i].item():.3g}")
