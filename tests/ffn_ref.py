"""Plain 64-bit implementations of the products around the finalize, and the
error bounds their GPU counterparts are held to.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value.  An fp32 sum
of K products of bf16 values (each exact in fp32) is off by at most K + 2
additions' errors, 2^-23 each to allow for truncation, relative to the sum of
the magnitudes.  The activations' fp32 forms are within 2^-16 of the value:
exp is off by (2 + 1.2 |q|) 2^-23 at argument q, |q| <= 88 before the result
leaves the range; erfc's argument rounding costs 2 x^2 2^-24 at x < 9.  Their
slopes are at most 1.13 and their second derivatives at most 0.8, which
carries an error of z into the value and the derivative.
"""
import math

import torch

BF16 = 2.0 ** -8
ADD = 2.0 ** -23
ACT = 2.0 ** -16
SLOPE, CURVE = 1.13, 0.8
TINY = 1e-30

ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")


def act(z, name):
    """The activation and its derivative in 64 bits."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z)), (z > 0).double()
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu":
        phi = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    b = 2 * math.sqrt(2 / math.pi)
    s = torch.sigmoid(b * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * b * (1 + 3 * 0.044715 * z ** 2)


def product(x, w, bias=None):
    """x w^T + bias, and the bound of its fp32 evaluation."""
    z = x.double() @ w.double().mT
    mag = x.double().abs() @ w.double().abs().mT
    if bias is not None:
        z = z + bias.double()
        mag = mag + bias.double().abs()
    return z, (x.shape[-1] + 2) * ADD * mag


def linear(x, w, bias=None, residual=None, name="none", fp32=False):
    """{"out": (value, bound), "preact": (value, bound)}."""
    z, dz = product(x, w, bias)
    a, _ = act(z, name)
    tol = SLOPE * dz + ACT * a.abs()
    if residual is not None:
        a = a + residual.double()
        tol = tol + ADD * a.abs()
    if not fp32:
        tol = tol + BF16 * (a.abs() + tol)
    return {"out": (a, tol + TINY), "preact": (z, dz + BF16 * (z.abs() + dz) + TINY)}


def gated(x, w, bias=None, name="silu"):
    z, dz = product(x, w, bias)
    g, u = z.chunk(2, dim=-1)
    eg, eu = dz.chunk(2, dim=-1)
    a, _ = act(g, name)
    ea = SLOPE * eg + ACT * a.abs()
    h = a * u
    tol = ea * (u.abs() + eu) + a.abs() * eu + ADD * h.abs()
    return {"out": (h, tol + BF16 * (h.abs() + tol) + TINY),
            "preact": (z, dz + BF16 * (z.abs() + dz) + TINY)}


def backward(dout, x, w, preact, name, is_gated):
    """Gradients of linear (or gated) from the saved preactivations."""
    d = dout.double()
    if is_gated:
        g, u = preact.double().chunk(2, dim=-1)
        a, da = act(g, name)
        dz = torch.cat([d * u * da, d * a], dim=-1)
        # a derivative is within 2^-16 of its terms' magnitudes, at most 1.13
        edz = torch.cat([2 * ACT * (d * u).abs() * SLOPE, 2 * ACT * (d * a).abs()], dim=-1)
    else:
        da = torch.ones_like(d) if preact is None else act(preact.double(), name)[1]
        dz = d * da
        edz = 2 * ACT * d.abs() * SLOPE
    rows = dz.shape[0]
    exact_z = not is_gated and (preact is None or name == "none")
    r = dz.abs() * (0 if exact_z else BF16) + (0 if exact_z else edz)   # dz as the products see it
    wd, xd = w.double(), x.double()
    dx, ex = dz @ wd, r @ wd.abs() + (dz.shape[1] + 2) * ADD * ((dz.abs() + r) @ wd.abs())
    dw, ew = dz.mT @ xd, r.mT @ xd.abs() + (rows + 2) * ADD * ((dz.abs() + r).mT @ xd.abs())
    db = dz.sum(0)
    eb = (0 if exact_z else edz.sum(0)) + (rows + 2) * ADD * dz.abs().sum(0)
    return {k: (v, e + BF16 * (v.abs() + e) + TINY)
            for k, v, e in (("dx", dx, ex), ("dweight", dw, ew), ("dbias", db, eb))}


def layout(ids, E, tile, P):
    """moe_permute in plain Python: (idx_map, row_token, offsets, counts)."""
    T, K = len(ids), len(ids[0]) if len(ids) else 0
    rows = [[] for _ in range(E)]
    for t in range(T):
        for k in range(K):
            if 0 <= ids[t][k] < E:
                rows[ids[t][k]].append((t, k))
    offsets, at = [], 0
    idx = [[-1] * K for _ in range(T)]
    token = [-1] * P
    for e in range(E):
        offsets.append(at)
        for j, (t, k) in enumerate(rows[e]):
            idx[t][k] = at + j
            token[at + j] = t
        at += -(-len(rows[e]) // tile) * tile
    return idx, token, offsets + [at], [len(r) for r in rows]


def check(got, ref, what=""):
    """Every element of got within its bound of the 64-bit value."""
    for key, t in got.items():
        value, tol = ref[key]
        g = t.double()
        assert g.shape == value.shape, (what, key, g.shape, value.shape)
        bad = ~((g - value).abs() <= tol)
        if bad.any():
            i = tuple(bad.nonzero()[0].tolist())
            raise AssertionError(
                f"{what} {key}: {int(bad.sum())} of {bad.numel()} off; first at {i}: "
                f"{g[i].item()!r}, expected {value[i].item()!r} +- {tol[i].item():.3g}")
