"""The activations far out: values and derivatives over |z| <= 14 against 64 bits,
at the ends of the number range, and at infinities and NaN.

Bounds, in units of 2^-23 (an fp32 rounding is half a unit, ex2.approx two, and
rcp.approx one), relative to the value:
  silu       exp's argument carries two roundings, |z| units into the sigmoid; with
             ex2, 1 + e, rcp and the product 4 more: |z| + 4
  gelu_tanh  the argument q = 2 sqrt(2/pi) (z + 0.044715 z^3) carries nine
             roundings (constants and products; both terms have one sign): 4.5 |q| + 4
  gelu       Phi(-u) = poly(t) exp(-u^2 / 2): three roundings of the argument
             u^2 / 2 give 0.75 u^2; the fit 2.9, t's 2.5 at a slope of at most 2.3
             5.8, Horner's steps 3, ex2 2 and two products 1: 0.75 z^2 + 15
Derivatives carry these into each of their terms; 1 - s of a sigmoid is off by 5
units whatever its size.  Below 2^-126 the sigmoid and the bell are 0, which costs
|z| 2^-125 at most.  z itself is exact: one product of two bf16 values.
"""
import math

import pytest
import torch

import ffn_ref as R

BF16 = torch.bfloat16
UNIT = 2.0 ** -23
FAR = [2.0 ** k for k in (5, 6, 7, 20, 63, 64, 100, 126, 127)] + [3.38e38]
NAMES = ("silu", "gelu", "gelu_tanh", "relu")


def grid(device="cpu"):
    """bf16 values: |z| <= 14, around 0, and far out."""
    near = torch.linspace(-14, 14, 701, dtype=torch.float64)
    tiny = torch.tensor([0.0, 1e-3, 1e-6, 2.0 ** -60, 2.0 ** -126], dtype=torch.float64)
    far = torch.tensor(FAR, dtype=torch.float64)
    z = torch.cat([near, tiny, -tiny, far, -far]).to(BF16)
    return torch.cat([z, z[:-z.numel() % 8]]).to(device)        # a multiple of 8


def units(z, name):
    """Relative error of act(z) in units."""
    a = z.abs()
    if name == "silu":
        return a + 4
    if name == "gelu":
        return 0.75 * a * a + 15
    if name == "gelu_tanh":
        return 4.5 * 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3) + 4
    return torch.zeros_like(a)


def value(z, name):
    """act(z) in 64 bits and the bound of the fp32 form."""
    v = R.act(z, name)[0]
    # above 30 the sigmoid is 1 to the last bit (exp(-30) < 2^-43); below -30 it is
    # still a number, down to -88 for silu, and its error keeps growing with |z|
    u = torch.where(z > 30, torch.full_like(z, 4.0), units(z.clamp(min=-200), name))
    return v, u * UNIT * v.abs() + (z.abs().clamp(max=200) + 1) * 2.0 ** -125


def slope(z, name):
    """act'(z) likewise."""
    v = R.act(z, name)[1]
    a = z.abs()
    u, flushed = units(z.clamp(min=-200), name), (a.clamp(max=200) ** 3 + 1) * 2.0 ** -125
    if name == "relu":
        return v, torch.zeros_like(v)
    if name == "silu":
        s = torch.sigmoid(z)
        e = s * (1 + a * (1 - s)) * u + s * a * 5
    elif name == "gelu":
        bell = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        e = 0.5 * torch.erfc(-z / math.sqrt(2)) * u + a * bell * u
    else:
        s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        outer = a * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        e = s * u + s * ((1 - s) * u + 5) * outer
        e = torch.where(s > 0, e, torch.zeros_like(e))
    e = torch.where(z > 30, torch.full_like(e, 1.0), e)        # the slope is 1
    return v, (e + 1) * UNIT * (e != 0) + flushed


def rounded(ref):
    v, e = ref
    return v, e + R.BF16 * (v.abs() + e) + 2.0 ** -133


def close(got, ref, what):
    v, tol = ref
    bad = ~((got.double() - v).abs() <= tol)
    assert not bad.any(), (what, [(got.flatten()[i].item(), v.flatten()[i].item(),
                                   tol.flatten()[i].item())
                                  for i in bad.flatten().nonzero()[:3, 0].tolist()])


@pytest.mark.parametrize("name", NAMES)
def test_bounds_are_small_next_to_a_bf16_rounding(name):
    """The bounds above stay below an eighth of a rounding to bf16 for |z| <= 9 in
    value, so that the tests below see the functions and not the bounds."""
    z = grid().double()
    z = z[(z.abs() <= 9) & (z != 0)]
    v, e = value(z, name)
    assert (e <= R.BF16 / 8 * v.abs() + 2.0 ** -120).all()
    _, e = slope(z, name)
    assert (e <= R.BF16 / 8).all()


FACTORS = (1.0, 255 / 256, 0.75, 129 / 256)


def operands(T, K, device="cuda"):
    """x [T, K] and w [N, K] with z[t, n] = factor of row t times grid value n."""
    w = torch.zeros(grid().numel(), K, dtype=BF16, device=device)
    w[:, 0] = grid(device)
    x = torch.zeros(T, K, dtype=BF16, device=device)
    x[:, 0] = torch.tensor([FACTORS[t % 4] for t in range(T)], dtype=BF16, device=device)
    return x, w, x[:, :1].double() * w[:, 0].double()


# decode kernel, tensor cores (single CTAs, pairs), single-value loads
FORMS = [(1, 8), (8, 8), (40, 8), (1030, 8), (5, 9)]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("T,K", FORMS)
def test_values(cuda_lib, name, T, K):
    x, w, z = operands(T, K)
    ref = value(z, name)
    close(cuda_lib.linear(x, w, activation=name, out_dtype=torch.float32)["out"], ref, "fp32")
    got = cuda_lib.linear(x, w, activation=name, save_preact=True)
    close(got["out"], rounded(ref), "bf16")
    assert torch.equal(got["preact"], z.to(BF16))
    # odd feature counts leave the wide epilogue
    close(cuda_lib.linear(x, w[:-1], activation=name)["out"], rounded((ref[0][:, :-1],
                                                                       ref[1][:, :-1])), "odd")


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("T,K", FORMS)
def test_gated_values(cuda_lib, name, T, K):
    x, w, z = operands(T, K)
    up = torch.zeros_like(w)
    up[:, 1] = 1
    x[:, 1] = 1
    got = cuda_lib.gated_ffn(x, torch.cat([w, up]), activation=name)["out"]
    close(got, rounded(value(z, name)), name)
    # one expert's rows
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    counts = torch.tensor([T], dtype=torch.int32, device="cuda")
    got = cuda_lib.expert_gated_ffn(x, None, offsets, counts, torch.cat([w, up])[None],
                                    activation=name)
    close(got, rounded(value(z, name)), name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("odd", [0, 1])
def test_slopes(cuda_lib, name, odd):
    """dout = 1 in one row: the bias gradient is dz itself, rounded once.  An odd
    number of features takes the single-value form of the pass."""
    pre = grid("cuda")[None, odd:].contiguous()
    n = pre.shape[1]
    z = pre.double()
    one = torch.ones(1, n, dtype=BF16, device="cuda")
    x, w = torch.ones(1, 8, dtype=BF16, device="cuda"), torch.zeros(n, 8, dtype=BF16, device="cuda")
    got = cuda_lib.linear_backward(one, x, w, activation=name, preact=pre, want_dbias=True)
    d = slope(z, name)
    close(got["dbias"][None], rounded(d), "dbias")
    close(got["dweight"], tuple(t.mT.expand(n, 8) for t in rounded(d)), "dweight")
    both = torch.cat([pre, one], dim=1)         # up = 1: dz is act' and act
    got = cuda_lib.gated_ffn_backward(one, x, torch.cat([w, w]), both, activation=name,
                                      want_dbias=True)
    close(got["dbias"][None, :n], rounded(d), "gate")
    close(got["dbias"][None, n:], rounded(value(z, name)), "up")


@pytest.mark.gpu
@pytest.mark.parametrize("name", ("none",) + NAMES)
@pytest.mark.parametrize("T,K", FORMS)
def test_infinities_and_nan(cuda_lib, name, T, K):
    """inf gives inf, NaN gives NaN; -inf gives what the formulas give in IEEE
    arithmetic: NaN (-inf times 0), 0 for relu and -inf for none.  Neighbouring
    features and the zeros beside them are not touched."""
    inf, nan = float("inf"), float("nan")
    x, w, z = operands(T, K)
    types = (torch.float32, BF16)
    clean = [cuda_lib.linear(x, w, activation=name, out_dtype=dt)["out"] for dt in types]
    w[3, 0], w[11, 0], w[17, 0] = inf, -inf, nan
    want = {3: inf, 11: {"none": -inf, "relu": 0.0}.get(name, nan), 17: nan}
    for dt, before in zip(types, clean):
        got = cuda_lib.linear(x, w, activation=name, out_dtype=dt)["out"]
        for n, v in want.items():
            col = got[:, n].float()
            assert (col.isnan() if v != v else col == v).all(), (n, dt)
        keep = [n for n in range(w.shape[0]) if n not in want]
        assert torch.equal(got[:, keep], before[:, keep])


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_slopes_at_infinities_and_nan(cuda_lib, name):
    """NaN gives NaN (relu: 0, as the comparison says); at infinities the limit or
    NaN, which the formulas give where they multiply one by 0."""
    pre = torch.tensor([[float("inf"), -float("inf"), float("nan"), 1.0] * 2], dtype=BF16,
                       device="cuda")
    one = torch.ones_like(pre)
    x, w = torch.ones(1, 8, dtype=BF16, device="cuda"), torch.zeros(8, 8, dtype=BF16, device="cuda")
    got = cuda_lib.linear_backward(one, x, w, activation=name, preact=pre,
                                   want_dbias=True)["dbias"].tolist()
    for at in (0, 4):
        assert got[at] == 1 or (got[at] != got[at] and name != "relu")
        assert got[at + 1] == 0 or (got[at + 1] != got[at + 1] and name != "relu")
        assert got[at + 2] == 0 if name == "relu" else got[at + 2] != got[at + 2]
        assert abs(got[at + 3] - R.act(torch.ones(1).double(), name)[1].item()) < 2.0 ** -7
