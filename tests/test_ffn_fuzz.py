"""Random sizes through every form of the products around the finalize: the
decode kernel, single CTAs and pairs, k in parts, both gradients together, odd
sizes and misaligned operands, ragged expert groups, each against the plain
64-bit implementation with its derived bound (ffn_ref)."""
import random

import pytest
import torch

import ffn_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def size(rng, lo, hi, odd=0.15):
    """Spread over the logarithm; mostly multiples of 8."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, v if rng.random() < odd else -(-v // 8) * 8)


def rows(rng):
    return rng.choice([rng.randint(1, 16), rng.randint(17, 300), rng.randint(300, 3000)])


class Inputs:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def __call__(self, *shape, scale=1.0, shift=False):
        """shift: at an address that is only 2-byte aligned."""
        n = 1
        for d in shape:
            n *= d
        t = torch.empty(n + 1, dtype=BF16, device="cuda")[int(shift):n + int(shift)].view(shape)
        return t.normal_(0.0, scale, generator=self.g)


def run_case(mf, seed):
    rng = random.Random(seed)
    rand = Inputs(seed)
    op = rng.choice(["linear", "linear", "gated", "linear_backward", "gated_backward", "experts"])
    name = rng.choice(R.ACTS)
    T = rows(rng)
    shift = [rng.random() < 0.1 for _ in range(4)]
    if op == "linear":
        N, K = size(rng, 1, 3000), size(rng, 1, 3000)
        x, w = rand(T, K, shift=shift[0]), rand(N, K, scale=K ** -0.5, shift=shift[1])
        b = rand(N) if rng.random() < 0.5 else None
        r = rand(T, N, shift=shift[2]) if rng.random() < 0.5 else None
        f32, save = rng.random() < 0.3, rng.random() < 0.3
        what = f"{op} T={T} N={N} K={K} {name} bias={b is not None} res={r is not None} f32={f32}"
        got = mf.linear(x, w, bias=b, residual=r, activation=name, save_preact=save,
                        out_dtype=torch.float32 if f32 else BF16)
        R.check(got, R.linear(x, w, b, r, name, f32), what)
    elif op == "gated":
        I, H = size(rng, 1, 2000), size(rng, 1, 3000)
        x, w = rand(T, H, shift=shift[0]), rand(2 * I, H, scale=H ** -0.5, shift=shift[1])
        b = rand(2 * I) if rng.random() < 0.5 else None
        what = f"{op} T={T} I={I} H={H} {name} bias={b is not None}"
        R.check(mf.gated_ffn(x, w, bias=b, activation=name, save_preact=rng.random() < 0.5),
                R.gated(x, w, b, name), what)
    elif op == "linear_backward":
        N, K = size(rng, 1, 2000), size(rng, 1, 2000)
        x, w = rand(T, K), rand(N, K, scale=K ** -0.5)
        d = rand(T, N, scale=0.1, shift=shift[0])
        pre = None if name == "none" else rand(T, N)
        got = mf.linear_backward(d, x, w, activation=name, preact=pre, want_dbias=True)
        R.check(got, R.backward(d, x, w, pre, name, False), f"{op} T={T} N={N} K={K} {name}")
    elif op == "gated_backward":
        I, H = size(rng, 1, 1200), size(rng, 1, 2000)
        x, w, d = rand(T, H), rand(2 * I, H, scale=H ** -0.5), rand(T, I, scale=0.1)
        pre = rand(T, 2 * I)
        got = mf.gated_ffn_backward(d, x, w, pre, activation=name, want_dbias=True)
        R.check(got, R.backward(d, x, w, pre, name, True), f"{op} T={T} I={I} H={H} {name}")
    else:
        E, K, tile = rng.randint(1, 40), rng.randint(1, 4), rng.choice([1, 3, 16, 128])
        H, I = size(rng, 8, 1000), size(rng, 1, 600)
        what = f"{op} T={T} K={K} E={E} tile={tile} H={H} I={I} {name}"
        ids = torch.randint(-1, E + 1, (T, K), generator=rand.g, device="cuda",
                            dtype=torch.int32)
        if rng.random() < 0.3:          # one expert takes most
            ids[torch.rand(T, K, generator=rand.g, device="cuda") < 0.8] = rng.randrange(E)
        m = mf.permute_tokens(ids, E, tile)
        ref = R.layout(ids.tolist(), E, tile, m["row_token"].numel())
        for key, r in zip(("idx_map", "row_token", "offsets", "counts"), ref):
            assert torch.equal(m[key].cpu(), torch.tensor(r, dtype=torch.int32)), (what, key)
        x, w13 = rand(T, H), rand(E, 2 * I, H, scale=H ** -0.5)
        w2 = rand(E, H, I, scale=I ** -0.5)
        b = rand(E, 2 * I) if rng.random() < 0.5 else None
        P = m["row_token"].numel()
        h = torch.full((P, I), 5.0, dtype=BF16, device="cuda")
        y = torch.full((P, H), 5.0, dtype=BF16, device="cuda")
        mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w13, bias=b,
                            activation=name, out=h)
        mf.expert_linear(h, m["offsets"], m["counts"], w2, out=y)
        unused = torch.ones(P, dtype=torch.bool, device="cuda")
        for e, (first, count) in enumerate(zip(ref[2], ref[3])):
            if count:
                s = slice(first, first + count)
                unused[s] = False
                xe = x[m["row_token"][s].long()]
                R.check({"out": h[s]}, R.gated(xe, w13[e], None if b is None else b[e], name),
                        f"{what} expert {e} up")
                R.check({"out": y[s]}, R.linear(h[s], w2[e]), f"{what} expert {e} down")
        assert (h[unused] == 5).all() and (y[unused] == 5).all(), what


@pytest.mark.parametrize("seed", range(60))
def test_random_case(cuda_lib, seed):
    run_case(cuda_lib, seed)
    assert cuda_lib.lost_waits() == 0
