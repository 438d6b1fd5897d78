"""The products around the finalize on the GPU, against plain 64-bit
implementations with bounds derived from their roundings (ffn_ref)."""
import pytest
import torch

import ffn_ref as R

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(0.0, scale, generator=g)


def misaligned(t):
    """The same values at an address that is only 2-byte aligned."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


# T, N, K: one token and one value, sizes off and on every tile, odd sizes
LINEAR_SHAPES = [(1, 1, 1), (1, 256, 512), (3, 8, 64), (7, 40, 72), (16, 128, 64), (17, 136, 200),
                 (64, 300, 128), (100, 1000, 24), (129, 257, 136), (255, 512, 512),
                 (256, 264, 1024), (300, 384, 4096), (513, 520, 328), (1100, 640, 256),
                 (5, 13, 77), (130, 67, 333)]


@pytest.mark.parametrize("T,N,K", LINEAR_SHAPES)
def test_linear_shapes(cuda_lib, T, N, K):
    x, w = rand(1, T, K), rand(2, N, K, scale=K ** -0.5)
    R.check(cuda_lib.linear(x, w), R.linear(x, w), f"{T}x{N}x{K}")


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("T,N,K", [(1, 264, 512), (37, 200, 136), (300, 520, 264), (9, 35, 51)])
def test_linear_epilogue(cuda_lib, name, T, N, K):
    x, w, b, r = rand(3, T, K), rand(4, N, K, scale=K ** -0.5), rand(5, N), rand(6, T, N, scale=2)
    for bias in (None, b):
        for res in (None, r):
            for dt in (BF16, torch.float32):
                got = cuda_lib.linear(x, w, bias=bias, residual=res, activation=name,
                                      out_dtype=dt, save_preact=True)
                assert got["out"].dtype == dt
                R.check(got, R.linear(x, w, bias, res, name, dt == torch.float32),
                        f"{name} bias={bias is not None} res={res is not None} {dt}")


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 192, 257,
                               1025])
def test_linear_every_row_count_class(cuda_lib, T):
    x, w = rand(7, T, 320), rand(8, 392, 320, scale=0.05)
    R.check(cuda_lib.linear(x, w), R.linear(x, w), f"T={T}")


def test_linear_in_place_residual_and_given_outputs(cuda_lib):
    x, w, r = rand(9, 70, 256), rand(10, 264, 256, scale=0.06), rand(11, 70, 264)
    ref = R.linear(x, w, None, r, "silu")
    pre = torch.empty(70, 264, dtype=BF16, device="cuda")
    got = cuda_lib.linear(x, w, residual=r, activation="silu", out=r, preact=pre)
    assert got["out"] is r and got["preact"] is pre
    R.check(got, ref)


@pytest.mark.parametrize("T,N,K", [(1, 264, 512), (5, 264, 512), (12, 640, 4096), (64, 264, 8192),
                                   (300, 264, 4096), (2000, 1000, 264)])
def test_in_place_residual_in_every_form(cuda_lib, T, N, K):
    """Decode kernel, single tiles, k in parts, pairs: out is the residual."""
    x, w, r = rand(18, T, K), rand(19, N, K, scale=K ** -0.5), rand(20, T, N)
    ref = R.linear(x, w, None, r, "gelu_tanh")
    want = cuda_lib.linear(x, w, residual=r, activation="gelu_tanh")["out"]
    got = cuda_lib.linear(x, w, residual=r, activation="gelu_tanh", out=r)
    R.check(got, ref)
    assert torch.equal(got["out"], want)


def test_linear_misaligned_operands(cuda_lib):
    x, w, b, r = rand(12, 33, 128), rand(13, 72, 128, scale=0.1), rand(14, 72), rand(15, 33, 72)
    ref = R.linear(x, w, b, r, "gelu")
    for k in range(4):
        a = [misaligned(t) if i == k else t for i, t in enumerate((x, w, b, r))]
        out = misaligned(torch.zeros(33, 72, dtype=BF16, device="cuda"))
        R.check(cuda_lib.linear(a[0], a[1], bias=a[2], residual=a[3], activation="gelu", out=out),
                ref, f"operand {k}")


def test_non_finite_rows_stay_in_their_rows(cuda_lib):
    x, w = rand(16, 40, 192), rand(17, 200, 192, scale=0.1)
    clean = cuda_lib.linear(x, w)["out"]
    x2 = x.clone()
    x2[5, 3] = float("nan")
    x2[11, 100] = float("inf")
    got = cuda_lib.linear(x2, w)["out"]
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[5] = keep[11] = False
    assert torch.equal(got[keep], clean[keep])
    assert got[5].isnan().all() and not got[11].isfinite().any()


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("T,I,H", [(1, 64, 256), (1, 8, 64), (5, 200, 136), (33, 136, 512),
                                   (300, 264, 264), (700, 72, 128), (6, 21, 35)])
def test_gated_ffn(cuda_lib, name, T, I, H):
    x, w, b = rand(20, T, H), rand(21, 2 * I, H, scale=H ** -0.5), rand(22, 2 * I)
    for bias in (None, b):
        for save in (False, True):
            got = cuda_lib.gated_ffn(x, w, bias=bias, activation=name, save_preact=save)
            assert set(got) == ({"out", "preact"} if save else {"out"})
            R.check(got, R.gated(x, w, bias, name), f"{name} bias={bias is not None}")


@pytest.mark.parametrize("T,I,H", [(1, 1, 1), (2, 2048, 1024), (64, 320, 2048), (200, 1024, 520),
                                   (1030, 264, 136)])
def test_gated_ffn_shapes(cuda_lib, T, I, H):
    x, w = rand(23, T, H), rand(24, 2 * I, H, scale=H ** -0.5)
    R.check(cuda_lib.gated_ffn(x, w, save_preact=True), R.gated(x, w), f"{T}x{I}x{H}")


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("T,N,K", [(1, 64, 128), (40, 72, 136), (300, 264, 520), (777, 128, 256),
                                   (33, 35, 51)])
def test_linear_backward(cuda_lib, name, T, N, K):
    x, w, d = rand(30, T, K), rand(31, N, K, scale=K ** -0.5), rand(32, T, N, scale=0.1)
    pre = None if name == "none" else cuda_lib.linear(x, w, save_preact=True)["preact"]
    got = cuda_lib.linear_backward(d, x, w, activation=name, preact=pre, want_dbias=True)
    R.check(got, R.backward(d, x, w, pre, name, False), name)


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("T,I,H", [(1, 64, 128), (40, 72, 136), (300, 264, 520), (777, 64, 256),
                                   (33, 19, 51)])
def test_gated_ffn_backward(cuda_lib, name, T, I, H):
    x, w, d = rand(33, T, H), rand(34, 2 * I, H, scale=H ** -0.5), rand(35, T, I, scale=0.1)
    pre = cuda_lib.gated_ffn(x, w, activation=name, save_preact=True)["preact"]
    got = cuda_lib.gated_ffn_backward(d, x, w, pre, activation=name, want_dbias=True)
    R.check(got, R.backward(d, x, w, pre, name, True), name)


@pytest.mark.parametrize("T", [16384, 16385, 40001])
@pytest.mark.parametrize("n", [1, 5, 8, 24, 64, 100, 264, 520])
def test_backward_of_many_rows(cuda_lib, T, n):
    """The column sums of many rows, over few and many columns."""
    x, w, d = rand(60, T, 64), rand(61, n, 64, scale=0.1), rand(62, T, n, scale=0.1)
    pre = cuda_lib.linear(x, w, save_preact=True)["preact"]
    got = cuda_lib.linear_backward(d, x, w, activation="silu", preact=pre, want_dbias=True)
    ref = R.backward(d, x, w, pre, "silu", False)
    R.check(got, ref, "linear")
    got = cuda_lib.linear_backward(d, x, w, activation="silu", preact=pre, want_dx=False,
                                   want_dweight=False, want_dbias=True)
    R.check(got, {"dbias": ref["dbias"]}, "dbias alone")
    w = rand(63, 2 * n, 64, scale=0.1)
    pre = cuda_lib.gated_ffn(x, w, save_preact=True)["preact"]
    got = cuda_lib.gated_ffn_backward(d, x, w, pre, want_dbias=True)
    R.check(got, R.backward(d, x, w, pre, "silu", True), "gated")


def test_backward_gives_what_is_wanted(cuda_lib):
    x, w, d = rand(36, 40, 64), rand(37, 48, 64), rand(38, 40, 48)
    full = cuda_lib.linear_backward(d, x, w, want_dbias=True)
    for key in ("dx", "dweight", "dbias"):
        want = {f"want_{k}": k == key for k in ("dx", "dweight", "dbias")}
        got = cuda_lib.linear_backward(d, x, w, **want)
        assert set(got) == {key} and torch.equal(got[key], full[key])
    ws = torch.empty(cuda_lib.linear_backward_workspace_bytes(40, 48), dtype=torch.uint8,
                     device="cuda")
    given = torch.empty(48, 64, dtype=BF16, device="cuda")
    got = cuda_lib.linear_backward(d, x, w, want_dx=False, dweight=given, workspace=ws)
    assert got["dweight"] is given and torch.equal(given, full["dweight"])


def test_backward_of_no_rows_is_zero(cuda_lib):
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    for gated, n in ((False, 48), (True, 24)):
        w = rand(39, 48, 64)
        d = torch.empty(0, n, dtype=BF16, device="cuda")
        if gated:
            got = cuda_lib.gated_ffn_backward(d, x, w, torch.empty(0, 48, dtype=BF16, device="cuda"),
                                              want_dbias=True)
        else:
            got = cuda_lib.linear_backward(d, x, w, want_dbias=True)
        assert got["dx"].shape == (0, 64)
        assert not got["dweight"].any() and got["dweight"].shape == (48, 64)
        assert not got["dbias"].any()
    assert cuda_lib.linear(x, rand(1, 8, 64))["out"].shape == (0, 8)
    assert cuda_lib.gated_ffn(x, rand(1, 8, 64))["out"].shape == (0, 4)


def test_gradient_against_differences(cuda_lib):
    """dx and dweight of a linear GELU layer against central differences of
    the fp32 forward.  x, the weights and the steps are multiples of 2^-6 below
    4, so x +- step is exact in bf16.  L = sum(dout * out): a central
    difference with step e is off by e^2 / 6 |L'''| from curvature and by the
    forward's own error over e."""
    g = torch.Generator().manual_seed(5)
    T, N, K, e = 24, 40, 64, 2.0 ** -5
    x = (torch.randint(-32, 33, (T, K), generator=g).double() / 32)
    w = (torch.randint(-16, 17, (N, K), generator=g).double() / 64)
    d = (torch.randint(-8, 9, (T, N), generator=g).double() / 8)
    vx = torch.randint(0, 2, (T, K), generator=g).double() * 2 - 1
    vw = torch.randint(0, 2, (N, K), generator=g).double() * 2 - 1

    def dev(t):
        b = t.to(BF16)
        assert torch.equal(b.double(), t)
        return b.cuda()

    def loss(xx, ww):
        out = cuda_lib.linear(dev(xx), dev(ww), activation="gelu",
                              out_dtype=torch.float32)["out"].cpu().double()
        return (d * out).sum().item()

    pre = cuda_lib.linear(dev(x), dev(w), activation="gelu", save_preact=True)["preact"]
    grads = cuda_lib.linear_backward(dev(d), dev(x), dev(w), activation="gelu", preact=pre)
    for key, (xx, ww), v in (("dx", (vx, 0 * w), vx), ("dweight", (0 * x, vw), vw)):
        diff = (loss(x + e * xx, w + e * ww) - loss(x - e * xx, w - e * ww)) / (2 * e)
        slope = (grads[key].cpu().double() * v).sum().item()
        dz = (xx @ w.mT + x @ ww.mT).abs()              # dz / de of each element
        curvature = (d.abs() * dz ** 3 * 2.0).sum().item() * e * e / 6   # |gelu'''| < 2
        zmag = x.abs() @ w.abs().mT
        forward = (d.abs() * (1.13 * (K + 2) * R.ADD * zmag * 2 + R.ACT * zmag)).sum().item() / e
        # dz's rounding, the saved preactivation's and the gradient's own
        ref = grads[key].cpu().double().abs().sum().item()
        path = (d.abs() @ w.abs()).sum().item() if key == "dx" else (d.abs().mT @ x.abs()).sum().item()
        rounding = R.BF16 * (ref + 1.13 * path) + 0.8 * R.BF16 * (
            (d.abs() * zmag) @ w.abs()).sum().item() * (key == "dx") + 0.8 * R.BF16 * (
            (d.abs() * zmag).mT @ x.abs()).sum().item() * (key == "dweight")
        assert abs(diff - slope) <= curvature + forward + rounding
        # a wrong sign, scale or missing derivative shows: the slope is large
        assert abs(slope) > 0 and abs(diff - slope) < 0.05 * (abs(slope) + abs(diff)) + 1.0


def test_equal_calls_give_equal_bits(cuda_lib):
    x, w, d = rand(40, 333, 512), rand(41, 400, 512, scale=0.05), rand(42, 333, 200)
    pre = cuda_lib.gated_ffn(x, w, save_preact=True)["preact"]
    first = cuda_lib.gated_ffn_backward(d, x, w, pre, want_dbias=True)
    for _ in range(3):
        again = cuda_lib.gated_ffn_backward(d, x, w, pre, want_dbias=True)
        for key in first:
            assert torch.equal(first[key], again[key]), key
    for T in (1, 9, 70):
        a = cuda_lib.linear(x[:T].contiguous(), w)["out"]
        assert torch.equal(a, cuda_lib.linear(x[:T].contiguous(), w)["out"])


# ---------------------------------------------------------------- row map


def ids_of(seed, T, K, E, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((T, K), E - 1, dtype=torch.int32)
    if kind == "none":
        return torch.full((T, K), -1, dtype=torch.int32)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)     # repeats in a token too
    if kind == "holes":
        ids[torch.rand(T, K, generator=g) < 0.3] = -1
        ids[torch.rand(T, K, generator=g) < 0.05] = E
        ids[torch.rand(T, K, generator=g) < 0.05] = 2 ** 31 - 1
    return ids


@pytest.mark.parametrize("kind", ["all", "holes", "one", "none"])
@pytest.mark.parametrize("T,K,E,tile", [(1, 1, 1, 1), (1, 8, 256, 128), (7, 3, 5, 4),
                                        (256, 8, 256, 128), (300, 6, 60, 16), (1000, 2, 8, 64),
                                        (5000, 8, 384, 1), (2049, 4, 1024, 7), (341, 6, 33, 3),
                                        (16384, 8, 256, 128), (16385, 8, 60, 2),
                                        (2200, 8, 1024, 3), (2048, 8, 1024, 1),
                                        (40000, 8, 128, 32)])
def test_permute(cuda_lib, kind, T, K, E, tile):
    ids = ids_of(T + K, T, K, E, kind)
    got = cuda_lib.permute_tokens(ids.cuda(), E, tile)
    P = got["row_token"].numel()
    assert P == cuda_lib.permute_rows(T, K, E, tile)
    ref = R.layout(ids.tolist(), E, tile, P)
    for key, r in zip(("idx_map", "row_token", "offsets", "counts"), ref):
        assert torch.equal(got[key].cpu(), torch.tensor(r, dtype=torch.int32)), key


def test_permute_larger_row_buffer_and_no_tokens(cuda_lib):
    ids = ids_of(3, 50, 4, 16, "all")
    row_token = torch.full((5000,), 77, dtype=torch.int32, device="cuda")
    got = cuda_lib.permute_tokens(ids.cuda(), 16, 8, row_token=row_token)
    ref = R.layout(ids.tolist(), 16, 8, 5000)
    assert torch.equal(got["row_token"].cpu(), torch.tensor(ref[1], dtype=torch.int32))
    empty = cuda_lib.permute_tokens(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 16, 8,
                                    row_token=row_token)
    assert not empty["offsets"].any() and not empty["counts"].any()
    assert (row_token == -1).all()


# --------------------------------------------------------- expert products


def experts_case(mf, T, K, E, tile, kind="holes", seed=50):
    ids = ids_of(seed, T, K, E, kind)
    return mf.permute_tokens(ids.cuda(), E, tile)


def check_experts(mf, T, K, E, tile, H, I, name, bias, kind):
    m = experts_case(mf, T, K, E, tile, kind)
    P = m["row_token"].numel()
    x = rand(51, T, H)
    w13, w2 = rand(52, E, 2 * I, H, scale=H ** -0.5), rand(53, E, H, I, scale=I ** -0.5)
    b13, b2 = (rand(54, E, 2 * I), rand(55, E, H)) if bias else (None, None)
    h = torch.full((P, I), 7.0, dtype=BF16, device="cuda")
    y = torch.full((P, H), 7.0, dtype=BF16, device="cuda")
    assert mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w13, bias=b13,
                               activation=name, out=h) is h
    mf.expert_linear(h, m["offsets"], m["counts"], w2, bias=b2, out=y)
    direct = mf.expert_linear(x, m["offsets"], m["counts"], w13, row_token=m["row_token"],
                              bias=b13, activation=name)
    valid = torch.zeros(P, dtype=torch.bool, device="cuda")
    for e, (first, count) in enumerate(zip(m["offsets"].tolist(), m["counts"].tolist())):
        if not count:
            continue
        rows = slice(first, first + count)
        valid[rows] = True
        xe = x[m["row_token"][rows].long()]
        R.check({"out": h[rows]}, R.gated(xe, w13[e], None if b13 is None else b13[e], name),
                f"expert {e} up")
        R.check({"out": y[rows]}, R.linear(h[rows], w2[e], None if b2 is None else b2[e]),
                f"expert {e} down")
        R.check({"out": direct[rows]}, R.linear(xe, w13[e], None if b13 is None else b13[e],
                                                name=name), f"expert {e} gathered linear")
    assert (h[~valid] == 7).all() and (y[~valid] == 7).all()


@pytest.mark.parametrize("T,K,E,tile,H,I", [(1, 8, 16, 128, 256, 64), (1, 1, 1, 1, 64, 8),
                                            (16, 4, 8, 16, 264, 136), (100, 2, 4, 1, 128, 72),
                                            (333, 3, 3, 64, 200, 264), (900, 2, 5, 7, 72, 40),
                                            (40, 4, 60, 8, 512, 128), (12, 2, 6, 4, 35, 21)])
def test_experts(cuda_lib, T, K, E, tile, H, I):
    check_experts(cuda_lib, T, K, E, tile, H, I, "silu", False, "holes")


@pytest.mark.parametrize("name", R.ACTS)
def test_experts_epilogues(cuda_lib, name):
    check_experts(cuda_lib, 60, 3, 5, 8, 136, 72, name, True, "all")


@pytest.mark.parametrize("kind", ["one", "none"])
def test_experts_all_rows_in_one_expert_and_none_at_all(cuda_lib, kind):
    check_experts(cuda_lib, 300, 2, 6, 16, 128, 64, "silu", False, kind)


@pytest.mark.parametrize("T,K,E,tile,H,I", [(1, 2, 128, 1, 3016, 256), (13, 8, 8, 128, 5400, 320),
                                            (5, 1, 3, 4, 4096, 72), (1, 1, 1, 1, 7168, 64),
                                            (2, 4, 8, 1, 2048, 1000), (90, 4, 16, 64, 3000, 184),
                                            (200, 1, 2, 1, 4104, 136), (3, 3, 7, 16, 2056, 2000)])
@pytest.mark.parametrize("kind", ["all", "holes", "one"])
def test_experts_with_few_tiles_and_long_sums(cuda_lib, T, K, E, tile, H, I, kind):
    check_experts(cuda_lib, T, K, E, tile, H, I, "gelu", True, kind)


def test_experts_graph_replays_where_the_split_differs(cuda_lib):
    """One captured call on routings from one group to many: equal to the eager
    call's bits, and the same again."""
    T, E, H, I = 24, 16, 4096, 264
    x, w = rand(5, T, H), rand(6, E, 2 * I, H, scale=0.02)
    wd = rand(7, E, 1000, I, scale=0.05)
    ids = ids_of(1, T, 1, E, "all").cuda()
    h = torch.zeros(cuda_lib.permute_rows(T, 1, E, 1), I, dtype=BF16, device="cuda")
    y = torch.zeros(h.shape[0], 1000, dtype=BF16, device="cuda")

    def step():
        m = cuda_lib.permute_tokens(ids, E, 1)
        cuda_lib.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w, out=h)
        cuda_lib.expert_linear(h, m["offsets"], m["counts"], wd, out=y)
        return m

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m = step()
    for groups in (1, 2, 3, 5, 11, 16, 4, 1):
        ids.copy_((torch.arange(T, device="cuda") % groups).int()[:, None])
        h.zero_()
        step()
        want = h.clone(), y.clone()
        for _ in range(3):
            h.zero_()
            y.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(h, want[0]) and torch.equal(y, want[1]), groups
        rows = slice(int(m["offsets"][0]), int(m["offsets"][0]) + int(m["counts"][0]))
        R.check({"out": h[rows]}, R.gated(x[m["row_token"][rows].long()], w[0]), f"{groups}")


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("T,K,N", [(3, 4096, 264), (40, 2048, 264), (70, 512, 136),
                                   (300, 128, 1032)])
def test_outputs_at_any_offset(cuda_lib, T, K, N, offset):
    """Aligned operands, outputs (and residual) of an allocation at 0, 2 and 8
    bytes: the same values, nothing written around them."""
    def view(rows, cols, fill):
        flat = torch.full((rows * cols + offset + 8,), fill, dtype=BF16, device="cuda")
        return flat, flat[offset:offset + rows * cols].view(rows, cols)

    def untouched(flat, rows, cols):
        return (flat[:offset] == 9).all() and (flat[offset + rows * cols:] == 9).all()

    x, w, b, r = rand(8, T, K), rand(9, 2 * N, K, scale=0.03), rand(10, 2 * N), rand(11, T, N)
    res = view(T, N, 9.0)[1].copy_(r)
    (of, out), (pf, pre) = view(T, N, 9.0), view(T, N, 9.0)
    cuda_lib.linear(x, w[:N], bias=b[:N], residual=res, activation="silu", out=out, preact=pre)
    R.check({"out": out, "preact": pre}, R.linear(x, w[:N], b[:N], r, "silu"), "linear")
    assert untouched(of, T, N) and untouched(pf, T, N)
    (of, out), (pf, pre) = view(T, N, 9.0), view(T, 2 * N, 9.0)
    cuda_lib.gated_ffn(x, w, bias=b, out=out, preact=pre)
    R.check({"out": out, "preact": pre}, R.gated(x, w, b), "gated")
    assert untouched(of, T, N) and untouched(pf, T, 2 * N)
    m = cuda_lib.permute_tokens(torch.arange(T, dtype=torch.int32, device="cuda")[:, None] % 2, 2)
    of, out = view(T, N, 9.0)
    cuda_lib.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"],
                              torch.stack([w, w.flip(0)]), out=out)
    rows = m["row_token"].long()
    split = int(m["offsets"][1])
    R.check({"out": out[:split]}, R.gated(x[rows[:split]], w), "expert 0")
    R.check({"out": out[split:]}, R.gated(x[rows[split:]], w.flip(0)), "expert 1")
    assert untouched(of, T, N)


def test_experts_at_the_most_experts(cuda_lib):
    check_experts(cuda_lib, 700, 2, 1024, 2, 64, 24, "silu", True, "holes")


def test_experts_rows_beyond_the_buffer_and_tokens_beyond_x(cuda_lib):
    """Rows at or past P are not computed; a row_token outside [0, T) is a row
    of zeros."""
    H, I, E = 128, 64, 2
    x, w = rand(60, 10, H), rand(61, E, 2 * I, H, scale=0.1)
    row_token = torch.tensor([0, 1, 12, -1, 4, 5, 6, 7], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 4, 40], dtype=torch.int32, device="cuda")
    counts = torch.tensor([4, 30], dtype=torch.int32, device="cuda")
    guard = torch.full((12, I), 3.0, dtype=BF16, device="cuda")
    got = cuda_lib.expert_gated_ffn(x, row_token, offsets, counts, w, out=guard[:8])
    xs = torch.cat([x[:2], torch.zeros(2, H, dtype=BF16, device="cuda"), x[4:8]])
    for e, rows in ((0, slice(0, 4)), (1, slice(4, 8))):
        R.check({"out": got[rows]}, R.gated(xs[rows], w[e]), f"expert {e}")
    assert (guard[8:] == 3).all()


# ------------------------------------------------------ streams and graphs


def test_calls_follow_the_given_and_the_current_stream(cuda_lib):
    s = torch.cuda.Stream()
    x, w = rand(70, 200, 2048), rand(71, 512, 2048, scale=0.02)
    want = cuda_lib.linear(x, w)["out"]
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    late = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            big.add_(1)                 # keeps s busy while the call is enqueued
        late.copy_(x)
        a = cuda_lib.linear(late, w)["out"]
    b = cuda_lib.linear(late, w, stream=s)["out"]
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want)


def test_two_captured_layers_replay_on_new_inputs(cuda_lib):
    """Two graphs of forward and backward over their own buffers, replayed in
    turn and at once on two streams, give what eager calls give."""
    T, H, I = 96, 256, 136
    states = []
    for k in range(2):
        x, w, d = rand(80 + k, T, H), rand(82 + k, 2 * I, H, scale=0.06), rand(84 + k, T, I)
        ws = torch.empty(cuda_lib.gated_ffn_backward_workspace_bytes(T, I), dtype=torch.uint8,
                         device="cuda")
        pre = torch.empty(T, 2 * I, dtype=BF16, device="cuda")

        def step(x=x, w=w, d=d, ws=ws, pre=pre):
            f = cuda_lib.gated_ffn(x, w, preact=pre)
            g = cuda_lib.gated_ffn_backward(d, x, w, pre, want_dbias=True, workspace=ws)
            return dict(out=f["out"], **g)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        states.append((graph, outs, x, w, d, pre, ws))      # the graph's buffers stay alive
    streams = [torch.cuda.Stream() for _ in states]
    for rnd in range(3):
        want = []
        for k, (_, _, x, w, d, *_) in enumerate(states):
            x.copy_(rand(90 + rnd * 2 + k, T, H))
            f = cuda_lib.gated_ffn(x, w, save_preact=True)
            g = cuda_lib.gated_ffn_backward(d, x, w, f["preact"], want_dbias=True)
            want.append(dict(out=f["out"], **g))
        torch.cuda.synchronize()
        for (graph, *_), s in zip(states, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, outs, *_), ref in zip(states, want):
            for key in ref:
                assert torch.equal(outs[key], ref[key]), (rnd, key)


def test_experts_graph_replays_on_new_routing(cuda_lib):
    """One graph of the row map and both expert products, replayed on other
    ids: counts and offsets change, nothing is read on the host."""
    T, K, E, H, I, tile = 50, 3, 12, 128, 64, 8
    x, w13, w2 = rand(1, T, H), rand(2, E, 2 * I, H, scale=0.1), rand(3, E, H, I, scale=0.1)
    ids = ids_of(1, T, K, E, "all").cuda()
    P = cuda_lib.permute_rows(T, K, E, tile)
    y = torch.zeros(P, H, dtype=BF16, device="cuda")

    def step():
        m = cuda_lib.permute_tokens(ids, E, tile)
        h = cuda_lib.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w13)
        cuda_lib.expert_linear(h, m["offsets"], m["counts"], w2, out=y)
        return m

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m = step()
    for seed, kind in ((4, "holes"), (5, "one"), (6, "none"), (7, "all")):
        ids.copy_(ids_of(seed, T, K, E, kind))
        y.zero_()
        graph.replay()
        got, got_map = y.clone(), {k: v.clone() for k, v in m.items()}
        y.zero_()
        ref_map = step()
        for key in ref_map:
            assert torch.equal(got_map[key], ref_map[key]), (kind, key)
        assert torch.equal(got, y), kind


# ------------------------------------------------------- the layer together


@pytest.mark.parametrize("T,H,I,E,K,tile", [(1, 256, 64, 16, 4, 16), (50, 264, 72, 12, 3, 8),
                                            (400, 512, 136, 32, 8, 128)])
def test_moe_layer(cuda_lib, T, H, I, E, K, tile):
    """Router, gate, row map, expert products, shared expert and finalize as
    one layer, against the layer in 64 bits on the same routing.  Bound: the
    finalize's own tolerance, widened by what the bf16 intermediates h, the
    expert rows and the shared output carry (three roundings of 2^-8 relative
    to the magnitudes that are summed)."""
    mf = cuda_lib
    x = rand(100, T, H)
    wr, w13, w2 = rand(101, E, H, scale=H ** -0.5), rand(102, E, 2 * I, H, scale=H ** -0.5), \
        rand(103, E, H, I, scale=I ** -0.5)
    s13, s2 = rand(104, 2 * I, H, scale=H ** -0.5), rand(105, H, I, scale=I ** -0.5)
    logits = mf.linear(x, wr, out_dtype=torch.float32)["out"]
    R.check({"out": logits}, R.linear(x, wr, fp32=True), "logits")
    route = mf.topk_route(logits, K, "sigmoid")
    m = mf.permute_tokens(route["expert_ids"], E, tile)
    h = mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w13)
    rows = mf.expert_linear(h, m["offsets"], m["counts"], w2)
    shared = mf.linear(mf.gated_ffn(x, s13)["out"], s2)["out"]
    bad = mf.check_indices(m["idx_map"], rows.shape[0])
    out = mf.moe_finalize(rows, m["idx_map"], route["weights"], "fp32", shared,
                          routed_scale=2.5)["out"]
    assert int(bad.item()) == 0

    def expert(w_up, w_down):
        z = x.double() @ w_up.double().mT
        g, u = z.chunk(2, dim=-1)
        hh = R.act(g, "silu")[0] * u
        return hh @ w_down.double().mT, hh.abs() @ w_down.double().abs().mT

    ref, mag = expert(s13, s2)
    for e in range(E):
        w = torch.where(route["expert_ids"] == e, route["weights"], 0.0).double().sum(1) * 2.5
        if w.any():
            y, ymag = expert(w13[e], w2[e])
            ref, mag = ref + w[:, None] * y, mag + w[:, None] * ymag
    bound = 2.0 ** -7 * ref.abs() + 2e-3 + 3 * R.BF16 * mag
    assert ((out.double() - ref).abs() <= bound).all()
    rel = ((out.double() - ref).norm() / ref.norm()).item()
    assert rel < 3 * R.BF16       # three roundings in a row, each at most 2^-8


@pytest.mark.parametrize("name", ["none", "gelu"])
@pytest.mark.parametrize("T,N,K", [(300, 1001, 264), (17, 9, 64), (129, 63, 136)])
def test_backward_of_odd_feature_counts(cuda_lib, name, T, N, K):
    x, w, d = rand(43, T, K), rand(44, N, K, scale=K ** -0.5), rand(45, T, N, scale=0.1)
    pre = None if name == "none" else cuda_lib.linear(x, w, save_preact=True)["preact"]
    got = cuda_lib.linear_backward(d, x, w, activation=name, preact=pre, want_dbias=True)
    R.check(got, R.backward(d, x, w, pre, name, False), name)
    if N > 60:
        w = rand(46, 2 * N, K, scale=K ** -0.5)
        pre = cuda_lib.gated_ffn(x, w, activation=name, save_preact=True)["preact"]
        got = cuda_lib.gated_ffn_backward(d, x, w, pre, activation=name, want_dbias=True)
        R.check(got, R.backward(d, x, w, pre, name, True), "gated " + name)


@pytest.mark.parametrize("T,N,K", [(2040, 1000, 1544), (3000, 2048, 2048), (64, 4096, 1024),
                                   (4096, 64, 1024), (1500, 3000, 264), (5000, 520, 72)])
def test_large_backward(cuda_lib, T, N, K):
    """Many tiles: both gradients in one launch, or each in its own."""
    x, w, d = rand(250, T, K), rand(251, N, K, scale=K ** -0.5), rand(252, T, N, scale=0.1)
    both = cuda_lib.linear_backward(d, x, w, want_dbias=True)
    ref = R.backward(d, x, w, None, "none", False)
    R.check(both, ref)
    alone = {**cuda_lib.linear_backward(d, x, w, want_dweight=False),
             **cuda_lib.linear_backward(d, x, w, want_dx=False)}
    R.check(alone, ref, "alone")


def test_backward_of_a_misaligned_dout(cuda_lib):
    x, w, d = rand(47, 50, 64), rand(48, 72, 64), rand(49, 50, 72)
    got = cuda_lib.linear_backward(misaligned(d), x, w, want_dbias=True)
    R.check(got, R.backward(d, x, w, None, "none", False))


def test_offsets_past_32_bits(cuda_lib):
    """Outputs of more than 2^31 elements: the first, middle and last rows."""
    T, N, K = 300_000, 8192, 64
    x, w = rand(200, T, K), rand(201, N, K, scale=0.1)
    out = cuda_lib.linear(x, w)["out"]
    for rows in (slice(0, 40), slice(262_120, 262_160), slice(T - 40, T)):
        R.check({"out": out[rows]}, R.linear(x[rows], w), f"rows {rows.start}")
    del out
    h = cuda_lib.gated_ffn(x, torch.cat([w, w.flip(0), w, w]), save_preact=True)
    rows = slice(T - 40, T)
    R.check({k: v[rows] for k, v in h.items()},
            R.gated(x[rows], torch.cat([w, w.flip(0), w, w])), "gated")


def test_expert_weights_past_32_bits(cuda_lib):
    E, H, I, T = 300, 4096, 1024, 8         # 2.5e9 weights
    w = torch.empty(E, 2 * I, H, dtype=BF16, device="cuda")
    for e in range(0, E, 50):
        w[e:e + 50].normal_(0.0, H ** -0.5)
    ids = torch.tensor([[0, E - 1], [E - 1, 255], [256, 257], [1, 2], [299, 298], [3, 4], [5, 6],
                        [7, 0]], dtype=torch.int32, device="cuda")
    m = cuda_lib.permute_tokens(ids, E, 4)
    x = rand(202, T, H)
    h = cuda_lib.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w)
    for t, k in ((0, 1), (1, 1), (2, 0), (4, 0), (7, 1)):
        row = int(m["idx_map"][t, k])
        R.check({"out": h[row:row + 1]}, R.gated(x[t:t + 1], w[int(ids[t, k])]), f"{t},{k}")


def test_finalize_may_read_the_routing_early_behind_these_kernels(cuda_lib):
    """moe_finalize with routing_ready reads the row map before the expert
    product in front of it has finished; the row map must be complete when
    that product starts, however early the launches overlap."""
    mf = cuda_lib
    T, K, E, H, I = 64, 4, 16, 256, 64
    x, w13, w2 = rand(210, T, H), rand(211, E, 2 * I, H, scale=0.1), rand(212, E, H, I, scale=0.1)
    shared = rand(213, T, H)
    wts = torch.rand(T, K, device="cuda")
    sets = [ids_of(220 + i, T, K, E, "all").cuda() for i in range(4)]
    P = mf.permute_rows(T, K, E, 8)
    bufs = {"idx_map": torch.zeros(T, K, dtype=torch.int32, device="cuda"),
            "row_token": torch.empty(P, dtype=torch.int32, device="cuda"),
            "offsets": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
            "counts": torch.empty(E, dtype=torch.int32, device="cuda")}
    h, y = (torch.zeros(P, n, dtype=BF16, device="cuda") for n in (I, H))

    def layer(ids, ready):
        m = mf.permute_tokens(ids, E, 8, **bufs)
        mf.expert_gated_ffn(x, m["row_token"], m["offsets"], m["counts"], w13, out=h)
        mf.expert_linear(h, m["offsets"], m["counts"], w2, out=y)
        return mf.moe_finalize(y, m["idx_map"], wts, "fp32", shared, routing_ready=ready)["out"]

    want = []
    for ids in sets:
        want.append(layer(ids, False))
        torch.cuda.synchronize()
    for _ in range(20):
        got = [layer(ids, True) for ids in sets]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_from_threads(cuda_lib):
    """Two host threads on their own streams at once."""
    import threading
    xs = [rand(230 + i, 40 + 100 * i, 512) for i in range(2)]
    w = rand(232, 640, 512, scale=0.05)
    want = [cuda_lib.linear(x, w)["out"] for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                out = cuda_lib.linear(xs[i], w)["out"]
                torch.cuda.current_stream().synchronize()
                if not torch.equal(out, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_python_and_one_pass_checks_agree(cuda_lib, monkeypatch):
    """The checked call through the extension and the Python checks with the
    ctypes call give the same bits and refuse the same calls."""
    from moe_deferred_finalize_gb300 import _abi
    x, w, b, r = rand(240, 20, 128), rand(241, 48, 128), rand(242, 48), rand(243, 20, 48)
    wx, bx = rand(244, 2, 48, 128), rand(245, 2, 48)
    token = torch.arange(12, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 8, 12], dtype=torch.int32, device="cuda")
    counts = torch.tensor([5, 4], dtype=torch.int32, device="cuda")
    filled = torch.zeros(12, 24, dtype=BF16, device="cuda")
    wide = torch.zeros(12, 48, dtype=BF16, device="cuda")
    calls = [lambda: cuda_lib.linear(x, w, bias=b, residual=r, activation="silu",
                                     save_preact=True),
             lambda: cuda_lib.linear(x, w, out_dtype=torch.float32),
             lambda: cuda_lib.gated_ffn(x, w, bias=b, save_preact=True),
             lambda: cuda_lib.linear_backward(r, x, w, activation="silu", preact=r,
                                              want_dbias=True),
             lambda: cuda_lib.linear_backward(r, x, w, preact=r, want_dx=False),
             lambda: cuda_lib.gated_ffn_backward(r[:, :24].contiguous(), x, w, r,
                                                 want_dbias=True),
             lambda: {"out": cuda_lib.expert_gated_ffn(x, token, offsets, counts, wx,
                                                       out=filled.clone())},
             lambda: {"out": cuda_lib.expert_linear(x[:12].contiguous(), offsets, counts, wx,
                                                    bias=bx, out=wide.clone())}]
    bad = [lambda: cuda_lib.linear(x.t(), w), lambda: cuda_lib.linear(x, w[:, :64]),
           lambda: cuda_lib.linear(x, w, bias=b[:40]), lambda: cuda_lib.linear(x.float(), w),
           lambda: cuda_lib.linear(x, w, residual=r[:10]), lambda: cuda_lib.linear(x, w, out=x),
           lambda: cuda_lib.linear(x, w, activation="tanh"),
           lambda: cuda_lib.linear(x, w, out_dtype=torch.float16),
           lambda: cuda_lib.linear(x.cpu(), w), lambda: cuda_lib.gated_ffn(x, w[:47]),
           lambda: cuda_lib.gated_ffn(x, w, out=r), lambda: cuda_lib.gated_ffn(x, w, bias=b[1:]),
           lambda: cuda_lib.gated_ffn(x, w, preact=x),
           lambda: cuda_lib.linear_backward(r, x, w, activation="silu"),
           lambda: cuda_lib.linear_backward(r, x, w, activation="silu", preact=x),
           lambda: cuda_lib.linear_backward(r[:10], x, w), lambda: cuda_lib.linear_backward(x, x, w),
           lambda: cuda_lib.linear_backward(r, x, w, dx=r),
           lambda: cuda_lib.linear_backward(r, x, w, dbias=b[:40]),
           lambda: cuda_lib.linear_backward(r, x, w, want_dx=False, want_dweight=False),
           lambda: cuda_lib.gated_ffn_backward(r, x, w, r),
           lambda: cuda_lib.expert_gated_ffn(x, token, offsets[:2], counts, wx),
           lambda: cuda_lib.expert_gated_ffn(x, token.long(), offsets, counts, wx),
           lambda: cuda_lib.expert_gated_ffn(x, token, offsets, counts, wx[0]),
           lambda: cuda_lib.expert_linear(x, offsets, counts, wx, out=filled),
           lambda: cuda_lib.expert_linear(x, offsets, counts, wx, bias=b),
           lambda: cuda_lib.expert_linear(x, offsets, counts, wx[:, :, :64])]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    fast = [f() for f in calls]
    monkeypatch.setattr(_abi, "_FAST", None)
    for f, ref in zip(calls, fast):
        got = f()
        assert set(got) == set(ref)
        for key in ref:
            assert got[key].dtype == ref[key].dtype and torch.equal(got[key], ref[key])
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()


def test_row_map_python_and_one_pass_checks_agree(cuda_lib, monkeypatch):
    from moe_deferred_finalize_gb300 import _abi
    ids = torch.randint(-1, 16, (50, 4), dtype=torch.int32, device="cuda")
    P = cuda_lib.permute_rows(50, 4, 16, 8)

    def i32(*shape):
        return torch.full(shape, -7, dtype=torch.int32, device="cuda")

    calls = [lambda: cuda_lib.permute_tokens(ids, 16, 8),
             lambda: cuda_lib.permute_tokens(ids[:0], 16, 8),
             lambda: cuda_lib.permute_tokens(ids, 16),
             lambda: cuda_lib.permute_tokens(ids.repeat(100, 1), 16, 8),
             lambda: cuda_lib.permute_tokens(ids, 16, 8, row_token=i32(P + 9), idx_map=i32(50, 4)),
             lambda: cuda_lib.permute_tokens(ids, 16, 8, offsets=i32(17), counts=i32(16))]
    bad = [lambda: cuda_lib.permute_tokens(ids.long(), 16, 8),
           lambda: cuda_lib.permute_tokens(ids.t(), 16, 8),
           lambda: cuda_lib.permute_tokens(ids[0], 16, 8),
           lambda: cuda_lib.permute_tokens(ids.cpu(), 16, 8),
           lambda: cuda_lib.permute_tokens(ids, 0, 8),
           lambda: cuda_lib.permute_tokens(ids, -3, 8),
           lambda: cuda_lib.permute_tokens(ids, 1025, 8),
           lambda: cuda_lib.permute_tokens(ids, 16, 0),
           lambda: cuda_lib.permute_tokens(ids, 16, 2 ** 32 + 8),
           lambda: cuda_lib.permute_tokens(ids, 16, 8, row_token=i32(P - 1)),
           lambda: cuda_lib.permute_tokens(ids, 16, 8, row_token=i32(P, 1)),
           lambda: cuda_lib.permute_tokens(ids, 16, 8, idx_map=i32(4, 50)),
           lambda: cuda_lib.permute_tokens(ids, 16, 8, offsets=i32(16)),
           lambda: cuda_lib.permute_tokens(ids, 16, 8, counts=i32(17)),
           lambda: cuda_lib.permute_tokens(ids.repeat(100, 1), 16, 8, workspace=i32(1))]

    def errors():
        kinds = []
        for f in bad:
            with pytest.raises((ValueError, TypeError, cuda_lib.MoefError)) as e:
                f()
            kinds.append(e.type)
        return kinds

    fast, kinds = [f() for f in calls], errors()
    monkeypatch.setattr(_abi, "_FAST", None)
    for f, ref in zip(calls, fast):
        got = f()
        assert list(got) == list(ref)
        for key in ref:
            assert got[key].dtype == torch.int32 and torch.equal(got[key], ref[key])
    assert errors() == kinds


def test_sizes_past_a_c_int_are_refused(cuda_lib):
    """2^32 + 5 rows must not become 5."""
    x = torch.empty(2 ** 32 + 5, 1, dtype=BF16, device="cuda")
    w = torch.ones(1, 1, dtype=BF16, device="cuda")
    with pytest.raises(cuda_lib.MoefError):
        cuda_lib.linear(x, w, out=x.view(2 ** 32 + 5, 1))
    with pytest.raises(cuda_lib.MoefError):
        cuda_lib.gated_ffn(x, torch.ones(2, 1, dtype=BF16, device="cuda"), out=x)
    with pytest.raises(cuda_lib.MoefError):
        cuda_lib.linear_backward(x, x, w, want_dx=False, want_dweight=True)


def test_expert_with_the_most_rows(cuda_lib):
    """One expert with 2^31 - 1 rows: nothing in the cut of the tiles may pass 31 bits."""
    P, K, N = 2 ** 31 - 1, 8, 8
    x = torch.zeros(P, K, dtype=BF16, device="cuda")
    some = [0, 1, 255, 256, P // 2, P - 257, P - 2, P - 1]
    x[some] = rand(3, len(some), K)
    w = rand(4, 1, N, K)
    offsets = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    counts = torch.tensor([P], dtype=torch.int32, device="cuda")
    out = torch.full((P, N), 7.0, dtype=BF16, device="cuda")
    cuda_lib.expert_linear(x, offsets, counts, w, out=out)
    R.check({"out": out[some]}, {"out": R.linear(x[some], w[0])["out"]}, "rows")
    assert int((out[: 2 ** 20] == 7.0).sum()) == 0 and int((out[-2 ** 20:] == 7.0).sum()) == 0


def test_lost_waits_waits_for_every_stream(cuda_lib):
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        done.record()
    assert cuda_lib.lost_waits() == 0
    assert done.query()


def test_no_barrier_wait_was_lost(cuda_lib):
    """Last: none of the launches above gave up a wait."""
    torch.cuda.synchronize()
    assert cuda_lib.lost_waits() == 0
