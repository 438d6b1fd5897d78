"""The products around the finalize without a GPU: argument errors of the C
entry points and of the binding, sizes of rows and workspaces, and the 64-bit
references themselves (gradients against differences).  No kernel runs."""
import ctypes
import itertools

import pytest
import torch

import ffn_ref as R
from moe_deferred_finalize_gb300 import build

A, ODD, HALF, NULL = 0x10000, 0x10001, 0x10002, None
OK, E_NULL, E_SHAPE, E_ALIGN, E_ARG = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    from moe_deferred_finalize_gb300 import _ffn
    return _ffn._lib()


def call(fn, base, **change):
    args = dict(base, **change)
    return fn(*args.values())


LINEAR = dict(x=A, w=A, bias=NULL, residual=NULL, act=0, out=A, out_type=0, preact=NULL, T=4, N=8,
              K=8, stream=NULL)


def test_linear_argument_errors(lib):
    f = lib.moe_linear
    assert call(f, LINEAR, T=0) == OK
    for k in ("x", "w", "out"):
        assert call(f, LINEAR, **{k: NULL}) == E_NULL
        assert call(f, LINEAR, **{k: ODD}) == E_ALIGN
    for k in ("bias", "residual", "preact"):
        assert call(f, LINEAR, **{k: ODD}) == E_ALIGN
    assert call(f, LINEAR, out=HALF, out_type=1) == E_ALIGN
    for k in ("N", "K"):
        for v in (0, -1, (1 << 24) + 1):
            assert call(f, LINEAR, **{k: v}) == E_SHAPE
    assert call(f, LINEAR, T=-1) == E_SHAPE
    for v in (-1, 5):
        assert call(f, LINEAR, act=v) == E_ARG
    for v in (-1, 2):
        assert call(f, LINEAR, out_type=v) == E_ARG


def test_gated_argument_errors(lib):
    f = lib.moe_gated_ffn
    base = dict(x=A, w=A, bias=NULL, act=1, out=A, preact=NULL, T=4, I=8, H=8, stream=NULL)
    assert call(f, base, T=0) == OK
    for k in ("x", "w", "out"):
        assert call(f, base, **{k: NULL}) == E_NULL
        assert call(f, base, **{k: ODD}) == E_ALIGN
    for k in ("bias", "preact"):
        assert call(f, base, **{k: ODD}) == E_ALIGN
    for k in ("I", "H"):
        for v in (0, -3, (1 << 24) + 1):
            assert call(f, base, **{k: v}) == E_SHAPE
    assert call(f, base, T=-1) == E_SHAPE
    assert call(f, base, act=9) == E_ARG


def test_backward_argument_errors(lib):
    for f, size in ((lib.moe_linear_backward, lib.moe_linear_backward_workspace_bytes),
                    (lib.moe_gated_ffn_backward, lib.moe_gated_ffn_backward_workspace_bytes)):
        base = dict(dout=A, x=A, w=A, act=1, preact=A, dx=A, dw=A, db=A, T=40, n=8, K=8, ws=A,
                    ws_bytes=1 << 20, stream=NULL)
        assert call(f, base, dx=NULL, dw=NULL, db=NULL) == E_NULL
        for k in ("dout", "x", "w", "preact", "ws"):
            assert call(f, base, **{k: NULL}) == E_NULL
        for k in ("dout", "x", "w", "preact", "dx", "dw", "db"):
            assert call(f, base, **{k: ODD}) == E_ALIGN
        assert call(f, base, ws=A + 8) == E_ALIGN
        assert call(f, base, ws_bytes=size(40, 8) - 1) == E_SHAPE
        for k in ("n", "K"):
            for v in (0, -1, (1 << 24) + 1):
                assert call(f, base, **{k: v}) == E_SHAPE
        assert call(f, base, T=-1) == E_SHAPE
        assert call(f, base, act=5) == E_ARG
        assert size(-1, 8) == 0 and size(4, 0) == 0 and size(0, 8) == 0
        assert size(2 ** 31 - 1, 1 << 24) > 2 ** 55       # 64-bit sizes
    assert call(lib.moe_linear_backward, base, act=0) == E_ARG     # a preact nobody reads


def test_permute_argument_errors(lib):
    f = lib.moe_permute
    base = dict(ids=A, T=4, K=2, E=8, tile=16, idx=A, rows=A, P=128, offsets=A, counts=A, ws=A,
                ws_bytes=1 << 20, stream=NULL)
    for k in ("ids", "idx", "rows", "offsets", "counts"):
        assert call(f, base, **{k: NULL}) == E_NULL
    many = dict(base, T=1 << 20, P=1 << 30)         # enough slots for the workspace to be used
    assert lib.moe_permute_workspace_bytes(4, 2, 8) == 0
    need = lib.moe_permute_workspace_bytes(1 << 20, 2, 8)
    assert need > 0
    assert call(f, many, ws=NULL) == E_NULL
    assert call(f, many, ws_bytes=need - 1) == E_SHAPE
    for k in ("ids", "idx", "rows", "offsets", "counts", "ws"):
        assert call(f, base, **{k: HALF}) == E_ALIGN
    for change in (dict(T=-1), dict(K=0), dict(K=33), dict(E=0), dict(E=1025), dict(tile=0),
                   dict(P=127), dict(P=1 << 31), dict(T=2 ** 31 - 1, K=32, P=2 ** 31 - 1)):
        assert call(f, base, **change) == E_SHAPE, change


def test_permute_rows_bounds_every_routing(lib):
    for T, K, E, tile in itertools.product((0, 1, 2, 3), (1, 2), (1, 2, 3), (1, 2, 3, 4)):
        most = 0
        for flat in itertools.product(range(E), repeat=T * K):
            most = max(most, sum(-(-flat.count(e) // tile) * tile for e in range(E)))
        rows = lib.moe_permute_rows(T, K, E, tile)
        assert most <= rows <= most + tile * E, (T, K, E, tile)
        assert rows % tile == 0
    assert lib.moe_permute_rows(2 ** 31 - 1, 32, 8, 1) == 0
    assert lib.moe_permute_rows(1, 1, 1, 2 ** 31 - 1) == 2 ** 31 - 1
    assert lib.moe_permute_rows(4, 2, 8, 16) == 128


def test_sizes_past_a_c_int_are_refused_not_cut_off(lib):
    """2^32 + 1 cut to 32 bits would be 1: a valid size of another problem."""
    import moe_deferred_finalize_gb300 as M
    big = 2 ** 32 + 1
    assert M.linear_backward_workspace_bytes(big, 8) == 0
    assert M.linear_backward_workspace_bytes(8, big) == 0
    assert M.gated_ffn_backward_workspace_bytes(big, 8) == 0
    for sizes in ((big, 1, 1, 1), (1, big, 1, 1), (1, 1, big, 1), (1, 1, 1, big)):
        assert M.permute_rows(*sizes) == 0, sizes
    assert M.permute_rows(1, 1, 1, 1) == 1


def test_lost_waits_needs_a_counter(lib):
    assert lib.moe_ffn_lost_waits(None) == E_NULL


def test_expert_argument_errors(lib):
    for f in (lib.moe_expert_gated_ffn, lib.moe_expert_linear):
        base = dict(x=A, T=16, rows=A, offsets=A, counts=A, w=A, bias=NULL, act=0, out=A, P=32,
                    E=4, M=8, K=8, stream=NULL)
        assert call(f, base, T=0) == OK and call(f, base, P=0) == OK
        for k in ("x", "offsets", "counts", "w", "out"):
            assert call(f, base, **{k: NULL}) == E_NULL
        for k in ("x", "w", "bias", "out"):
            assert call(f, base, **{k: ODD}) == E_ALIGN
        for k in ("rows", "offsets", "counts"):
            assert call(f, base, **{k: HALF}) == E_ALIGN
        for change in (dict(T=-1), dict(P=-1), dict(P=1 << 31), dict(T=1 << 31), dict(E=0),
                       dict(E=1025), dict(M=0), dict(K=0), dict(M=(1 << 24) + 1),
                       dict(rows=NULL)):        # without row_token x has P rows
            assert call(f, base, **change) == E_SHAPE, change
        assert call(f, base, act=-1) == E_ARG


def test_binding_refuses_cpu_tensors_and_bad_names():
    import moe_deferred_finalize_gb300 as mf
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for fn in (lambda: mf.linear(x, w), lambda: mf.gated_ffn(x, w),
               lambda: mf.linear_backward(x, x, w), lambda: mf.gated_ffn_backward(x, x, w, x),
               lambda: mf.permute_tokens(ids, 8), lambda: mf.expert_linear(x, ids, ids, w)):
        with pytest.raises(ValueError):
            fn()
    with pytest.raises(TypeError):
        mf.linear([[1.0]], w)
    from moe_deferred_finalize_gb300 import _ffn
    with pytest.raises(ValueError, match="activation"):
        _ffn._activation("tanh")


@pytest.mark.parametrize("name", R.ACTS)
@pytest.mark.parametrize("is_gated", [False, True])
def test_reference_gradients_against_differences(name, is_gated):
    """The 64-bit gradient formulas against central differences of the 64-bit
    forward: step 1e-5, so e^2 / 6 |f'''| and 2^-52 |f| / e are both below
    1e-9 of the sums."""
    g = torch.Generator().manual_seed(7)
    T, n, K, e = 5, 4, 6, 1e-5
    cols = 2 * n if is_gated else n
    x = torch.randn(T, K, generator=g, dtype=torch.float64)
    w = torch.randn(cols, K, generator=g, dtype=torch.float64)
    b = torch.randn(cols, generator=g, dtype=torch.float64)
    d = torch.randn(T, n, generator=g, dtype=torch.float64)

    def loss(x, w, b):
        z = x @ w.mT + b
        if is_gated:
            p, u = z.chunk(2, dim=-1)
            return (d * R.act(p, name)[0] * u).sum()
        return (d * R.act(z, name)[0]).sum()

    grads = R.backward(d, x, w, x @ w.mT + b, name, is_gated)
    for i, key in enumerate(("dx", "dweight", "dbias")):
        args = [x, w, b]
        value = grads[key][0]
        for at in range(args[i].numel()):
            lo, hi = [a.clone() for a in args], [a.clone() for a in args]
            lo[i].view(-1)[at] -= e
            hi[i].view(-1)[at] += e
            diff = (loss(*hi) - loss(*lo)) / (2 * e)
            assert abs(diff - value.view(-1)[at]) < 1e-7 * (1 + value.abs().max())


def test_reference_layout_by_hand():
    idx, token, offsets, counts = R.layout([[1, 0], [1, -1], [3, 1]], 4, 2, 10)
    assert idx == [[2, 0], [3, -1], [6, 4]]
    assert token == [0, -1, 0, 1, 2, -1, 2, -1, -1, -1]
    assert offsets == [0, 2, 6, 6, 8] and counts == [1, 3, 0, 1]


def test_header_struct_free_interface_matches_the_binding(lib):
    """Every entry point of moe_ffn.h has a signature in the binding."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_ffn.h")).read(),
                  flags=re.S)
    found = re.findall(r"^(?:\w+)\s+(moe_\w+)\(([^;]*)\);", text, flags=re.M)
    assert len(found) == 12
    for name, params in found:
        fn = getattr(lib, name)
        assert len(fn.argtypes) == len(params.split(",")), name
        assert fn.restype is not ctypes.c_int or name not in ("moe_permute_rows",)
