"""The MoE layer's training side without a GPU: argument errors of the C entry
points and of the binding, workspace sizes, given streams, and the 64-bit
references themselves (gradients against differences).  No kernel runs."""
import ctypes

import pytest
import torch

import train_ref as T_
from moe_deferred_finalize_gb300 import build

A, ODD, HALF, NULL = 0x10000, 0x10001, 0x10002, None
OK, E_NULL, E_SHAPE, E_ALIGN, E_ARG = 0, 1, 2, 3, 4
BF16, F32 = torch.bfloat16, torch.float32
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    from moe_deferred_finalize_gb300 import _ffn, _train
    _ffn._lib()
    return _train._lib()


def call(fn, base, **change):
    return fn(*dict(base, **change).values())


FINALIZE = dict(rows=A, P=16, idx=A, w=A, wkind=0, scale=1.0, r=A, gamma=A, eps=1e-6, dout=A,
                dres=A, dnorm=A, drows=A, dweights=A, dshared=A, dresidual=A, dgamma=A, T=40, K=2,
                H=8, ws=A, ws_bytes=1 << 20, stream=NULL)


def test_finalize_backward_argument_errors(lib):
    f = lib.moe_finalize_backward
    assert call(f, FINALIZE, T=0, dgamma=NULL) == OK
    none = dict(drows=NULL, dweights=NULL, dshared=NULL, dresidual=NULL, dgamma=NULL)
    assert call(f, FINALIZE, **none) == E_NULL
    for k in ("idx", "w", "rows", "ws"):
        assert call(f, FINALIZE, **{k: NULL}) == E_NULL, k
    assert call(f, FINALIZE, dout=NULL, dres=NULL, dnorm=NULL, r=NULL, gamma=NULL,
                dgamma=NULL) == E_NULL
    for k in ("r", "gamma", "dnorm"):       # all three or none
        assert call(f, FINALIZE, **{k: NULL}) == E_ARG, k
    assert call(f, FINALIZE, r=NULL, gamma=NULL, dnorm=NULL) == E_ARG     # dgamma without dnorm
    for k in ("rows", "r", "gamma", "dout", "dres", "dnorm", "drows", "dshared", "dresidual",
              "dgamma"):
        assert call(f, FINALIZE, **{k: ODD}) == E_ALIGN, k
    for k in ("idx", "w", "dweights"):
        assert call(f, FINALIZE, **{k: HALF}) == E_ALIGN, k
    assert call(f, FINALIZE, ws=A + 8) == E_ALIGN
    need = lib.moe_finalize_backward_workspace_bytes(40, 8)
    assert call(f, FINALIZE, ws_bytes=need - 1) == E_SHAPE
    for k, vs in (("T", (-1,)), ("K", (0, 33)), ("H", (0, -1, (1 << 30) + 1)), ("P", (0, -1))):
        for v in vs:
            assert call(f, FINALIZE, **{k: v}) == E_SHAPE, (k, v)
    for v in (-1, 3):
        assert call(f, FINALIZE, wkind=v) == E_ARG
    for v in (-1.0, float("nan"), float("inf")):
        assert call(f, FINALIZE, eps=v) == E_ARG
    # a row that one cluster cannot hold
    assert call(f, FINALIZE, H=8 * 32768 + 8, ws_bytes=1 << 40) == E_SHAPE
    assert call(f, FINALIZE, H=32768 + 1, ws_bytes=1 << 40) == E_SHAPE
    assert call(f, FINALIZE, H=32768 + 8, dout=HALF, ws_bytes=1 << 40) == E_SHAPE


def test_batches_of_nothing(lib):
    """Arrays without elements may have no address: without tokens and rows, outputs of
    none are not missing ones."""
    f = lib.moe_finalize_backward
    none = dict(drows=NULL, dweights=NULL, dshared=NULL, dresidual=NULL, dgamma=NULL)
    assert call(f, FINALIZE, **none, T=0) == call(f, FINALIZE, **none, T=0, P=0) == OK
    assert call(f, FINALIZE, **none, T=1) == E_NULL
    none = dict(dx=NULL, dw=NULL, db=NULL)
    for f in (lib.moe_expert_gated_ffn_backward, lib.moe_expert_linear_backward):
        assert call(f, EXPERT, **none, T=0, P=0) == call(f, EXPERT, **none, P=0) == OK
        assert call(f, EXPERT, **none, T=0) == call(f, EXPERT, **none) == E_NULL


def test_finalize_backward_workspace(lib):
    size = lib.moe_finalize_backward_workspace_bytes
    assert size(0, 8) == size(4, 0) == size(-1, 8) == 0
    assert size(1, 8) == size(32, 8) == size(16, 9) == 0
    assert size(33, 8) == 33 * 32 and size(17, 9) == 17 * 36
    assert size(INT_MAX, 7168) == size(5000, 7168) == 1024 * 7168 * 4


UNPERMUTE = dict(rows=A, P=8, idx=A, add0=NULL, add1=NULL, out=A, T=4, K=2, H=8, stream=NULL)


def test_unpermute_argument_errors(lib):
    f = lib.moe_unpermute
    assert call(f, UNPERMUTE, T=0) == OK
    for k in ("rows", "idx", "out"):
        assert call(f, UNPERMUTE, **{k: NULL}) == E_NULL
    for k in ("rows", "add0", "add1", "out"):
        assert call(f, UNPERMUTE, **{k: ODD}) == E_ALIGN
    assert call(f, UNPERMUTE, idx=HALF) == E_ALIGN
    for k, vs in (("T", (-1,)), ("P", (-1,)), ("K", (0, 33)), ("H", (0, (1 << 30) + 1))):
        for v in vs:
            assert call(f, UNPERMUTE, **{k: v}) == E_SHAPE
    assert call(f, UNPERMUTE, T=INT_MAX, H=129) == E_SHAPE


GATE = dict(dw=A, w=A, ids=A, logits=A, T=4, E=8, K=2, kind=1, out=A, out_type=0, stream=NULL)


def test_gate_backward_argument_errors(lib):
    f = lib.moe_topk_route_backward
    assert call(f, GATE, T=0) == OK
    for k in ("dw", "w", "ids", "logits", "out"):
        assert call(f, GATE, **{k: NULL}) == E_NULL
    for k in ("dw", "w", "ids", "logits"):
        assert call(f, GATE, **{k: HALF}) == E_ALIGN
    assert call(f, GATE, out=ODD) == E_ALIGN
    assert call(f, GATE, out=HALF, out_type=1) == E_ALIGN
    for k, vs in (("T", (-1,)), ("E", (0, 1025)), ("K", (0, 33, 9))):
        for v in vs:
            assert call(f, GATE, **{k: v}) == E_SHAPE
    for k in ("kind", "out_type"):
        for v in (-1, 2):
            assert call(f, GATE, **{k: v}) == E_ARG


EXPERT = dict(dout=A, x=A, T=16, row_token=A, offsets=A, counts=A, w=A, act=1, preact=A, dx=A,
              dw=A, db=A, P=40, E=4, n=8, K=8, ws=A, ws_bytes=1 << 20, stream=NULL)


@pytest.mark.parametrize("gated", [False, True])
def test_expert_backward_argument_errors(lib, gated):
    f = lib.moe_expert_gated_ffn_backward if gated else lib.moe_expert_linear_backward
    cols = 16 if gated else 8
    for k in ("dout", "x", "offsets", "counts", "w", "preact", "ws"):
        assert call(f, EXPERT, **{k: NULL}) == E_NULL, k
    assert call(f, EXPERT, dx=NULL, dw=NULL, db=NULL) == E_NULL
    for k in ("dout", "x", "w", "preact", "dx", "dw", "db"):
        assert call(f, EXPERT, **{k: ODD}) == E_ALIGN, k
    for k in ("row_token", "offsets", "counts"):
        assert call(f, EXPERT, **{k: HALF}) == E_ALIGN, k
    assert call(f, EXPERT, ws=A + 8) == E_ALIGN
    size = lib.moe_expert_backward_workspace_bytes
    assert size(40, cols, 0) == 40 * cols * 2 and size(40, cols, 8) == 40 * (cols + 8) * 2
    assert size(40, 9, 17) == 40 * (16 + 24) * 2
    assert size(-1, 8, 0) == size(40, 0, 0) == size(40, 8, -1) == size(40, -1, 8) == 0
    # rows of x are laid out with a row map, an odd width, a misaligned x
    assert call(f, EXPERT, ws_bytes=size(40, cols, 8) - 1) == E_SHAPE
    in_layout = dict(row_token=NULL, T=40, ws_bytes=size(40, cols, 0) - 1)
    assert call(f, EXPERT, **in_layout) == E_SHAPE
    in_layout["ws_bytes"] += 1
    assert call(f, EXPERT, **in_layout, x=HALF) == E_SHAPE
    assert call(f, EXPERT, **in_layout, K=9) == E_SHAPE
    for k, vs in (("T", (-1, 1 << 31)), ("P", (-1, 1 << 31)), ("E", (0, 1025)),
                  ("n", (0, (1 << 24) + 1)), ("K", (0, (1 << 24) + 1))):
        for v in vs:
            assert call(f, EXPERT, **{k: v}) == E_SHAPE, (k, v)
    assert call(f, EXPERT, row_token=NULL) == E_SHAPE       # then T = P
    for v in (-1, 5):
        assert call(f, EXPERT, act=v) == E_ARG
    if not gated:
        assert call(f, EXPERT, act=0) == E_ARG              # no preact then


def test_expert_save_argument_errors(lib):
    base = dict(x=A, T=16, row_token=A, offsets=A, counts=A, w=A, bias=NULL, act=1, out=A,
                preact=A, P=40, E=4, n=8, K=8, stream=NULL)
    for f in (lib.moe_expert_gated_ffn_save, lib.moe_expert_linear_save):
        assert call(f, base, T=0) == call(f, base, P=0) == OK
        for k in ("x", "offsets", "counts", "w", "out"):
            assert call(f, base, **{k: NULL}) == E_NULL
        assert call(f, base, preact=ODD) == E_ALIGN
        assert call(f, base, P=-1) == E_SHAPE


def test_adamw_argument_errors(lib):
    from moe_deferred_finalize_gb300._train import AdamWConfig, AdamWTensor

    def step(n=1, config=None, rows=None, **tensor):
        t = dict(param=A, master=NULL, grad=A, exp_avg=A, exp_avg_sq=A, exp_avg_scale=NULL,
                 exp_avg_sq_scale=NULL, n=100)
        table = (AdamWTensor * 2)(AdamWTensor(**{**t, **tensor}), AdamWTensor(**(rows or t)))
        c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1,
                 state_bits=32, param_type=0, grad_type=0)
        return lib.moe_adamw_step(table, n, ctypes.byref(AdamWConfig(**{**c, **(config or {})})),
                                  NULL)

    assert step(n=0) == OK
    assert step(**{k: NULL for k in ("param", "grad", "exp_avg", "exp_avg_sq")}, n=1) == E_NULL
    assert lib.moe_adamw_step(NULL, 1, ctypes.byref(AdamWConfig(
        beta1=0.9, beta2=0.9, step=1, state_bits=32)), NULL) == E_NULL
    assert lib.moe_adamw_step(NULL, 0, NULL, NULL) == E_NULL
    assert step(n=-1) == E_SHAPE
    for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert step(**{k: NULL}) == E_NULL
        assert step(**{k: ODD}) == E_ALIGN
    for k in ("exp_avg", "exp_avg_sq", "master"):
        assert step(**{k: HALF}) == E_ALIGN
    assert step(param=HALF, config=dict(param_type=1)) == E_ALIGN
    assert step(grad=HALF, config=dict(grad_type=1)) == E_ALIGN
    eight = dict(exp_avg_scale=A, exp_avg_sq_scale=A)
    for k in eight:
        assert step(**{**eight, k: NULL}, config=dict(state_bits=8)) == E_NULL
        assert step(**{**eight, k: HALF}, config=dict(state_bits=8)) == E_ALIGN
        assert step(**{k: A}) == E_ARG          # scales without 8 bits
    assert step(master=A, config=dict(param_type=1)) == E_ARG
    assert step(n=2, master=A) == E_ARG         # a master for one of two
    for k in ("lr", "eps", "weight_decay"):
        for v in (-1.0, float("nan"), float("inf")):
            assert step(config={k: v}) == E_ARG
    for k in ("beta1", "beta2"):
        for v in (-0.1, 1.0, float("nan")):
            assert step(config={k: v}) == E_ARG
    for c in (dict(step=0), dict(state_bits=16), dict(param_type=2), dict(grad_type=-1)):
        assert step(config=c) == E_ARG
    for k in ("device_step", "device_lr", "grad_scale"):
        assert step(config={k: HALF}) == E_ALIGN


def test_adamw_numbers_past_fp32(lib):
    """Numbers that are infinite in fp32, which the step is taken in, are refused."""
    from moe_deferred_finalize_gb300._train import AdamWConfig, AdamWTensor
    t = (AdamWTensor * 1)(AdamWTensor(param=A, grad=A, exp_avg=A, exp_avg_sq=A, n=0))
    c = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, state_bits=32)
    for k in ("lr", "eps", "weight_decay"):
        for v, want in ((3.4e38, OK), (3.5e38, E_ARG), (1e300, E_ARG)):
            config = AdamWConfig(**{**c, k: v})
            assert lib.moe_adamw_step(t, 1, ctypes.byref(config), NULL) == want, (k, v)


# ---------------------------------------------------------------- binding


def cpu(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors_and_bad_choices(lib):
    import moe_deferred_finalize_gb300 as mf
    i32 = torch.int32
    calls = [
        lambda: mf.moe_finalize_backward(cpu(8, 8), cpu(4, 2, dtype=i32), cpu(4, 2, dtype=F32),
                                         "fp32", cpu(4, 8)),
        lambda: mf.moe_finalize_backward(cpu(8, 8), cpu(4, 2, dtype=i32), cpu(4, 2, dtype=F32),
                                         "fp16", cpu(4, 8)),
        lambda: mf.unpermute_tokens(cpu(8, 8), cpu(4, 2, dtype=i32)),
        lambda: mf.topk_route_backward(cpu(4, 2, dtype=F32), cpu(4, 2, dtype=F32),
                                       cpu(4, 2, dtype=i32), 8, "softmax"),
        lambda: mf.topk_route_backward(cpu(4, 2, dtype=F32), cpu(4, 2, dtype=F32),
                                       cpu(4, 2, dtype=i32), 8, "top1"),
        lambda: mf.expert_linear_backward(cpu(8, 8), cpu(8, 8), cpu(3, dtype=i32),
                                          cpu(2, dtype=i32), cpu(2, 8, 8)),
        lambda: mf.bind_adamw([], [], [], []),
        lambda: mf.bind_adamw([cpu(4)], [cpu(4)], [cpu(4, dtype=F32)], [cpu(4, dtype=F32)]),
        lambda: mf.adamw_state([cpu(4)], bits=16),
    ]
    for f in calls:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        mf.unpermute_tokens(None, None)


def test_adamw_state_on_the_host():
    import moe_deferred_finalize_gb300 as mf
    p = [torch.ones(3, 100, dtype=BF16), torch.ones(1, dtype=BF16)]
    s = mf.adamw_state(p, bits=8, master=True)
    assert [t.dtype for t in s["exp_avg"]] == [torch.float8_e4m3fn] * 2
    assert [t.shape for t in s["exp_avg_scale"]] == [(2,), (1,)]
    assert s["masters"][0].dtype == F32 and s["masters"][0].shape == (3, 100)
    s = mf.adamw_state(p)
    assert set(s) == {"exp_avg", "exp_avg_sq"} and not s["exp_avg"][0].any()


def test_adamw_masters_are_copies_of_their_own():
    """Of parameters that record gradients too: numbers, not part of a graph."""
    import moe_deferred_finalize_gb300 as mf
    for dtype in (BF16, F32):
        p = torch.nn.Parameter(torch.arange(6, dtype=dtype).view(2, 3))
        m = mf.adamw_state([p], master=True)["masters"][0]
        assert m.dtype == F32 and torch.equal(m, p.detach().float())
        assert not m.requires_grad and m.data_ptr() != p.data_ptr()


# ---------------------------------------------------------- given streams

CURRENT, OTHER = 0x70, 0x90     # stream handles


class Entered(Exception):
    """The given stream was made the current one."""


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    device = property(lambda self: torch.device("cuda", 0))


def fake(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def i32(*shape):
    return fake(*shape, dtype=torch.int32)


def f32(*shape):
    return fake(*shape, dtype=F32)


FINALIZE_ARGS = lambda: (fake(8, 8), i32(4, 2), f32(4, 2), "fp32", fake(4, 8))   # noqa: E731
NORM = lambda: dict(dnorm_out=fake(4, 8), residual_out=fake(4, 8), gamma=fake(8))   # noqa: E731
# name, required arguments, all that the call would allocate, options
ALLOCATING = [
    ("moe_finalize_backward", FINALIZE_ARGS, dict(drows=(8, 8), dweights=(4, 2)), dict),
    ("moe_finalize_backward", FINALIZE_ARGS,
     dict(drows=(8, 8), dweights=(4, 2), dshared=(4, 8), dresidual=(4, 8), dgamma=(8,),
          workspace=(4096,)), NORM),
    ("moe_finalize_backward", FINALIZE_ARGS,
     dict(drows=(8, 8), dweights=(4, 2), dshared=(4, 8), dresidual=(4, 8), workspace=(4096,)),
     lambda: dict(NORM(), dgamma=fake(8), want_dgamma=False)),
    ("unpermute_tokens", lambda: (fake(8, 8), i32(4, 2)), dict(out=(4, 8)), dict),
    ("topk_route_backward", lambda: (f32(4, 2), f32(4, 2), i32(4, 2), 8, "softmax"),
     dict(dlogits=(4, 8)), dict),
    ("expert_linear_backward", lambda: (fake(8, 8), fake(8, 8), i32(3), i32(2), fake(2, 8, 8)),
     dict(dx=(8, 8), dweight=(2, 8, 8), dbias=(2, 8), workspace=(4096,)),
     lambda: dict(want_dbias=True)),
    ("expert_gated_ffn_backward",
     lambda: (fake(8, 8), fake(4, 8), i32(8), i32(3), i32(2), fake(2, 16, 8), fake(8, 16)),
     dict(dx=(8, 8), dweight=(2, 16, 8), dbias=(2, 16), workspace=(4096,)),
     lambda: dict(want_dbias=True)),
]


@pytest.mark.parametrize("name,args,outputs,options", ALLOCATING)
def test_allocations_belong_to_the_given_stream(monkeypatch, name, args, outputs, options):
    import moe_deferred_finalize_gb300 as mf
    from moe_deferred_finalize_gb300 import _abi, _train

    def enter(stream):
        if stream is not None:          # None: the current one, set again on the way out
            raise Entered(stream)

    def library():
        raise RuntimeError("these tensors must not reach the library")

    monkeypatch.setattr(_abi, "_lib", library)
    monkeypatch.setattr(_train, "_lib", library)
    monkeypatch.setattr(_abi, "_FAST", None)
    monkeypatch.setattr(_abi, "_RAW_STREAM", lambda index: CURRENT)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "set_stream", enter)
    fn, a, options = getattr(mf, name), args(), options()
    given = {k: fake(*s) for k, s in outputs.items()}
    with pytest.raises(Entered) as e:
        fn(*a, **options, stream=OTHER)
    assert e.value.args == ((OTHER, torch.device("cuda", 0)),)
    for missing in given:
        some = {k: v for k, v in given.items() if k != missing}
        with pytest.raises(Entered):
            fn(*a, **options, **some, stream=OTHER)
    # nothing to allocate, or the current stream: straight on to the checks
    for kw in (dict(given, stream=OTHER), dict(stream=CURRENT), {}):
        with pytest.raises(Exception) as e:
            fn(*a, **options, **kw)
        assert e.type is not Entered


# ------------------------------------------------------------- references


def test_finalize_reference_against_differences():
    g = torch.Generator().manual_seed(0)
    T, K, P, H = 3, 2, 7, 5
    idx = torch.randperm(P, generator=g)[:T * K].view(T, K).int()
    idx[1, 0] = -1

    def rand(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    x = {"rows": rand(P, H), "w": rand(T, K), "base": rand(T, H), "res": rand(T, H),
         "gamma": rand(H)}
    d = {k: rand(T, H) for k in ("out", "res", "norm")}

    def forward(x):
        rows = torch.where((idx >= 0)[:, :, None], x["rows"][idx.clamp(min=0).long()], 0.0)
        m = 1.5 * (x["w"][:, :, None] * rows).sum(1) + x["base"]
        r = m + x["res"]
        return m, r, r * (r.square().mean(1, keepdim=True) + 1e-2) ** -0.5 * x["gamma"]

    def loss(x):
        return sum((a * b).sum() for a, b in zip(forward(x), (d["out"], d["res"], d["norm"])))

    ref = T_.finalize_backward(x["rows"], idx, x["w"], 1.5, d["out"], d["res"], d["norm"],
                               forward(x)[1], x["gamma"], 1e-2)
    drows = torch.zeros(P, H, dtype=torch.float64)
    drows[idx[idx >= 0].long()] = ref["drows"][0][idx >= 0]
    got = {"rows": drows, "w": ref["dweights"][0], "base": ref["dshared"][0],
           "res": ref["dresidual"][0], "gamma": ref["dgamma"][0]}
    for name, v in x.items():
        for i in range(v.numel()):
            up, down = v.clone(), v.clone()
            up.view(-1)[i] += 1e-6
            down.view(-1)[i] -= 1e-6
            diff = (loss({**x, name: up}) - loss({**x, name: down})) / 2e-6
            assert abs(got[name].reshape(-1)[i] - diff) < 1e-6, (name, i)


def test_gate_reference_against_autograd():
    g = torch.Generator().manual_seed(1)
    z = torch.randn(5, 9, generator=g, dtype=torch.float64, requires_grad=True)
    ids = z.topk(3, dim=1).indices
    dw = torch.randn(5, 3, generator=g, dtype=torch.float64)
    for kind in ("softmax", "sigmoid"):
        c = z.gather(1, ids)
        w = torch.softmax(c, 1) if kind == "softmax" else \
            torch.sigmoid(c) / torch.sigmoid(c).sum(1, keepdim=True)
        want, = torch.autograd.grad((w * dw).sum(), z)
        got = T_.gate_backward(dw, w.detach(), ids.int(), 9, kind, z.detach())[0]
        assert (got - want).abs().max() < 1e-12


def test_adamw_reference_against_torch():
    g = torch.Generator().manual_seed(2)
    p = torch.randn(50, generator=g, dtype=torch.float64)
    q = torch.nn.Parameter(p.clone())
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.8, 0.95), eps=1e-3, weight_decay=0.3)
    m = v = torch.zeros_like(p)
    for step in (1, 2, 3):
        grad = torch.randn(50, generator=g, dtype=torch.float64)
        q.grad = grad.clone()
        opt.step()
        r = T_.adamw(p, grad, m, v, 1e-2, (0.8, 0.95), 1e-3, 0.3, step)
        p, m, v = r["master"][0], r["m"][0], r["v"][0]
        assert (p - q.detach()).abs().max() < 1e-12


def test_eight_bit_reference():
    """Codes of torch's own conversion lie within the bounds."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1000, generator=g, dtype=torch.float64) * 10.0 ** torch.randint(
        -5, 1, (1000,), generator=g)
    for root in (False, True):
        v = x.abs() if root else x
        (y, tol), (scale, _) = T_.code(v, torch.zeros_like(v), root)
        code = y.float().to(torch.float8_e4m3fn).double()
        if root:
            code = torch.where(y > 0, code.clamp(min=2.0 ** -9), code)
        assert ((code - y).abs() <= tol).all()
        assert len(scale) == 4
