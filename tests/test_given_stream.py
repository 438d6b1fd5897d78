"""Calls on a given stream (``stream=``) that allocate: what they allocate
belongs to that stream, so that neither a workspace freed on return nor a
recycled block is shared with work on the current stream."""
import ctypes

import pytest
import torch

import ffn_ref as R

BF16 = torch.bfloat16
CURRENT, OTHER = 0x70, 0x90     # stream handles


class Entered(Exception):
    """The given stream was made the current one."""


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on cuda:0."""
    device = property(lambda self: torch.device("cuda", 0))


def fake(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


@pytest.fixture
def entry_points(monkeypatch):
    """The package with streams that only tell whether they were entered."""
    import moe_deferred_finalize_gb300 as mf
    from moe_deferred_finalize_gb300 import _abi, _ffn

    def enter(stream):
        if stream is not None:          # None: the current one, set again on the way out
            raise Entered(stream)

    def library():
        raise RuntimeError("these tensors must not reach the library")

    monkeypatch.setattr(_abi, "_lib", library)
    monkeypatch.setattr(_ffn, "_lib", library)
    monkeypatch.setattr(_abi, "_FAST", None)
    monkeypatch.setattr(_abi, "_RAW_STREAM", lambda index: CURRENT)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "set_stream", enter)
    return mf


def i32(*shape):
    return fake(*shape, dtype=torch.int32)


# name, required arguments, all that the call would allocate
PRODUCTS = [
    ("linear", lambda: (fake(4, 8), fake(8, 8)),
     dict(out=(4, 8), preact=(4, 8)), dict(save_preact=True)),
    ("linear_backward", lambda: (fake(4, 8), fake(4, 8), fake(8, 8)),
     dict(dx=(4, 8), dweight=(8, 8), dbias=(8,), workspace=(4096,)), dict(want_dbias=True)),
    ("gated_ffn", lambda: (fake(4, 8), fake(16, 8)),
     dict(out=(4, 8), preact=(4, 16)), dict(save_preact=True)),
    ("gated_ffn_backward", lambda: (fake(4, 8), fake(4, 8), fake(16, 8), fake(4, 16)),
     dict(dx=(4, 8), dweight=(16, 8), dbias=(16,), workspace=(4096,)), dict(want_dbias=True)),
    ("permute_tokens", lambda: (i32(4, 2), 8),
     dict(row_token=(8,), idx_map=(4, 2), offsets=(9,), counts=(8,), workspace=(4096,)), {}),
    ("expert_gated_ffn", lambda: (fake(4, 8), i32(4), i32(3), i32(2), fake(2, 16, 8)),
     dict(out=(4, 8)), {}),
    ("expert_linear", lambda: (fake(4, 8), i32(3), i32(2), fake(2, 8, 8)), dict(out=(4, 8)), {}),
]


def f32(*shape):
    return fake(*shape, dtype=torch.float32)


def finalize_args():
    return fake(8, 8), i32(4, 2), f32(4, 2), "fp32", fake(4, 8)


def norm():
    return dict(residual=fake(4, 8), gamma=fake(8))


def one_rank():
    x, idx, w, _, shared = finalize_args()
    return [dict(permuted_out=x, idx_map=idx, weights=w, shared_out=shared)], "fp32"


NORM_OUTPUTS = dict(out=(4, 8), residual_out=(4, 8), norm_out=(4, 8))
FINALIZE = [
    ("moe_finalize", finalize_args, dict(out=(4, 8)), {}),
    ("moe_finalize", finalize_args, NORM_OUTPUTS, norm),
    ("moe_finalize_unfused", finalize_args, dict(out=(4, 8), workspace=(4096,)), {}),
    ("bind", finalize_args, NORM_OUTPUTS, norm),
    ("moe_finalize_partial", finalize_args, dict(partial=(4, 8)), {}),
    ("moe_finalize_allreduce", one_rank, NORM_OUTPUTS, norm),
    ("moe_finalize_allreduce_reduce", lambda: ([f32(4, 8)],), NORM_OUTPUTS, norm),
    ("pack_topk_ids", lambda: (i32(4, 2), f32(4, 2)), dict(packed=(4, 2)), {}),
    ("unpack_topk_ids", lambda: (i32(4, 2),), dict(expert_ids=(4, 2), weights=(4, 2)), {}),
    ("check_indices", lambda: (i32(4, 2), 8), dict(counter=(1,)), {}),
]


def test_gate_outputs_belong_to_the_given_stream(entry_points):
    with pytest.raises(Entered):
        entry_points.topk_route(f32(4, 8), 2, stream=OTHER)


@pytest.mark.parametrize("name,args,outputs,options", PRODUCTS + FINALIZE,
                         ids=[p[0] for p in PRODUCTS + FINALIZE])
def test_allocations_belong_to_the_given_stream(entry_points, monkeypatch, name, args, outputs,
                                                options):
    # some take their device from the outputs too, or the current one
    monkeypatch.setattr(OnDevice, "is_cuda", True, raising=False)
    monkeypatch.setattr(OnDevice, "get_device", lambda self: 0, raising=False)
    fn, a = getattr(entry_points, name), args()
    options = options() if callable(options) else options
    integers = name == "permute_tokens"
    given = {k: fake(*s, dtype=torch.int32 if integers else BF16) for k, s in outputs.items()}
    with pytest.raises(Entered) as e:
        fn(*a, **options, stream=OTHER)
    assert e.value.args == ((OTHER, torch.device("cuda", 0)),)
    for missing in given:
        some = {k: v for k, v in given.items() if k != missing}
        with pytest.raises(Entered):
            fn(*a, **options, **some, stream=OTHER)
    # nothing to allocate, or the current stream: straight on to the checks
    monkeypatch.setattr(OnDevice, "is_cuda", False)
    for kw in (dict(given, stream=OTHER), dict(stream=CURRENT), {}):
        with pytest.raises(Exception) as e:
            fn(*a, **options, **kw)
        assert e.type is not Entered


def test_a_stream_of_another_device_is_refused(entry_points, monkeypatch):
    class Stream:
        cuda_stream, device = OTHER, torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    with pytest.raises(ValueError, match="cuda:1"):
        entry_points.linear(fake(4, 8), fake(8, 8), stream=Stream())


# ----------------------------------------------------------------- on a GPU


def rand(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF16, device="cuda").normal_(0.0, scale, generator=g)


def busy(stream):
    """Some 25 ms of work on the stream."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(50_000_000)


def handles(stream):
    return [stream, stream.cuda_stream]


def fill_like(nbytes, value):
    """The current stream takes and fills whatever block of that size is free."""
    return [torch.full((nbytes,), value, dtype=torch.uint8, device="cuda") for _ in range(6)]


@pytest.mark.gpu
@pytest.mark.parametrize("is_gated", [False, True])
def test_backward_workspace_is_not_shared(cuda_lib, is_gated):
    T, n, K = 600, 256, 128
    cols = 2 * n if is_gated else n
    x, w, d, pre = rand(1, T, K), rand(2, cols, K, scale=0.1), rand(3, T, n), rand(4, T, cols)
    ref = R.backward(d, x, w, pre, "gelu", is_gated)
    if is_gated:
        nbytes = cuda_lib.gated_ffn_backward_workspace_bytes(T, n)
    else:
        nbytes = cuda_lib.linear_backward_workspace_bytes(T, n)
    side = torch.cuda.Stream()
    for stream in handles(side):
        torch.cuda.synchronize()
        busy(side)
        if is_gated:
            got = cuda_lib.gated_ffn_backward(d, x, w, pre, activation="gelu", want_dbias=True,
                                              stream=stream)
        else:
            got = cuda_lib.linear_backward(d, x, w, activation="gelu", preact=pre,
                                           want_dbias=True, stream=stream)
        kept = fill_like(nbytes, 0x41)          # bf16 12.06, were it read as dz
        torch.cuda.synchronize()
        R.check(got, ref)
        del kept


@pytest.mark.gpu
def test_row_map_workspace_is_not_shared(cuda_lib):
    T, K, E, tile = 5000, 4, 32, 8              # 20000 slots: two kernels, counts between them
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ids = torch.randint(-1, E, (T, K), dtype=torch.int32, device="cuda", generator=g)
    want = cuda_lib.permute_tokens(ids, E, tile)
    side = torch.cuda.Stream()
    for stream in handles(side):
        torch.cuda.synchronize()
        busy(side)
        got = cuda_lib.permute_tokens(ids, E, tile, stream=stream)
        kept = fill_like(4096, 0) + fill_like(65536, 0)
        torch.cuda.synchronize()
        for key in want:
            assert torch.equal(got[key], want[key]), key
        del kept


def finalize_case(T=128, K=2, H=4096, E=8):
    """Arguments of moe_finalize: token t's slots are rows t K .. of x."""
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    idx = torch.randperm(T * K, device="cuda", generator=g).int().view(T, K)
    return rand(12, T * K, H), idx, torch.rand(T, K, device="cuda", generator=g), "fp32", \
        rand(13, T, H)


@pytest.mark.gpu
def test_unfused_workspace_is_not_shared(cuda_lib):
    args = finalize_case()
    T, H = args[4].shape
    want = cuda_lib.moe_finalize_unfused(*args)["out"]
    side = torch.cuda.Stream()
    for stream in handles(side):
        torch.cuda.synchronize()
        busy(side)
        got = cuda_lib.moe_finalize_unfused(*args, stream=stream)["out"]
        kept = fill_like(cuda_lib.unfused_workspace_bytes(T, H), 0x41)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del kept


@pytest.mark.gpu
def test_every_call_on_another_stream_gives_the_same_bits(cuda_lib):
    args = finalize_case()
    x, idx, w, _, shared = args
    res = dict(residual=rand(14, *shared.shape), gamma=rand(15, shared.shape[1]))
    logits = torch.rand(40, 16, device="cuda")
    ids = torch.randint(0, 16, (40, 2), dtype=torch.int32, device="cuda")
    words = cuda_lib.pack_topk_ids(ids, w[:40].contiguous())
    ranks = [dict(permuted_out=x, idx_map=idx, weights=w, shared_out=shared)] * 2
    partial = cuda_lib.moe_finalize_partial(*args)
    calls = [lambda **s: cuda_lib.moe_finalize(*args, **s),
             lambda **s: cuda_lib.moe_finalize(*args, **res, write_out=False, **s),
             lambda **s: cuda_lib.moe_finalize_unfused(*args, **res, **s),
             lambda **s: cuda_lib.bind(*args, **res, **s)(),
             lambda **s: cuda_lib.moe_finalize_partial(*args, **s),
             lambda **s: cuda_lib.moe_finalize_allreduce(ranks, "fp32", **res, **s),
             lambda **s: cuda_lib.moe_finalize_allreduce_reduce([partial, partial], **res, **s),
             lambda **s: cuda_lib.topk_route(logits, 4, want_packed=True, **s),
             lambda **s: cuda_lib.pack_topk_ids(ids, w[:40].contiguous(), **s),
             lambda **s: cuda_lib.unpack_topk_ids(words, **s),
             lambda **s: cuda_lib.check_indices(idx, idx.numel() - 3, **s)]

    def tensors(r):
        r = list(r.values()) if isinstance(r, dict) else r
        r = r if isinstance(r, (list, tuple)) else [r]
        return [t.clone() for t in r if t is not None]

    for i, call in enumerate(calls):
        want = tensors(call())
        side = torch.cuda.Stream()
        for stream in handles(side):
            side.wait_stream(torch.cuda.current_stream())
            r = call(stream=stream)
            torch.cuda.current_stream().wait_stream(side)
            got = tensors(r)
            assert len(got) == len(want)
            for a, b in zip(got, want):
                assert torch.equal(a, b), i


@pytest.mark.gpu
def test_outputs_do_not_take_blocks_still_in_use(cuda_lib):
    """A block freed by the host while the current stream has yet to read it
    does not become an output of a call on another stream."""
    T, n, K = 200, 512, 256
    x, w, w2 = rand(6, T, K), rand(7, n, K, scale=0.06), rand(8, 2 * n, K, scale=0.06)
    we, offsets = w.view(1, n, K), torch.tensor([0, T], dtype=torch.int32, device="cuda")
    counts = torch.tensor([T], dtype=torch.int32, device="cuda")
    idx = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    one = torch.ones(T, 1, device="cuda")
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    calls = [lambda s: cuda_lib.linear(x, w, save_preact=True, stream=s),
             lambda s: cuda_lib.gated_ffn(x, w2, stream=s),
             lambda s: {"out": cuda_lib.expert_linear(x, offsets, counts, we, stream=s)},
             lambda s: cuda_lib.moe_finalize(x, idx, one, "fp32", x, stream=s)]
    for call in calls:
        want = call(None)
        for stream in handles(side):
            old = [torch.full((T, n), 3.0, dtype=BF16, device="cuda") for _ in range(8)]
            read = torch.empty(8, T, n, dtype=BF16, device="cuda")
            torch.cuda.synchronize()
            busy(current)
            torch.stack(old, out=read)
            del old
            got = call(stream)
            torch.cuda.synchronize()
            assert (read == 3).all()
            for key in want:
                assert torch.equal(got[key], want[key])


@pytest.mark.gpu
def test_the_current_stream_stays_current(cuda_lib):
    """Also when the call is refused, and from a stream that is not the default."""
    x, w = rand(9, 20, 64), rand(10, 32, 64)
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(mine):
        for stream in handles(side):
            cuda_lib.linear(x, w, stream=stream)
            assert torch.cuda.current_stream() == mine
            with pytest.raises(ValueError):
                cuda_lib.linear(x, w[:, :32], stream=stream)
            assert torch.cuda.current_stream() == mine
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_handles_of_every_kind(cuda_lib):
    """The legacy default stream by its handles, from another current stream; a
    ctypes pointer; a graph whose capture the given stream has joined."""
    x, w = rand(9, 20, 64), rand(10, 32, 64)
    want = cuda_lib.linear(x, w)["out"]
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(mine):
        for stream in (0, torch.cuda.default_stream(), ctypes.c_void_p(0),
                       ctypes.c_void_p(side.cuda_stream)):
            got = cuda_lib.linear(x, w, stream=stream)["out"]
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    ws = {}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        ws["out"] = cuda_lib.linear(x, w, stream=side)["out"]
        ws["grads"] = cuda_lib.linear_backward(ws["out"], x, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    x.copy_(rand(11, 20, 64))
    graph.replay()
    torch.cuda.synchronize()
    want = cuda_lib.linear(x, w)["out"]
    assert torch.equal(ws["out"], want)
    for key, t in cuda_lib.linear_backward(want, x, w).items():
        assert torch.equal(ws["grads"][key], t)


@pytest.mark.gpu
def test_results_may_be_dropped_while_the_current_stream_reads_them(cuda_lib):
    x, w = rand(9, 200, 256), rand(10, 512, 256, scale=0.06)
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    want = cuda_lib.linear(x, w)["out"]
    for stream in handles(side):
        torch.cuda.synchronize()
        got = cuda_lib.linear(x, w, stream=stream)["out"]
        current.wait_stream(side)
        busy(current)
        copy = got * 1.0
        del got
        with torch.cuda.stream(side):
            kept = fill_like(want.numel() * 2, 0x41)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
        del kept
