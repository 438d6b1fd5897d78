"""Binding of include/moe_ffn.h: the matrix products around the finalize.

Argument marshalling only, as in ``_abi``: shape and dtype checks, output and
workspace allocation through torch, the current CUDA stream, status ->
exception.  Every step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _abi
from ._abi import MoefError, _check, _device, _elsewhere, _on, _ptr, _stream, _under

ACTIVATION = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}

_BF16 = (torch.bfloat16,)
_I32 = (torch.int32,)
_OUT_TYPE = {torch.bfloat16: 0, torch.float32: 1}

_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        lib = _abi._lib()
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        signatures = {
            "moe_linear": (i32, [vp] * 4 + [i32, vp, i32, vp, i32, i32, i32, vp]),
            "moe_linear_backward": (i32, [vp] * 3 + [i32] + [vp] * 4 + [i32] * 3 + [vp, sz, vp]),
            "moe_linear_backward_workspace_bytes": (sz, [i32, i32]),
            "moe_gated_ffn": (i32, [vp] * 3 + [i32, vp, vp, i32, i32, i32, vp]),
            "moe_gated_ffn_backward": (i32,
                                       [vp] * 3 + [i32] + [vp] * 4 + [i32] * 3 + [vp, sz, vp]),
            "moe_gated_ffn_backward_workspace_bytes": (sz, [i32, i32]),
            "moe_permute_rows": (i64, [i32] * 4),
            "moe_permute_workspace_bytes": (sz, [i32] * 3),
            "moe_permute": (i32, [vp] + [i32] * 4 + [vp, vp, i64, vp, vp, vp, sz, vp]),
            "moe_expert_gated_ffn": (i32, [vp, i64] + [vp] * 5 + [i32, vp, i64, i32, i32, i32,
                                                                  vp]),
            "moe_expert_linear": (i32, [vp, i64] + [vp] * 5 + [i32, vp, i64, i32, i32, i32, vp]),
            "moe_expert_gated_ffn_save": (i32, [vp, i64] + [vp] * 5 + [i32, vp, vp, i64, i32, i32,
                                                                       i32, vp]),
            "moe_expert_linear_save": (i32, [vp, i64] + [vp] * 5 + [i32, vp, vp, i64, i32, i32,
                                                                    i32, vp]),
            "moe_ffn_lost_waits": (i32, [ctypes.POINTER(ctypes.c_uint)]),
        }
        for name, (restype, argtypes) in signatures.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = restype, argtypes
        _LIB = lib
    return _LIB


def _int(n):
    """n as a C int; what does not fit becomes -1, which every entry point
    refuses (ctypes would drop the high bits)."""
    return n if -1 <= n <= 0x7FFFFFFF else -1


_ADDRESS = {}


def _address(name):
    """The entry point's address, for the _fastcall extension."""
    if name not in _ADDRESS:
        _ADDRESS[name] = ctypes.cast(getattr(_lib(), name), ctypes.c_void_p).value
    return _ADDRESS[name]


def _call(kind, name, *args):
    """An entry point's status: through the _fastcall extension's ``kind``
    (direct argument conversion) when it was built, else through ctypes."""
    fast = _abi._fastcall()
    if fast is not None:
        return getattr(fast, kind)(_address(name), *args)
    return getattr(_lib(), name)(*args)


def _fast_device(fast, x):
    """The device index of x when the one-pass check of the _fastcall
    extension can take the call (x on the current device), else None."""
    if fast is None or not isinstance(x, torch.Tensor):
        return None
    dev = x.get_device()
    return dev if dev >= 0 and dev == torch.cuda.current_device() else None


def _raw_stream(stream, dev):
    if stream is None and _abi._RAW_STREAM is not None:
        return _abi._RAW_STREAM(dev)
    return _stream(stream, torch.device("cuda", dev))


def _activation(name):
    if name not in ACTIVATION:
        raise ValueError(f"activation must be one of {sorted(ACTIVATION)}")
    return ACTIVATION[name]


def _matrix(t, name, what):
    """The shape of a 2-D CUDA tensor argument that fixes a call's device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda" or t.dim() != 2:
        raise ValueError(f"{name} is a CUDA {what} tensor")
    return t.shape


def _output(t, name, dtype, shape, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check(t, name, (dtype,), shape, device)
    return t


def _optional(t, name, shape, device):
    if t is not None:
        _check(t, name, _BF16, shape, device)


def _workspace_bytes(workspace, device):
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    return workspace.numel() * workspace.element_size()


def _raise(status, where):
    if status != 0:
        raise MoefError(status, where)


def linear(x: torch.Tensor, weight: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, activation: str = "none",
           out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
           save_preact: bool = False, preact: Optional[torch.Tensor] = None,
           stream=None) -> dict:
    """act(x weight^T + bias) + residual in one kernel (include/moe_ffn.h).

    x bf16 [T, K]; weight bf16 [N, K]; bias bf16 [N]; residual bf16 [T, N].
    ``activation``: "none", "silu", "gelu", "gelu_tanh" or "relu".  Returns a
    dict with "out" [T, N] (``out_dtype`` bfloat16 or float32; a given bf16
    ``out`` may be the residual) and, with ``save_preact`` or a given
    ``preact``, "preact" bf16 [T, N] (x weight^T + bias, for
    ``linear_backward``, which gives the gradients: no call here is recorded
    by autograd).  Enqueued on the current stream (or ``stream``, on which
    what the call allocates is then allocated too)."""
    if stream is not None and (out is None or save_preact and preact is None) and \
            _elsewhere(stream, _device(x)):
        return _under(linear, x.device, dict(locals()))
    res = _fast_linear(x, weight, bias, residual, activation, out, out_dtype, save_preact,
                       preact, stream)
    if res is not None:
        return res
    T, K = _matrix(x, "x", "[T, K]")
    N = _matrix(weight, "weight", "[N, K]")[0]
    dev = x.device
    act = _activation(activation)
    _check(x, "x", _BF16, (T, K), dev)
    _check(weight, "weight", _BF16, (N, K), dev)
    _optional(bias, "bias", (N,), dev)
    _optional(residual, "residual", (T, N), dev)
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _OUT_TYPE:
        raise ValueError("out_dtype must be bfloat16 or float32")
    out = _output(out, "out", out_dtype, (T, N), dev)
    res = {"out": out}
    if save_preact or preact is not None:
        res["preact"] = preact = _output(preact, "preact", torch.bfloat16, (T, N), dev)
    with _on(dev):
        st = _lib().moe_linear(_ptr(x), _ptr(weight), _ptr(bias), _ptr(residual), act, _ptr(out),
                               _OUT_TYPE[out_dtype], _ptr(preact), _int(T), _int(N), _int(K),
                               _stream(stream, dev))
    _raise(st, "moe_linear")
    return res


def _fast_linear(x, weight, bias, residual, activation, out, out_dtype, save_preact, preact,
                 stream):
    """linear in one pass through the _fastcall extension, which checks DLPack
    descriptions of the tensors (outputs allocated here are passed by address:
    describing a new tensor costs more than all the rest); None when it is
    missing or a check fails (the Python checks then name the problem)."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, x)
        if dev is None:
            return None
        act = ACTIVATION[activation]
        d = _abi._TO_DLPACK
        out_at = pre_at = None
        if out is None:
            out = torch.empty((x.shape[0], weight.shape[0]), dtype=out_dtype, device=x.device)
            out_at = out.data_ptr()
        if preact is not None:
            pre_at = d(preact)
        elif save_preact:
            preact = torch.empty((x.shape[0], weight.shape[0]), dtype=x.dtype, device=x.device)
            pre_at = preact.data_ptr()
        st = fast.checked_linear(_address("moe_linear"), act, _OUT_TYPE[out.dtype], dev,
                                 _raw_stream(stream, dev), d(x), d(weight),
                                 None if bias is None else d(bias),
                                 None if residual is None else d(residual),
                                 d(out) if out_at is None else out_at, pre_at)
    except (AttributeError, IndexError, KeyError, TypeError, RuntimeError, BufferError):
        return None
    if st < 0:
        return None
    _raise(st, "moe_linear")
    return {"out": out} if preact is None else {"out": out, "preact": preact}


def _fast_gated(x, weight, bias, activation, out, save_preact, preact, stream):
    """gated_ffn likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, x)
        if dev is None:
            return None
        act = ACTIVATION[activation]
        rows = weight.shape[0]
        d = _abi._TO_DLPACK
        out_at = pre_at = None
        if out is None:
            out = torch.empty((x.shape[0], rows // 2), dtype=x.dtype, device=x.device)
            out_at = out.data_ptr()
        if preact is not None:
            pre_at = d(preact)
        elif save_preact:
            preact = torch.empty((x.shape[0], rows), dtype=x.dtype, device=x.device)
            pre_at = preact.data_ptr()
        st = fast.checked_gated(_address("moe_gated_ffn"), act, dev, _raw_stream(stream, dev),
                                d(x), d(weight), None if bias is None else d(bias),
                                d(out) if out_at is None else out_at, pre_at)
    except (AttributeError, IndexError, KeyError, TypeError, RuntimeError, BufferError):
        return None
    if st < 0:
        return None
    _raise(st, "moe_gated_ffn")
    return {"out": out} if preact is None else {"out": out, "preact": preact}


_GRADS = ("dx", "dweight", "dbias")


def _fast_backward(where, gated, dout, x, weight, preact, activation, want, given, workspace,
                   stream):
    """A backward call likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, dout)
        if dev is None:
            return None
        act = ACTIVATION[activation]
        T, n = dout.shape
        d, device = _abi._TO_DLPACK, dout.device
        res, at = {}, []
        for name, wanted, t, like in zip(_GRADS, want, given, (x, weight, weight)):
            if t is not None:
                res[name] = t
                at.append(d(t))
            elif wanted:
                res[name] = t = torch.empty(like.shape if name != "dbias" else like.shape[:1],
                                            dtype=torch.bfloat16, device=device)
                at.append(t.data_ptr())
            else:
                at.append(None)
        if workspace is not None:
            nbytes = _workspace_bytes(workspace, device)
        else:
            nbytes = fast.call_size(_address(where + "_workspace_bytes"), T, n)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        if not res:
            return None
        st = fast.checked_backward(_address(where), gated, act, dev, _raw_stream(stream, dev),
                                   d(dout), d(x), d(weight), None if preact is None else d(preact),
                                   *at, None if workspace is None else workspace.data_ptr(),
                                   nbytes)
    except (AttributeError, IndexError, KeyError, TypeError, ValueError, RuntimeError,
            BufferError):
        return None
    if st < 0:
        return None
    _raise(st, where)
    return res


def _backward(where, gated, dout, x, weight, preact, activation, want_dx, want_dweight,
              want_dbias, dx, dweight, dbias, workspace, stream):
    res = _fast_backward(where, gated, dout, x, weight, preact, activation,
                         (want_dx, want_dweight, want_dbias), (dx, dweight, dbias), workspace,
                         stream)
    if res is not None:
        return res
    T, n = _matrix(dout, "dout", "[T, features]")
    dev = dout.device
    K = _matrix(x, "x", "[T, inputs]")[1]
    act = _activation(activation)
    cols = 2 * n if gated else n
    _check(dout, "dout", _BF16, (T, n), dev)
    _check(x, "x", _BF16, (T, K), dev)
    _check(weight, "weight", _BF16, (cols, K), dev)
    if preact is None:
        if gated or act != 0:
            raise ValueError("preact is needed for the activation's derivative")
    else:
        _check(preact, "preact", _BF16, (T, cols), dev)
        if not gated and act == 0:
            preact = None       # the derivative is 1
    res = {}
    for name, want, t, shape in (("dx", want_dx, dx, (T, K)),
                                 ("dweight", want_dweight, dweight, (cols, K)),
                                 ("dbias", want_dbias, dbias, (cols,))):
        if want or t is not None:
            res[name] = _output(t, name, torch.bfloat16, shape, dev)
    if not res:
        raise ValueError("no gradient is wanted")
    lib = _lib()
    size = lib.moe_gated_ffn_backward_workspace_bytes if gated \
        else lib.moe_linear_backward_workspace_bytes
    nbytes = int(size(_int(T), _int(n)))
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    else:
        nbytes = _workspace_bytes(workspace, dev)
    with _on(dev):
        st = _call("call_backward", where, _ptr(dout), _ptr(x), _ptr(weight), act, _ptr(preact),
                   _ptr(res.get("dx")), _ptr(res.get("dweight")), _ptr(res.get("dbias")), _int(T),
                   _int(n), _int(K), _ptr(workspace), nbytes, _stream(stream, dev))
    _raise(st, where)
    return res


def linear_backward_workspace_bytes(T: int, N: int) -> int:
    """Bytes of workspace linear_backward needs for T rows of N features."""
    return int(_lib().moe_linear_backward_workspace_bytes(_int(int(T)), _int(int(N))))


def linear_backward(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *,
                    activation: str = "none", preact: Optional[torch.Tensor] = None,
                    want_dx: bool = True, want_dweight: bool = True, want_dbias: bool = False,
                    dx: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                    dbias: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``linear`` for dout bf16 [T, N]: the requested of "dx"
    bf16 [T, K], "dweight" bf16 [N, K] and "dbias" bf16 [N].  ``preact``:
    what the forward call saved, needed unless the activation is "none".
    The gradient of the residual is ``dout`` itself.  ``workspace``: at least
    ``linear_backward_workspace_bytes`` bytes, allocated when not given."""
    if stream is not None and (workspace is None or want_dx and dx is None or
                               want_dweight and dweight is None or
                               want_dbias and dbias is None) and \
            _elsewhere(stream, _device(dout)):
        return _under(linear_backward, dout.device, dict(locals()))
    return _backward("moe_linear_backward", False, dout, x, weight, preact, activation, want_dx,
                     want_dweight, want_dbias, dx, dweight, dbias, workspace, stream)


def gated_ffn(x: torch.Tensor, weight: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
              activation: str = "silu", out: Optional[torch.Tensor] = None,
              save_preact: bool = False, preact: Optional[torch.Tensor] = None,
              stream=None) -> dict:
    """act(x Wg^T + bg) * (x Wu^T + bu) in one kernel (include/moe_ffn.h).

    x bf16 [T, H]; weight bf16 [2I, H], the I gate rows and then the I up
    rows; bias bf16 [2I].  Returns a dict with "out" bf16 [T, I] and, with
    ``save_preact`` or a given ``preact``, "preact" bf16 [T, 2I] (both
    projections with their bias, for ``gated_ffn_backward``; not recorded by
    autograd)."""
    if stream is not None and (out is None or save_preact and preact is None) and \
            _elsewhere(stream, _device(x)):
        return _under(gated_ffn, x.device, dict(locals()))
    res = _fast_gated(x, weight, bias, activation, out, save_preact, preact, stream)
    if res is not None:
        return res
    T, H = _matrix(x, "x", "[T, H]")
    rows = _matrix(weight, "weight", "[2I, H]")[0]
    if rows % 2:
        raise ValueError("weight is [2I, H]: the gate rows, then the up rows")
    I = rows // 2
    dev = x.device
    act = _activation(activation)
    _check(x, "x", _BF16, (T, H), dev)
    _check(weight, "weight", _BF16, (rows, H), dev)
    _optional(bias, "bias", (rows,), dev)
    out = _output(out, "out", torch.bfloat16, (T, I), dev)
    res = {"out": out}
    if save_preact or preact is not None:
        res["preact"] = preact = _output(preact, "preact", torch.bfloat16, (T, rows), dev)
    with _on(dev):
        st = _lib().moe_gated_ffn(_ptr(x), _ptr(weight), _ptr(bias), act, _ptr(out),
                                  _ptr(preact), _int(T), _int(I), _int(H),
                                  _stream(stream, dev))
    _raise(st, "moe_gated_ffn")
    return res


def gated_ffn_backward_workspace_bytes(T: int, I: int) -> int:
    """Bytes of workspace gated_ffn_backward needs for T rows of I features."""
    return int(_lib().moe_gated_ffn_backward_workspace_bytes(_int(int(T)), _int(int(I))))


def gated_ffn_backward(dout: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                       preact: torch.Tensor, *, activation: str = "silu", want_dx: bool = True,
                       want_dweight: bool = True, want_dbias: bool = False,
                       dx: Optional[torch.Tensor] = None,
                       dweight: Optional[torch.Tensor] = None,
                       dbias: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``gated_ffn`` for dout bf16 [T, I] and the saved preact
    bf16 [T, 2I]: the requested of "dx" bf16 [T, H], "dweight" bf16 [2I, H]
    and "dbias" bf16 [2I].  ``workspace``: at least
    ``gated_ffn_backward_workspace_bytes`` bytes, allocated when not given."""
    if stream is not None and (workspace is None or want_dx and dx is None or
                               want_dweight and dweight is None or
                               want_dbias and dbias is None) and \
            _elsewhere(stream, _device(dout)):
        return _under(gated_ffn_backward, dout.device, dict(locals()))
    return _backward("moe_gated_ffn_backward", True, dout, x, weight, preact, activation,
                     want_dx, want_dweight, want_dbias, dx, dweight, dbias, workspace, stream)


def _permute_sizes(T, K, E, tile):
    """(rows of the layout at most, bytes of workspace)."""
    fast = _abi._fastcall()
    if fast is not None:
        return fast.permute_sizes(_address("moe_permute_rows"),
                                  _address("moe_permute_workspace_bytes"), T, K, E, tile)
    lib = _lib()
    T, K, E, tile = _int(T), _int(K), _int(E), _int(tile)
    return lib.moe_permute_rows(T, K, E, tile), lib.moe_permute_workspace_bytes(T, K, E)


def _fast_permute(expert_ids, E, tile, row_token, idx_map, offsets, counts, workspace, stream):
    """permute_tokens likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, expert_ids)
        if dev is None:
            return None
        E, tile = int(E), int(tile)
        T, K = expert_ids.shape
        P, nbytes = _permute_sizes(T, K, E, tile)
        d, device, i32 = _abi._TO_DLPACK, expert_ids.device, torch.int32
        res, at = {}, []
        for name, t, shape in (("idx_map", idx_map, (T, K)), ("row_token", row_token, (P,)),
                               ("offsets", offsets, (E + 1,)), ("counts", counts, (E,))):
            if t is None:
                res[name] = t = torch.empty(shape, dtype=i32, device=device)
                at.append(t.data_ptr())
            else:
                res[name] = t
                at.append(d(t))
        if workspace is not None:
            nbytes = _workspace_bytes(workspace, device)
        elif nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        st = fast.checked_permute(_address("moe_permute"), dev, _raw_stream(stream, dev), E, tile,
                                  P, d(expert_ids), *at,
                                  None if workspace is None else workspace.data_ptr(), nbytes)
    except (AttributeError, IndexError, KeyError, TypeError, ValueError, RuntimeError,
            BufferError):
        return None
    if st < 0:
        return None
    _raise(st, "moe_permute")
    return res


def permute_rows(T: int, K: int, E: int, tile: int) -> int:
    """The most rows the grouped layout of T x K slots over E experts can need."""
    return int(_permute_sizes(int(T), int(K), int(E), int(tile))[0])


def permute_tokens(expert_ids: torch.Tensor, E: int, tile: int = 1, *,
                   row_token: Optional[torch.Tensor] = None,
                   idx_map: Optional[torch.Tensor] = None,
                   offsets: Optional[torch.Tensor] = None,
                   counts: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """The padded, expert-grouped layout of expert ids int32 [T, K]
    (include/moe_ffn.h): "idx_map" int32 [T, K] for ``moe_finalize``,
    "row_token" int32 [P] (-1 on padding; P = ``permute_rows`` unless given),
    "offsets" int32 [E + 1] and "counts" int32 [E].  Ids outside [0, E) get
    no row: idx_map is -1 there, which ``moe_finalize`` must not be given
    (leave such tokens out of its T; ``check_indices`` counts them)."""
    if stream is not None and \
            (row_token is None or idx_map is None or offsets is None or counts is None or
             workspace is None) and _elsewhere(stream, _device(expert_ids)):
        return _under(permute_tokens, expert_ids.device, dict(locals()))
    res = _fast_permute(expert_ids, E, tile, row_token, idx_map, offsets, counts, workspace,
                        stream)
    if res is not None:
        return res
    T, K = _matrix(expert_ids, "expert_ids", "[T, K]")
    dev = expert_ids.device
    E, tile = int(E), int(tile)
    _check(expert_ids, "expert_ids", _I32, (T, K), dev)
    P, nbytes = _permute_sizes(T, K, E, tile)
    if row_token is not None:
        P = row_token.numel()
    res = {"idx_map": _output(idx_map, "idx_map", torch.int32, (T, K), dev),
           "row_token": _output(row_token, "row_token", torch.int32, (P,), dev),
           "offsets": _output(offsets, "offsets", torch.int32, (max(E, 0) + 1,), dev),
           "counts": _output(counts, "counts", torch.int32, (max(E, 0),), dev)}
    if workspace is not None:
        nbytes = _workspace_bytes(workspace, dev)
    elif nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    with _on(dev):
        st = _call("call_permute", "moe_permute", _ptr(expert_ids), _int(T), _int(K), _int(E),
                   _int(tile), _ptr(res["idx_map"]), _ptr(res["row_token"]), P, _ptr(res["offsets"]),
                   _ptr(res["counts"]), _ptr(workspace), nbytes, _stream(stream, dev))
    _raise(st, "moe_permute")
    return res


def _fast_expert(where, gated, x, row_token, offsets, counts, weight, bias, activation, out,
                 stream):
    """An expert product likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, x)
        if dev is None:
            return None
        act = ACTIVATION[activation]
        d = _abi._TO_DLPACK
        if out is None:
            M = weight.shape[1]
            out = torch.empty(((x if row_token is None else row_token).shape[0],
                               M // 2 if gated else M), dtype=x.dtype, device=x.device)
            at = out.data_ptr()
        else:
            at = d(out)
        st = fast.checked_expert(_address(where), gated, act, dev, _raw_stream(stream, dev), d(x),
                                 None if row_token is None else d(row_token), d(offsets),
                                 d(counts), d(weight), None if bias is None else d(bias), at)
    except (AttributeError, IndexError, KeyError, TypeError, RuntimeError, BufferError):
        return None
    if st < 0:
        return None
    _raise(st, where)
    return out


def _expert(where, gated, x, row_token, offsets, counts, weight, bias, activation, out, preact,
            stream):
    if preact is None:
        res = _fast_expert(where, gated, x, row_token, offsets, counts, weight, bias, activation,
                           out, stream)
        if res is not None:
            return res
    T, K = _matrix(x, "x", "[T, inputs]")
    dev = x.device
    if not isinstance(weight, torch.Tensor) or weight.dim() != 3:
        raise ValueError("weight is a CUDA [E, features, inputs] tensor")
    E, rows = weight.shape[:2]
    if gated and rows % 2:
        raise ValueError("weight is [E, 2I, H]: the gate rows, then the up rows")
    M = rows // 2 if gated else rows
    act = _activation(activation)
    _check(x, "x", _BF16, (T, K), dev)
    _check(weight, "weight", _BF16, (E, rows, K), dev)
    _check(offsets, "offsets", _I32, (E + 1,), dev)
    _check(counts, "counts", _I32, (E,), dev)
    _optional(bias, "bias", (E, rows), dev)
    P = T
    if row_token is not None:
        P = row_token.numel()
        _check(row_token, "row_token", _I32, (P,), dev)
    out = _output(out, "out", torch.bfloat16, (P, M), dev)
    if preact is not None:
        _check(preact, "preact", _BF16, (P, rows), dev)
        with _on(dev):
            st = getattr(_lib(), where + "_save")(
                _ptr(x), T, _ptr(row_token), _ptr(offsets), _ptr(counts), _ptr(weight),
                _ptr(bias), act, _ptr(out), _ptr(preact), P, _int(E), _int(M), _int(K),
                _stream(stream, dev))
        _raise(st, where + "_save")
        return out
    with _on(dev):
        st = _call("call_expert", where, _ptr(x), T, _ptr(row_token), _ptr(offsets), _ptr(counts),
                   _ptr(weight), _ptr(bias), act, _ptr(out), P, _int(E), _int(M), _int(K),
                   _stream(stream, dev))
    _raise(st, where)
    return out


def expert_gated_ffn(x: torch.Tensor, row_token: Optional[torch.Tensor], offsets: torch.Tensor,
                     counts: torch.Tensor, weight: torch.Tensor, *,
                     bias: Optional[torch.Tensor] = None, activation: str = "silu",
                     out: Optional[torch.Tensor] = None,
                     preact: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``gated_ffn`` over rows grouped by expert (include/moe_ffn.h): out
    bf16 [P, I], row r of expert e from x row ``row_token[r]`` (row r itself
    with ``row_token=None``) and weight[e].

    x bf16 [T, H]; row_token int32 [P], offsets int32 [E + 1] and counts int32
    [E] as from ``permute_tokens``; weight bf16 [E, 2I, H]; bias bf16 [E, 2I].
    Rows of no expert are left as they were (unset when ``out`` is allocated
    here).  ``preact``: a bf16 [P, 2I] tensor that receives both projections
    with their bias, for ``expert_gated_ffn_backward``."""
    if stream is not None and out is None and _elsewhere(stream, _device(x)):
        return _under(expert_gated_ffn, x.device, dict(locals()))
    return _expert("moe_expert_gated_ffn", True, x, row_token, offsets, counts, weight, bias,
                   activation, out, preact, stream)


def expert_linear(x: torch.Tensor, offsets: torch.Tensor, counts: torch.Tensor,
                  weight: torch.Tensor, *, row_token: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, activation: str = "none",
                  out: Optional[torch.Tensor] = None, preact: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """act(x weight[e]^T + bias[e]) over rows grouped by expert: out bf16
    [P, N], the ``permuted_out`` of ``moe_finalize``.  x bf16 [P, K] in the
    layout itself, or [T, K] with ``row_token``; weight bf16 [E, N, K]; bias
    bf16 [E, N]; ``preact`` bf16 [P, N].  Otherwise as ``expert_gated_ffn``."""
    if stream is not None and out is None and _elsewhere(stream, _device(x)):
        return _under(expert_linear, x.device, dict(locals()))
    return _expert("moe_expert_linear", False, x, row_token, offsets, counts, weight, bias,
                   activation, out, preact, stream)


def lost_waits(device=None) -> int:
    """Barrier waits of the tensor-core kernels that were given up on the
    current device (or ``device``) since the library was loaded: 0 unless
    something is broken.  Waits for the device."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    count = ctypes.c_uint()
    with _on(dev):
        st = _lib().moe_ffn_lost_waits(ctypes.byref(count))
    _raise(st, "moe_ffn_lost_waits")
    return count.value
