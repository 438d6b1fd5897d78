"""Binding of include/moe_train.h: the MoE layer's training side.

Argument marshalling only, as in ``_abi`` and ``_ffn``.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _abi
from ._abi import (_WCODE, _WDTYPE, GATE, WKIND, _check, _device, _elsewhere, _on, _ptr,
                   _stream, _under)
from ._ffn import (_BF16, _I32, _OUT_TYPE, ACTIVATION, _activation, _fast_device, _int, _matrix,
                   _optional, _output, _raise, _raw_stream, _workspace_bytes)

_F32 = (torch.float32,)
BLOCK = 256         # values of an 8-bit AdamW state that share a scale


class AdamWTensor(ctypes.Structure):
    """moef_adamw_tensor."""
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("n", ctypes.c_int64)]


class AdamWConfig(ctypes.Structure):
    """moef_adamw_config."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("device_step", ctypes.c_void_p), ("device_lr", ctypes.c_void_p),
                ("grad_scale", ctypes.c_void_p), ("step", ctypes.c_int),
                ("state_bits", ctypes.c_int), ("param_type", ctypes.c_int),
                ("grad_type", ctypes.c_int)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        lib = _abi._lib()
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        f32 = ctypes.c_float
        expert = [vp, vp, i64] + [vp] * 4 + [i32] + [vp] * 4 + [i64] + [i32] * 3 + [vp, sz, vp]
        signatures = {
            "moe_finalize_backward_workspace_bytes": (sz, [i32, i32]),
            "moe_finalize_backward": (i32, [vp, i64, vp, vp, i32, f32, vp, vp, f32] + [vp] * 8 +
                                      [i32] * 3 + [vp, sz, vp]),
            "moe_unpermute": (i32, [vp, i64] + [vp] * 4 + [i32] * 3 + [vp]),
            "moe_topk_route_backward": (i32, [vp] * 4 + [i32] * 4 + [vp, i32, vp]),
            "moe_expert_backward_workspace_bytes": (sz, [i64, i32, i32]),
            "moe_expert_gated_ffn_backward": (i32, expert),
            "moe_expert_linear_backward": (i32, expert),
            "moe_adamw_step": (i32, [ctypes.POINTER(AdamWTensor), i32,
                                     ctypes.POINTER(AdamWConfig), vp]),
        }
        for name, (restype, argtypes) in signatures.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = restype, argtypes
        _LIB = lib
    return _LIB


_ADDRESS = {}


def _address(name):
    """The entry point's address, for the _fastcall extension."""
    if name not in _ADDRESS:
        _ADDRESS[name] = ctypes.cast(getattr(_lib(), name), ctypes.c_void_p).value
    return _ADDRESS[name]


# what the one-pass calls below leave to the checks that name the problem
_REFUSED = (AttributeError, IndexError, KeyError, TypeError, ValueError, RuntimeError,
            BufferError)


def _describe(t):
    return None if t is None else _abi._TO_DLPACK(t)


def finalize_backward_workspace_bytes(T: int, H: int) -> int:
    """Bytes of workspace moe_finalize_backward needs for dgamma."""
    return int(_lib().moe_finalize_backward_workspace_bytes(_int(int(T)), _int(int(H))))


def moe_finalize_backward(permuted_out: torch.Tensor, idx_map: torch.Tensor,
                          weights: torch.Tensor, wkind: str,
                          dout: Optional[torch.Tensor] = None, *, routed_scale: float = 1.0,
                          dresidual_out: Optional[torch.Tensor] = None,
                          dnorm_out: Optional[torch.Tensor] = None,
                          residual_out: Optional[torch.Tensor] = None,
                          gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          want_drows: bool = True, want_dweights: bool = True,
                          want_dgamma: bool = True, drows: Optional[torch.Tensor] = None,
                          dweights: Optional[torch.Tensor] = None,
                          dshared: Optional[torch.Tensor] = None,
                          dresidual: Optional[torch.Tensor] = None,
                          dgamma: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``moe_finalize`` (include/moe_train.h) from those of its
    outputs: ``dout``, ``dresidual_out`` and ``dnorm_out``, bf16 [T, H], each
    optional.  permuted_out, idx_map, weights, wkind, routed_scale, gamma and
    eps as in the forward call; ``residual_out`` as it returned it (with
    dnorm_out).

    Returns a dict with "drows" bf16 [P, H] (rows that no slot names are left as
    they were: unset when allocated here), "dweights" fp32 [T, K] (0 for slots
    outside [0, P)); with dresidual_out or dnorm_out "dresidual" and "dshared"
    bf16 [T, H], one tensor when dout is not given (without them, dshared is
    dout itself); with dnorm_out "dgamma" bf16 [H].  ``dshared`` and
    ``dresidual`` may be ``dout`` or ``dresidual_out``.  ``workspace``: at least
    ``finalize_backward_workspace_bytes`` bytes, allocated when not given."""
    norm = dnorm_out is not None
    residual = norm or dresidual_out is not None
    separate = residual and dout is not None
    if stream is not None and \
            (want_drows and drows is None or want_dweights and dweights is None or
             residual and dresidual is None or separate and dshared is None or
             norm and (want_dgamma or dgamma is not None) and
             (dgamma is None or workspace is None)) and \
            _elsewhere(stream, _device(permuted_out)):
        args = dict(locals())
        for name in ("norm", "residual", "separate"):
            del args[name]
        return _under(moe_finalize_backward, permuted_out.device, args)
    res = _fast_finalize_backward(permuted_out, idx_map, weights, wkind, dout, routed_scale,
                                  dresidual_out, dnorm_out, residual_out, gamma, eps, want_drows,
                                  want_dweights, want_dgamma, drows, dweights, dshared,
                                  dresidual, dgamma, workspace, stream)
    if res is not None:
        return res
    if wkind not in WKIND:
        raise ValueError(f"wkind must be one of {sorted(WKIND)}")
    P, H = _matrix(permuted_out, "permuted_out", "[P, H]")
    T, K = _matrix(idx_map, "idx_map", "[T, K]")
    dev = permuted_out.device
    _check(permuted_out, "permuted_out", _BF16, (P, H), dev)
    _check(idx_map, "idx_map", _I32, (T, K), dev)
    _check(weights, "weights", _WDTYPE[wkind], (T, K), dev)
    if dout is None and not residual:
        raise ValueError("no gradient is given: dout, dresidual_out or dnorm_out")
    for name, t in (("dout", dout), ("dresidual_out", dresidual_out), ("dnorm_out", dnorm_out)):
        _optional(t, name, (T, H), dev)
    if norm:
        _check(residual_out, "residual_out", _BF16, (T, H), dev)
        _check(gamma, "gamma", _BF16, (H,), dev)
    elif residual_out is not None or gamma is not None:
        raise ValueError("residual_out and gamma go with dnorm_out")
    res = {}
    if want_drows or drows is not None:
        res["drows"] = drows = _output(drows, "drows", torch.bfloat16, (P, H), dev)
    if want_dweights or dweights is not None:
        res["dweights"] = dweights = _output(dweights, "dweights", torch.float32, (T, K), dev)
    if residual:
        if not separate:        # one value, one buffer
            dresidual = dshared if dresidual is None else dresidual
        dresidual = _output(dresidual, "dresidual", torch.bfloat16, (T, H), dev)
        if separate or dshared is not None and dshared is not dresidual:
            dshared = _output(dshared, "dshared", torch.bfloat16, (T, H), dev)
        else:
            dshared = None
        res["dresidual"] = dresidual
        res["dshared"] = dresidual if dshared is None else dshared
    elif dshared is not None or dresidual is not None:
        raise ValueError("dshared and dresidual are dout itself without dresidual_out and dnorm_out")
    nbytes = 0
    if norm and (want_dgamma or dgamma is not None):
        res["dgamma"] = dgamma = _output(dgamma, "dgamma", torch.bfloat16, (H,), dev)
        if workspace is None:
            nbytes = finalize_backward_workspace_bytes(T, H)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        else:
            nbytes = _workspace_bytes(workspace, dev)
    elif dgamma is not None:
        raise ValueError("dgamma needs dnorm_out")
    if not res:
        raise ValueError("no gradient is wanted")
    with _on(dev):
        st = _lib().moe_finalize_backward(
            _ptr(permuted_out), P, _ptr(idx_map), _ptr(weights), WKIND[wkind],
            float(routed_scale), _ptr(residual_out), _ptr(gamma), float(eps), _ptr(dout),
            _ptr(dresidual_out), _ptr(dnorm_out), _ptr(drows), _ptr(dweights), _ptr(dshared),
            _ptr(dresidual), _ptr(dgamma), _int(T), _int(K), _int(H), _ptr(workspace), nbytes,
            _stream(stream, dev))
    _raise(st, "moe_finalize_backward")
    return res


def _fast_finalize_backward(permuted_out, idx_map, weights, wkind, dout, routed_scale,
                            dresidual_out, dnorm_out, residual_out, gamma, eps, want_drows,
                            want_dweights, want_dgamma, drows, dweights, dshared, dresidual,
                            dgamma, workspace, stream):
    """moe_finalize_backward in one pass through the _fastcall extension, which
    checks DLPack descriptions of the tensors; None when it is missing or a check
    fails."""
    fast = _abi._fastcall()
    norm = dnorm_out is not None
    residual = norm or dresidual_out is not None
    if not residual and (dout is None or dshared is not None or dresidual is not None) or \
            dgamma is not None and not norm:
        return None
    try:
        dev = _fast_device(fast, permuted_out)
        if dev is None:
            return None
        device, d, empty_like = permuted_out.device, _abi._TO_DLPACK, torch.empty_like
        like = dnorm_out if norm else dresidual_out
        separate = residual and dout is not None
        if residual and not separate and dshared is not None:
            return None
        # what the extension is given for an output: the description of one that the
        # caller gave, the address of one made here
        res, at = {}, [None] * 5
        if drows is not None:
            res["drows"], at[0] = drows, d(drows)
        elif want_drows:
            res["drows"] = drows = empty_like(permuted_out)
            at[0] = drows.data_ptr()
        if dweights is not None:
            res["dweights"], at[1] = dweights, d(dweights)
        elif want_dweights:
            res["dweights"] = dweights = torch.empty(idx_map.shape, dtype=torch.float32,
                                                     device=device)
            at[1] = dweights.data_ptr()
        if residual:
            if dresidual is None:
                dresidual = empty_like(like)
                at[3] = dresidual.data_ptr()
            else:
                at[3] = d(dresidual)
            res["dresidual"] = dresidual
            if not separate:
                res["dshared"] = dresidual
            elif dshared is None:
                res["dshared"] = dshared = empty_like(like)
                at[2] = dshared.data_ptr()
            else:
                res["dshared"], at[2] = dshared, d(dshared)
        nbytes, ws = 0, None
        if norm and (want_dgamma or dgamma is not None):
            if dgamma is None:
                dgamma = empty_like(gamma)
                at[4] = dgamma.data_ptr()
            else:
                at[4] = d(dgamma)
            res["dgamma"] = dgamma
            if workspace is not None:
                nbytes = _workspace_bytes(workspace, device)
            else:
                nbytes = fast.call_size(_address("moe_finalize_backward_workspace_bytes"),
                                        idx_map.shape[0], permuted_out.shape[1])
                if nbytes:
                    workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            ws = None if workspace is None else workspace.data_ptr()
        if not res:
            return None
        code, bits = _WCODE[wkind]
        st = fast.checked_finalize_backward(
            _address("moe_finalize_backward"), WKIND[wkind], code, bits, routed_scale, eps, dev,
            _raw_stream(stream, dev), ws, nbytes, d(permuted_out), d(idx_map), d(weights),
            None if residual_out is None else d(residual_out), None if gamma is None else d(gamma),
            None if dout is None else d(dout),
            None if dresidual_out is None else d(dresidual_out),
            None if dnorm_out is None else d(dnorm_out), *at)
    except _REFUSED:
        return None
    if st < 0:
        return None
    _raise(st, "moe_finalize_backward")
    return res


def _fast_unpermute(rows, idx_map, adds, out, stream):
    """unpermute_tokens likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, rows)
        if dev is None:
            return None
        if out is None:
            out = torch.empty((idx_map.shape[0], rows.shape[1]), dtype=torch.bfloat16,
                              device=rows.device)
            at = out.data_ptr()
        else:
            at = _abi._TO_DLPACK(out)
        st = fast.checked_unpermute(_address("moe_unpermute"), dev, _raw_stream(stream, dev),
                                    _abi._TO_DLPACK(rows), _abi._TO_DLPACK(idx_map),
                                    _describe(adds[0]), _describe(adds[1]), at)
    except _REFUSED:
        return None
    if st < 0:
        return None
    _raise(st, "moe_unpermute")
    return out


def unpermute_tokens(rows: torch.Tensor, idx_map: torch.Tensor, *, add=None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows grouped by expert back to their tokens (include/moe_train.h): out
    bf16 [T, H], out[t] = sum_k rows[idx_map[t, k]] + add[t], where a slot outside
    [0, P) adds nothing.  The gradient of the gather of ``expert_gated_ffn`` and
    ``expert_linear``: rows is their backward calls' "dx".

    rows bf16 [P, H]; idx_map int32 [T, K]; ``add``: a bf16 [T, H] tensor, or a
    sequence of at most two; ``out`` may be one of them."""
    if stream is not None and out is None and _elsewhere(stream, _device(rows)):
        return _under(unpermute_tokens, rows.device, dict(locals()))
    adds = [] if add is None else [add] if isinstance(add, torch.Tensor) else list(add)
    if len(adds) > 2:
        raise ValueError("add is at most two tensors")
    adds += [None] * (2 - len(adds))
    res = _fast_unpermute(rows, idx_map, adds, out, stream)
    if res is not None:
        return res
    P, H = _matrix(rows, "rows", "[P, H]")
    T, K = _matrix(idx_map, "idx_map", "[T, K]")
    dev = rows.device
    _check(rows, "rows", _BF16, (P, H), dev)
    _check(idx_map, "idx_map", _I32, (T, K), dev)
    for t in adds:
        _optional(t, "add", (T, H), dev)
    out = _output(out, "out", torch.bfloat16, (T, H), dev)
    with _on(dev):
        st = _lib().moe_unpermute(_ptr(rows), P, _ptr(idx_map), _ptr(adds[0]), _ptr(adds[1]),
                                  _ptr(out), _int(T), _int(K), _int(H), _stream(stream, dev))
    _raise(st, "moe_unpermute")
    return out


def _fast_gate_backward(dweights, weights, expert_ids, E, kind, logits, out_dtype, dlogits,
                        stream):
    """topk_route_backward likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, dweights)
        if dev is None:
            return None
        if dlogits is None:
            dlogits = torch.empty((dweights.shape[0], E), dtype=out_dtype, device=dweights.device)
            at = dlogits.data_ptr()
        else:
            at = _abi._TO_DLPACK(dlogits)
        st = fast.checked_gate_backward(
            _address("moe_topk_route_backward"), dev, _raw_stream(stream, dev), E, GATE[kind],
            _OUT_TYPE[dlogits.dtype], _abi._TO_DLPACK(dweights), _abi._TO_DLPACK(weights),
            _abi._TO_DLPACK(expert_ids), _describe(logits), at)
    except _REFUSED:
        return None
    if st < 0:
        return None
    _raise(st, "moe_topk_route_backward")
    return dlogits


def topk_route_backward(dweights: torch.Tensor, weights: torch.Tensor, expert_ids: torch.Tensor,
                        E: int, kind: str = "sigmoid", *, logits: Optional[torch.Tensor] = None,
                        out_dtype: torch.dtype = torch.bfloat16,
                        dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of ``topk_route``'s weights (include/moe_train.h): dlogits
    [T, E], ``out_dtype`` bfloat16 (as ``linear_backward`` takes it) or float32.

    dweights, weights fp32 [T, K] and expert_ids int32 [T, K] as the gate
    returned them; ``logits`` fp32 [T, E], needed for the sigmoid gate.  Slots
    whose id is outside [0, E) (padding) count for nothing."""
    if stream is not None and dlogits is None and _elsewhere(stream, _device(dweights)):
        return _under(topk_route_backward, dweights.device, dict(locals()))
    res = _fast_gate_backward(dweights, weights, expert_ids, E, kind, logits, out_dtype, dlogits,
                              stream)
    if res is not None:
        return res
    if kind not in GATE:
        raise ValueError(f"kind must be one of {sorted(GATE)}")
    T, K = _matrix(dweights, "dweights", "[T, K]")
    dev, E = dweights.device, int(E)
    _check(dweights, "dweights", _F32, (T, K), dev)
    _check(weights, "weights", _F32, (T, K), dev)
    _check(expert_ids, "expert_ids", _I32, (T, K), dev)
    if logits is not None:
        _check(logits, "logits", _F32, (T, E), dev)
    elif kind == "sigmoid":
        raise ValueError("the sigmoid gate's gradient needs logits")
    if dlogits is not None:
        out_dtype = dlogits.dtype
    if out_dtype not in _OUT_TYPE:
        raise ValueError("out_dtype must be bfloat16 or float32")
    dlogits = _output(dlogits, "dlogits", out_dtype, (T, max(E, 0)), dev)
    with _on(dev):
        st = _lib().moe_topk_route_backward(
            _ptr(dweights), _ptr(weights), _ptr(expert_ids), _ptr(logits), _int(T), _int(E),
            _int(K), GATE[kind], _ptr(dlogits), _OUT_TYPE[out_dtype], _stream(stream, dev))
    _raise(st, "moe_topk_route_backward")
    return dlogits


def expert_backward_workspace_bytes(P: int, cols: int, inputs: int = 0) -> int:
    """Bytes of workspace the expert products' backward calls need for P rows of
    ``cols`` features before the activation (2I gated, N linear; 0 for a linear
    product without one whose dout is 16-byte aligned, N a multiple of 8).
    ``inputs``: the width of x, when dweight is wanted and x has a row map, a
    width that is not a multiple of 8, or is not 16-byte aligned."""
    return int(_lib().moe_expert_backward_workspace_bytes(int(P), _int(int(cols)),
                                                          _int(int(inputs))))


def _expert_workspace(res, dout, x, row_token, P, cols, K, act, gated):
    """The arguments of expert_backward_workspace_bytes for a call with these
    outputs."""
    products = "dx" in res or "dweight" in res
    makes_dz = products and (gated or act or cols % 8 or dout.data_ptr() % 16)
    copies_x = "dweight" in res and (row_token is not None or K % 8 or x.data_ptr() % 16)
    return P, cols if makes_dz else 0, K if copies_x else 0


def _fast_expert_backward(where, gated, dout, x, row_token, offsets, counts, weight, preact,
                          activation, want, given, workspace, stream):
    """An expert product's backward call likewise."""
    fast = _abi._fastcall()
    try:
        dev = _fast_device(fast, dout)
        if dev is None:
            return None
        act, device = ACTIVATION[activation], dout.device
        P, (E, cols, K) = dout.shape[0], weight.shape
        d, res, at = _abi._TO_DLPACK, {}, []
        for name, wanted, t, shape in zip(("dx", "dweight", "dbias"), want, given,
                                          ((P, K), (E, cols, K), (E, cols))):
            if t is not None:
                res[name] = t
                at.append(d(t))
            elif wanted:
                res[name] = t = torch.empty(shape, dtype=torch.bfloat16, device=device)
                at.append(t.data_ptr())
            else:
                at.append(None)
        if not res:
            return None
        if workspace is not None:
            nbytes = _workspace_bytes(workspace, device)
        else:
            nbytes = fast.call_size3(
                _address("moe_expert_backward_workspace_bytes"),
                *_expert_workspace(res, dout, x, row_token, P, cols, K, act, gated))
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
        st = fast.checked_expert_backward(
            _address(where), gated, act, dev, _raw_stream(stream, dev), _ptr(workspace), nbytes,
            d(dout), d(x), _describe(row_token), d(offsets), d(counts), d(weight),
            _describe(preact), *at)
    except _REFUSED:
        return None
    if st < 0:
        return None
    _raise(st, where)
    return res


def _expert_backward(where, gated, dout, x, row_token, offsets, counts, weight, preact,
                     activation, want_dx, want_dweight, want_dbias, dx, dweight, dbias,
                     workspace, stream):
    res = _fast_expert_backward(where, gated, dout, x, row_token, offsets, counts, weight, preact,
                                activation, (want_dx, want_dweight, want_dbias),
                                (dx, dweight, dbias), workspace, stream)
    if res is not None:
        return res
    P, n = _matrix(dout, "dout", "[P, features]")
    dev = dout.device
    T, K = _matrix(x, "x", "[T, inputs]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 3:
        raise ValueError("weight is a CUDA [E, features, inputs] tensor")
    E, cols = weight.shape[0], 2 * n if gated else n
    act = _activation(activation)
    _check(dout, "dout", _BF16, (P, n), dev)
    _check(x, "x", _BF16, (T, K), dev)
    _check(weight, "weight", _BF16, (E, cols, K), dev)
    _check(offsets, "offsets", _I32, (E + 1,), dev)
    _check(counts, "counts", _I32, (E,), dev)
    if row_token is not None:
        _check(row_token, "row_token", _I32, (P,), dev)
    elif T != P:
        raise ValueError(f"x has {T} rows, dout {P}: without row_token both are in the layout")
    if preact is None:
        if gated or act != 0:
            raise ValueError("preact is needed for the activation's derivative")
    else:
        _check(preact, "preact", _BF16, (P, cols), dev)
        if not gated and act == 0:
            preact = None       # the derivative is 1
    res = {}
    for name, want, t, shape in (("dx", want_dx, dx, (P, K)),
                                 ("dweight", want_dweight, dweight, (E, cols, K)),
                                 ("dbias", want_dbias, dbias, (E, cols))):
        if want or t is not None:
            res[name] = _output(t, name, torch.bfloat16, shape, dev)
    if not res:
        raise ValueError("no gradient is wanted")
    if workspace is None:
        nbytes = expert_backward_workspace_bytes(
            *_expert_workspace(res, dout, x, row_token, P, cols, K, act, gated))
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    else:
        nbytes = _workspace_bytes(workspace, dev)
    with _on(dev):
        st = getattr(_lib(), where)(
            _ptr(dout), _ptr(x), T, _ptr(row_token), _ptr(offsets), _ptr(counts), _ptr(weight),
            act, _ptr(preact), _ptr(res.get("dx")), _ptr(res.get("dweight")),
            _ptr(res.get("dbias")), P, _int(E), _int(n), _int(K), _ptr(workspace), nbytes,
            _stream(stream, dev))
    _raise(st, where)
    return res


def expert_gated_ffn_backward(dout: torch.Tensor, x: torch.Tensor,
                              row_token: Optional[torch.Tensor], offsets: torch.Tensor,
                              counts: torch.Tensor, weight: torch.Tensor, preact: torch.Tensor,
                              *, activation: str = "silu", want_dx: bool = True,
                              want_dweight: bool = True, want_dbias: bool = False,
                              dx: Optional[torch.Tensor] = None,
                              dweight: Optional[torch.Tensor] = None,
                              dbias: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``expert_gated_ffn`` (include/moe_train.h) for dout bf16
    [P, I] and the saved preact bf16 [P, 2I]: the requested of "dx" bf16 [P, H]
    (per row of the layout; ``unpermute_tokens`` sums them to tokens; rows of no
    expert are left as they were), "dweight" bf16 [E, 2I, H] (zeros for an
    expert without rows) and "dbias" bf16 [E, 2I].  x, row_token, offsets,
    counts and weight as in the forward call.  ``workspace``: at least
    ``expert_backward_workspace_bytes(P, 2I, H)`` bytes, allocated when not given."""
    if stream is not None and (workspace is None or want_dx and dx is None or
                               want_dweight and dweight is None or
                               want_dbias and dbias is None) and \
            _elsewhere(stream, _device(dout)):
        return _under(expert_gated_ffn_backward, dout.device, dict(locals()))
    return _expert_backward("moe_expert_gated_ffn_backward", True, dout, x, row_token, offsets,
                            counts, weight, preact, activation, want_dx, want_dweight,
                            want_dbias, dx, dweight, dbias, workspace, stream)


def expert_linear_backward(dout: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                           counts: torch.Tensor, weight: torch.Tensor, *,
                           row_token: Optional[torch.Tensor] = None, activation: str = "none",
                           preact: Optional[torch.Tensor] = None, want_dx: bool = True,
                           want_dweight: bool = True, want_dbias: bool = False,
                           dx: Optional[torch.Tensor] = None,
                           dweight: Optional[torch.Tensor] = None,
                           dbias: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of ``expert_linear`` for dout bf16 [P, N]: the requested of
    "dx" bf16 [P, K], "dweight" bf16 [E, N, K] and "dbias" bf16 [E, N].
    ``preact`` bf16 [P, N]: what the forward call saved, needed unless the
    activation is "none".  Otherwise as ``expert_gated_ffn_backward``."""
    if stream is not None and (workspace is None or want_dx and dx is None or
                               want_dweight and dweight is None or
                               want_dbias and dbias is None) and \
            _elsewhere(stream, _device(dout)):
        return _under(expert_linear_backward, dout.device, dict(locals()))
    return _expert_backward("moe_expert_linear_backward", False, dout, x, row_token, offsets,
                            counts, weight, preact, activation, want_dx, want_dweight,
                            want_dbias, dx, dweight, dbias, workspace, stream)


# ------------------------------------------------------------------ AdamW


def _number(t, name, dtype, device):
    """A device number (a one-element tensor), or None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.numel() != 1:
        raise ValueError(f"{name} must be a one-element tensor")
    _check(t, name, (dtype,), t.shape, device)
    return t


class BoundAdamW:
    """An AdamW step whose tensors were checked and marshalled once (``bind_adamw``).

    Calling it enqueues one step over them.  The tensors must stay alive and
    keep their storage while the object is used."""

    def __init__(self, table, kept, types, device):
        self._table, self._kept, self._types, self._device = table, kept, types, device
        self._fn = _lib().moe_adamw_step

    def __call__(self, *, step, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, grad_scale: Optional[torch.Tensor] = None,
                 stream=None) -> None:
        """One step.  ``step``: the number of this step, from 1, or an int32
        device number; ``lr``: a number, or a float32 device number;
        ``grad_scale``: a float32 device number that multiplies the gradients."""
        dev = self._device
        device_step = device_lr = None
        if isinstance(step, torch.Tensor):
            device_step, step = _ptr(_number(step, "step", torch.int32, dev)), 1
        if isinstance(lr, torch.Tensor):
            device_lr, lr = _ptr(_number(lr, "lr", torch.float32, dev)), 0.0
        config = AdamWConfig(lr, betas[0], betas[1], eps, weight_decay, device_step, device_lr,
                             _ptr(_number(grad_scale, "grad_scale", torch.float32, dev)),
                             _int(int(step)), *self._types)
        with _on(dev):
            st = self._fn(self._table, len(self._table), ctypes.byref(config),
                          _stream(stream, dev))
        _raise(st, "moe_adamw_step")


def bind_adamw(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor], *,
               masters: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_scale: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_sq_scale: Optional[Sequence[torch.Tensor]] = None) -> BoundAdamW:
    """Check and marshal the tensors of an AdamW step once (include/moe_train.h);
    the returned object takes a step over them each time it is called.

    params: bf16, or float32 without ``masters``; grads: bf16 or float32, of the
    params' shapes, as their backward calls write them; ``masters``: float32, the
    values that are updated, their bf16 rounding goes to params.  States: float32
    (no scales), or 8-bit: float8_e4m3fn with float32 scales [ceil(n / 256)], one
    for each 256 values (``adamw_state`` makes either).  Types are the same for all
    tensors; all are contiguous and on one device, and none overlaps another."""
    lists = {"grads": grads, "exp_avg": exp_avg, "exp_avg_sq": exp_avg_sq, "masters": masters,
             "exp_avg_scale": exp_avg_scale, "exp_avg_sq_scale": exp_avg_sq_scale}
    params = list(params)
    if not params:
        raise ValueError("params is empty")
    for name, ts in lists.items():
        if ts is None:
            if name in ("grads", "exp_avg", "exp_avg_sq"):
                raise ValueError(f"{name} is needed")
            continue
        lists[name] = ts = list(ts)
        if len(ts) != len(params):
            raise ValueError(f"{name} has {len(ts)} tensors, params {len(params)}")
    first = params[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError("params are CUDA tensors")
    dev, dtype, state = first.device, first.dtype, getattr(lists["exp_avg"][0], "dtype", None)
    if dtype not in _OUT_TYPE:
        raise ValueError("params must be bfloat16 or float32")
    if masters is not None and dtype != torch.bfloat16:
        raise ValueError("masters go with bfloat16 params")
    eight = state == torch.float8_e4m3fn
    if not eight and state != torch.float32:
        raise ValueError("states are float32 or float8_e4m3fn")
    for name in ("exp_avg_scale", "exp_avg_sq_scale"):
        if eight != (lists[name] is not None):
            raise ValueError("8-bit states have exp_avg_scale and exp_avg_sq_scale, others none")
    grad_dtype = getattr(lists["grads"][0], "dtype", None)
    if grad_dtype not in _OUT_TYPE:
        raise ValueError("grads must be bfloat16 or float32")
    kept = [params] + [ts for ts in lists.values() if ts is not None]
    # the table's columns in its order: name, tensors, type, one value a block
    columns = [("params", params, dtype, False), ("masters", lists["masters"], torch.float32, False),
               ("grads", lists["grads"], grad_dtype, False),
               ("exp_avg", lists["exp_avg"], state, False),
               ("exp_avg_sq", lists["exp_avg_sq"], state, False),
               ("exp_avg_scale", lists["exp_avg_scale"], torch.float32, True),
               ("exp_avg_sq_scale", lists["exp_avg_sq_scale"], torch.float32, True)]
    table, index = (AdamWTensor * len(params))(), dev.index
    for i, p in enumerate(params):
        shape, n = p.shape, p.numel()
        blocks, row = (-(-n // BLOCK),), []
        for name, ts, t_dtype, per_block in columns:
            if ts is None:
                row.append(None)
                continue
            t, want = ts[i], blocks if per_block else shape
            if not isinstance(t, torch.Tensor) or t.get_device() != index or \
                    t.dtype is not t_dtype or t.shape != want or not t.is_contiguous():
                _check(t, f"{name}[{i}]", (t_dtype,), want, dev)    # names the problem
            row.append(t.data_ptr())
        table[i] = tuple(row) + (n,)
    return BoundAdamW(table, kept, (8 if eight else 32, _OUT_TYPE[dtype], _OUT_TYPE[grad_dtype]),
                      dev)


def adamw_state(params: Sequence[torch.Tensor], bits: int = 32, master: bool = False) -> dict:
    """The state of an AdamW run over ``params`` before its first step, as
    keyword arguments of ``bind_adamw`` and ``adamw_step``: zeros in 32 or 8
    ``bits``, and with ``master`` float32 copies of the params."""
    if bits not in (8, 32):
        raise ValueError("bits is 8 or 32")
    dtype = torch.float8_e4m3fn if bits == 8 else torch.float32

    def zeros(like):
        return torch.zeros(like.shape, dtype=torch.uint8 if bits == 8 else dtype,
                           device=like.device).view(dtype)

    res = {"exp_avg": [zeros(p) for p in params], "exp_avg_sq": [zeros(p) for p in params]}
    if master:
        res["masters"] = [p.detach().to(torch.float32, copy=True) for p in params]
    if bits == 8:
        for name in ("exp_avg_scale", "exp_avg_sq_scale"):
            res[name] = [torch.zeros(-(-p.numel() // BLOCK), device=p.device) for p in params]
    return res


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               exp_avg: Sequence[torch.Tensor], exp_avg_sq: Sequence[torch.Tensor], *, step,
               lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2,
               masters: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_scale: Optional[Sequence[torch.Tensor]] = None,
               exp_avg_sq_scale: Optional[Sequence[torch.Tensor]] = None,
               grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step over many tensors, in place: ``bind_adamw`` and one call
    of what it returns."""
    bound = bind_adamw(params, grads, exp_avg, exp_avg_sq, masters=masters,
                       exp_avg_scale=exp_avg_scale, exp_avg_sq_scale=exp_avg_sq_scale)
    bound(step=step, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
          grad_scale=grad_scale, stream=stream)
