"""Muon optimizer step on MI355X: Python binding of libmuon.so.

Thin argument marshalling over the C ABI declared in include/muon.h; every
step of the computation runs in the library's HIP kernels.  Tensors are torch
tensors on the current HIP device: fp32 params/grads/momentum, bf16 for the
Newton-Schulz entry; the gradients of the norm, clip and AdamW calls may be
bf16 or fp16 too, and the layers' products take bf16 and fp16 activations.
Calls enqueue on torch's current stream (or `stream`) and return without
synchronising.
"""
from __future__ import annotations

import ctypes

from . import _lib

__all__ = [
    "DEFAULT_COEFFS", "MuonError", "matrix_shape", "muon_step", "muon_step_noalloc", "muon_newton_schulz", "muon_adamw_step", "muon_adamw_untie",
    "muon_grad_norm", "muon_grad_clip",
    "muon_linear", "muon_linear_dx", "muon_linear_dw", "muon_dropout",
    "muon_workspace_bytes",
    "muon_set_workspace", "muon_release", "muon_plan_stats", "muon_set_lanes", "muon_timing_enable", "muon_timing_read", "muon_last_error",
    "KERNEL_MOMENTUM", "KERNEL_CAST", "KERNEL_GRAM", "KERNEL_POLY", "KERNEL_UPDATE", "KERNEL_APPLY",
    "KERNEL_ADAMW", "KERNEL_GRAD_NORM", "KERNEL_GRAD_CLIP", "KERNEL_LINEAR", "KERNEL_LINEAR_DW", "KERNEL_DROPOUT",
]

DEFAULT_COEFFS = (3.4445, -4.7750, 2.0315)
KERNEL_MOMENTUM, KERNEL_CAST, KERNEL_GRAM, KERNEL_POLY, KERNEL_UPDATE, KERNEL_APPLY, KERNEL_ADAMW = range(7)
KERNEL_GRAD_NORM, KERNEL_GRAD_CLIP = 7, 8
KERNEL_LINEAR, KERNEL_LINEAR_DW, KERNEL_DROPOUT = 9, 10, 11
GRAD_WORKSPACE_BYTES = 16640
_CODES = {-1: "MUON_EINVAL", -2: "MUON_ENOMEM", -3: "MUON_EHIP"}


class MuonError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_CODES.get(code, code)}: {msg}")
        self.code = code


def muon_last_error() -> str:
    return (_lib.load().muon_last_error() or b"").decode()


def _check(rc: int) -> None:
    if rc != 0:
        raise MuonError(rc, muon_last_error())


def _current_device():
    """torch's current GPU, or -1 where there is none (then no tensor is on it)."""
    import torch
    if torch.cuda.is_initialized() or torch.cuda.is_available():
        return torch.cuda.current_device()
    return -1


def _device_and_stream():
    """The current GPU and the handle of torch's current stream on it; -1 and 0 where there is none."""
    import torch
    if torch.cuda.is_initialized() or torch.cuda.is_available():
        dev = torch.cuda.current_device()
        handle = torch._C._cuda_getCurrentRawStream(dev)
        _refuse_per_thread(handle)  # a workspace would belong to one stream and be used on several
        return dev, handle
    return -1, 0


def _stream_handle(stream):
    if stream is None:
        import torch
        # what torch.cuda.current_stream().cuda_stream gives, 2.8 us sooner
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def matrix_shape(shape):
    """The matrix a parameter of rank >= 2 is orthogonalised as: its first
    dimension by the product of the others (for a convolution filter
    out x in x kh x kw, the out x (in kh kw) matrix of its im2col form).  A
    contiguous row-major tensor already is that matrix in memory."""
    shape = tuple(int(d) for d in shape)
    if len(shape) < 2:
        raise ValueError("rank >= 2 expected (1-D parameters belong to another optimizer)")
    cols = 1
    for d in shape[1:]:
        cols *= d
    return shape[0], cols


def _fp32_matrix(t, what):
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() < 2:
        raise ValueError(f"{what}: expected a tensor of rank >= 2 (1-D parameters belong to another optimizer)")
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous float32 tensor on the GPU")
    return t.data_ptr()


def _bf16_matrix(t, what):
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() < 2:
        raise ValueError(f"{what}: expected a tensor of rank >= 2")
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous bfloat16 tensor on the GPU")
    return t.data_ptr()


def _coeff_arg(coeffs, ns_steps):
    """(is a schedule, ctypes float array): one (a, b, c) for every iteration,
    or ns_steps triples, triple k for iteration k."""
    rows = [list(c) if hasattr(c, "__len__") else None for c in coeffs]
    if all(r is None for r in rows):
        vals = [float(c) for c in coeffs]
        if len(vals) != 3:
            raise ValueError("coeffs: expected (a, b, c) or one (a, b, c) per iteration")
        return False, _lib.float3(vals)
    if any(r is None or len(r) != 3 for r in rows) or len(rows) != ns_steps:
        raise ValueError(f"coeffs schedule: expected {ns_steps} triples (a, b, c)")
    return True, _lib.float_array([float(v) for r in rows for v in r])


def _update_ptrs(updates, params):
    if updates is None:
        return None
    updates = list(updates)
    if len(updates) != len(params):
        raise ValueError("updates must have one entry per matrix")
    ptrs = []
    for i, u in enumerate(updates):
        if u is None:
            ptrs.append(None)
            continue
        _bf16_matrix(u, f"updates[{i}]")
        if u.shape != params[i].shape:
            raise ValueError(f"updates[{i}]: shape differs from params[{i}]")
        ptrs.append(u.data_ptr())
    return _lib.ptr_array(ptrs)


def muon_step(params, grads, momentum, lr=0.02, beta=0.95, ns_steps=5, coeffs=DEFAULT_COEFFS,
              updates=None, stream=None, clip=None) -> None:
    """One Muon step over lists of fp32 tensors of rank >= 2 (params and
    momentum updated in place; rank > 2 is taken as the matrix_shape view).
    `coeffs` is one (a, b, c) or a schedule of ns_steps triples.  `updates`, if
    given, is a list of bf16 tensors (or None entries) of the params' shapes
    receiving the applied update.  `clip`, if given, is the record of
    muon_grad_norm: the step then takes the gradients clipped, and changes
    nothing when the record's norm is not finite."""
    params, grads, momentum = list(params), list(grads), list(momentum)  # this call's own, whatever becomes of the lists
    n = len(params)
    if len(grads) != n or len(momentum) != n:
        raise ValueError("params, grads and momentum must have the same length")
    shapes = []
    for i, (p, g, m) in enumerate(zip(params, grads, momentum)):
        _fp32_matrix(p, f"params[{i}]"), _fp32_matrix(g, f"grads[{i}]"), _fp32_matrix(m, f"momentum[{i}]")
        if g.shape != p.shape or m.shape != p.shape:
            raise ValueError(f"matrix {i}: shapes differ")
        shapes.append(matrix_shape(p.shape))
    lib = _lib.load()
    P = _lib.ptr_array([p.data_ptr() for p in params])
    G = _lib.ptr_array([g.data_ptr() for g in grads])
    M = _lib.ptr_array([m.data_ptr() for m in momentum])
    S = _lib.shape_array(shapes)
    sched, C = _coeff_arg(coeffs, ns_steps)
    st = ctypes.c_void_p(_stream_handle(stream))
    if clip is not None:
        record = _record_ptr(clip)
        if not sched:  # the same triple every iteration (a count out of range is the library's to refuse)
            C = _lib.float_array(list(C) * min(max(int(ns_steps), 0), 65))
        rc = lib.muon_step_clip(P, G, M, S, n, float(lr), float(beta), int(ns_steps), C, _update_ptrs(updates, params),
                                record, st)
    elif updates is None:
        if sched:
            rc = lib.muon_step_sched(P, G, M, S, n, float(lr), float(beta), int(ns_steps), C, None, st)
        else:
            rc = lib.muon_step(P, G, M, S, n, float(lr), float(beta), int(ns_steps), C, st)
    else:
        U = _update_ptrs(updates, params)
        entry = lib.muon_step_sched if sched else lib.muon_step_ex
        rc = entry(P, G, M, S, n, float(lr), float(beta), int(ns_steps), C, U, st)
    _check(rc)


def muon_step_noalloc(params, grads, momentum, lr=0.02, beta=0.95, ns_steps=5, coeffs=DEFAULT_COEFFS,
                      stream=None) -> None:
    """muon_step for callers that cannot allocate device memory: workspace and
    tables in the library's static scratch array (MUON_NOALLOC_SCRATCH_BYTES
    per device); one fixed (a, b, c) triple."""
    n = len(params)
    if len(grads) != n or len(momentum) != n:
        raise ValueError("params, grads and momentum must have the same length")
    shapes = []
    for i, (p, g, m) in enumerate(zip(params, grads, momentum)):
        _fp32_matrix(p, f"params[{i}]"), _fp32_matrix(g, f"grads[{i}]"), _fp32_matrix(m, f"momentum[{i}]")
        if g.shape != p.shape or m.shape != p.shape:
            raise ValueError(f"matrix {i}: shapes differ")
        shapes.append(matrix_shape(p.shape))
    sched, C = _coeff_arg(coeffs, ns_steps)
    if sched:
        raise ValueError("muon_step_noalloc takes one (a, b, c) triple")
    rc = _lib.load().muon_step_noalloc(_lib.ptr_array([p.data_ptr() for p in params]),
                                       _lib.ptr_array([g.data_ptr() for g in grads]),
                                       _lib.ptr_array([m.data_ptr() for m in momentum]), _lib.shape_array(shapes), n,
                                       float(lr), float(beta), int(ns_steps), C,
                                       ctypes.c_void_p(_stream_handle(stream)))
    _check(rc)


def muon_newton_schulz(xs, outs, ns_steps=5, coeffs=DEFAULT_COEFFS, stream=None) -> None:
    """The Newton-Schulz core alone on bf16 matrices (no normalisation);
    `coeffs` is one (a, b, c) or a schedule of ns_steps triples."""
    n = len(xs)
    if len(outs) != n:
        raise ValueError("xs and outs must have the same length")
    shapes = []
    for i, (x, o) in enumerate(zip(xs, outs)):
        _bf16_matrix(x, f"xs[{i}]"), _bf16_matrix(o, f"outs[{i}]")
        if x.shape != o.shape:
            raise ValueError(f"matrix {i}: shapes differ")
        shapes.append(matrix_shape(x.shape))
    lib = _lib.load()
    sched, C = _coeff_arg(coeffs, ns_steps)
    entry = lib.muon_newton_schulz_sched if sched else lib.muon_newton_schulz
    rc = entry(_lib.ptr_array([x.data_ptr() for x in xs]), _lib.ptr_array([o.data_ptr() for o in outs]),
               _lib.shape_array(shapes), n, int(ns_steps), C, ctypes.c_void_p(_stream_handle(stream)))
    _check(rc)


def _fp32_flat(t, what, i=None):
    import torch
    if isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    # put together for a refusal alone: names of every tensor were 49 of 337 us of a call on 148 tensors
    where = what if i is None else f"{what}[{i}]"
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: expected a tensor")
    raise ValueError(f"{where}: expected a contiguous float32 tensor on the GPU")


def _any_16_bit(ts):
    import torch
    halves = (torch.bfloat16, torch.float16)
    return any(getattr(t, "dtype", None) in halves for t in ts)


def _as_list(ts):
    return ts if isinstance(ts, (list, tuple)) else list(ts)


def _record_ptr(record):
    import torch
    if (not isinstance(record, torch.Tensor) or record.dtype != torch.float32 or record.numel() != 2
            or not record.is_contiguous() or record.get_device() != torch.cuda.current_device()):
        raise ValueError("record: expected the contiguous float32 tensor of 2 of muon_grad_norm, on the current GPU")
    return record.data_ptr()


def _refuse_per_thread(handle):
    if handle == 2:
        raise ValueError("stream: hipStreamPerThread is another stream in every host thread; pass a stream of your own")


def _on_stream(stream):
    """A context in which `stream` is torch's current one, so that what a call
    allocates belongs to the stream that uses it."""
    import torch
    if isinstance(stream, int):
        _refuse_per_thread(stream)
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


# One norm workspace per device and stream of torch's own: calls on one stream
# are ordered, so each finds it as the one before left it; calls on two
# streams share none.  torch's streams are never destroyed, so these handles
# never come to name another stream, and they are few.
_norm_workspaces = {}


def _norm_workspace(dev, handle):
    """The workspace of a norm on torch's current stream.  A captured call
    takes one of its own from the graph's memory, cleared by the graph, so
    that graphs share none either; so does a call on a stream that is not
    torch's own, whose handle may name another stream by the next call."""
    import torch
    _refuse_per_thread(handle)
    if dev < 0:
        return torch.empty(0)
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(GRAD_WORKSPACE_BYTES // 8, dtype=torch.float64, device=dev)
    ws = _norm_workspaces.get((dev, handle))
    if ws is None:
        ws = torch.zeros(GRAD_WORKSPACE_BYTES // 8, dtype=torch.float64, device=dev)
        # the id of a stream that torch did not make is its handle
        if handle == 0 or torch.cuda.current_stream(dev).stream_id != handle:
            _norm_workspaces[dev, handle] = ws
    return ws


def muon_adamw_step(params, grads, exp_avg, exp_avg_sq, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                    step=1, stream=None, clip=None) -> None:
    """One AdamW step over tensors of any shape (each contiguous fp32, taken
    flat; the gradients may be bf16 or fp16); exp_avg and exp_avg_sq start at
    zero and `step` counts from 1.  `weight_decay` is one value or one per
    tensor.  `clip`, if given, is the record of muon_grad_norm: the step then
    takes the gradients clipped, and changes nothing when the record's norm is
    not finite."""
    n = len(params)
    if not (len(grads) == len(exp_avg) == len(exp_avg_sq) == n):
        raise ValueError("params, grads, exp_avg and exp_avg_sq must have the same length")
    if clip is not None or _any_16_bit(grads):
        dev = _current_device()
        wd = weight_decay if not hasattr(weight_decay, "__len__") else _as_list(weight_decay)
        b1, b2 = betas
        _check(_lib.load_tensor_calls().adamw_clip(
            _as_list(params), _as_list(grads), _as_list(exp_avg), _as_list(exp_avg_sq), wd, float(lr), float(b1),
            float(b2), float(eps), int(step), clip, dev, _stream_handle(stream) if dev >= 0 else 0))
        return
    if hasattr(weight_decay, "__len__"):
        wds = [float(w) for w in weight_decay]
        if len(wds) != n:
            raise ValueError("weight_decay: expected one value or one per tensor")
    else:
        wds = [float(weight_decay)] * n
    ptrs = ([], [], [], [])
    numels = []
    for i in range(n):
        ts = (params[i], grads[i], exp_avg[i], exp_avg_sq[i])
        names = ("params", "grads", "exp_avg", "exp_avg_sq")
        for k, (t, name) in enumerate(zip(ts, names)):
            ptrs[k].append(_fp32_flat(t, name, i))
        if len({t.numel() for t in ts}) != 1:
            raise ValueError(f"tensor {i}: element counts differ")
        numels.append(params[i].numel())
    b1, b2 = betas
    rc = _lib.load().muon_adamw_step(*(_lib.ptr_array(p) for p in ptrs), _lib.int64_array(numels),
                                     _lib.float_array(wds), n, float(lr), float(b1), float(b2), float(eps),
                                     int(step), ctypes.c_void_p(_stream_handle(stream)))
    _check(rc)


def muon_grad_norm(grads, max_norm=float("inf"), scale=1.0, record=None, stream=None):
    """The global norm of a list of gradients and the factor that clips it:
    a float32 tensor {norm, factor} on the GPU with
        norm = scale * sqrt(sum of g^2),  factor = scale * min(1, max_norm / (norm + 1e-6)).
    Gradients are float32, bfloat16 or float16, mixed as needed, each dense in
    memory (any order of dimensions).  `scale` is 1 / micro-batches under
    gradient accumulation, 1 / loss scale under loss scaling.  Pass the result
    as `clip` to muon_step and muon_adamw_step, which then take the gradients
    clipped without a pass that writes them back.  `record` is a tensor of 2
    to fill instead of a new one.  `stream`, if not torch's current one, is a
    torch stream or a raw handle, of a stream that lives until the call's work
    is done; hipStreamPerThread is refused."""
    if stream is not None:
        with _on_stream(stream):
            return muon_grad_norm(grads, max_norm, scale, record)
    dev = _current_device()
    handle = _stream_handle(None) if dev >= 0 else 0
    ws = _norm_workspace(dev, handle)
    rc, record = _lib.load_tensor_calls().grad_norm(_as_list(grads), max_norm, scale, record, ws.data_ptr(), dev, handle)
    _check(rc)
    return record


def muon_grad_clip(grads, max_norm, scale=1.0, outs=None, record=None, stream=None):
    """Clip a list of gradients by their global norm: every gradient times the
    factor of muon_grad_norm, in place, or rounded into `outs`, tensors of the
    same shapes and memory order and of any of the three types (16-bit
    gradients into float32 ones, say).  Returns the record {norm, factor};
    the norm is the one before clipping.  Autograd takes what is written as
    changed.  `stream` as in muon_grad_norm."""
    if stream is not None:
        with _on_stream(stream):
            return muon_grad_clip(grads, max_norm, scale, outs, record)
    dev = _current_device()
    handle = _stream_handle(None) if dev >= 0 else 0
    ws = _norm_workspace(dev, handle)
    rc, record = _lib.load_tensor_calls().grad_clip(_as_list(grads), None if outs is None else _as_list(outs), max_norm,
                                                    scale, record, ws.data_ptr(), dev, handle)
    _check(rc)
    return record


_ACTS = {None: 0, "gelu": 1, "relu": 2, "relu2": 3}


def _act_code(act):
    try:
        return _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act: {act!r} is none of None, 'gelu', 'relu', 'relu2'") from None


def _dtype_code(dtype):
    if dtype is None:
        return -1
    import torch
    codes = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    if dtype not in codes:
        raise ValueError(f"out_dtype: expected float32, bfloat16 or float16, not {dtype}")
    return codes[dtype]


def muon_linear(x, w, bias=None, act=None, dropout=0.0, rng=None, site=0, residual=None, out=None, out_dtype=None,
                preact=None, stream=None):
    """A layer's forward product: residual + drop(act(x w + bias)).

    `x` is bfloat16 or float16, (..., inputs); `w` is inputs x outputs in either
    memory order (the transposed view of an outputs x inputs weight is one),
    of x's type or float32 (rounded to x's type).  `act` is None, 'gelu' (the
    tanh form), 'relu' or 'relu2' (its square).  With `dropout` > 0, `rng` is
    (seed, step), or an int64 tensor of the two on the GPU, read when the call
    runs (under a captured graph: at every replay); `site` tells the dropouts of
    a model apart.  The mask is never stored: the same dropout, rng and site in
    muon_linear_dx or muon_dropout, on a matrix as wide, make it again.  It goes by
    the row within the call: micro-batches and ranks need a step or seed of their own.
    `residual` and the result are of x's type or float32 (`out_dtype`; by default the
    residual's type, or x's); `out` is a tensor to fill, and may be the residual.
    `preact`, of x's type, receives x w + bias for the backward pass.  Rows may
    lie apart in memory and start anywhere; the fastest kernels take rows
    that are 16-byte aligned and multiples of 8 elements long, and large products copy
    others (and float32 weights) first.  `stream` as in muon_grad_norm.  No autograd graph is
    recorded, whatever requires a gradient: muon_linear_dx, muon_linear_dw and muon_dropout are the
    backward pass."""
    return _linear(x, w, bias, act, dropout, rng, site, residual, out, out_dtype, preact, 0, stream)


def muon_linear_dx(dz, w, act=None, preact=None, dropout=0.0, rng=None, site=0, residual=None, out=None,
                   out_dtype=None, stream=None):
    """The gradient of a layer's input from that of its z = x w + bias:
    residual + drop(dz w^T) act'(preact).

    `act` and `preact` (both or neither), `dropout`, `rng` and `site` are those of the
    layer whose output x is, so that the result is the gradient of that layer's z;
    `residual` is a gradient that reaches x another way.  Types, memory
    orders, `out` (which may be the residual or preact) and `stream` as in muon_linear.
    No autograd graph is recorded."""
    return _linear(dz, w, None, act, dropout, rng, site, residual, out, out_dtype, preact, 1, stream)


def _linear(x, w, bias, act, dropout, rng, site, residual, out, out_dtype, preact, backward, stream):
    if stream is not None:
        with _on_stream(stream):
            return _linear(x, w, bias, act, dropout, rng, site, residual, out, out_dtype, preact, backward, None)
    rc, y = _lib.load_tensor_calls().linear(x, w, bias, _act_code(act), dropout, rng, site, residual, out,
                                            _dtype_code(out_dtype), preact, backward, *_device_and_stream())
    _check(rc)
    return y


def muon_linear_dw(x, dz, dw, dbias=None, accumulate=False, stream=None) -> None:
    """The gradients of a layer's weight and bias: dw = x^T dz and dbias = the sums of
    dz over its rows, or both added to what the tensors hold (`accumulate`: the
    micro-batches of a step).  `x` and `dz` are bfloat16 or float16, (..., inputs) and
    (..., outputs); `dw` is float32, inputs x outputs in either memory order,
    as muon_step reads it, and `dbias` float32, as muon_adamw_step does.  No autograd
    graph is recorded; autograd takes what is written as changed.  `stream` as in muon_grad_norm."""
    if stream is not None:
        with _on_stream(stream):
            return muon_linear_dw(x, dz, dw, dbias, accumulate)
    _check(_lib.load_tensor_calls().linear_dw(x, dz, dw, dbias, accumulate, *_device_and_stream()))


def muon_dropout(x, p, rng, site=0, act=None, preact=None, residual=None, out=None, out_dtype=None, stream=None):
    """residual + drop(x) act'(preact), elementwise: dropout of any tensor, its
    gradient (the same call on the gradient), or with `act` and `preact` the gradient dz of a
    layer's z behind activation and dropout.  float32, bfloat16 or float16; the
    mask goes by the last dimension and the rows before it, as in muon_linear.
    `out` may be x, preact or residual.  No autograd graph is recorded.  `stream` as in
    muon_grad_norm."""
    if stream is not None:
        with _on_stream(stream):
            return muon_dropout(x, p, rng, site, act, preact, residual, out, out_dtype)
    rc, y = _lib.load_tensor_calls().dropout(x, p, rng, site, _act_code(act), preact, residual, out,
                                             _dtype_code(out_dtype), *_device_and_stream())
    _check(rc)
    return y


def muon_adamw_untie(param, exp_avg, exp_avg_sq, transpose=False, stream=None):
    """Delayed untying: new (param, exp_avg, exp_avg_sq) tensors copied from
    a shared 2-D parameter and its AdamW moments, transposed if asked, so the
    untied parameter continues from the shared point.  Returns the three new
    tensors (allocated here, filled by the library on the stream)."""
    import torch
    for t, name in ((param, "param"), (exp_avg, "exp_avg"), (exp_avg_sq, "exp_avg_sq")):
        _fp32_flat(t, name)
        if t.dim() != 2 or t.shape != param.shape:
            raise ValueError(f"{name}: expected a 2-D tensor of the parameter's shape")
    rows, cols = param.shape
    shape = (cols, rows) if transpose else (rows, cols)
    out = [torch.empty(shape, dtype=torch.float32, device=param.device) for _ in range(3)]
    rc = _lib.load().muon_adamw_untie(param.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(),
                                      out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), rows, cols,
                                      1 if transpose else 0, ctypes.c_void_p(_stream_handle(stream)))
    _check(rc)
    return tuple(out)


def muon_workspace_bytes(shapes) -> int:
    lib = _lib.load()
    b = lib.muon_workspace_bytes(_lib.shape_array(shapes), len(shapes))
    if b == 0 and len(shapes) > 0:
        raise MuonError(-1, muon_last_error())
    return int(b)


def muon_set_workspace(ptr: int | None, nbytes: int = 0) -> None:
    _check(_lib.load().muon_set_workspace(ctypes.c_void_p(ptr or 0), int(nbytes)))


def muon_release() -> None:
    _lib.load().muon_release()
    _norm_workspaces.clear()


PLAN_STATS = ("plan_builds", "uploads", "pointer_patches", "device_syncs", "evictions", "workspace_allocs")


def muon_plan_stats() -> dict:
    """Counters of the current device's plan cache (diagnostics)."""
    arr = (ctypes.c_int64 * 6)()
    _check(_lib.load().muon_plan_stats(arr))
    return dict(zip(PLAN_STATS, (int(v) for v in arr)))


def muon_set_lanes(lanes: int) -> None:
    """Concurrency of a call: up to `lanes` shape groups run at once on the
    library's internal streams (1 = everything on the caller's stream)."""
    _check(_lib.load().muon_set_lanes(int(lanes)))


def muon_timing_enable(kernel: int) -> None:
    _check(_lib.load().muon_timing_enable(int(kernel)))


def muon_timing_read():
    """(total milliseconds, number of launches) of the timed kernel family since the last read."""
    ms = ctypes.c_double()
    cnt = ctypes.c_int64()
    _check(_lib.load().muon_timing_read(ctypes.byref(ms), ctypes.byref(cnt)))
    return ms.value, cnt.value
