"""One AdamW step over many tensors at once, moments in 8 bits or in 32.

Binding of ``include/lowbit_adamw.h``; argument marshalling only:

  adamw_state(params, bits=8, master=False) -> state    zero moments (and an fp32 copy)
  adamw(params, grads, state, lr, betas, eps, weight_decay, step, rounding=)    one step, in place
  adamw_moments(state) -> m, v                          the moments as fp32 values

The moments of all tensors lie in one buffer each, in blocks of 256 values; every tensor
begins with a block.
"""
from __future__ import annotations

import ctypes
from array import array
from itertools import chain

import numpy as np

from . import LowbitError, load_library as _load_library
from .w8a8 import _check_tensor, _run, _torch

ADAMW_BLOCK = 256
ADAMW_RANDOM = 256
F16, BF16, F32 = 0, 1, 3

EXPORTED_ADAMW = ("lowbit_adamw", "lowbit_adamw_moments")


class AdamwState(ctypes.Structure):
    _fields_ = [("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("m_max", ctypes.c_void_p),
                ("v_max", ctypes.c_void_p), ("master", ctypes.c_void_p)]


class AdamwOptions(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("lr_or_null", ctypes.c_void_p),
                ("step_or_null", ctypes.c_void_p), ("grad_scale_or_null", ctypes.c_void_p)]


_declared = None


def _lib() -> ctypes.CDLL:
    global _declared
    lib = _load_library()
    if _declared is lib:
        return lib
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.lowbit_adamw.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp]
    lib.lowbit_adamw_moments.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp]
    lib.lowbit_adamw.restype = lib.lowbit_adamw_moments.restype = i32
    _declared = lib
    return lib


# ---------------------------------------------------------------------------
# raw entry points (addresses as ints; the caller owns every buffer)
# ---------------------------------------------------------------------------
def adamw_raw(tensors, count, param_dtype, grad_dtype, bits, state, options, stream) -> int:
    """``tensors``: the host address of ``count`` triples of 64-bit words (param, grad, n);
    ``state`` and ``options``: AdamwState and AdamwOptions, or None."""
    return _lib().lowbit_adamw(tensors, count, param_dtype, grad_dtype, bits,
                               None if state is None else ctypes.byref(state),
                               None if options is None else ctypes.byref(options), stream)


def adamw_moments_raw(m, v, m_max, v_max, blocks, m_out, v_out, stream) -> int:
    return _lib().lowbit_adamw_moments(m, v, m_max, v_max, blocks, m_out, v_out, stream)


# ---------------------------------------------------------------------------
# tensor front end
# ---------------------------------------------------------------------------
def _type_of(dtype, name: str) -> int:
    torch = _torch()
    kinds = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
    if dtype not in kinds:
        raise TypeError(f"{name} must be torch.float32, torch.float16 or torch.bfloat16, got {dtype}")
    return kinds[dtype]


def _blocks(params) -> int:
    return sum(-(-p.numel() // ADAMW_BLOCK) for p in params)


def adamw_state(params, bits: int = 8, master: bool = False) -> dict:
    """Moments of zero for ``params``, tensors of one type on one GPU: a dict with ``m`` and
    ``v`` (uint8, or fp32 with ``bits=32``, 256 values for each block), for 8 bits ``m_max`` and
    ``v_max`` (fp32, one for each block), and with ``master`` the parameters in fp32."""
    torch = _torch()
    params = list(params)
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    if not params:
        raise ValueError("params must not be empty")
    dev = params[0].device
    _list_type(params, "params", dev)
    blocks = _blocks(params)
    n = blocks * ADAMW_BLOCK
    kind = torch.uint8 if bits == 8 else torch.float32
    state = {"m": torch.zeros(n, dtype=kind, device=dev), "v": torch.zeros(n, dtype=kind, device=dev)}
    if bits == 8:
        state["m_max"] = torch.zeros(blocks, dtype=torch.float32, device=dev)
        state["v_max"] = torch.zeros(blocks, dtype=torch.float32, device=dev)
    if master:
        copy = torch.zeros(n, dtype=torch.float32, device=dev)
        at = 0
        for p in params:
            copy[at:at + p.numel()] = p.detach().reshape(-1)
            at += -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
        state["master"] = copy
    return state


def _list_type(tensors, name: str, device) -> int:
    """The type of a list of dense tensors on ``device``, checked.  A model's adapters are
    hundreds of tensors: each is asked by a call that needs no Python frame."""
    Tensor = _torch().Tensor
    try:
        fine = (tensors[0].is_cuda and set(map(Tensor.get_device, tensors)) == {device.index}
                and all(map(Tensor.is_contiguous, tensors))
                and len(set(map(Tensor.dtype.__get__, tensors))) == 1)
    except (AttributeError, TypeError):
        raise TypeError(f"{name} must be torch.Tensors") from None
    if fine:
        return _type_of(tensors[0].dtype, name)
    dtype = tensors[0].dtype
    if not tensors[0].is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    for i, t in enumerate(tensors):
        if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != device.index:
            raise ValueError(f"{name}[{i}] must be contiguous, {dtype} and on {device}, as {name}[0] is; "
                             f"got {t.dtype} on {t.device}")


def _refuse_shared(params, grads, state: dict, scalars) -> None:
    """Names what shares memory with something that a step writes."""
    torch = _torch()
    written = [(f"params[{i}]", p) for i, p in enumerate(params)]
    names = ("m", "v", "m_max", "v_max", "master") if state["m"].dtype is torch.uint8 else ("m", "v", "master")
    written += [(name, state[name]) for name in names if state.get(name) is not None]
    read = [(f"grads[{i}]", g) for i, g in enumerate(grads)]
    read += [(name, t) for name, t in zip(("lr", "step", "grad_scale"), scalars) if isinstance(t, torch.Tensor)]
    pieces = sorted((t.data_ptr(), t.data_ptr() + t.nbytes, name, i < len(written))
                    for i, (name, t) in enumerate(written + read) if t.nbytes)
    ends = {True: (0, ""), False: (0, "")}  # of the pieces so far that are written, and are read: the last end
    for lo, hi, name, write in pieces:
        for other in (True, False) if write else (True,):
            if ends[other][0] > lo:
                raise ValueError(f"{ends[other][1]} and {name} must not share memory: a step writes to one of them")
        ends[write] = max(ends[write], (hi, name))


def adamw(params, grads, state: dict, lr, betas=(0.9, 0.999), eps: float = 1e-8,
          weight_decay: float = 0.01, step=1, grad_scale=None, rounding: str = "nearest") -> None:
    """One AdamW step, in place: ``params`` (tensors of one type: fp32, fp16 or bf16) and
    ``state`` (of ``adamw_state``) from ``grads`` (tensors of one type, one for each parameter).
    A gradient has as many values as its parameter, and they pair up in the order of memory: a flat or
    reshaped gradient is fine, and a transposed one, which has the values in another order, is not told
    from it (comparing the shapes of 448 pairs takes 34 us more).
    ``step`` counts from 1.  ``lr`` (fp32) and ``step`` (int32) may be GPU tensors of one
    element, read when the step runs, and ``grad_scale`` is one (fp32) that multiplies the gradients:
    a captured step follows them.  A grad_scale of infinity or NaN leaves everything as it was.
    ``rounding`` of 8-bit moments: "nearest", or "random", up or down by a number made of the
    step and the place, so that the same calls still give the same bits.  To the nearest code a second
    moment cannot follow gradients that change against the rest of their block (72 times too large
    after 7000 steps at a tenth of the gradient); rounded at random it follows in the mean.  Train
    with "random" or with 32 bits unless blocks' gradients keep their proportions.
    What a step writes shares memory with nothing else of the call; gradients may with each other."""
    torch = _torch()
    if rounding not in ("nearest", "random"):
        raise ValueError(f"rounding must be 'nearest' or 'random', got {rounding!r}")
    params, grads = list(params), list(grads)
    count = len(params)
    if count != len(grads):
        raise ValueError(f"params and grads must be as many, got {count} and {len(grads)}")
    if not params:
        return
    Tensor = torch.Tensor
    dev = getattr(params[0], "device", None)
    p_kind = _list_type(params, "params", dev)
    g_kind = _list_type(grads, "grads", dev)
    columns = (map(Tensor.data_ptr, params), map(Tensor.data_ptr, grads), map(Tensor.numel, params))
    if count < 64:  # a few tensors: 4 us less without numpy, hundreds: 24 us more
        sizes = [p.numel() for p in params]
        same = sizes == [g.numel() for g in grads]
        blocks = sum(-(-n // ADAMW_BLOCK) for n in sizes)
        table = array("q", chain.from_iterable(zip(*columns)))
        at = table.buffer_info()[0]
    else:
        table = np.empty((count, 3), np.int64)
        for i, values in enumerate(columns):
            table[:, i] = np.fromiter(values, np.int64, count)
        sizes = table[:, 2]
        same = (sizes == np.fromiter(map(Tensor.numel, grads), np.int64, count)).all()
        blocks = int((sizes + (ADAMW_BLOCK - 1) >> 8).sum())
        at = table.ctypes.data
    if not same:
        raise ValueError("each gradient must have its parameter's size")
    n = blocks * ADAMW_BLOCK
    m = state["m"]
    if m.dtype is torch.uint8:
        bits = 8
        _check_tensor(state["m_max"], "m_max", torch.float32, dev, (blocks,))
        _check_tensor(state["v_max"], "v_max", torch.float32, dev, (blocks,))
        tops = (state["m_max"].data_ptr(), state["v_max"].data_ptr())
    else:
        bits = 32
        tops = (None, None)
        if rounding != "nearest":
            raise ValueError("32-bit moments are not rounded: rounding must be 'nearest'")
    kind = torch.uint8 if bits == 8 else torch.float32
    _check_tensor(m, "m", kind, dev, (n,))
    _check_tensor(state["v"], "v", kind, dev, (n,))
    master = state.get("master")
    if master is not None:
        _check_tensor(master, "master", torch.float32, dev, (n,))

    def scalar(t, name, dtype):
        _check_tensor(t, name, dtype, dev, tuple(t.shape))
        if t.numel() != 1:
            raise ValueError(f"{name} must have one element")
        return t.data_ptr()

    lr_at = scalar(lr, "lr", torch.float32) if isinstance(lr, torch.Tensor) else None
    step_at = scalar(step, "step", torch.int32) if isinstance(step, torch.Tensor) else None
    scale_at = None if grad_scale is None else scalar(grad_scale, "grad_scale", torch.float32)
    options = AdamwOptions(0.0 if lr_at else lr, betas[0], betas[1], eps, weight_decay,
                           1 if step_at else step, lr_at, step_at, scale_at)
    place = AdamwState(m.data_ptr(), state["v"].data_ptr(), *tops,
                       None if master is None else master.data_ptr())
    _lib()
    try:
        _run("lowbit_adamw", None, (at, count, p_kind, g_kind,
                                    bits | ADAMW_RANDOM if rounding == "random" else bits,
                                    ctypes.addressof(place), ctypes.addressof(options)), dev)
    except LowbitError:
        _refuse_shared(params, grads, state, (lr, step, grad_scale))
        raise
    torch.autograd.graph.increment_version(params)


def adamw_moments(state: dict):
    """(m, v), the moments of a state as fp32 values, 256 for each block: of 8-bit ones what
    the codes stand for, in new tensors; 32-bit ones are the state's own buffers, and what is
    written into them is written into the state."""
    torch = _torch()
    m, v = state["m"], state["v"]
    if m.dtype is torch.float32:
        return m, v
    _check_tensor(m, "m", torch.uint8, None, tuple(m.shape))
    dev = m.device
    blocks = m.numel() // ADAMW_BLOCK
    _check_tensor(m, "m", torch.uint8, dev, (blocks * ADAMW_BLOCK,))
    _check_tensor(v, "v", torch.uint8, dev, (blocks * ADAMW_BLOCK,))
    _check_tensor(state["m_max"], "m_max", torch.float32, dev, (blocks,))
    _check_tensor(state["v_max"], "v_max", torch.float32, dev, (blocks,))
    m_out = torch.empty(m.shape, dtype=torch.float32, device=dev)
    v_out = torch.empty_like(m_out)
    _lib()
    _run("lowbit_adamw_moments", None,
         (m.data_ptr(), v.data_ptr(), state["m_max"].data_ptr(), state["v_max"].data_ptr(), blocks,
          m_out.data_ptr(), v_out.data_ptr()), dev)
    return m_out, v_out
