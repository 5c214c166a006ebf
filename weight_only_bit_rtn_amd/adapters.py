"""Low-rank adapters of many requests beside a shared projection, and their gradients.

Binding of ``include/lowbit_lora.h``; argument marshalling only.  Adapters lie in
pools a[L][R][K] and b[L][N][R] with a scale for each; every token goes through one
adapter or none:

  lora_plan(ids, L) -> plan                            the batch's tokens sorted by adapter
  lora(x, a, b, scales, plan, y) -> out                y + s_l b_l (a_l x)
  lora_grad(dy, x, v, a, b, scales, plan, dx) -> dx, da, db

y is the output of ``qgemv``, ``qgemm`` or ``linear_w8a8`` on the same x.  One plan holds
for every layer that the batch passes.  The calls are outside autograd, as those of
``include/lowbit_w8a8.h`` are.
"""
from __future__ import annotations

import ctypes

from . import _check, load_library as _load_library
from .w8a8 import _apart, _check_tensor, _float_type, _out, _stream_handle, _torch

LORA_MAX_R = 128
LORA_MAX_L = 1024
LORA_MIN_N = 8

EXPORTED_LORA = ("lowbit_lora_plan", "lowbit_lora_workspace_bytes", "lowbit_lora",
                 "lowbit_lora_grad_workspace_bytes", "lowbit_lora_grad")

_declared = None
_entry = {}  # name: (entry point, its workspace size)


def _lib() -> ctypes.CDLL:
    global _declared
    lib = _load_library()
    if _declared is lib:
        return lib
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.lowbit_lora_plan.argtypes = [vp, i64, i64, vp, vp, vp]
    lib.lowbit_lora_workspace_bytes.argtypes = [i64] * 5
    lib.lowbit_lora.argtypes = [vp, i32, i64, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp,
                                vp, i64, vp]
    lib.lowbit_lora_grad_workspace_bytes.argtypes = [i64] * 5
    lib.lowbit_lora_grad.argtypes = [vp, vp, vp, i32, i64, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                     vp, vp, vp, vp, vp, i64, vp]
    for name in EXPORTED_LORA:
        getattr(lib, name).restype = i64 if name.endswith("_bytes") else i32
    # at once: another thread's first call sees all of them or none
    _entry.update({name: (getattr(lib, name), getattr(lib, name + "_workspace_bytes", None))
                   for name in ("lowbit_lora_plan", "lowbit_lora", "lowbit_lora_grad")})
    _declared = lib
    return lib


# ---------------------------------------------------------------------------
# raw entry points (device pointers as ints; the caller owns every buffer)
# ---------------------------------------------------------------------------
def lora_plan_raw(ids, T, L, order, starts, stream) -> int:
    return _lib().lowbit_lora_plan(ids, T, L, order, starts, stream)


def lora_workspace_bytes(T: int, N: int, K: int, R: int, L: int) -> int:
    return _lib().lowbit_lora_workspace_bytes(T, N, K, R, L)


def lora_raw(x, dtype, T, order, starts, a, b, scales, L, R, N, K, y, out, v, workspace,
             workspace_bytes, stream) -> int:
    return _lib().lowbit_lora(x, dtype, T, order, starts, a, b, scales, L, R, N, K, y, out, v,
                              workspace, workspace_bytes, stream)


def lora_grad_workspace_bytes(T: int, N: int, K: int, R: int, L: int) -> int:
    return _lib().lowbit_lora_grad_workspace_bytes(T, N, K, R, L)


def lora_grad_raw(dy, x, v, dtype, T, order, starts, a, b, scales, L, R, N, K, base, dx, da, db,
                  workspace, workspace_bytes, stream) -> int:
    return _lib().lowbit_lora_grad(dy, x, v, dtype, T, order, starts, a, b, scales, L, R, N, K,
                                   base, dx, da, db, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------
# tensor front end
# ---------------------------------------------------------------------------
def lora_plan(ids, L: int, out: dict | None = None) -> dict:
    """The plan of a batch whose token t goes through adapter ``ids[t]`` (int32; an id
    outside [0, L): none) of ``L``: a dict with ``order`` (int32 [T], the tokens sorted by
    adapter, those without one last) and ``starts`` (int32 [L + 1], where an adapter's tokens
    begin in it).  ``out``: such a dict to write into."""
    torch = _torch()
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch.Tensor")
    if ids.dim() != 1:
        raise ValueError("ids must have 1 dimension")
    T, dev = ids.shape[0], ids.device
    _check_tensor(ids, "ids", torch.int32, None, (T,))
    if out is None:
        order = torch.empty_like(ids)
        starts = torch.empty(L + 1, dtype=torch.int32, device=dev)
    else:
        order = _out(out.get("order"), "order", (T,), torch.int32, dev)
        starts = _out(out.get("starts"), "starts", (L + 1,), torch.int32, dev)
        _apart(order, "order", ids, starts)
        _apart(starts, "starts", ids)
    _call("lowbit_lora_plan", None, (ids.data_ptr(), T, L, order.data_ptr(), starts.data_ptr()), dev)
    if out is not None:
        torch.autograd.graph.increment_version((order, starts))
    return {"order": order, "starts": starts}


def _fine(device, *tensors) -> None:
    """Checks (tensor, name, type, shape) one after the other: dense GPU tensors on ``device`` whose
    gradients nobody waits for.  Decoding takes some microseconds, so a call's tensors are looked at in
    one loop, and spelled out by ``_check_tensor`` only when one is wrong."""
    index = device.index
    recorded = _torch().is_grad_enabled()
    for t, name, dtype, shape in tensors:
        try:
            if (t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()
                    and not (recorded and t.requires_grad)):
                continue
        except AttributeError:
            pass
        _check_tensor(t, name, dtype, device, shape)


def _sizes(x, a, b):
    """T, N, K, R, L from the tensors' shapes."""
    try:
        (T, K), (L, R, _), (_, N, _) = x.shape, a.shape, b.shape
        return T, N, K, R, L
    except (AttributeError, ValueError):
        torch = _torch()
        if not all(isinstance(t, torch.Tensor) for t in (x, a, b)):
            raise TypeError("x, a and b must be torch.Tensors") from None
        raise ValueError("x must have 2 dimensions, a and b 3") from None


def _call(name: str, sizes, args, device) -> None:
    """Calls an entry point on ``args``, its workspace (for ``sizes``; None: it takes none) and the
    current stream of the tensors' device, which it makes the current one."""
    torch = _torch()
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, sizes, args, device)
    if not _entry:
        _lib()
    call, need_of = _entry[name]
    if sizes is None:  # no workspace
        return _check(call(*args, _stream_handle(device)), name)
    need = need_of(*sizes)
    if need > 0:
        # torch's caching allocator hands out blocks aligned to 512 bytes
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        at = workspace.data_ptr()
    else:
        _check(need, name + "_workspace_bytes")
        at = None
    status = call(*args, at, need, _stream_handle(device))
    if status:
        _check(status, name)


def lora(x, a, b, scales, plan, y=None, out=None, save: bool = False):
    """out[T][N] = y + s_l b_l (a_l x), each token through the adapter l that the plan
    (of ``lora_plan``) names; a token without one keeps y.  ``x`` [T][K], ``y`` [T][N] and the
    pools ``a`` [L][R][K] and ``b`` [L][N][R] are all fp16 or all bf16, ``scales`` fp32 [L].
    Without ``y`` the adapters' part alone.  ``out``: a tensor to write into, y itself
    allowed.  ``save``: (out, v), v = a_l x in fp32 [T][R], which ``lora_grad`` takes."""
    torch = _torch()
    kind = _float_type(x, "x")
    T, N, K, R, L = _sizes(x, a, b)
    dtype, dev = x.dtype, x.device
    order, starts = plan["order"], plan["starts"]
    if not x.is_cuda:
        raise ValueError("x must live on the GPU")
    _fine(dev, (x, "x", dtype, (T, K)), (a, "a", dtype, (L, R, K)), (b, "b", dtype, (L, N, R)),
          (scales, "scales", torch.float32, (L,)), (order, "order", torch.int32, (T,)),
          (starts, "starts", torch.int32, (L + 1,)))
    if y is not None:
        _fine(dev, (y, "y", dtype, (T, N)))
    if out is None:
        o = torch.empty((T, N), dtype=dtype, device=dev) if y is None else torch.empty_like(y)
    else:
        o = _out(out, "out", (T, N), dtype, dev)
        inputs = (x, a, b, scales, order, starts)
        if y is not None and y.data_ptr() != o.data_ptr():
            inputs += (y,)
        _apart(o, "out", *inputs)
    v = torch.empty((T, R), dtype=torch.float32, device=dev) if save else None
    _call("lowbit_lora", (T, N, K, R, L),
          (x.data_ptr(), kind, T, order.data_ptr(), starts.data_ptr(), a.data_ptr(), b.data_ptr(),
           scales.data_ptr(), L, R, N, K, None if y is None else y.data_ptr(), o.data_ptr(),
           v.data_ptr() if save else None), dev)
    if out is not None:  # a recorded operation that saved it notices
        torch.autograd.graph.increment_version(o)
    return (o, v) if save else o


def lora_grad(dy, x, v, a, b, scales, plan, dx=None, out=None):
    """(dx, da, db), the gradients of ``lora`` from dy [T][N], its x and the v that it
    saved.  ``dx``: the gradient through the shared projection (of ``linear_w8a8_grad``),
    which the adapters' part is added to; without it that part alone.  ``out``: where dx is
    written, ``dx`` itself allowed.  da [L][R][K] and db [L][N][R] are fp32, the sums as they
    are; an adapter without tokens has zeros.  fp16: u and v enter them with 22 bits each, and not
    below 2^-39 of the largest among up to 64 ranks and all tokens of an adapter (bf16: 24 bits each)."""
    torch = _torch()
    kind = _float_type(x, "x")
    T, N, K, R, L = _sizes(x, a, b)
    dtype, dev = x.dtype, x.device
    order, starts = plan["order"], plan["starts"]
    if not x.is_cuda:
        raise ValueError("x must live on the GPU")
    _fine(dev, (x, "x", dtype, (T, K)), (a, "a", dtype, (L, R, K)), (b, "b", dtype, (L, N, R)),
          (scales, "scales", torch.float32, (L,)), (order, "order", torch.int32, (T,)),
          (starts, "starts", torch.int32, (L + 1,)), (dy, "dy", dtype, (T, N)),
          (v, "v", torch.float32, (T, R)))
    if dx is not None:
        _fine(dev, (dx, "dx", dtype, (T, K)))
    if out is None:
        o = torch.empty_like(x)
    else:
        o = _out(out, "out", (T, K), dtype, dev)
        inputs = (dy, x, v, a, b, scales, order, starts)
        if dx is not None and dx.data_ptr() != o.data_ptr():
            inputs += (dx,)
        _apart(o, "out", *inputs)
    da = torch.empty((L, R, K), dtype=torch.float32, device=dev)
    db = torch.empty((L, N, R), dtype=torch.float32, device=dev)
    _call("lowbit_lora_grad", (T, N, K, R, L),
          (dy.data_ptr(), x.data_ptr(), v.data_ptr(), kind, T, order.data_ptr(), starts.data_ptr(),
           a.data_ptr(), b.data_ptr(), scales.data_ptr(), L, R, N, K,
           None if dx is None else dx.data_ptr(), o.data_ptr(), da.data_ptr(), db.data_ptr()), dev)
    if out is not None:
        torch.autograd.graph.increment_version(o)
    return o, da, db
