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
from .w8a8 import _apart, _check_tensor, _float_type, _out, _run, _stream_handle, _torch

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
    for name in ("lowbit_lora", "lowbit_lora_grad"):
        _entry[name] = (getattr(lib, name), getattr(lib, name + "_workspace_bytes"))
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
    out = out or {}
    order = _out(out.get("order"), "order", (T,), torch.int32, dev)
    starts = _out(out.get("starts"), "starts", (L + 1,), torch.int32, dev)
    if out:
        _apart(order, "order", ids, starts)
        _apart(starts, "starts", ids)
    _lib()
    _run("lowbit_lora_plan", None, (ids.data_ptr(), T, L, order.data_ptr(), starts.data_ptr()), dev)
    return {"order": order, "starts": starts}


def _adapters(x, a, b, scales, plan, name: str):
    """(element type, T, N, K, R, L, device) and the shared pointers, checked."""
    torch = _torch()
    kind = _float_type(x, name)
    dtype = x.dtype
    _check_tensor(x, name, dtype)
    T, K = x.shape
    dev = x.device
    if not (isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor)):
        raise TypeError("a and b must be torch.Tensors")
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must have 3 dimensions")
    L, R, _ = a.shape
    N = b.shape[1]
    _check_tensor(a, "a", dtype, dev, (L, R, K))
    _check_tensor(b, "b", dtype, dev, (L, N, R))
    _check_tensor(scales, "scales", torch.float32, dev, (L,))
    order, starts = plan["order"], plan["starts"]
    _check_tensor(order, "order", torch.int32, dev, (T,))
    _check_tensor(starts, "starts", torch.int32, dev, (L + 1,))
    shared = (order.data_ptr(), starts.data_ptr(), a.data_ptr(), b.data_ptr(), scales.data_ptr(),
              L, R, N, K)
    return kind, T, N, K, R, L, dev, shared


def _call(name: str, sizes, args, device) -> None:
    """Calls an entry point on ``args``, its workspace and the current stream of the tensors'
    device, which it makes the current one."""
    torch = _torch()
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, sizes, args, device)
    if not _entry:
        _lib()
    call, need_of = _entry[name]
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
    kind, T, N, K, R, L, dev, shared = _adapters(x, a, b, scales, plan, "x")
    if y is not None:
        _check_tensor(y, "y", x.dtype, dev, (T, N))
    if out is None:
        o = torch.empty((T, N), dtype=x.dtype, device=dev) if y is None else torch.empty_like(y)
    else:
        o = _out(out, "out", (T, N), x.dtype, dev)
        inputs = (x, a, b, scales, plan["order"], plan["starts"])
        if y is not None and y.data_ptr() != o.data_ptr():
            inputs += (y,)
        _apart(o, "out", *inputs)
    v = torch.empty((T, R), dtype=torch.float32, device=dev) if save else None
    _call("lowbit_lora", (T, N, K, R, L),
         (x.data_ptr(), kind, T, *shared, None if y is None else y.data_ptr(), o.data_ptr(),
          v.data_ptr() if save else None), dev)
    return (o, v) if save else o


def lora_grad(dy, x, v, a, b, scales, plan, dx=None, out=None):
    """(dx, da, db), the gradients of ``lora`` from dy [T][N], its x and the v that it
    saved.  ``dx``: the gradient through the shared projection (of ``linear_w8a8_grad``),
    which the adapters' part is added to; without it that part alone.  ``out``: where dx is
    written, ``dx`` itself allowed.  da [L][R][K] and db [L][N][R] are fp32, the sums as they
    are; an adapter without tokens has zeros."""
    torch = _torch()
    kind, T, N, K, R, L, dev, shared = _adapters(x, a, b, scales, plan, "x")
    _check_tensor(dy, "dy", x.dtype, dev, (T, N))
    _check_tensor(v, "v", torch.float32, dev, (T, R))
    if dx is not None:
        _check_tensor(dx, "dx", x.dtype, dev, (T, K))
    if out is None:
        o = torch.empty_like(x)
    else:
        o = _out(out, "out", (T, K), x.dtype, dev)
        inputs = (dy, x, v, a, b, scales, plan["order"], plan["starts"])
        if dx is not None and dx.data_ptr() != o.data_ptr():
            inputs += (dx,)
        _apart(o, "out", *inputs)
    da = torch.empty((L, R, K), dtype=torch.float32, device=dev)
    db = torch.empty((L, N, R), dtype=torch.float32, device=dev)
    _call("lowbit_lora_grad", (T, N, K, R, L),
         (dy.data_ptr(), x.data_ptr(), v.data_ptr(), kind, T, *shared,
          None if dx is None else dx.data_ptr(), o.data_ptr(), da.data_ptr(), db.data_ptr()), dev)
    return o, da, db
