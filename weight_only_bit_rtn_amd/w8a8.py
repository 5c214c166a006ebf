"""Products in 8-bit integers: 8-bit weights, activations quantized per token.

Binding of ``include/lowbit_w8a8.h``; argument marshalling only, as in the
package's other functions.  Weights are the 8-bit per-row codes of
``quantize_rtn(w, 8, 0)`` (either grid) or ``quantize_gptq(w, x, 8, 0)``:

  quantize_act(x) -> dict                            codes, scales, sums of each token
  linear_w8a8(x, packed, scales, zeros) -> y         x fp16 / bf16, or a quantize_act dict
  gated_w8a8(x, gate's three, up's three, act) -> h  act(x G^T) * (x U^T), one kernel
  linear_w8a8_grad(dy, packed, scales, zeros) -> dx
  gated_w8a8_grad(dh, gate, up, gate's three, up's three, act) -> dx

The gradients are with respect to x; the weights are constants, and the
rounding of the activations is passed through unchanged.  The calls are outside
autograd: where gradients are recorded, a tensor that requires grad is refused,
as its gradient would end there.  An autograd function's forward and backward,
and torch.no_grad(), take any tensor.
"""
from __future__ import annotations

import ctypes

from . import _check, _ptr, _require_gpu_tensor, load_library as _load_library

W8A8_MAX_K = 131072
W8A8_MAX_TN = 1 << 20
F16, BF16, I8 = 0, 1, 2
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}

EXPORTED_W8A8 = ("lowbit_quantize_act", "lowbit_linear_w8a8_workspace_bytes", "lowbit_linear_w8a8",
                 "lowbit_gated_w8a8_workspace_bytes", "lowbit_gated_w8a8",
                 "lowbit_linear_w8a8_grad_workspace_bytes", "lowbit_linear_w8a8_grad",
                 "lowbit_gated_w8a8_grad_workspace_bytes", "lowbit_gated_w8a8_grad")

_declared = None
_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(device) -> int:
    """The current stream's handle, without the stream object where torch offers that (1.8 us less)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(device.index) if raw is not None else torch.cuda.current_stream(device).cuda_stream


def _lib() -> ctypes.CDLL:
    global _declared
    lib = _load_library()
    if _declared is lib:
        return lib
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.lowbit_quantize_act.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp]
    lib.lowbit_linear_w8a8_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.lowbit_linear_w8a8.argtypes = [vp, i32, vp, vp, i64, vp, vp, vp, i64, i64, vp, i32, vp,
                                       i64, vp]
    lib.lowbit_gated_w8a8_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.lowbit_gated_w8a8.argtypes = [vp, i32, vp, vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i32,
                                      vp, vp, vp, i32, vp, i64, vp]
    lib.lowbit_linear_w8a8_grad_workspace_bytes.argtypes = [i64, i64, i64]
    lib.lowbit_linear_w8a8_grad.argtypes = [vp, i32, i64, vp, vp, vp, i64, i64, vp, vp, i64, vp]
    lib.lowbit_gated_w8a8_grad_workspace_bytes.argtypes = [i64, i64, i64]
    lib.lowbit_gated_w8a8_grad.argtypes = [vp, vp, vp, i32, i64, vp, vp, vp, vp, vp, vp, i64, i64,
                                           i32, vp, vp, vp, vp, i64, vp]
    for name in EXPORTED_W8A8:
        getattr(lib, name).restype = i64 if name.endswith("_bytes") else i32
    _declared = lib
    return lib


# ---------------------------------------------------------------------------
# raw entry points (device pointers as ints; the caller owns every buffer)
# ---------------------------------------------------------------------------
def quantize_act_raw(x, dtype, T, K, codes, scales, sums, stream) -> int:
    return _lib().lowbit_quantize_act(x, dtype, T, K, codes, scales, sums, stream)


def linear_w8a8_workspace_bytes(T: int, N: int, K: int, dtype: int) -> int:
    return _lib().lowbit_linear_w8a8_workspace_bytes(T, N, K, dtype)


def linear_w8a8_raw(x, dtype, x_scales, x_sums, T, packed, scales, zeros, N, K, y, out_dtype,
                    workspace, workspace_bytes, stream) -> int:
    return _lib().lowbit_linear_w8a8(x, dtype, x_scales, x_sums, T, packed, scales, zeros, N, K, y,
                                     out_dtype, workspace, workspace_bytes, stream)


def gated_w8a8_workspace_bytes(T: int, N: int, K: int, dtype: int) -> int:
    return _lib().lowbit_gated_w8a8_workspace_bytes(T, N, K, dtype)


def gated_w8a8_raw(x, dtype, x_scales, x_sums, T, packed_gate, scales_gate, zeros_gate, packed_up,
                   scales_up, zeros_up, N, K, act, h, gate, up, out_dtype, workspace,
                   workspace_bytes, stream) -> int:
    return _lib().lowbit_gated_w8a8(x, dtype, x_scales, x_sums, T, packed_gate, scales_gate,
                                    zeros_gate, packed_up, scales_up, zeros_up, N, K, act, h, gate,
                                    up, out_dtype, workspace, workspace_bytes, stream)


def linear_w8a8_grad_workspace_bytes(T: int, N: int, K: int) -> int:
    return _lib().lowbit_linear_w8a8_grad_workspace_bytes(T, N, K)


def linear_w8a8_grad_raw(dy, dtype, T, packed, scales, zeros, N, K, dx, workspace,
                         workspace_bytes, stream) -> int:
    return _lib().lowbit_linear_w8a8_grad(dy, dtype, T, packed, scales, zeros, N, K, dx, workspace,
                                          workspace_bytes, stream)


def gated_w8a8_grad_workspace_bytes(T: int, N: int, K: int) -> int:
    return _lib().lowbit_gated_w8a8_grad_workspace_bytes(T, N, K)


def gated_w8a8_grad_raw(dh, gate, up, dtype, T, packed_gate, scales_gate, zeros_gate, packed_up,
                        scales_up, zeros_up, N, K, act, dx, dgate, dup, workspace,
                        workspace_bytes, stream) -> int:
    return _lib().lowbit_gated_w8a8_grad(dh, gate, up, dtype, T, packed_gate, scales_gate,
                                         zeros_gate, packed_up, scales_up, zeros_up, N, K, act, dx,
                                         dgate, dup, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------
# tensor front end: a decoding step's kernels take some microseconds, so the
# checks look at each tensor once and spell out what is wrong only when it is
# ---------------------------------------------------------------------------
def _float_type(t, name: str) -> int:
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    return F16 if t.dtype == torch.float16 else BF16


def _wrong(t, name: str, dtype, device, shape) -> None:
    """Says what is wrong with a tensor."""
    torch = _torch()
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires grad, and the call is outside autograd: its gradient would end "
                         "here; make the call under torch.no_grad() and the *_grad call for the gradient")
    _require_gpu_tensor(t, name, dtype)
    if device is not None and t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    if t.dim() != (2 if shape is None else len(shape)):
        raise ValueError(f"{name} must have {2 if shape is None else len(shape)} dimensions")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _check_tensor(t, name: str, dtype, device=None, shape=None) -> None:
    """``t`` is a dense GPU tensor of this type, place and shape (any matrix where None)
    whose gradient nobody waits for."""
    try:
        fine = (t.dtype is dtype and t.is_contiguous()
                and not (t.requires_grad and _torch().is_grad_enabled())
                and (t.dim() == 2 if shape is None else t.shape == shape)
                and (t.is_cuda if device is None else t.get_device() == device.index))
    except AttributeError:
        fine = False
    if not fine:
        _wrong(t, name, dtype, device, shape)


def _weights(packed, scales, zeros, device, N=None, K=None):
    """N, K of one 8-bit per-row weight matrix, checked."""
    torch = _torch()
    _check_tensor(packed, "packed", torch.int32, device)
    n, words = packed.shape
    if N is not None and (n, 4 * words) != (N, K):
        raise ValueError(f"the two weight matrices must have one shape, got {[N, K]} and "
                         f"{[n, 4 * words]}")
    _check_tensor(scales, "scales", torch.float16, device, (n, 1))
    _check_tensor(zeros, "zeros", torch.int32, device, (n, 1))
    return n, 4 * words


def _activations(x, out_dtype):
    """(pointers and type), T, K, device, output type of a tensor or a quantize_act dict."""
    torch = _torch()
    if isinstance(x, dict):
        codes, scales, sums = x["codes"], x["scales"], x["sums"]
        _check_tensor(codes, "codes", torch.int8)
        T, K = codes.shape
        dev = codes.device
        _check_tensor(scales, "scales of x", torch.float32, dev, (T,))
        _check_tensor(sums, "sums of x", torch.int32, dev, (T,))
        if out_dtype is None:
            out_dtype = torch.float16
        ptrs = (codes.data_ptr(), I8, scales.data_ptr(), sums.data_ptr())
    else:
        kind = _float_type(x, "x")
        _check_tensor(x, "x", x.dtype)
        T, K = x.shape
        dev = x.device
        if out_dtype is None:
            out_dtype = x.dtype
        ptrs = (x.data_ptr(), kind, None, None)
    if out_dtype == torch.float16:
        out_kind = F16
    elif out_dtype == torch.bfloat16:
        out_kind = BF16
    else:
        raise TypeError(f"out_dtype must be torch.float16 or torch.bfloat16, got {out_dtype}")
    return ptrs, T, K, dev, out_dtype, out_kind


def _run(name: str, sizes, args, device) -> None:
    """Calls an entry point on ``args``, its workspace (for ``sizes``; None: it
    takes none) and the current stream of the tensors' device, which it makes
    the current one: launches go there."""
    torch = _torch()
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _run(name, sizes, args, device)
    lib = _lib()
    if sizes is None:
        return _check(getattr(lib, name)(*args, _stream_handle(device)), name)
    need = getattr(lib, name + "_workspace_bytes")(*sizes)
    if need > 0:
        # torch's caching allocator hands out blocks aligned to 512 bytes
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        at = workspace.data_ptr()
    else:
        _check(need, name + "_workspace_bytes")
        at = None
    _check(getattr(lib, name)(*args, at, need, _stream_handle(device)), name)


def _out(out, name, shape, dtype, device):
    if out is None:
        return _torch().empty(shape, dtype=dtype, device=device)
    _check_tensor(out, name, dtype, device, shape)
    return out


def _apart(out, name, *inputs) -> None:
    """Refuses an output that shares memory with an input of its device."""
    lo = out.data_ptr()
    hi = lo + out.nbytes
    for t in inputs:
        at = t.data_ptr()
        if at < hi and lo < at + t.nbytes:
            raise ValueError(f"{name} must not share memory with an input")


def _act(act) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


def quantize_act(x, out: dict | None = None) -> dict:
    """Per-token int8 quantization of fp16 or bf16 ``x[T][K]``: a dict with
    ``codes`` (int8 [T][K]), ``scales`` (fp32 [T]) and ``sums`` (int32 [T], the
    sum of a token's codes), which the products take instead of x.  ``out``: such
    a dict to write into."""
    torch = _torch()
    kind = _float_type(x, "x")
    _check_tensor(x, "x", x.dtype)
    T, K = x.shape
    dev = x.device
    out = out or {}
    codes = _out(out.get("codes"), "codes", (T, K), torch.int8, dev)
    scales = _out(out.get("scales"), "scales", (T,), torch.float32, dev)
    sums = _out(out.get("sums"), "sums", (T,), torch.int32, dev)
    if out:
        _apart(codes, "codes", x)
        _apart(scales, "scales", x, codes)
        _apart(sums, "sums", x, codes, scales)
    _run("lowbit_quantize_act", None,
         (x.data_ptr(), kind, T, K, codes.data_ptr(), scales.data_ptr(), sums.data_ptr()), dev)
    return {"codes": codes, "scales": scales, "sums": sums}


def linear_w8a8(x, packed, scales, zeros, out_dtype=None, out=None):
    """y[T][N] = x * deq(packed)^T in 8-bit integers.  ``x``: fp16 or bf16
    [T][K], quantized on the way, or the dict of ``quantize_act``.  ``out_dtype``
    is x's type, or fp16 for a dict, unless given."""
    ptrs, T, K, dev, out_dtype, out_kind = _activations(x, out_dtype)
    N, k = _weights(packed, scales, zeros, dev)
    if k != K:
        raise ValueError("x and the weights must have the same K")
    y = _out(out, "out", (T, N), out_dtype, dev)
    if out is not None:
        _apart(y, "out", *((x["codes"], x["scales"], x["sums"]) if isinstance(x, dict) else (x,)),
               packed, scales, zeros)
    _run("lowbit_linear_w8a8", (T, N, K, ptrs[1]),
         (*ptrs, T, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), N, K, y.data_ptr(),
          out_kind), dev)
    return y


def gated_w8a8(x, packed_gate, scales_gate, zeros_gate, packed_up, scales_up, zeros_up,
               act: str = "silu", save: bool = False, out_dtype=None):
    """h[T][N] = act(x * deq(gate)^T) * (x * deq(up)^T), both projections in
    one kernel; ``act``: "silu" or "gelu_tanh"; ``x`` as for ``linear_w8a8``.
    ``save``: (h, gate, up), the projections rounded to the output type, which
    ``gated_w8a8_grad`` takes."""
    torch = _torch()
    kind = _act(act)
    ptrs, T, K, dev, out_dtype, out_kind = _activations(x, out_dtype)
    N, k = _weights(packed_gate, scales_gate, zeros_gate, dev)
    if k != K:
        raise ValueError("x and the weights must have the same K")
    _weights(packed_up, scales_up, zeros_up, dev, N, K)
    outs = [torch.empty((T, N), dtype=out_dtype, device=dev) for _ in range(3 if save else 1)]
    _run("lowbit_gated_w8a8", (T, N, K, ptrs[1]),
         (*ptrs, T, packed_gate.data_ptr(), scales_gate.data_ptr(), zeros_gate.data_ptr(),
          packed_up.data_ptr(), scales_up.data_ptr(), zeros_up.data_ptr(), N, K, kind,
          outs[0].data_ptr(), outs[1].data_ptr() if save else None,
          outs[2].data_ptr() if save else None, out_kind), dev)
    return tuple(outs) if save else outs[0]


def linear_w8a8_grad(dy, packed, scales, zeros, out=None):
    """dx[T][K] = dy[T][N] * deq(packed), of dy's type: the gradient of
    ``linear_w8a8`` with respect to x."""
    kind = _float_type(dy, "dy")
    _check_tensor(dy, "dy", dy.dtype)
    dev = dy.device
    N, K = _weights(packed, scales, zeros, dev)
    T = dy.shape[0]
    if dy.shape[1] != N:
        raise ValueError("dy.shape[1] must be the weights' N")
    dx = _out(out, "out", (T, K), dy.dtype, dev)
    if out is not None:
        _apart(dx, "out", dy, packed, scales, zeros)
    _run("lowbit_linear_w8a8_grad", (T, N, K),
         (dy.data_ptr(), kind, T, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(), N, K,
          dx.data_ptr()), dev)
    return dx


def gated_w8a8_grad(dh, gate, up, packed_gate, scales_gate, zeros_gate, packed_up, scales_up,
                    zeros_up, act: str = "silu", parts: bool = False):
    """dx[T][K], the gradient of ``gated_w8a8`` with respect to x, from dh and
    the projections that the forward call saved (one type).  ``parts``: (dx,
    dgate, dup), with the gradients of both projections' outputs, from which
    those of adapters beside them follow."""
    torch = _torch()
    code = _act(act)
    kind = _float_type(dh, "dh")
    _check_tensor(dh, "dh", dh.dtype)
    dev = dh.device
    N, K = _weights(packed_gate, scales_gate, zeros_gate, dev)
    _weights(packed_up, scales_up, zeros_up, dev, N, K)
    T = dh.shape[0]
    if dh.shape[1] != N:
        raise ValueError("dh.shape[1] must be the weights' N")
    _check_tensor(gate, "gate", dh.dtype, dev, dh.shape)
    _check_tensor(up, "up", dh.dtype, dev, dh.shape)
    dx = torch.empty((T, K), dtype=dh.dtype, device=dev)
    dgate = torch.empty_like(dh) if parts else None
    dup = torch.empty_like(dh) if parts else None
    _run("lowbit_gated_w8a8_grad", (T, N, K),
         (dh.data_ptr(), gate.data_ptr(), up.data_ptr(), kind, T, packed_gate.data_ptr(),
          scales_gate.data_ptr(), zeros_gate.data_ptr(), packed_up.data_ptr(),
          scales_up.data_ptr(), zeros_up.data_ptr(), N, K, code, dx.data_ptr(), _ptr(dgate),
          _ptr(dup)), dev)
    return (dx, dgate, dup) if parts else dx
