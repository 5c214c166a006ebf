"""The adapters and the AdamW step in 64 bits, from their definition (numpy).

Shared by the CPU and GPU tests; no code of the library.  The adapters' functions work on
float64; the moments of the AdamW step are numpy float32, one rounded operation at a time, as
the definition has them.
"""
from __future__ import annotations

import numpy as np

#: half a step of a 16-bit type, relative to the value, and half its smallest subnormal
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}
U32 = 2.0 ** -24
BLOCK = 256


def plan(ids, L):
    """order, starts of a batch."""
    ids = list(ids)
    order, starts = [], []
    for l in range(L):
        starts.append(len(order))
        order += [t for t, i in enumerate(ids) if i == l]
    starts.append(len(order))
    order += [t for t, i in enumerate(ids) if not 0 <= i < L]
    return np.array(order, np.int32), np.array(starts, np.int32)


def lora(x, a, b, scales, ids, y=None):
    """out, v."""
    T, L = len(x), len(a)
    out = np.zeros((T, b.shape[1])) if y is None else np.array(y, np.float64)
    v = np.zeros((T, a.shape[1]))
    for l in range(L):
        t = np.flatnonzero(ids == l)
        v[t] = x[t] @ a[l].T
        out[t] += scales[l] * (v[t] @ b[l].T)
    return out, v


def lora_grad(dy, x, v, a, b, scales, ids, base=None):
    """dx, da, db."""
    dx = np.zeros(x.shape) if base is None else np.array(base, np.float64)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    for l in range(len(a)):
        t = np.flatnonzero(ids == l)
        u = scales[l] * (dy[t] @ b[l])
        dx[t] += u @ a[l]
        da[l] = u.T @ x[t]
        db[l] = scales[l] * (dy[t].T @ v[t])
    return dx, da, db


# ---------------------------------------------------------------------------
# how far the kernels may be from that
# ---------------------------------------------------------------------------
def depth(n):
    """Roundings that a sum of n products can pass through: one for each 32 terms, and the joins of
    waves and shares (16 at most).  Each is off by 2^-23 of the sum of the terms' absolute values
    at most, whether the adder rounds or cuts."""
    return (n / 32 + 16) * 2.0 ** -23


def split(kind, parts):
    """Relative error of an fp32 value as a sum of 16-bit parts (each leaves half a step of itself)."""
    return max(HALF_STEP[kind] ** parts, U32)


def lora_bound(x, a, b, scales, ids, out, kind):
    """How far out and v may be off."""
    T, N = out.shape
    R, K = a.shape[1:]
    far, far_v = np.zeros((T, N)), np.zeros((T, R))
    for l in range(len(a)):
        t = np.flatnonzero(ids == l)
        v, absolute = x[t] @ a[l].T, np.abs(x[t]) @ np.abs(a[l]).T
        far_v[t] = depth(K) * absolute
        # the parts' error (and of fp16 values far below the token's largest), then the sum
        parts = split(kind, 2) * np.abs(v) + 2.0 ** -39 * np.abs(v).max(1, keepdims=True, initial=0)
        far[t] = np.abs(scales[l]) * ((far_v[t] + parts + depth(2 * R) * np.abs(v)) @ np.abs(b[l]).T)
    far += 2 * U32 * (np.abs(out) + far)
    return far * 1.01 + HALF_STEP[kind] * (np.abs(out) + far) + HALF_TINY[kind], far_v * 1.01 + 1e-300


def lora_grad_bound(dy, x, v, a, b, scales, ids, dx, kind):
    """How far dx, da and db may be off."""
    R, K = a.shape[1:]
    N = b.shape[1]
    far, far_a, far_b = np.zeros(dx.shape), np.zeros(a.shape), np.zeros(b.shape)
    three = split(kind, 3 if kind == "bf16" else 2)
    for l in range(len(a)):
        t = np.flatnonzero(ids == l)
        s = np.abs(scales[l])
        u, absolute = dy[t] @ b[l], np.abs(dy[t]) @ np.abs(b[l])
        far_u = depth(N) * absolute
        top = np.abs(u).max(1, keepdims=True, initial=0)
        parts = split(kind, 2) * np.abs(u) + 2.0 ** -39 * top
        far[t] = s * ((far_u + parts + depth(2 * R) * np.abs(u)) @ np.abs(a[l]))
        # a chunk's largest value is at most the adapter's
        parts = three * np.abs(u) + 2.0 ** -39 * np.abs(u).max(initial=0)
        far_a[l] = s * ((far_u + parts + depth(3 * len(t)) * np.abs(u)).T @ np.abs(x[t]))
        w = np.abs(v[t])
        parts = (three + depth(3 * len(t))) * w + 2.0 ** -39 * w.max(initial=0)
        far_b[l] = s * (np.abs(dy[t]).T @ parts)
    far += 2 * U32 * (np.abs(dx) + far)
    return (far * 1.01 + HALF_STEP[kind] * (np.abs(dx) + far) + HALF_TINY[kind],
            far_a * 1.01 + 2.0 ** -140, far_b * 1.01 + 2.0 ** -140)


# ---------------------------------------------------------------------------
# the AdamW step
# ---------------------------------------------------------------------------
def numbers(bits):
    """What the codes of m's magnitude (bits = 7) and of v (bits = 8) stand for, block maximum 1."""
    codes = np.arange(1 << bits, dtype=np.uint32)
    out = ((codes + np.uint32(0x3F8 - ((1 << bits) - 1))) << np.uint32(20)).view(np.float32).copy()
    out[0] = 0
    return out


def decode(m, v, m_max, v_max):
    """fp32 values of 8-bit moments."""
    m, v = m.reshape(-1, BLOCK), v.reshape(-1, BLOCK)
    with np.errstate(invalid="ignore"):
        fm = numbers(7)[m & 127] * m_max[:, None]
        fv = numbers(8)[v] * v_max[:, None]
    return np.where(m > 127, -fm, fm).astype(np.float32).reshape(-1), fv.astype(np.float32).reshape(-1)


def encode(x, bits):
    """Codes and maxima of fp32 values (bits = 7: signed, 8: never 0 but for 0)."""
    x = x.reshape(-1, BLOCK)
    mag = np.abs(x)
    finite = np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        top = np.where(finite, mag.max(1), np.float32(np.nan)).astype(np.float32)
        top = np.where(top < np.float32(2.0 ** -126), np.float32(0), top)
        inverse = np.where(top > 0, np.float32(1) / top, np.float32(0)).astype(np.float32)
        q = (np.where(finite[:, None], mag, 0) * inverse[:, None]).astype(np.float32)
    tab = numbers(bits).astype(np.float64)
    border = np.concatenate([[tab[1] - (tab[2] - tab[1]) / 2], (tab[1:-1] + tab[2:]) / 2])
    code = np.searchsorted(border, q.astype(np.float64), side="right")
    if bits == 8:
        code = np.maximum(code, (q > 0).astype(code.dtype))
    else:
        code = np.where((code > 0) & np.signbit(x), code + 128, code)
    return code.astype(np.uint8).reshape(-1), top


def moments(m, v, g, beta1, beta2, scale=None):
    """m', v', float32: every operation rounded by itself."""
    f = np.float32
    g = g.astype(f)
    with np.errstate(all="ignore"):
        if scale is not None:
            g = g * f(scale)
        m = f(beta1) * m + f(1 - beta1) * g
        v = f(beta2) * v + f(1 - beta2) * (g * g)
    return m.astype(f), v.astype(f)


def update(p, m, v, lr, beta1, beta2, eps, decay, step):
    """p', and the step that was taken, float64."""
    with np.errstate(all="ignore"):
        taken = lr / (1 - beta1 ** step) * m.astype(np.float64) / (
            np.sqrt(np.maximum(v.astype(np.float64), 2.0 ** -126)) / np.sqrt(1 - beta2 ** step) + eps)
        taken = np.where(np.isnan(v), np.nan, taken)
    return p.astype(np.float64) * (1 - lr * decay) - taken, taken
