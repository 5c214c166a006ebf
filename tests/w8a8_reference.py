"""The 8-bit activation operators in 64 bits, from their definition (numpy).

Shared by the CPU and GPU tests of the operators; no code of the library.
Every function works on float64 values and on codes; the only 32-bit steps are
the ones the definition has (a token's scale and the quotients).
"""
from __future__ import annotations

import numpy as np

#: half a step, relative to the value, and half the smallest subnormal
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134}
U32 = 2.0 ** -24


def quantize_act(x32: np.ndarray):
    """codes int8 [T][K], scales fp32 [T], sums int32 [T] of fp32-widened activations."""
    x32 = np.asarray(x32, np.float32)
    finite = np.isfinite(x32).all(1)
    safe = np.where(finite[:, None], x32, np.float32(0))
    s = np.abs(safe).max(1) / np.float32(127)
    s = np.where(s == 0, np.float32(1), s).astype(np.float32)
    a = np.clip(np.rint((safe / s[:, None]).astype(np.float32)), -127, 127).astype(np.int8)
    return a, np.where(finite, s, np.float32(np.nan)), a.sum(1, dtype=np.int32)


def product(a, s, codes, scales, zeros):
    """S_t s_n sum_k a (c - z): exact integer sums, then 64-bit products."""
    w = codes.astype(np.float64) - zeros.reshape(-1, 1)
    d = a.astype(np.float64) @ w.T          # integers below 2^53: exact
    return d * (s.astype(np.float64)[:, None] * scales.astype(np.float64).reshape(1, -1))


def two_q(v, act):
    """2q of v * sigma, sigma = 1 / (1 + exp(-2q))."""
    return v if act == "silu" else 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)


def _sigma(q2):
    return 1 / (1 + np.exp(-np.clip(q2, -700, 700)))


def act_value(v, act):
    return v * _sigma(two_q(v, act))


def act_slope(v, act):
    s = _sigma(two_q(v, act))
    d = 1.0 if act == "silu" else 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * v ** 2)
    return s + v * s * (1 - s) * d


def deq(codes, scales, zeros):
    return (codes.astype(np.float64) - zeros.reshape(-1, 1)) * scales.astype(np.float64).reshape(-1, 1)


def linear_grad(dy, codes, scales, zeros):
    return dy @ deq(codes, scales, zeros)


def gated_parts(dh, gate, up, act):
    """dgate, dup"""
    return dh * up * act_slope(gate, act), dh * act_value(gate, act)


# ---------------------------------------------------------------------------
# how far a kernel's output may be off
# ---------------------------------------------------------------------------
def linear_bound(ref, kind):
    """One rounding to the output type; in 32 bits the sum's conversion, the two scales' product and the last
    product (the integer sum is exact): three half steps, and their products."""
    return np.abs(ref) * (HALF_STEP[kind] * (1 + 2 ** -10) + 4 * U32) + HALF_TINY[kind]


def gated_bound(ref, gate, kind, act):
    """As linear_bound for g and u (4 half steps each), then sigma: an error of r in 2q moves sigma by at most
    r relative, 2q has the relative errors of g (cubed for GELU: 12) and of its own steps (6) and of
    exp's argument (2); exp, the sum, the reciprocal and the three products: under 12 half steps more."""
    q = np.minimum(np.abs(two_q(gate, act)), 104.0)   # beyond, sigma is its limit in 32 bits
    r = (20 + 20 * q) * U32
    # e^-2q overflows 32 bits from 88.7 on: sigma is 0 there, at most 2^-127
    lost = np.where(two_q(gate, act) < -87, np.abs(ref), 0)
    return np.abs(ref) * (HALF_STEP[kind] * (1 + 2 ** -10) + r) + lost + HALF_TINY[kind]


def grad_bound(ref, parts, kind, extra=None):
    """``parts``: list of (d [T][N] in 64 bits, codes, scales, zeros).  Each factor d s is rounded to fp16 (half a
    step 2^-11, or half of 2^-24 below the token's largest / 2^29), after a few 32-bit steps (``extra``, relative,
    [T][N], for those of the activation); the 32-bit sums of n terms lose at most n steps each of 2^-23."""
    slack = np.zeros_like(ref)
    top = np.zeros((ref.shape[0], 1))
    terms = 0
    for d, codes, scales, zeros in parts:
        a = np.abs(d * scales.astype(np.float64).reshape(1, -1))
        if a.size:
            top = np.maximum(top, a.max(1, keepdims=True))
        terms += codes.shape[0]
    for i, (d, codes, scales, zeros) in enumerate(parts):
        a = np.abs(d * scales.astype(np.float64).reshape(1, -1))
        rel = 2.0 ** -11 + 8 * U32 + terms * 2.0 ** -23
        err = a * (rel + (extra[i] if extra is not None else 0)) + top * 2.0 ** -39
        # the kernel's two sums: over code - 128, and over 128 - z
        size = np.abs(codes.astype(np.float64) - 128) + np.abs(128.0 - zeros.reshape(-1, 1))
        slack = slack + err @ size
    return np.abs(ref) * HALF_STEP[kind] * (1 + 2 ** -8) + slack * (1 + HALF_STEP[kind]) + HALF_TINY[kind]
