"""The 8-bit activation operators without a GPU: the header and the binding
agree, bad arguments are refused on the host before anything is launched, and
the 64-bit reference of the GPU tests is what it says (hand-worked numbers,
exact rationals, differences)."""
from __future__ import annotations

import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest

import w8a8_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lowbit_w8a8.h")


@pytest.fixture(scope="module")
def lw():
    import weight_only_bit_rtn_amd as lw
    if not os.path.exists(lw.LIB_PATH):
        from weight_only_bit_rtn_amd import build
        build.build()
    lw.load_library()
    return lw


def test_header_library_and_binding_agree(lw):
    text = open(HEADER).read()
    declared = set(re.findall(r"LOWBIT_API\s+[\w\s\*]+?\b(lowbit_\w+)\s*\(", text))
    assert declared == set(lw.EXPORTED_W8A8)
    lib = ctypes.CDLL(lw.LIB_PATH)
    for name in declared:
        assert hasattr(lib, name), name
    consts = dict(re.findall(r"#define\s+(LOWBIT_\w+)\s+(\d+)", text))
    from weight_only_bit_rtn_amd import w8a8
    assert int(consts["LOWBIT_W8A8_MAX_K"]) == lw.W8A8_MAX_K
    assert int(consts["LOWBIT_W8A8_MAX_TN"]) == lw.W8A8_MAX_TN
    assert (int(consts["LOWBIT_F16"]), int(consts["LOWBIT_BF16"]), int(consts["LOWBIT_I8"])) == (
        w8a8.F16, w8a8.BF16, w8a8.I8)
    assert {"silu": int(consts["LOWBIT_ACT_SILU"]),
            "gelu_tanh": int(consts["LOWBIT_ACT_GELU_TANH"])} == w8a8.ACTIVATIONS


# Addresses that are never dereferenced: each call is refused, or empty.  (100 tokens: the products then need a
# workspace.)
P = 0x7F0000000000
MIS = P + 2
BIG = 1 << 40


def quant(lw, x=P, dtype=0, T=4, K=64, codes=P, scales=P, sums=P):
    return lw.quantize_act_raw(x, dtype, T, K, codes, scales, sums, None)


def linear(lw, x=P, dtype=0, xs=None, sums=None, T=100, packed=P, scales=P, zeros=P, N=8, K=64, y=P, out=0, ws=P,
           size=BIG):
    return lw.linear_w8a8_raw(x, dtype, xs, sums, T, packed, scales, zeros, N, K, y, out, ws, size, None)


def gated(lw, x=P, dtype=0, xs=None, sums=None, T=100, pg=P, sg=P, zg=P, pu=P, su=P, zu=P, N=8, K=64, act=0, h=P, g=None,
          u=None, out=0, ws=P, size=BIG):
    return lw.gated_w8a8_raw(x, dtype, xs, sums, T, pg, sg, zg, pu, su, zu, N, K, act, h, g, u, out, ws, size, None)


def linear_grad(lw, dy=P, dtype=0, T=4, packed=P, scales=P, zeros=P, N=8, K=64, dx=P, ws=P, size=BIG):
    return lw.linear_w8a8_grad_raw(dy, dtype, T, packed, scales, zeros, N, K, dx, ws, size, None)


def gated_grad(lw, dh=P, gate=P, up=P, dtype=0, T=4, pg=P, sg=P, zg=P, pu=P, su=P, zu=P, N=8, K=64, act=0, dx=P,
               dgate=None, dup=None, ws=P, size=BIG):
    return lw.gated_w8a8_grad_raw(dh, gate, up, dtype, T, pg, sg, zg, pu, su, zu, N, K, act, dx, dgate, dup, ws, size,
                                  None)


ARG, SHAPE, UNSUPPORTED = -1, -2, -3
ALL = (quant, linear, gated, linear_grad, gated_grad)
REFUSED = (
    [(f, dict(dtype=d), UNSUPPORTED) for f in ALL for d in (-1, 3, 7)]
    + [(f, dict(dtype=2), UNSUPPORTED) for f in (quant, linear_grad, gated_grad)]
    + [(f, dict(out=2), UNSUPPORTED) for f in (linear, gated)]
    + [(f, dict(act=a), UNSUPPORTED) for f in (gated, gated_grad) for a in (-1, 2)]
    + [(f, dict(T=-1), ARG) for f in ALL] + [(f, dict(K=-32), ARG) for f in ALL]
    + [(f, dict(N=-1), ARG) for f in ALL if f is not quant]
    + [(f, dict(K=k), SHAPE) for f in ALL for k in (0, 16, 65, 100, 131072 + 32)]
    + [(f, dict(T=(1 << 20) + 1), SHAPE) for f in ALL]
    + [(f, dict(N=(1 << 20) + 1), SHAPE) for f in ALL if f is not quant]
    + [(f, dict(T=1 << 20, N=1 << 17), SHAPE) for f in ALL if f is not quant]
    + [(f, dict(T=1 << 20, K=65536 + 32), SHAPE) for f in ALL]
    + [(quant, {a: v}, ARG) for a in ("x", "codes", "scales", "sums") for v in (None, MIS)]
    + [(linear, {a: v}, ARG) for a in ("x", "packed", "scales", "zeros", "y", "ws") for v in (None, MIS)]
    + [(gated, {a: v}, ARG) for a in ("x", "pg", "sg", "zg", "pu", "su", "zu", "h", "ws") for v in (None, MIS)]
    + [(linear_grad, {a: v}, ARG) for a in ("dy", "packed", "scales", "zeros", "dx", "ws") for v in (None, MIS)]
    + [(gated_grad, {a: v}, ARG) for a in ("dh", "gate", "up", "pg", "sg", "zg", "pu", "su", "zu", "dx", "ws")
       for v in (None, MIS)]
    + [(f, dict(xs=P, sums=P), ARG) for f in (linear, gated)]          # scales beside values
    + [(f, dict(dtype=2), ARG) for f in (linear, gated)]               # codes without scales
    + [(f, dict(dtype=2, xs=P, sums=MIS), ARG) for f in (linear, gated)]
    + [(gated, dict(g=P), ARG), (gated, dict(u=P), ARG), (gated, dict(g=P, u=MIS), ARG),
       (gated_grad, dict(dgate=P), ARG), (gated_grad, dict(dup=P), ARG), (gated_grad, dict(dgate=MIS, dup=P), ARG)]
    + [(f, dict(size=0), ARG) for f in ALL if f is not quant]
    + [(f, dict(ws=P + 16), ARG) for f in ALL if f is not quant])


@pytest.mark.parametrize("f,args,status", REFUSED)
def test_refused_on_the_host(lw, f, args, status):
    assert f(lw, **args) == status


@pytest.mark.parametrize("f", ALL)
def test_empty_problems_launch_nothing(lw, f):
    assert f(lw, T=0) == 0
    if f in (linear, gated):
        assert f(lw, N=0) == 0


def test_workspace_sizes(lw):
    sizes = (lw.linear_w8a8_workspace_bytes, lw.gated_w8a8_workspace_bytes)
    grads = (lw.linear_w8a8_grad_workspace_bytes, lw.gated_w8a8_grad_workspace_bytes)
    for f in sizes:
        assert f(0, 8, 64, 0) == 0
        assert f(8, 8, 65, 0) == SHAPE and f(-1, 8, 64, 0) == ARG and f(8, 8, 64, 5) == UNSUPPORTED
        # the codes of long inputs need room, and room for more tokens is never less
        assert f(4096, 64, 1024, 0) >= 4096 * 1024
        last = 0
        for T in (1, 2, 63, 64, 65, 500, 5000):
            assert 0 <= f(T, 4096, 1024, 2) <= f(T, 4096, 1024, 0)
    for f in grads:
        assert f(0, 8, 64) == 0 and f(8, 8, 65) == SHAPE
        for T, N in ((1, 1), (3, 65), (100, 1000)):
            assert f(T, N, 64) >= 2 * T * N


def test_one_workspace_too_small_by_a_byte(lw):
    for f, need in ((linear, lw.linear_w8a8_workspace_bytes(4000, 8, 64, 0)),
                    (gated, lw.gated_w8a8_workspace_bytes(4000, 8, 64, 0)),
                    (linear_grad, lw.linear_w8a8_grad_workspace_bytes(4000, 8, 64)),
                    (gated_grad, lw.gated_w8a8_grad_workspace_bytes(4000, 8, 64))):
        assert need > 0 and f(lw, T=4000, size=need - 1) == ARG


def test_binding_refuses_what_is_not_on_the_gpu(lw):
    import torch
    x = torch.zeros(2, 64, dtype=torch.float16)
    w = (torch.zeros(8, 16, dtype=torch.int32), torch.ones(8, 1, dtype=torch.float16),
         torch.zeros(8, 1, dtype=torch.int32))
    for call in (lambda: lw.quantize_act(x), lambda: lw.linear_w8a8(x, *w), lambda: lw.gated_w8a8(x, *w, *w),
                 lambda: lw.linear_w8a8_grad(x[:, :8].contiguous(), *w)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        lw.quantize_act(x.float())
    with pytest.raises(TypeError):
        lw.linear_w8a8([1, 2], *w)


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------
def test_codes_by_hand():
    # scale 1: the quotient is x itself, halves go to the even code
    a, s, total = ref.quantize_act(np.array([[127, 0.5, 1.5, -2.5, -0.5, 63.5, 3, -127]], np.float32))
    assert s[0] == 1 and a[0].tolist() == [127, 0, 2, -2, 0, 64, 3, -127] and total[0] == 67
    a, s, total = ref.quantize_act(np.array([[0, 0], [np.inf, 1], [-1e-45, 0]], np.float32))
    assert s[0] == 1 and np.isnan(s[1]) and total.tolist() == [0, 0, a[2].sum()] and a[:2].tolist() == [[0, 0], [0, 0]]


def test_codes_are_the_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 64)).astype(np.float32)
    a, s, _ = ref.quantize_act(x)
    for i in range(20):
        assert abs(float(s[i]) * 127 / np.abs(x[i]).max() - 1) < 2.0 ** -23
        for j in range(64):
            q = Fraction(float(x[i, j])) / Fraction(float(s[i]))
            assert abs(q - int(a[i, j])) <= Fraction(1, 2) + Fraction(1, 2 ** 16)


def test_product_in_rationals():
    rng = np.random.default_rng(1)
    a = rng.integers(-127, 128, (3, 32)).astype(np.int8)
    codes = rng.integers(0, 256, (4, 32)).astype(np.uint8)
    scales, zeros = rng.uniform(0.1, 1, 4).astype(np.float16), np.array([0, 128, -5000, 255], np.int32)
    s = rng.uniform(0.1, 1, 3).astype(np.float32)
    y = ref.product(a, s, codes, scales, zeros)
    for t in range(3):
        for n in range(4):
            d = sum(int(a[t, k]) * (int(codes[n, k]) - int(zeros[n])) for k in range(32))
            assert abs(Fraction(float(y[t, n])) / (d * Fraction(float(s[t])) * Fraction(float(scales[n]))) - 1) < 2 ** -50


def test_activations_by_hand():
    assert ref.act_value(np.array([0.0]), "silu")[0] == 0 and ref.act_slope(np.array([0.0]), "silu")[0] == 0.5
    assert ref.act_slope(np.array([0.0]), "gelu_tanh")[0] == 0.5
    v = np.linspace(-6, 6, 25)
    p = np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
    assert np.allclose(ref.act_value(v, "gelu_tanh"), 0.5 * v * (1 + np.tanh(p)), rtol=0, atol=1e-15)
    assert np.allclose(ref.act_value(v, "silu"), 0.5 * v * (1 + np.tanh(v / 2)), rtol=0, atol=1e-15)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(act):
    """The gated block without the rounding of x: central differences of sum(dh * h) by every element of x."""
    rng = np.random.default_rng(2)
    T, N, K = 3, 5, 32
    ws = []
    for _ in range(2):
        ws.append((rng.integers(0, 256, (N, K)).astype(np.uint8), rng.uniform(0.001, 0.01, N).astype(np.float16),
                   rng.integers(100, 150, N).astype(np.int32)))
    x, dh = rng.standard_normal((T, K)), rng.standard_normal((T, N))
    wg, wu = (ref.deq(*w) for w in ws)

    def loss(x):
        return (dh * ref.act_value(x @ wg.T, act) * (x @ wu.T)).sum()

    dg, du = ref.gated_parts(dh, x @ wg.T, x @ wu.T, act)
    dx = ref.linear_grad(dg, *ws[0]) + ref.linear_grad(du, *ws[1])
    e = 1e-5
    for t in range(T):
        for k in range(K):
            step = np.zeros_like(x)
            step[t, k] = e
            d = (loss(x + step) - loss(x - step)) / (2 * e)
            assert abs(d - dx[t, k]) <= 1e-7 * np.abs(dx).max()


def test_outputs_apart_from_inputs():
    """Sharing a byte is refused, lying next to each other is not."""
    import torch
    from weight_only_bit_rtn_amd import w8a8
    buf = torch.zeros(64, dtype=torch.float16)
    w8a8._apart(buf[:32], "out", buf[32:], torch.zeros(64))
    w8a8._apart(buf[32:], "out", buf[:32])
    for out, x in [(buf, buf), (buf[:33], buf[32:]), (buf[10:12], buf), (buf.view(torch.int8)[63:64], buf[31:40])]:
        with pytest.raises(ValueError):
            w8a8._apart(out, "out", x)
