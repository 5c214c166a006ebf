"""Gradients near the end of bf16's range: factors dy s below fp32's normal
range keep their 11 bits, for every length of a row, and tokens of other sizes
beside them are what they are alone."""
from __future__ import annotations

import numpy as np
import pytest

import w8a8_reference as ref
from test_w8a8_gpu import check, f64, gpu, lw, on_gpu, say  # noqa: F401

# rows that a thread holds one, two and four chunks of, and longer ones; whole chunks of eight values and not
ROWS = [40, 2003, 11008, 9001, 20000, 20001, 40000, 40001]
#: dx leaves fp32 by way of a power of two: below fp32's normal range half a step of 2^-149 more
HALF_LAST = 2.0 ** -150


def one_signed(rng, N, K):
    """Weights of small scales whose products add up, by far zero points to what bf16 can hold."""
    codes = rng.integers(0, 256, (N, K)).astype(np.uint8)
    scales = (np.array([1, 3, 5, 7])[rng.integers(0, 4, N)] * 2.0 ** -24).astype(np.float16)
    return codes, scales, -rng.integers(20000, 40000, N).astype(np.int32)


def tokens(rng, N):
    """A smallest normal one, random ones near 1e-38, subnormal ones, zeros, and one of ordinary size."""
    d = np.stack([np.full(N, 2.0 ** -126), rng.uniform(0.5, 4, N) * 1e-38, np.full(N, 2.0 ** -133),
                  rng.integers(1, 100, N) * 2.0 ** -133, np.zeros(N), rng.standard_normal(N), np.full(N, -2.0 ** -112)])
    return gpu(d.astype(np.float32), "bf16")


def test_the_bounds_see_lost_bits():
    """Factors rounded to fp32 as they come, without a power of two, lie outside the bounds of these tests."""
    for N in ROWS:
        rng = np.random.default_rng(N)
        codes, scales, zeros = one_signed(rng, N, 64)
        d = np.stack([np.full(N, 2.0 ** -126), np.full(N, 2.0 ** -133)])
        want = ref.linear_grad(d, codes, scales, zeros)
        bound = ref.grad_bound(want, [(d, codes, scales, zeros)], "bf16") + HALF_LAST
        a = (d * scales.astype(np.float64)).astype(np.float32).astype(np.float64)
        assert (np.abs(a @ (codes - zeros[:, None].astype(np.float64)) - want) > bound).any()


@pytest.mark.gpu
@pytest.mark.parametrize("N", ROWS)
def test_linear_grad_of_tiny_gradients(lw, N):  # noqa: F811
    K = 64
    say("tiny linear", N)
    rng = np.random.default_rng(N)
    w = one_signed(rng, N, K)
    dy = tokens(rng, N)
    want = ref.linear_grad(f64(dy), *w)
    dx = lw.linear_w8a8_grad(dy, *on_gpu(w))
    check(dx, want, ref.grad_bound(want, [(f64(dy), *w)], "bf16") + HALF_LAST, f"N={N}")
    assert bool((dx[4] == 0).all()) and bool((dx[0] > 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("N", ROWS)
def test_gated_grad_of_tiny_gradients(lw, N, act):  # noqa: F811
    """dg and du above 2^-126 (they are fp32 values), their factors below."""
    K = 64
    say("tiny gated", N, act)
    rng = np.random.default_rng([N, 1])
    wg, wu = one_signed(rng, N, K), one_signed(rng, N, K)
    T = 4
    size = np.array([2.0 ** -125, 2.0 ** -124, 0, 1])[:, None]
    # gates where value and slope are above 1/2 and without cancellation; the first token's values all alike, so
    # that lost bits do not even out over the rows
    dh, gate, up = size * rng.uniform(1, 2, (T, N)), rng.uniform(0.75, 3, (T, N)), rng.uniform(1, 3, (T, N))
    dh[0], gate[0], up[0] = size[0], 0.75, 1
    dh, gate, up = (gpu(a.astype(np.float32), "bf16") for a in (dh, gate, up))
    dg, du = ref.gated_parts(f64(dh), f64(gate), f64(up), act)
    want = ref.linear_grad(dg, *wg) + ref.linear_grad(du, *wu)
    dx, pg, pu = lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu), act=act, parts=True)
    # act's value and slope: sigma's error as in gated_bound (2q below 8: under 320 half steps), a few more steps
    few = 400 * ref.U32
    for got, v in ((pg, dg), (pu, du)):
        check(got, v, np.abs(v) * (ref.HALF_STEP["bf16"] * 1.01 + few) + ref.HALF_TINY["bf16"], "parts")
    check(dx, want, ref.grad_bound(want, [(dg, *wg), (du, *wu)], "bf16", [few, few]) + HALF_LAST, f"N={N}")
    assert bool((dx[2] == 0).all()) and bool((dx[0] > 0).all())
    assert bool((lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu), act=act) == dx).all())


@pytest.mark.gpu
def test_fp16_block_behind_closed_gates(lw):  # noqa: F811
    """fp16 gradients get this small where every gate of a token is far below zero."""
    N, K = 96, 64
    rng = np.random.default_rng(5)
    wg, wu = one_signed(rng, N, K), one_signed(rng, N, K)
    dh = gpu(np.full((2, N), 2.0 ** -14, np.float32), "fp16")
    gate = gpu(np.array([[-70.0], [-1.0]]) * np.ones((2, N)), "fp16")
    up = gpu(np.ones((2, N)), "fp16")
    dg, du = ref.gated_parts(f64(dh), f64(gate), f64(up), "silu")
    want = ref.linear_grad(dg, *wg) + ref.linear_grad(du, *wu)
    dx = lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu))
    # sigma: 20 + 20 * 2q half steps, the slope's terms each that much
    few = (20 + 20 * 70) * 2 * ref.U32
    check(dx, want, ref.grad_bound(want, [(dg, *wg), (du, *wu)], "fp16", [few, few]), "closed gates")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 100, 300])
def test_among_other_tokens(lw, T):  # noqa: F811
    """Tiny tokens between ordinary ones, in every kernel that multiplies: each as close as alone."""
    N, K = 130, 160
    say("tiny among others", T)
    rng = np.random.default_rng(T)
    w = one_signed(rng, N, K)
    d = rng.standard_normal((T, N))
    d[::3] = np.abs(d[::3]) * 1e-38
    dy = gpu(d.astype(np.float32), "bf16")
    want = ref.linear_grad(f64(dy), *w)
    check(lw.linear_w8a8_grad(dy, *on_gpu(w)), want, ref.grad_bound(want, [(f64(dy), *w)], "bf16") + HALF_LAST, f"T={T}")
