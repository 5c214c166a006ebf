"""The AdamW step where eps is near 0: gradients whose second moments lie below fp32's normal range, and
none at all.  The update is the definition in 64 bits from the moments in 32, with no least second
moment: lr / (1 - beta1^t) * m' / (sqrt(v') / sqrt(1 - beta2^t) + fl32(eps)), and no step where that
denominator is 0."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import adapters_reference as ref

LR, BETAS = 1e-3, (0.9, 0.999)


@pytest.fixture(scope="module")
def lw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_bit_rtn_amd as lw
    if not os.path.exists(lw.LIB_PATH):
        from weight_only_bit_rtn_amd import build
        build.build()
    lw.load_library()
    return lw


def defined_step(m, v, eps, step):
    """What p loses, float64, from fp32 moments."""
    m, v = m.astype(np.float64), v.astype(np.float64)
    under = np.sqrt(v) / np.sqrt(1 - BETAS[1] ** step) + float(np.float32(eps))
    with np.errstate(all="ignore"):
        taken = LR / (1 - BETAS[0] ** step) * m / under
    return np.where(under == 0, m * 0, taken)


def test_the_definition_by_hand():
    """The first step is lr in the gradient's direction, however small the gradient; no gradient, no step."""
    for g in (2.0, 1e-3, 1e-18, 1e-19, 3e-22):
        m, v = ref.moments(np.zeros(1, np.float32), np.zeros(1, np.float32), np.array([g]), *BETAS)
        # v' is c2 g^2 rounded to fp32's subnormals, steps of 2^-149
        off = 2.0 ** -20 + 2.0 ** -149 / max(1e-3 * g * g, 2.0 ** -149)
        assert v[0] == 0 or abs(defined_step(m, v, 0.0, 1)[0] / LR - 1) < off
    zero = np.zeros(1, np.float32)
    assert defined_step(zero, zero, 0.0, 1)[0] == 0
    m, v = ref.moments(zero, zero, np.array([1e-18]), *BETAS)
    assert 0.98 * LR < defined_step(m, v, 1e-20, 1)[0] < LR


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-30, 1e-20, 1e-12, 1e-8])
def test_small_gradients(lw, bits, eps):
    print(f"[adamw] eps {eps} {bits} bits", flush=True)
    rng = np.random.default_rng(7)
    n = 1000
    # from none at all over squares that are 0 or subnormal in fp32 to ordinary ones, both signs, next to each other
    g = (10.0 ** rng.uniform(-24, -2, n) * rng.choice([-1, 1], n)).astype(np.float32)
    g[rng.random(n) < 0.1] = 0
    g[512:768] = rng.standard_normal(256) * 1e-19   # a block of subnormal second moments alone
    p = torch.zeros(n, device="cuda")
    state = lw.adamw_state([p], bits=bits)
    m, v = np.zeros(1024, np.float32), np.zeros(1024, np.float32)
    wide = np.zeros(1024, np.float32)
    wide[:n] = g
    for step in (1, 2):
        m, v = ref.moments(m, v, wide, *BETAS)
        had = p.cpu().numpy().astype(np.float64)
        lw.adamw([p], [torch.from_numpy(g).cuda()], state, lr=LR, betas=BETAS, eps=eps, weight_decay=0.0, step=step)
        taken = defined_step(m, v, eps, step)[:n]
        want = had - taken
        # 2^-21 of the step, and the sum of step and p rounded once
        far = 2.0 ** -21 * np.abs(taken) + 2.0 ** -24 * (np.abs(want) + np.abs(taken)) + 2.0 ** -149
        got = p.cpu().numpy().astype(np.float64)
        fits = np.abs(want) < 3.4e38
        assert np.isfinite(got[fits]).all()
        assert (np.abs(got - want) <= far)[fits].all()
        assert (np.abs(got[~fits]) >= 3.4e38).all()
        p.copy_(torch.where(p.isfinite(), p, torch.zeros_like(p)))
        if bits == 8:
            codes_m, top_m = ref.encode(m, 7)
            codes_v, top_v = ref.encode(v, 8)
            m, v = ref.decode(codes_m, codes_v, top_m, top_v)
    # what the last block has beyond the tensor is zero
    assert not state["m"][n:].any() and not state["v"][n:].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_no_gradient_and_no_eps(lw, kind):
    """0 / 0: nothing but the decay happens, and nothing becomes a NaN."""
    for bits in (8, 32):
        p = torch.full((300,), 1.5, dtype=kind, device="cuda")
        state = lw.adamw_state([p], bits=bits, master=kind is not torch.float32)
        for step in (1, 2):
            lw.adamw([p], [torch.zeros_like(p)], state, lr=0.5, eps=0.0, weight_decay=0.0, step=step)
        assert (p == 1.5).all() and not state["m"].any() and not state["v"].any()


@pytest.mark.gpu
def test_a_moment_that_is_no_number_stays_one(lw):
    p = torch.ones(256, device="cuda")
    state = lw.adamw_state([p], bits=32)
    state["m"][3], state["v"][4], state["m"][5] = float("nan"), float("nan"), float("inf")
    lw.adamw([p], [torch.zeros_like(p)], state, lr=0.5, eps=0.0, weight_decay=0.0, step=1)
    assert not p[3:6].isfinite().any() and p.isfinite().sum() == 253
