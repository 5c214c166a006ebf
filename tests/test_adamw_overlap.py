"""Memory that an AdamW step writes (parameters, moments, their maxima, the fp32 copy) is shared with nothing
else that the step reads or writes, whatever the offset: refused on the host before anything is
launched.  Gradients are read only, and may share memory with one another."""
from __future__ import annotations

import os
import random

import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import test_adapters_host as host

GAP = 1 << 20  # far more than any of these tensors


@pytest.fixture(scope="module")
def lw():
    import weight_only_bit_rtn_amd as lw
    if not os.path.exists(lw.LIB_PATH):
        from weight_only_bit_rtn_amd import build
        build.build()
    lw.load_library()
    return lw


def places(count):
    """Addresses far apart, never dereferenced: each call here is refused."""
    return [host.P + i * GAP for i in range(count)]


P0, G0, P1, G1, M, V, MM, VM, MASTER, AT = places(10)
N = 1000                 # fp32: 4000 bytes, four blocks of moments
STATE = dict(m=M, v=V, m_max=MM, v_max=VM)
PAIRS = ((P0, G0, N), (P1, G1, N))

SHARED = (
    # a parameter twice, or a part of it, from either side and inside
    [dict(tensors=((P0, G0, N), (P0 + d, G1, N))) for d in (0, 16, 3984)]
    + [dict(tensors=((P0 + d, G0, N), (P0, G1, N))) for d in (16, 3984)]
    + [dict(tensors=((P0, G0, N), (P0 + 160, G1, 4))), dict(tensors=((P0 + 160, G0, 4), (P0, G1, N)))]
    # a gradient that is a parameter, its own or another one's, or a part of one
    + [dict(tensors=((P0, P0 + d, N),)) for d in (0, 16, -16, 3984, -3984)]
    + [dict(tensors=((P0, G0, N), (P1, P0 + 320, 8)))]
    # moments, maxima and copy against parameters, gradients and each other
    + [dict(tensors=PAIRS, **{**STATE, k: at}) for k in STATE for at in (P0, P1 + 3984, G1, G0 - 16 if k in ("m", "v") else G0)]
    + [dict(tensors=PAIRS, **STATE, master=at) for at in (P0, P1 + 3984, G1, G0 - 16, M, V + 2032, MM, VM + 16)]
    + [dict(tensors=PAIRS, **{**STATE, "v": at}) for at in (M, M + 2032, M - 2032)]
    + [dict(tensors=PAIRS, **{**STATE, "v_max": at}) for at in (MM, MM + 16, M, V + 16)]
    + [dict(tensors=PAIRS, bits=32, m=M, v=M + 8176, m_max=None, v_max=None)]
    # the step's own scalars
    + [dict(tensors=PAIRS, **STATE, **{k: at}) for k in ("lr_at", "step_at", "scale_at") for at in (P0 + 3996, M + 2044, MM)])


@pytest.mark.parametrize("args", SHARED)
def test_shared_memory_is_refused(lw, args):
    args = {**STATE, **args}
    assert host.adamw(lw, **args) == host.ARG


# what test_adapters_host refuses with one address in every place, each with memory of its own
ALONE = (
    [dict(lr=-1e-3), dict(eps=host.NAN), dict(decay=host.INF), dict(beta1=1.0), dict(step=0), dict(master=MASTER + 2),
     dict(lr_at=AT + 1), dict(m=None), dict(v=M + 2), dict(m_max=None), dict(v_max=VM + 4), dict(bits=32)]
    + [dict(tensors=((P0, G0, 5), t)) for t in ((None, G1, 3), (P1, None, 3), (P1 + 2, G1, 3), (P1, G1 + 8, 3), (P1, G1, -1))])


@pytest.mark.parametrize("args", ALONE)
def test_other_refusals_are_not_that_one(lw, args):
    assert host.adamw(lw, **{**STATE, "tensors": PAIRS, **args}) == host.ARG


def test_one_pair_among_many_is_found(lw):
    """Hundreds of tensors in any order of addresses, one of them shared."""
    rng = random.Random(0)
    for count in (3, 100, 128, 129, 1000):
        at = places(2 * count + 4)
        rng.shuffle(at)
        rest = dict(zip(STATE, at[2 * count:]))
        tensors = [(at[2 * i], at[2 * i + 1], rng.randrange(1, 5000)) for i in range(count)]
        a, b = rng.sample(range(count), 2)
        last = (tensors[a][2] * 4 - 1) // 16 * 16
        for shared in ((tensors[a][0] + last, tensors[b][1], tensors[b][2]), (tensors[b][0], tensors[a][0] + last, tensors[b][2])):
            assert host.adamw(lw, tensors=[shared if i == b else t for i, t in enumerate(tensors)], **rest) == host.ARG


def test_tensors_of_no_values_share_nothing(lw):
    """They have no memory: the call gets as far as the refusal of what it is given besides."""
    assert host.adamw(lw, tensors=((P0, G0, 0), (P0, G0, 0)), **STATE) == 0


@pytest.mark.gpu
def test_refused_by_the_binding(lw):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    flat = torch.ones(4096, device="cuda")
    g = torch.ones(512, device="cuda")
    p = [flat[:512], flat[512:1024]]
    with torch.no_grad():
        state = lw.adamw_state(p)
        wide = lw.adamw_state(p, bits=32)
    before = flat.clone()
    for params, grads, s in (([flat[:512], flat[256:768]], [g, g], state), ([flat[256:768], flat[:512]], [g, g], state),
                             (p, [g, flat[:512]], state), (p, [flat[508:1020], g], state), (p, [flat[512:1024], g], state),
                             (p, [g, g], {**state, "v": state["m"]}), (p, [g, g], {**state, "v_max": state["m_max"]}),
                             (p, [g, g], {**state, "master": flat[:1024]}), (p, [g, g], {**wide, "m": flat[1020:2044]}),
                             ([flat[512 * (i % 70 % 8):][:512] for i in range(80)], [g] * 80, lw.adamw_state([g] * 80))):
        with pytest.raises(ValueError, match="share memory"):
            lw.adamw(params, grads, s, lr=0.5)
    torch.cuda.synchronize()
    assert torch.equal(flat, before) and not state["m"].any() and not wide["m"].any()


@pytest.mark.gpu
def test_neighbours_and_shared_gradients_are_fine(lw):
    """Tensors side by side in one buffer, one gradient for several of them: as apart."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for count in (2, 100):
        flat = torch.ones(256 * count, device="cuda")
        g = torch.linspace(-1, 1, 512, device="cuda")
        p = [flat[256 * i:256 * i + 256] for i in reversed(range(count))]
        q = [t.clone() for t in p]
        grads = [g[4 * (i % 64):][:256] for i in range(count)]
        s, t = lw.adamw_state(p), lw.adamw_state(q)
        lw.adamw(p, grads, s, lr=0.5)
        lw.adamw(q, [x.clone() for x in grads], t, lr=0.5)
        assert all(torch.equal(a, b) for a, b in zip((*p, *s.values()), (*q, *t.values())))
