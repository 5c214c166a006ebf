"""Tensors that a caller gives the adapter calls to write into are marked as changed: a recorded operation
that saved one refuses its backward pass, and none goes on with overwritten values.  Under
torch.inference_mode(), where tensors have no versions, the calls write as elsewhere."""
from __future__ import annotations

import os

import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

pytestmark = pytest.mark.gpu

T, N, K, R, L = 40, 72, 64, 16, 2


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


def inputs(lw):
    print("[adapters] versions", flush=True)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").half()

    ids = (torch.arange(T, device="cuda") % 3 - 1).int()
    return normal(T, K), normal(L, R, K), normal(L, N, R), torch.ones(L, device="cuda"), ids, normal(T, N)


def saved(shape):
    """A tensor that a recorded operation saved, and that operation's output."""
    t = torch.ones(shape, dtype=torch.float16, device="cuda", requires_grad=True) * 2
    return t, (t * t).sum()


def refused(loss):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("in_place", [True, False])
def test_forward(lw, in_place):
    x, a, b, s, ids, y = inputs(lw)
    plan = lw.lora_plan(ids, L)
    out, loss = saved((T, N))
    with torch.no_grad():
        lw.lora(x, a, b, s, plan, y=out if in_place else y, out=out)
    refused(loss)


@pytest.mark.parametrize("in_place", [True, False])
def test_backward(lw, in_place):
    x, a, b, s, ids, dy = inputs(lw)
    plan = lw.lora_plan(ids, L)
    _, v = lw.lora(x, a, b, s, plan, save=True)
    out, loss = saved((T, K))
    with torch.no_grad():
        lw.lora_grad(dy, x, v, a, b, s, plan, dx=out if in_place else torch.zeros_like(x), out=out)
    refused(loss)


def test_plan(lw):
    ids = inputs(lw)[4]
    plan = lw.lora_plan(ids, L)
    for name, n in (("order", T), ("starts", T + 1)):
        w = torch.ones(n, 4, device="cuda", requires_grad=True)
        loss = (w.index_select(0, plan[name]) ** 2).sum()
        assert lw.lora_plan(ids, L, out=plan)[name] is plan[name]
        refused(loss)


def test_only_what_is_written(lw):
    """Inputs, and outputs that the calls make themselves, keep their versions."""
    x, a, b, s, ids, y = inputs(lw)
    plan = lw.lora_plan(ids, L)
    out, v = lw.lora(x, a, b, s, plan, y=y, save=True)
    into = torch.empty_like(y)
    lw.lora(x, a, b, s, plan, y=y, out=into)
    lw.lora_grad(y, x, v, a, b, s, plan, dx=x.clone(), out=torch.empty_like(x))
    assert [t._version for t in (x, a, b, s, ids, y, v, out, plan["order"], plan["starts"])] == [0] * 10
    assert into._version == 1


def test_inference_mode(lw):
    x, a, b, s, ids, y = inputs(lw)
    plan = lw.lora_plan(ids, L)
    out, v = lw.lora(x, a, b, s, plan, y=y, save=True)
    dx = lw.lora_grad(y, x, v, a, b, s, plan, dx=x)[0]
    with torch.inference_mode():
        plan = lw.lora_plan(ids, L, out={k: t.clone() for k, t in plan.items()})
        mine, base = y.clone(), x.clone()
        lw.lora(x, a, b, s, plan, y=mine, out=mine)
        lw.lora_grad(y, x, v, a, b, s, plan, dx=base, out=base)
        params = [a.clone(), b.clone()]
        lw.adamw(params, [a, b], lw.adamw_state(params), lr=1e-2)
    assert torch.equal(mine, out) and torch.equal(base, dx) and not torch.equal(params[0], a)
