"""The 8-bit activation calls are outside autograd: where gradients are
recorded they refuse a tensor that requires grad, whose gradient would end
there without a word; in an autograd function they take part in a backward
pass."""
from __future__ import annotations

import pytest

import w8a8_reference as ref


@pytest.fixture(scope="module")
def lw():
    import weight_only_bit_rtn_amd as lw
    return lw


def tensors(device, T=3, N=8, K=64):
    import torch
    g = torch.Generator().manual_seed(0)
    w = (torch.randint(0, 256, (N, K), generator=g, dtype=torch.uint8).view(torch.int32),
         (torch.rand(N, 1, generator=g) * 1e-3 + 1e-3).half(), torch.randint(100, 156, (N, 1), generator=g).int())
    x, d, gate, up = (torch.randn(s, generator=g).half() for s in ((T, K), (T, N), (T, N), (T, N)))
    return [t.to(device) for t in w], *(t.to(device) for t in (x, d, gate, up))


def calls(lw, device):
    """(what requires grad, the call) of every tensor that a gradient could be wanted of."""
    w, x, d, gate, up = tensors(device)
    grad = lambda t: t.clone().requires_grad_()
    ws = [w[0], grad(w[1]), w[2]]
    q = {"codes": x.char(), "scales": x[:, 0].float().contiguous(), "sums": x[:, 0].int().contiguous()}
    yield "x", lambda: lw.quantize_act(grad(x))
    yield "x", lambda: lw.linear_w8a8(grad(x), *w)
    yield "scales", lambda: lw.linear_w8a8(x, *ws)
    yield "scales of x", lambda: lw.linear_w8a8({**q, "scales": grad(q["scales"])}, *w)
    yield "out", lambda: lw.linear_w8a8(x, *w, out=grad(d))
    yield "x", lambda: lw.gated_w8a8(grad(x), *w, *w)
    yield "scales", lambda: lw.gated_w8a8(x, *w, *ws)
    yield "dy", lambda: lw.linear_w8a8_grad(grad(d), *w)
    yield "dh", lambda: lw.gated_w8a8_grad(grad(d), gate, up, *w, *w)
    yield "gate", lambda: lw.gated_w8a8_grad(d, grad(gate), up, *w, *w)
    yield "up", lambda: lw.gated_w8a8_grad(d, gate, grad(up), *w, *w)


def refused(lw, device, name, call):
    import torch
    with pytest.raises(ValueError, match=f"^{name} requires grad"):
        call()


def test_a_lost_gradient_is_refused(lw):
    """On the host's tensors: what requires grad is refused as such where it is the first tensor of its call,
    and a call without it, or under no_grad, is refused for its place only."""
    import torch
    for name, call in calls(lw, "cpu"):
        if name in ("x", "dy", "dh"):
            refused(lw, "cpu", name, call)
        with torch.no_grad(), pytest.raises(ValueError, match="must live on the GPU"):
            call()


@pytest.mark.gpu
def test_a_lost_gradient_is_refused_on_the_gpu(lw):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    for name, call in calls(lw, "cuda:0"):
        refused(lw, "cuda:0", name, call)
        with torch.no_grad():
            call()


@pytest.mark.gpu
def test_in_an_autograd_function(lw):
    """y = x + linear(x) with the calls in a function's forward and backward: both terms of the gradient."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    w, x, *_ = tensors("cuda:0", T=5, N=64)

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return lw.linear_w8a8(x, *w)

        @staticmethod
        def backward(ctx, dy):
            return lw.linear_w8a8_grad(dy.contiguous(), *w)

    leaf = x.clone().requires_grad_()
    dy = torch.randn(5, 64, generator=torch.Generator().manual_seed(1)).half().cuda()
    (leaf + Linear.apply(leaf)).backward(dy)
    codes, scales, zeros = (t.cpu().numpy() for t in w)
    codes = codes.view("uint8").reshape(64, 64)
    d = dy.double().cpu().numpy()
    want = ref.linear_grad(d, codes, scales, zeros)
    bound = ref.grad_bound(want, [(d, codes, scales, zeros)], "fp16")
    total = d + want
    # the sum of the two terms is rounded once more
    off = abs(leaf.grad.double().cpu().numpy() - total)
    assert (off <= bound + (abs(total) + bound) * ref.HALF_STEP["fp16"] + ref.HALF_TINY["fp16"]).all()
