"""Workspace sizes hold for one T, N and K: they do not grow with T throughout,
a call with less than its own size is refused, and one workspace of the largest
of several sizes serves all of them."""
from __future__ import annotations

import os

import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import test_w8a8_host as host
from test_w8a8_host import lw  # noqa: F401

N, K = 4096, 4096
QUERIES = [("linear", lambda lw, T: lw.linear_w8a8_workspace_bytes(T, N, K, 0)),
           ("codes", lambda lw, T: lw.linear_w8a8_workspace_bytes(T, N, K, 2)),
           ("gated", lambda lw, T: lw.gated_w8a8_workspace_bytes(T, N, K, 0)),
           ("linear_grad", lambda lw, T: lw.linear_w8a8_grad_workspace_bytes(T, N, K)),
           ("gated_grad", lambda lw, T: lw.gated_w8a8_grad_workspace_bytes(T, N, K))]
CALLS = {"linear": lambda lw, T, size: host.linear(lw, T=T, N=N, K=K, size=size),
         "codes": lambda lw, T, size: host.linear(lw, T=T, N=N, K=K, dtype=2, xs=host.P, sums=host.P, size=size),
         "gated": lambda lw, T, size: host.gated(lw, T=T, N=N, K=K, size=size),
         "linear_grad": lambda lw, T, size: host.linear_grad(lw, T=T, N=N, K=K, size=size),
         "gated_grad": lambda lw, T, size: host.gated_grad(lw, T=T, N=N, K=K, size=size)}


@pytest.mark.parametrize("name,query", QUERIES, ids=lambda v: v if isinstance(v, str) else "")
def test_sizes_are_each_tokens_counts_own(lw, name, query):  # noqa: F811
    sizes = {T: query(lw, T) for T in range(1, 1100)}
    assert all(query(lw, T) == s for T, s in sizes.items())
    # the codes of values, or the factors, at the least
    if name in ("linear", "gated"):
        assert all(s >= T * K for T, s in sizes.items() if T > 4)
    if name.endswith("grad"):
        assert all(s >= 2 * T * N * (2 if name == "gated_grad" else 1) for T, s in sizes.items())
    # a longer call's size may be less, and is refused then
    T = max(sizes, key=sizes.get)
    if T < 1099:
        assert CALLS[name](lw, T, sizes[1099]) == host.ARG
    assert CALLS[name](lw, T, sizes[T] - 1) == host.ARG


def test_the_header_says_so(lw):  # noqa: F811
    assert lw.linear_w8a8_workspace_bytes(256, N, K, 0) > lw.linear_w8a8_workspace_bytes(1000, N, K, 0)
    text = " ".join(open(os.path.join(host.ROOT, "include", "lowbit_w8a8.h")).read().replace(" * ", " ").split())
    assert "A size holds for its T, N and K only: it does not grow with T throughout" in text
    for T, size in ((256, "17.0 MiB for 256 tokens"), (1000, "3.9 for 1000")):
        assert size in text and f"{lw.linear_w8a8_workspace_bytes(T, N, K, 0) / 2 ** 20:.1f}" == size.split()[0]


@pytest.mark.gpu
def test_one_workspace_of_the_largest_size_serves_all(lw):  # noqa: F811
    """Calls of many token counts in turn, each with what the others left in their one workspace."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from test_w8a8_gpu import random_weights
    n, k = 1000, 2048
    counts = [300, 5, 64, 1, 700, 130, 33]
    g = torch.Generator(device="cuda").manual_seed(0)
    wg, wu = random_weights(g, n, k), random_weights(g, n, k)
    need = max(max(lw.linear_w8a8_workspace_bytes(T, n, k, 0), lw.gated_w8a8_workspace_bytes(T, n, k, 0),
                   lw.linear_w8a8_grad_workspace_bytes(T, n, k), lw.gated_w8a8_grad_workspace_bytes(T, n, k))
               for T in counts)
    ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    at, st = ws.data_ptr(), torch.cuda.current_stream().cuda_stream
    assert at % 256 == 0

    def p(w):
        return tuple(t.data_ptr() for t in w)

    for T in counts:
        print("[w8a8] one workspace", T, flush=True)
        x = torch.randn(T, k, generator=g, device="cuda").half()
        y, h, gate, up = (torch.empty(T, n, dtype=torch.float16, device="cuda") for _ in range(4))
        dx, dx2 = (torch.empty(T, k, dtype=torch.float16, device="cuda") for _ in range(2))
        assert lw.linear_w8a8_raw(x.data_ptr(), 0, None, None, T, *p(wg), n, k, y.data_ptr(), 0, at, need, st) == 0
        assert lw.gated_w8a8_raw(x.data_ptr(), 0, None, None, T, *p(wg), *p(wu), n, k, 0, h.data_ptr(),
                                 gate.data_ptr(), up.data_ptr(), 0, at, need, st) == 0
        assert lw.linear_w8a8_grad_raw(y.data_ptr(), 0, T, *p(wg), n, k, dx.data_ptr(), at, need, st) == 0
        assert lw.gated_w8a8_grad_raw(h.data_ptr(), gate.data_ptr(), up.data_ptr(), 0, T, *p(wg), *p(wu), n, k, 0,
                                      dx2.data_ptr(), None, None, at, need, st) == 0
        assert bool((y == lw.linear_w8a8(x, *wg)).all())
        assert bool((h == lw.gated_w8a8(x, *wg, *wu)).all())
        assert bool((dx == lw.linear_w8a8_grad(y, *wg)).all())
        assert bool((dx2 == lw.gated_w8a8_grad(h, gate, up, *wg, *wu)).all())
    assert bool((ws[need:] == 0xA5).all())
