"""One to four tokens at the longest rows that the product's kernel quantizes
itself (T K = 16384) and the shortest that it does not: bit for bit the
definition's values, and what codes handed over give."""
from __future__ import annotations

import numpy as np
import pytest

import w8a8_reference as ref
from test_w8a8_gpu import activations, gpu, lw, on_gpu, say, types, weights  # noqa: F401

pytestmark = pytest.mark.gpu


def value(a, s, w, kind):
    """fl32(fl32(S s) d), rounded to the output type: d is an exact integer."""
    import torch
    codes, scales, zeros = w
    d = a.astype(np.float64) @ (codes.astype(np.float64) - zeros[:, None]).T
    y = (s[:, None] * scales.astype(np.float32)[None]).astype(np.float32) * d.astype(np.float32)
    return torch.from_numpy(y.astype(np.float32)).to(types()[kind]).cuda()


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,K", [(1, 32), (1, 992), (1, 1024), (1, 15392), (1, 16384), (1, 16416), (2, 64), (2, 7200),
                                 (2, 8192), (2, 8224), (3, 1056), (3, 5152), (3, 5440), (3, 5472), (4, 3104), (4, 4096),
                                 (4, 4128)])
def test_rows_around_the_fused_quantizer(lw, T, K, kind):  # noqa: F811
    say("few", T, K, kind)
    rng = np.random.default_rng([T, K])
    for N in (1, 7, 5000):
        wg, wu = weights(rng, N, K, "minmax"), weights(rng, N, K, "sym")
        x = activations(rng, T, K, kind)
        a, s, _ = ref.quantize_act(x.float().cpu().numpy())
        y = lw.linear_w8a8(x, *on_gpu(wg))
        assert bool((y == value(a, s, wg, kind)).all()), f"linear {N}"
        h, gate, up = lw.gated_w8a8(x, *on_gpu(wg), *on_gpu(wu), save=True)
        assert bool((gate == value(a, s, wg, kind)).all()) and bool((up == value(a, s, wu, kind)).all()), f"gated {N}"
        q = lw.quantize_act(x)
        assert bool((lw.linear_w8a8(q, *on_gpu(wg), out_dtype=x.dtype) == y).all())
        again = lw.gated_w8a8(q, *on_gpu(wg), *on_gpu(wu), out_dtype=x.dtype)
        assert bool((again == h).all())
