"""The 8-bit activation operators on the GPU against their definition in 64
bits (tests/w8a8_reference.py): per-token quantization, the linear product,
the gated block and their input gradients.

Codes, scales and sums are bit-exact; products and gradients lie within the
roundings that their definitions name (see the bounds of w8a8_reference).
"""
from __future__ import annotations

import numpy as np
import pytest

import w8a8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lw():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import weight_only_bit_rtn_amd as lw
    lw.load_library()
    return lw


def say(*a):
    print("[w8a8]", *a, flush=True)


def types():
    import torch
    return {"fp16": torch.float16, "bf16": torch.bfloat16}


def gpu(a, kind=None):
    """A numpy array on the GPU; with ``kind``, float values rounded to that type."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")
    return t if kind is None else t.to(types()[kind])


def f64(t):
    return t.double().cpu().numpy()


def weights(rng, N, K, grid):
    """codes uint8 [N][K], scales fp16 [N], zeros int32 [N]: what the quantizers produce."""
    if grid == "sym":
        codes = rng.integers(1, 256, (N, K))
        zeros = np.full(N, 128)
    else:
        codes = rng.integers(0, 256, (N, K))
        zeros = rng.integers(0, 256, N)
        if grid == "far":      # one-signed rows: zero points far outside the codes, some at the fp16 extremes
            zeros = np.where(np.arange(N) % 3 == 0, zeros, rng.integers(-522240, 522241, N))
    # far zero points with small scales, as such rows have them: (code - zero) * scale stays below one
    scales = (rng.uniform(0.5, 2, N) * (1e-6 if grid == "far" else 2e-4)).astype(np.float16)
    return codes.astype(np.uint8), scales, zeros.astype(np.int32)


def on_gpu(w):
    codes, scales, zeros = w
    N = codes.shape[0]
    packed = codes.view(np.int32) if N else np.empty((0, codes.shape[1] // 4), np.int32)
    return gpu(packed), gpu(scales.reshape(N, 1)), gpu(zeros.reshape(N, 1))


def check(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        at = np.argwhere(bad)[:4]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; " + ", ".join(
            f"{tuple(i)}: {got[tuple(i)]!r} want {want[tuple(i)]!r} +- {bound[tuple(i)]:.3g}" for i in at))


def activations(rng, T, K, kind):
    x = rng.standard_normal((T, K)) * np.exp(rng.uniform(-6, 3, (T, 1)))
    x[:, rng.integers(0, K, max(1, K // 100))] *= 10
    return gpu(x.astype(np.float32), kind)


# ---------------------------------------------------------------------------
# quantize_act
# ---------------------------------------------------------------------------
def check_codes(lw, x, what):
    want = ref.quantize_act(x.float().cpu().numpy())
    q = lw.quantize_act(x)
    for name, w in zip(("codes", "scales", "sums"), want):
        got = q[name].cpu().numpy()
        assert got.shape == w.shape and got.dtype == w.dtype, (what, name)
        if name == "scales":
            assert np.array_equal(got.view(np.uint32)[np.isfinite(w)], w.view(np.uint32)[np.isfinite(w)]), what
            assert np.array_equal(np.isnan(got), np.isnan(w)), what
        else:
            assert np.array_equal(got, w), f"{what}: {name} differ at {np.argwhere(got != w)[:5].tolist()}"


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("K", [32, 64, 96, 512, 544, 1024, 1056, 4096, 11008, 16384, 16416, 32768, 32800, 131072])
def test_quantize_act(lw, K, kind):
    say("quantize", K, kind)
    rng = np.random.default_rng(K)
    for T in (1, 3, 70):
        if T * K <= 1 << 22:
            check_codes(lw, activations(rng, T, K, kind), f"{T}x{K} {kind}")


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_quantize_act_edges(lw, kind):
    import torch
    K = 256
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, K)).astype(np.float32)
    x[0] = 0
    x[1] = -3
    x[2] = 0
    x[2, 77] = 6e-8 if kind == "fp16" else 1e-40            # one subnormal
    x[3] *= 1e-7 if kind == "fp16" else 1e-39
    x[4] *= 1e4 if kind == "fp16" else 1e38
    x[5, 9] = np.inf
    x[6, 255] = -np.inf
    x[7, 0] = np.nan
    x[8] = np.arange(K) - 127                                # maximum 127 + 1: all kinds of halves
    x[9] = (np.arange(K) - 128) / 2
    x[10, :] = np.where(np.arange(K) % 2, 127, np.arange(K) / 2 - 60)  # scale 1: exact ties
    x[11] = -x[10]
    x[12, :] = 65504 if kind == "fp16" else 3.3e38
    say("quantize edges", kind)
    check_codes(lw, gpu(x, kind), kind)
    # every finite positive value of the type as an element under several maxima
    bits = torch.arange(0, 0x7c00 if kind == "fp16" else 0x7f80, dtype=torch.int32).to(torch.int16)
    v = bits.view(types()[kind])
    n = v.numel() // 32 * 32
    for top in (1.0, 127.0, 381.0, 0.0999, 3.17e-3):
        row = torch.where(v[:n].float() <= top, v[:n].float(), torch.tensor(top)).to(types()[kind])
        check_codes(lw, row.reshape(1, n).cuda(), f"{kind} all values to {top}")


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------
SHAPES = [(1, 1, 32), (1, 256, 256), (1, 515, 1056), (2, 3, 64), (3, 64, 96), (5, 33, 4128), (8, 130, 512),
          (15, 100, 160), (16, 16, 128), (17, 127, 288), (31, 272, 2048), (33, 65, 1024), (63, 257, 192),
          (64, 128, 256), (65, 129, 224), (100, 1000, 512), (127, 63, 128), (129, 300, 416), (200, 64, 4096),
          (257, 130, 160), (300, 515, 352), (513, 257, 288), (600, 1030, 96), (1025, 511, 640)]


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(lw, shape, kind):
    T, N, K = shape
    for grid in ("sym", "minmax", "far"):
        say("linear", shape, kind, grid)
        rng = np.random.default_rng([T, N, K])
        w = weights(rng, N, K, grid)
        x = activations(rng, T, K, kind)
        a, s, _ = ref.quantize_act(x.float().cpu().numpy())
        want = ref.product(a, s, *w)
        y = lw.linear_w8a8(x, *on_gpu(w))
        assert y.dtype == x.dtype
        check(y, want, ref.linear_bound(want, kind), f"linear {shape} {kind} {grid}")
        # codes handed over: the same bits
        q = lw.quantize_act(x)
        y2 = lw.linear_w8a8(q, *on_gpu(w), out_dtype=x.dtype)
        assert bool((y2 == y).all()), f"codes and values differ at {shape}"


@pytest.mark.parametrize("T", [1, 3, 20, 70, 600])
def test_linear_longest_rows(lw, T):
    """K at its limit with the largest codes: the integer sums come near 2^31."""
    K, N = lw.W8A8_MAX_K, 5
    say("longest rows", T)
    codes = np.empty((N, K), np.uint8)
    codes[0] = 0
    codes[1] = 255
    codes[2:] = np.random.default_rng(0).integers(0, 256, (N - 2, K))
    w = codes, np.full(N, 1e-6, np.float16), np.array([128, 128, 0, 255, -522240], np.int32)
    x = np.ones((T, K), np.float32)
    x[T // 2:] *= -1
    x = gpu(x, "bf16")
    a, s, _ = ref.quantize_act(x.float().cpu().numpy())
    want = ref.product(a, s, *w)
    check(lw.linear_w8a8(x, *on_gpu(w)), want, ref.linear_bound(want, "bf16"), f"T={T}")


@pytest.mark.parametrize("T", [1, 9, 40, 100, 520])
def test_linear_rows_apart(lw, T):
    """Zero tokens give zeros, tokens with an infinity or a NaN give NaN, and neither touches other tokens."""
    N, K = 70, 320
    rng = np.random.default_rng(T)
    w = weights(rng, N, K, "minmax")
    x = activations(rng, T, K, "fp16")
    clean = lw.linear_w8a8(x, *on_gpu(w))
    bad = x.clone()
    bad[0, 3] = float("inf")
    if T > 4:
        bad[T // 2, K - 1] = float("nan")
        bad[T - 1] = 0
    say("rows apart", T)
    y = lw.linear_w8a8(bad, *on_gpu(w))
    assert bool(y[0].isnan().all())
    if T > 4:
        assert bool(y[T // 2].isnan().all()) and bool((y[T - 1] == 0).all())
        keep = [t for t in range(1, T - 1) if t != T // 2]
        assert bool((y[keep] == clean[keep]).all())


def test_linear_of_the_quantizers_codes(lw):
    """quantize_rtn's packed words, scales and zeros go in as they come."""
    rng = np.random.default_rng(3)
    N, K, T = 300, 544, 70
    for sym in (False, True):
        wf = (rng.standard_normal((N, K)) * 0.02).astype(np.float16)
        wf[5] = 0.25          # constant rows
        wf[6] = 0
        q = lw.quantize_rtn(gpu(wf), 8, 0, symmetric=sym)
        x = activations(rng, T, K, "fp16")
        a, s, _ = ref.quantize_act(x.float().cpu().numpy())
        want = ref.product(a, s, q["codes"].cpu().numpy(), q["scales"].cpu().numpy()[:, 0],
                           q["zeros"].cpu().numpy()[:, 0])
        y = lw.linear_w8a8(x, q["packed"], q["scales"], q["zeros"])
        check(y, want, ref.linear_bound(want, "fp16"), f"sym={sym}")


# ---------------------------------------------------------------------------
# gated
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated(lw, shape, kind):
    T, N, K = shape
    for grid, act in (("sym", "silu"), ("minmax", "gelu_tanh"), ("far", "silu")):
        say("gated", shape, kind, grid, act)
        rng = np.random.default_rng([T, N, K, 1])
        wg, wu = weights(rng, N, K, grid), weights(rng, N, K, grid)
        x = activations(rng, T, K, kind)
        a, s, _ = ref.quantize_act(x.float().cpu().numpy())
        g, u = ref.product(a, s, *wg), ref.product(a, s, *wu)
        want = ref.act_value(g, act) * u
        top = 65504.0 if kind == "fp16" else 3.3e38
        h, hg, hu = lw.gated_w8a8(x, *on_gpu(wg), *on_gpu(wu), act=act, save=True)
        fits = np.abs(want) < top
        got = np.where(fits, f64(h), 0)
        bound = ref.gated_bound(want, g, kind, act)
        assert (np.abs(got - np.where(fits, want, 0)) <= bound).all(), f"h {shape} {kind} {grid} {act}"
        check(hg, g, ref.linear_bound(g, kind), "gate")
        check(hu, u, ref.linear_bound(u, kind), "up")
        alone = lw.gated_w8a8(x, *on_gpu(wg), *on_gpu(wu), act=act)
        assert bool(((alone == h) | (alone.isnan() & h.isnan())).all())


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def norm_of(d):
    return float(np.sqrt((d * d).sum()))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_grad(lw, shape, kind):
    T, N, K = shape
    for grid in ("sym", "minmax", "far"):
        say("linear grad", shape, kind, grid)
        rng = np.random.default_rng([T, N, K, 2])
        w = weights(rng, N, K, grid)
        size = np.exp(rng.uniform(-4, 2, (T, 1)))
        dy = gpu((rng.standard_normal((T, N)) * size * 0.05).astype(np.float32), kind)
        want = ref.linear_grad(f64(dy), *w)
        dx = lw.linear_w8a8_grad(dy, *on_gpu(w))
        assert dx.dtype == dy.dtype
        check(dx, want, ref.grad_bound(want, [(f64(dy), *w)], kind), f"{shape} {kind} {grid}")
        if grid == "sym" and N >= 64:
            # independent roundings: half a step is their largest, not their common size
            assert norm_of(f64(dx) - want) <= norm_of(want) * (2.0 ** -11 + ref.HALF_STEP[kind])


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_grad(lw, shape, kind):
    T, N, K = shape
    for grid, act in (("sym", "gelu_tanh"), ("minmax", "silu")):
        say("gated grad", shape, kind, grid, act)
        rng = np.random.default_rng([T, N, K, 3])
        wg, wu = weights(rng, N, K, grid), weights(rng, N, K, grid)
        dh = gpu((rng.standard_normal((T, N)) * 0.05).astype(np.float32), kind)
        gate = gpu((rng.standard_normal((T, N)) * 2).astype(np.float32), kind)
        up = gpu(rng.standard_normal((T, N)).astype(np.float32), kind)
        dg, du = ref.gated_parts(f64(dh), f64(gate), f64(up), act)
        want = ref.linear_grad(dg, *wg) + ref.linear_grad(du, *wu)
        dx, pg, pu = lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu), act=act, parts=True)
        # sigma as in gated_bound; the slope is a difference of terms, each with such an error
        g = f64(gate)
        q = np.abs(ref.two_q(g, act))
        r = (24 + 24 * q) * ref.U32
        s = 1 / (1 + np.exp(-ref.two_q(g, act)))
        rise = np.abs(ref.act_slope(g, act) - s)
        slope_err = (s + rise) * r
        ag, au = np.abs(f64(dh) * f64(up)) * slope_err, np.abs(du) * r
        check(pg, dg, np.abs(dg) * ref.HALF_STEP[kind] * 1.01 + 2 * ag + ref.HALF_TINY[kind], "dgate")
        check(pu, du, np.abs(du) * ref.HALF_STEP[kind] * 1.01 + 2 * au + ref.HALF_TINY[kind], "dup")
        bound = ref.grad_bound(want, [(dg, *wg), (du, *wu)], kind)
        for e, w in ((ag, wg), (au, wu)):
            size = np.abs(w[0].astype(np.float64) - 128) + np.abs(128.0 - w[2].reshape(-1, 1))
            bound += (2 * e * w[1].astype(np.float64)) @ size
        check(dx, want, bound, f"{shape} {kind} {grid} {act}")
        if grid == "sym" and N >= 64:
            assert norm_of(f64(dx) - want) <= norm_of(want) * (2.0 ** -11 + ref.HALF_STEP[kind])
        alone = lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu), act=act)
        assert bool((alone == dx).all())


@pytest.mark.parametrize("T", [1, 40, 100, 520])
def test_grad_of_any_size(lw, T):
    """Gradients far below and above the fp16 operands' range, zero tokens, and tokens with infinities or NaN."""
    N, K = 130, 160
    rng = np.random.default_rng(T)
    w = weights(rng, N, K, "sym")
    for scale in (1e-30, 1e-12, 1.0, 1e25):
        say("grad size", T, scale)
        dy = gpu((rng.standard_normal((T, N)) * scale).astype(np.float32), "bf16")
        want = ref.linear_grad(f64(dy), *w)
        dx = lw.linear_w8a8_grad(dy, *on_gpu(w))
        check(dx, want, ref.grad_bound(want, [(f64(dy), *w)], "bf16"), f"{scale}")
        bad = dy.clone()
        bad[0, N - 1] = float("nan") if scale == 1.0 else float("inf")
        if T > 2:
            bad[T - 1] = 0
        got = lw.linear_w8a8_grad(bad, *on_gpu(w))
        assert bool(got[0].isnan().all())
        if T > 2:
            assert bool((got[T - 1] == 0).all()) and bool((got[1:T - 1] == dx[1:T - 1]).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_far_gates(lw, act):
    """Gates where sigma is at its limits: no infinities or NaN from intermediate steps."""
    N, K, T = 96, 64, 5
    rng = np.random.default_rng(8)
    wg, wu = weights(rng, N, K, "sym"), weights(rng, N, K, "sym")
    g = np.concatenate([[0, 1e-30, -1e-30, 5, -5, 12, -12, 20, -20, 88, -88, 90, -90, 110, -110, 3e4, -3e4, 1e15, -1e15,
                         1e30, -1e30], rng.standard_normal(N - 21)])
    gate = gpu(np.tile(g, (T, 1)).astype(np.float32), "bf16")
    up = gpu(rng.standard_normal((T, N)).astype(np.float32), "bf16")
    dh = gpu(np.where(np.abs(g) > 1e3, 1e-28, 0.05).astype(np.float32) * rng.standard_normal((T, N)).astype(np.float32),
             "bf16")
    say("far gates", act)
    dx, pg, pu = lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu), act=act, parts=True)
    with np.errstate(over="ignore", invalid="ignore"):
        dg, du = ref.gated_parts(f64(dh), np.clip(f64(gate), -600, 600), f64(up), act)
        du = f64(dh) * ref.act_value(np.where(f64(gate) < -600, -600, f64(gate)), act)
    # below e^-88 sigma is zero in 32 bits
    tol = 2e-36
    assert bool(dx.isfinite().all()) and bool(pg.isfinite().all()) and bool(pu.isfinite().all())
    near = ref.HALF_STEP["bf16"] + 3e-5
    assert (np.abs(f64(pg) - dg) <= near * np.abs(dg) + 3e-6 * np.abs(f64(dh) * f64(up)) + tol).all()
    assert (np.abs(f64(pu) - du) <= near * np.abs(du) + tol).all()


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------
def block(rng, N, K):
    """The three matrices of a gated feed-forward block."""
    return [weights(rng, *s, "minmax") for s in ((N, K), (N, K), (K, N))]


def run_block(lw, x, w):
    h, g, u = lw.gated_w8a8(x, *w[0], *w[1], save=True)
    y = lw.linear_w8a8(h, *w[2])
    dh = lw.linear_w8a8_grad(y, *w[2])
    return h, y, dh, lw.gated_w8a8_grad(dh, g, u, *w[0], *w[1])


@pytest.mark.parametrize("T", [1, 12, 50, 100, 600])
def test_block_repeats_on_streams_and_in_graphs(lw, T):
    """A feed-forward block forward and backward: the same bits again, on a side stream, with two calls at once,
    and from a captured graph replayed between eager work of its own."""
    import torch
    say("block", T)
    rng = np.random.default_rng(T)
    w = [on_gpu(m) for m in block(rng, 352, 160)]
    x = activations(rng, T, 160, "bf16")
    x2 = activations(rng, T, 160, "bf16")
    want, want2 = run_block(lw, x, w), run_block(lw, x2, w)
    torch.cuda.synchronize()
    assert all(bool(t.isfinite().all()) for t in want)

    def same(a, b):
        return all(bool((p == q).all()) for p, q in zip(a, b))

    assert same(run_block(lw, x, w), want)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s1):
        a = run_block(lw, x, w)
    with torch.cuda.stream(s2):
        b = run_block(lw, x2, w)
    torch.cuda.synchronize()
    assert same(a, want) and same(b, want2)

    held = x.clone()
    with torch.cuda.stream(s1):
        run_block(lw, held, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_block(lw, held, w)
    for i in range(4):
        src, expect = (x, want) if i % 2 == 0 else (x2, want2)
        held.copy_(src)
        graph.replay()
        other = run_block(lw, x2 if i % 2 == 0 else x, w)      # eager work between the replays
        torch.cuda.synchronize()
        assert same(out, expect), f"replay {i}"
        assert same(other, want2 if i % 2 == 0 else want)


@pytest.mark.parametrize("T,N,K", [(1, 33, 64), (20, 65, 96), (70, 130, 160), (520, 259, 288)])
def test_nothing_written_past_the_end(lw, T, N, K):
    """Raw calls with every output and workspace of exactly its size inside guarded memory."""
    import torch
    say("guards", T, N, K)
    rng = np.random.default_rng(N)
    wg, wu = (on_gpu(weights(rng, N, K, "minmax")) for _ in range(2))
    x = activations(rng, T, K, "fp16")
    guards = []

    def room(nbytes):
        t = torch.full((nbytes + 1024,), 0xA5, dtype=torch.uint8, device="cuda")
        guards.append((t, nbytes))
        return t[512:].data_ptr()

    def p(w):
        return tuple(t.data_ptr() for t in w)

    st = torch.cuda.current_stream().cuda_stream
    assert lw.quantize_act_raw(x.data_ptr(), 0, T, K, room(T * K), room(T * 4), room(T * 4), st) == 0
    need = lw.linear_w8a8_workspace_bytes(T, N, K, 0)
    y = room(2 * T * N)
    assert lw.linear_w8a8_raw(x.data_ptr(), 0, None, None, T, *p(wg), N, K, y, 0, room(need), need, st) == 0
    need = lw.gated_w8a8_workspace_bytes(T, N, K, 0)
    h, g, u = (room(2 * T * N) for _ in range(3))
    assert lw.gated_w8a8_raw(x.data_ptr(), 0, None, None, T, *p(wg), *p(wu), N, K, 0, h, g, u, 0, room(need), need,
                             st) == 0
    need = lw.linear_w8a8_grad_workspace_bytes(T, N, K)
    assert lw.linear_w8a8_grad_raw(y, 0, T, *p(wg), N, K, room(2 * T * K), room(need), need, st) == 0
    need = lw.gated_w8a8_grad_workspace_bytes(T, N, K)
    assert lw.gated_w8a8_grad_raw(h, g, u, 0, T, *p(wg), *p(wu), N, K, 1, room(2 * T * K), room(2 * T * N),
                                  room(2 * T * N), room(need), need, st) == 0
    torch.cuda.synchronize()
    for t, n in guards:
        assert bool((t[:512] == 0xA5).all()) and bool((t[512 + n:] == 0xA5).all())


def test_empty_problems(lw):
    import torch
    rng = np.random.default_rng(0)
    w = on_gpu(weights(rng, 8, 64, "sym"))
    none = on_gpu(weights(rng, 0, 64, "sym"))
    x = activations(rng, 3, 64, "fp16")
    assert lw.linear_w8a8(x[:0], *w).shape == (0, 8)
    assert lw.linear_w8a8(x, *none).shape == (3, 0)
    assert lw.gated_w8a8(x[:0], *w, *w).shape == (0, 8)
    assert lw.gated_w8a8(x, *none, *none).shape == (3, 0)
    assert lw.quantize_act(x[:0])["codes"].shape == (0, 64)
    dy = torch.zeros(0, 8, dtype=torch.float16, device="cuda")
    assert lw.linear_w8a8_grad(dy, *w).shape == (0, 64)
    dy = torch.zeros(3, 0, dtype=torch.float16, device="cuda")
    out = torch.full((3, 64), 7, dtype=torch.float16, device="cuda")
    assert bool((lw.linear_w8a8_grad(dy, *none, out=out) == 0).all())
    assert bool((lw.gated_w8a8_grad(dy, dy, dy, *none, *none) == 0).all())


def test_refusals(lw):
    import torch
    rng = np.random.default_rng(0)
    w = on_gpu(weights(rng, 8, 64, "sym"))
    x = activations(rng, 3, 64, "fp16")
    dy = torch.zeros(3, 8, dtype=torch.float16, device="cuda")
    other = on_gpu(weights(rng, 9, 64, "sym"))
    for call, error in [
            (lambda: lw.linear_w8a8(x.float(), *w), TypeError),
            (lambda: lw.linear_w8a8(x.cpu(), *w), ValueError),
            (lambda: lw.linear_w8a8(x.t(), *w), ValueError),
            (lambda: lw.linear_w8a8(x[0], *w), ValueError),
            (lambda: lw.linear_w8a8(x[:, :32].contiguous(), *w), ValueError),
            (lambda: lw.linear_w8a8(x, w[0], w[1].float(), w[2]), TypeError),
            (lambda: lw.linear_w8a8(x, w[0], w[1][:4], w[2]), ValueError),
            (lambda: lw.linear_w8a8(x, w[0], w[1], w[2].cpu()), ValueError),
            (lambda: lw.linear_w8a8(x, *w, out_dtype=torch.float32), TypeError),
            (lambda: lw.linear_w8a8(x, *w, out=torch.empty(3, 9, dtype=torch.float16, device="cuda")), ValueError),
            (lambda: lw.gated_w8a8(x, *w, *other), ValueError),
            (lambda: lw.gated_w8a8(x, *w, *w, act="relu"), ValueError),
            (lambda: lw.linear_w8a8_grad(dy[:, :7].contiguous(), *w), ValueError),
            (lambda: lw.gated_w8a8_grad(dy, dy.bfloat16(), dy, *w, *w), TypeError),
            (lambda: lw.gated_w8a8_grad(dy, dy, dy[:2], *w, *w), ValueError),
            (lambda: lw.quantize_act(x.double()), TypeError),
            (lambda: lw.quantize_act(torch.zeros(2, 40, dtype=torch.float16, device="cuda")), lw.LowbitError),
            (lambda: lw.quantize_act(torch.zeros(1, lw.W8A8_MAX_K + 32, dtype=torch.float16, device="cuda")),
             lw.LowbitError)]:
        with pytest.raises(error):
            call()


# ---------------------------------------------------------------------------
# larger sizes: every tile shape, whole and shared out, and long index ranges
# (the 64-bit reference on the GPU)
# ---------------------------------------------------------------------------
LARGE = [(70, 21, 1504), (400, 8273, 1632), (644, 6956, 4416), (1289, 8336, 64), (2526, 6531, 992), (184, 8255, 5088),
         (1035, 7325, 64), (2834, 8215, 3328), (133, 8211, 1600), (396, 5143, 4416), (545, 8245, 32),
         (798, 8247, 1632), (399, 5628, 3680), (398, 8230, 128), (2072, 5437, 3104), (2322, 6432, 2304),
         (812, 8211, 2432), (2074, 7217, 32), (3105, 7520, 1504), (784, 8508, 64), (1337, 8245, 1728)]
LARGE_GRAD = [(65, 917, 544), (1026, 1153, 3616), (689, 4793, 4064), (2314, 44, 4832), (3257, 1258, 5024),
              (131, 4413, 4768), (1694, 46, 4640), (2339, 2268, 4832), (74, 496, 160), (773, 609, 4672),
              (642, 2338, 4064), (3082, 839, 4896), (138, 2603, 3232), (2334, 1101, 4864)]


def random_weights(g, N, K):
    """Packed words, scales, zero points near the middle, on the GPU."""
    import torch
    codes = torch.randint(0, 256, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(N, 1, generator=g, device="cuda") * 1.5 + 0.5) * 2e-4).half()
    zeros = torch.randint(110, 146, (N, 1), generator=g, device="cuda", dtype=torch.int32)
    return codes.view(torch.int32), scales, zeros


def integers(w):
    import torch
    packed, _, zeros = w
    return packed.view(torch.uint8).view(packed.shape[0], -1).double() - zeros.double()


def inside(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {bad.nonzero()[:3].tolist()}"


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_every_tile_plan(lw, shape):
    import torch
    T, N, K = shape
    say("tile plans", shape)
    g = torch.Generator(device="cuda").manual_seed(T)
    wg, wu = random_weights(g, N, K), random_weights(g, N, K)
    x = torch.randn(T, K, generator=g, device="cuda").half()
    q = lw.quantize_act(x)
    a, s = q["codes"].double(), q["scales"].double()[:, None]
    gate = (a @ integers(wg).t()) * (s * wg[1].double().t())
    bound = 2.0 ** -11 * 1.001 + 4 * ref.U32

    def linear_bound(v):
        return v.abs() * bound + ref.HALF_TINY["fp16"]

    y = lw.linear_w8a8(x, *wg)
    inside(y, gate, linear_bound(gate), f"linear {shape}")
    assert bool((lw.linear_w8a8(q, *wg) == y).all())
    up = (a @ integers(wu).t()) * (s * wu[1].double().t())
    h, hg, hu = lw.gated_w8a8(x, *wg, *wu, save=True)
    inside(hg, gate, linear_bound(gate), f"gate {shape}")
    inside(hu, up, linear_bound(up), f"up {shape}")
    want = gate * torch.sigmoid(gate) * up
    r = (20 + 20 * gate.abs().clamp(max=104)) * ref.U32
    inside(h, want, want.abs() * (2.0 ** -11 * 1.001 + r) + ref.HALF_TINY["fp16"], f"h {shape}")


@pytest.mark.parametrize("shape", LARGE_GRAD, ids=str)
def test_every_gradient_plan(lw, shape):
    import torch
    T, N, K = shape
    say("gradient plans", shape)
    g = torch.Generator(device="cuda").manual_seed(T)
    ws = [random_weights(g, N, K) for _ in range(2)]
    dy = (torch.randn(T, N, generator=g, device="cuda") * 0.05).half()

    def bound(want, parts, extra):
        terms = N * len(parts)
        out = want.abs() * 2.0 ** -11 * 1.01 + ref.HALF_TINY["fp16"]
        top = torch.stack([(d.abs() * w[1].double().t()).amax(1) for d, w in parts]).amax(0)[:, None]
        for (d, w), e in zip(parts, extra):
            size = (integers(w) + w[2].double() - 128).abs() + (128 - w[2].double()).abs()
            f = d.abs() * w[1].double().t()
            out += (f * (2.0 ** -11 + 8 * ref.U32 + terms * 2.0 ** -23 + e) + top * 2.0 ** -39) @ size * 1.001
        return out

    def product(parts):
        return sum((d * w[1].double().t()) @ integers(w) for d, w in parts)

    parts = [(dy.double(), ws[0])]
    want = product(parts)
    dx = lw.linear_w8a8_grad(dy, *ws[0])
    inside(dx, want, bound(want, parts, [0]), f"linear {shape}")
    if N >= 512:     # sums of independent roundings: half a step each at the most, in the 2-norm
        assert float((dx.double() - want).norm()) <= float(want.norm()) * 2.0 ** -10
    assert bool((lw.linear_w8a8_grad(dy, *ws[0]) == dx).all())
    gate = torch.randn(T, N, generator=g, device="cuda").half()
    up = torch.randn(T, N, generator=g, device="cuda").half()
    v = gate.double()
    s = torch.sigmoid(v)
    parts = [(dy.double() * up.double() * (s + v * s * (1 - s)), ws[0]), (dy.double() * v * s, ws[1])]
    want = product(parts)
    # the slope's relative error where its terms cancel is bounded by their size: 64 half steps of dy up
    slope = (dy.double() * up.double()).abs() * 64 * ref.U32 / parts[0][0].abs().clamp(min=1e-30)
    inside(lw.gated_w8a8_grad(dy, gate, up, *ws[0], *ws[1]), want, bound(want, parts, [slope, 64 * ref.U32]),
           f"gated {shape}")


@pytest.mark.parametrize("N", [32769, 40000, 65544])
def test_gradients_of_long_rows(lw, N):
    """More weight rows than a preparation holds in registers, whole 16-byte chunks and not."""
    T, K = 3, 64
    say("long rows", N)
    rng = np.random.default_rng(N)
    wg, wu = weights(rng, N, K, "minmax"), weights(rng, N, K, "minmax")
    dh, gate, up = (gpu(rng.standard_normal((T, N)).astype(np.float32), "bf16") for _ in range(3))
    dh = dh * 0.01
    want = ref.linear_grad(f64(dh), *wg)
    check(lw.linear_w8a8_grad(dh, *on_gpu(wg)), want, ref.grad_bound(want, [(f64(dh), *wg)], "bf16"), f"linear {N}")
    dg, du = ref.gated_parts(f64(dh), f64(gate), f64(up), "silu")
    dx, pg, pu = lw.gated_w8a8_grad(dh, gate, up, *on_gpu(wg), *on_gpu(wu), parts=True)
    want = ref.linear_grad(dg, *wg) + ref.linear_grad(du, *wu)
    size = np.abs(f64(dh) * f64(up)) * 64 * ref.U32
    extra = [size / np.maximum(np.abs(dg), 1e-30), 64 * ref.U32]
    check(dx, want, ref.grad_bound(want, [(dg, *wg), (du, *wu)], "bf16", extra), f"gated {N}")
    check(pg, dg, np.abs(dg) * 2.0 ** -8 * 1.01 + 2 * size + ref.HALF_TINY["bf16"], "dgate")
    check(pu, du, np.abs(du) * (2.0 ** -8 * 1.01 + 64 * ref.U32) + ref.HALF_TINY["bf16"], "dup")


def test_more_outputs_than_32_bits_count(lw):
    """T N and T K above 2^31 elements (offsets above 2^32 bytes): the last tokens and rows are right."""
    import torch
    T, N, K = 46000, 49153, 64
    say("many outputs", T, N, K)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = random_weights(g, N, K)
    x = torch.randn(T, K, generator=g, device="cuda").half()
    y = lw.linear_w8a8(x, *w)
    some = torch.tensor([0, 1, 22000, 43689, 43690, 43691, T - 2, T - 1], device="cuda")
    q = lw.quantize_act(x[some])
    want = (q["codes"].double() @ integers(w).t()) * (q["scales"].double()[:, None] * w[1].double().t())
    inside(y[some], want, want.abs() * (2.0 ** -11 * 1.001 + 4 * ref.U32) + ref.HALF_TINY["fp16"], "linear")
    dx = lw.linear_w8a8_grad(y, *w)
    alone = lw.linear_w8a8_grad(y[some].contiguous(), *w)
    # other tile shapes: the same sums in another order
    assert float((dx[some] - alone).double().norm()) <= float(alone.double().norm()) * 2.0 ** -10
    del dx, alone, y
    torch.cuda.empty_cache()
    w = random_weights(g, 64, 65536)
    d = torch.randn(40000, 64, generator=g, device="cuda").half()
    dx = lw.linear_w8a8_grad(d, *w)
    rows = torch.tensor([0, 32767, 32768, 39999], device="cuda")
    want = (d[rows].double() * w[1].double().t()) @ integers(w)
    assert float((dx[rows].double() - want).norm()) <= float(want.norm()) * 2.0 ** -10


def test_first_calls_captured():
    """In a new process, the very first calls go into a graph."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    say("first calls captured")
    code = """
import torch, sys
sys.path.insert(0, %r)
import weight_only_bit_rtn_amd as lw
g = torch.Generator(device="cuda").manual_seed(0)
codes = torch.randint(0, 256, (256, 256), generator=g, device="cuda", dtype=torch.uint8)
w = codes.view(torch.int32), torch.full((256, 1), 1e-3, device="cuda").half(), torch.full((256, 1), 128, device="cuda", dtype=torch.int32)
xs = [torch.randn(T, 256, generator=g, device="cuda").half() for T in (1, 20, 300)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = [(lw.gated_w8a8(x, *w, *w), lw.linear_w8a8(x, *w), lw.linear_w8a8_grad(x, *w)) for x in xs]
for _ in range(3):
    graph.replay()
    torch.cuda.synchronize()
    for x, o in zip(xs, out):
        for p, q in zip(o, (lw.gated_w8a8(x, *w, *w), lw.linear_w8a8(x, *w), lw.linear_w8a8_grad(x, *w))):
            assert bool((p == q).all())
print("captured")
""" % root
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_outputs_that_share_memory_are_refused(lw):
    rng = np.random.default_rng(0)
    w = on_gpu(weights(rng, 64, 64, "sym"))
    x = activations(rng, 64, 64, "fp16")
    q = lw.quantize_act(x)
    both = activations(rng, 96, 64, "fp16")
    for call in [lambda: lw.linear_w8a8(x, *w, out=x), lambda: lw.linear_w8a8_grad(x, *w, out=x),
                 lambda: lw.linear_w8a8(both[:64], *w, out=both[32:]),
                 lambda: lw.quantize_act(x, out={"codes": q["codes"], "scales": q["sums"].view(q["scales"].dtype),
                                                 "sums": q["sums"]}),
                 lambda: lw.quantize_act(x, out={"codes": x.view(q["codes"].dtype).view(-1)[:4096].view(64, 64)})]:
        with pytest.raises(ValueError):
            call()
    want = lw.linear_w8a8(both[:32], *w)
    assert bool((lw.linear_w8a8(both[:32], *w, out=both[64:]) == want).all())


@pytest.mark.parametrize("T", [3, 70])
def test_factors_past_the_range(lw, T):
    """A token whose factors dy s leave fp32's range is NaN; the others are as ever."""
    import torch
    rng = np.random.default_rng(1)
    codes, scales, zeros = weights(rng, 40, 64, "sym")
    scales[7] = 4.0
    w = on_gpu((codes, scales, zeros))
    dy = activations(rng, T, 40, "bf16")
    want = lw.linear_w8a8_grad(dy, *w)
    dy[1, 7] = 3e38
    got = lw.linear_w8a8_grad(dy, *w)
    assert bool(got[1].isnan().all())
    keep = torch.arange(T, device="cuda") != 1
    assert bool((got[keep] == want[keep]).all()) and not bool(got[keep].isnan().any())


@pytest.mark.parametrize("shape", [(516, 8057, 3200), (130, 5497, 3424), (396, 8456, 32), (147, 9000, 4448),
                                   (132, 2715, 3424), (131, 8564, 32), (533, 8187, 3136)], ids=str)
def test_every_plan_of_small_tiles(lw, shape):
    """192 x 192 tiles: whole and shared out, linear and gated."""
    test_every_tile_plan(lw, shape)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 2000, 512), (2, 1999, 544), (4, 1000, 96), (13, 1501, 544), (33, 1000, 544),
                                   (64, 777, 1056), (100, 500, 320), (520, 1031, 4096), (516, 8057, 224)])
def test_products_are_the_fp32_value(lw, T, N, K, kind):
    """fl32(fl32(S s) d), rounded to the output type: one value, bit for bit, whichever kernel makes it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    w, wu = random_weights(g, N, K), random_weights(g, N, K)
    x = torch.randn(T, K, generator=g, device="cuda").to(types()[kind])
    q = lw.quantize_act(x)

    def value(w):
        d = q["codes"].double() @ integers(w).t()
        return (q["scales"][:, None] * w[1].float().t() * d.float()).to(x.dtype)

    assert bool((lw.linear_w8a8(x, *w) == value(w)).all())
    assert bool((lw.linear_w8a8(q, *w, out_dtype=x.dtype) == value(w)).all())
    _, gate, up = lw.gated_w8a8(x, *w, *wu, save=True)
    assert bool((gate == value(w)).all()) and bool((up == value(wu)).all())


@pytest.mark.parametrize("shape", [(85, 22, 2464), (630, 20, 32), (2562, 26, 4032), (205, 8807, 32), (407, 8200, 4256),
                                   (670, 5380, 96), (528, 6586, 4128), (1287, 5405, 96), (520, 6782, 32),
                                   (1366, 8139, 32), (2087, 7317, 32), (129, 5767, 32), (275, 5468, 4064),
                                   (138, 8885, 96), (419, 8308, 3552), (129, 8218, 3744), (305, 8827, 96),
                                   (523, 8348, 3552), (129, 8335, 32), (562, 8736, 32), (1371, 5479, 2016),
                                   (806, 8360, 32), (1289, 8190, 1568), (21, 30, 32)], ids=str)
def test_every_plan_of_long_steps(lw, shape):
    """Steps of 64 and 128 values, every shape whole and shared out, linear and gated."""
    test_every_tile_plan(lw, shape)


@pytest.mark.parametrize("shape", [(24, 10852, 9568), (61, 8037, 8032), (19, 22688, 960), (52, 17920, 960),
                                   (31, 36162, 4608), (60, 33771, 2560), (52, 39997, 992), (23, 8151, 9472),
                                   (61, 4065, 12768), (32, 12369, 1024), (64, 10635, 1024), (30, 34159, 5120),
                                   (54, 18606, 4480), (63, 24569, 1280)], ids=str)
def test_few_tokens_by_large_weights(lw, shape):
    """17 to 64 tokens where tiles take over from the rings, whole and shared out."""
    test_every_tile_plan(lw, shape)


@pytest.mark.parametrize("shape", [(1, 2614, 32), (1, 174, 32), (17, 1468, 32), (24, 22, 32), (33, 1473, 32), (35, 61, 32),
                                   (34, 2117, 6624), (139, 1009, 64), (113, 49, 32), (391, 1249, 8224),
                                   (133, 1849, 5504), (588, 21, 6624), (2363, 5107, 160), (1258, 20, 7296),
                                   (129, 8681, 8160), (1844, 24, 6368), (2199, 1241, 7200)], ids=str)
def test_every_gradient_shape(lw, shape):
    """Every tile shape of the gradients, whole and shared out."""
    test_every_gradient_plan(lw, shape)
