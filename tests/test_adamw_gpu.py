"""The AdamW step on the GPU against the definition: moments bit for bit in 8 and 32 bits, parameters
within their bound, over types, odd sizes and many tensors; infinities, skipped steps, graphs and
long tensors."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import adapters_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {**ref.HALF_STEP, "fp32": ref.U32}
TINY = {**ref.HALF_TINY, "fp32": 2.0 ** -150}


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


class Run:
    """A list of tensors, its state, and the same in numpy."""

    def __init__(self, lw, sizes, kind, grads, bits, master, seed=0):
        print(f"[adamw] {len(sizes)} tensors to {max(sizes)} {kind} grads {grads} {bits} bits master {master}", flush=True)
        self.lw, self.sizes, self.kind, self.bits, self.master = lw, sizes, kind, bits, master
        self.rng = np.random.default_rng(seed)
        self.grad_type = TYPES[grads]
        self.params = [torch.from_numpy(self.rng.standard_normal(n).astype(np.float32) * 0.1).cuda().to(TYPES[kind]) for n in sizes]
        self.state = lw.adamw_state(self.params, bits=bits, master=master)
        self.blocks = [-(-n // 256) for n in sizes]
        self.at = np.concatenate([[0], np.cumsum(self.blocks)]) * 256

    def flat(self, tensors):
        out = np.zeros(self.at[-1], np.float32)
        for a, n, t in zip(self.at, self.sizes, tensors):
            out[a:a + n] = t.float().cpu().numpy()
        return out

    def grads(self, by=1e-2):
        return [torch.from_numpy((self.rng.standard_normal(n) * np.exp(2 * self.rng.standard_normal(n)) * by).astype(np.float32))
                .cuda().to(self.grad_type) for n in self.sizes]

    def held(self):
        """m, v in fp32, and the parameters a step starts from."""
        s = {k: t.cpu().numpy() for k, t in self.state.items()}
        m, v = ref.decode(s["m"], s["v"], s["m_max"], s["v_max"]) if self.bits == 8 else (s["m"], s["v"])
        return m, v, s["master"] if self.master else self.flat(self.params)

    def check(self, grads, step, lr=1e-2, betas=(0.9, 0.999), eps=1e-8, decay=0.05, scale=None):
        m, v, p = self.held()
        m, v = ref.moments(m, v, self.flat(grads), *betas, scale)
        inside = self.flat([torch.ones(n) for n in self.sizes]) > 0
        m, v = np.where(inside, m, np.float32(0)), np.where(inside, v, np.float32(0))
        want, taken = ref.update(p, m, v, lr, *betas, eps, decay, step)
        self.lw.adamw(self.params, grads, self.state, lr=lr, betas=betas, eps=eps, weight_decay=decay, step=step,
                      grad_scale=None if scale is None else torch.tensor([scale], device="cuda"))
        s = {k: t.cpu().numpy() for k, t in self.state.items()}
        if self.bits == 8:
            for name, x, bits in (("m", m, 7), ("v", v, 8)):
                code, top = ref.encode(x, bits)
                assert np.array_equal(s[name], code) and np.array_equal(s[name + "_max"], top, equal_nan=True), name
            got = [t.cpu().numpy() for t in self.lw.adamw_moments(self.state)]
            assert all(np.array_equal(g, w, equal_nan=True)
                       for g, w in zip(got, ref.decode(s["m"], s["v"], s["m_max"], s["v_max"])))
        else:
            assert np.array_equal(s["m"], m, equal_nan=True) and np.array_equal(s["v"], v, equal_nan=True)
        # decay and step rounded to fp32, the sum once; the root, the reciprocal and their products
        far = 4 * ref.U32 * (np.abs(want) + np.abs(p)) + 2.0 ** -21 * np.abs(taken) + 2.0 ** -149
        got = self.flat(self.params)
        if self.master:
            assert within(s["master"], want, far)
        far = far + HALF[self.kind] * (np.abs(want) + far) + TINY[self.kind]
        assert within(got, want, far)


def within(got, want, far):
    return (np.isnan(got) == np.isnan(want)).all() and (np.isnan(want) | (np.abs(got - want) <= far)).all()


SIZES = [1, 2, 3, 4, 5, 255, 256, 257, 511, 1000, 1023, 1024, 1025, 4097, 70000]


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grads", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
def test_steps(lw, kind, grads, bits, master):
    run = Run(lw, SIZES, kind, grads, bits, master)
    for step in (1, 2, 3):
        run.check(run.grads(), step, scale=0.25 if step == 2 else None)


@pytest.mark.parametrize("count", [1, 127, 128, 129, 300])
def test_many_tensors(lw, count):
    rng = np.random.default_rng(count)
    run = Run(lw, [int(n) for n in rng.integers(1, 3000, count)], "fp32", "fp32", 8, False)
    run.check(run.grads(), 7)


@pytest.mark.parametrize("bits", [8, 32])
def test_options(lw, bits):
    run = Run(lw, [3000, 77], "fp32", "fp32", bits, False)
    run.check(run.grads(), 1, lr=0.0)
    run.check(run.grads(), 100000, betas=(0.0, 0.0), eps=0.0, decay=0.0)
    run.check(run.grads(), 2, betas=(0.99, 0.9999), eps=1e-3, decay=10.0)


def test_lr_and_step_on_the_gpu(lw):
    """As the same numbers given from the host."""
    for step in (1, 37, 2000000):
        a, b = (Run(lw, [3000, 77], "fp32", "fp32", 8, False, seed=2) for _ in range(2))
        g = a.grads()
        lw.adamw(a.params, g, a.state, lr=0.125, step=step)
        lw.adamw(b.params, g, b.state, lr=torch.tensor(0.125, device="cuda"), step=torch.tensor([step], dtype=torch.int32, device="cuda"))
        assert all(torch.equal(p, q) for p, q in zip((*a.params, *a.state.values()), (*b.params, *b.state.values())))


@pytest.mark.parametrize("bits", [8, 32])
def test_zeros(lw, bits):
    """No gradient ever: nothing but the decay happens."""
    run = Run(lw, [600], "fp32", "fp32", bits, False)
    run.check([torch.zeros(600, device="cuda")], 1)
    assert not run.state["m"].any() and not run.state["v"].any()


@pytest.mark.parametrize("by", [1e-21, 1e-19, 1e-17, 1e15])
def test_far_gradients(lw, by):
    """Second moments below fp32's normal range, and first ones far above them."""
    for bits in (8, 32):
        run = Run(lw, [1000], "fp32", "fp32", bits, False)
        for step in (1, 2):
            run.check(run.grads(by), step, eps=1e-8)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_gradients(lw, bits, bad):
    run = Run(lw, [1000, 300], "fp32", "fp32", bits, False)
    run.check(run.grads(), 1)
    g = run.grads()
    g[0][300] = bad
    run.check(g, 2)
    assert run.params[0][300].isnan()
    assert run.params[1].isfinite().all() and run.params[0][:300].isfinite().all()
    run.check(run.grads(), 3)
    # in 8 bits the value's block goes with it
    assert run.params[0].isnan().sum() == (256 if bits == 8 else 1)


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -float("inf")])
def test_a_step_that_overflowed_is_skipped(lw, scale):
    run = Run(lw, [1000, 30], "bf16", "bf16", 8, True)
    run.check(run.grads(), 1)
    before = [t.clone() for t in (*run.params, *run.state.values())]
    lw.adamw(run.params, run.grads(), run.state, lr=1e-2, step=2, grad_scale=torch.tensor([scale], device="cuda"))
    assert all(torch.equal(p, q) for p, q in zip(before, (*run.params, *run.state.values())))


def test_empty_tensors_and_repeats(lw):
    a, b = (Run(lw, [300, 40], "fp32", "fp32", 8, False, seed=4) for _ in range(2))
    g = a.grads()
    empty = torch.empty(0, device="cuda")
    lw.adamw(a.params, g, a.state, lr=1e-2, step=1)
    lw.adamw([empty, b.params[0], empty, b.params[1]], [empty, g[0], empty, g[1]], b.state, lr=1e-2, step=1)
    assert all(torch.equal(p, q) for p, q in zip((*a.params, *a.state.values()), (*b.params, *b.state.values())))


def test_captured(lw):
    """A captured step replayed with new gradients, rates and counts, eager steps of another state in between."""
    a, b = (Run(lw, [3000, 77, 130000], "bf16", "bf16", 8, True, seed=5) for _ in range(2))
    g = [torch.zeros_like(p) for p in a.params]
    lr, step, scale = torch.tensor([0.1], device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lw.adamw(a.params, g, a.state, lr=lr, step=step, grad_scale=scale)
    for i in range(1, 6):
        for to, fresh in zip(g, b.grads()):
            to.copy_(fresh)
        lr.fill_(0.1 / i)
        step.fill_(i)
        scale.fill_(0.5 if i != 3 else float("inf"))
        graph.replay()
        lw.adamw(b.params, g, b.state, lr=lr, step=step, grad_scale=scale)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((*a.params, *a.state.values()), (*b.params, *b.state.values()))), i


def test_more_values_than_32_bits_count(lw):
    """The largest tensor is several launches: places on either side of their borders."""
    n = (1 << 32) + 1000
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    places = [0, (1 << 30) - 1, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1]
    g[places] = 0.5
    blocks = -(-n // 256)
    state = {k: torch.zeros(blocks * 256, dtype=torch.uint8, device="cuda") for k in ("m", "v")}
    state.update({k: torch.zeros(blocks, device="cuda") for k in ("m_max", "v_max")})
    lw.adamw([p], [g], state, lr=0.5, weight_decay=0.0, step=1)
    assert (p[places] == -0.5).all() and (state["m"][places] == 127).all() and (state["v"][places] == 255).all()
    assert int((p != 0).sum()) == len(places) and int((state["v_max"] > 0).sum()) == len({i // 256 for i in places})


def test_nothing_written_past_the_end(lw):
    n, blocks = 1001, 4
    raw = {k: torch.full((512 + size + 512,), 0xA5, dtype=torch.uint8, device="cuda")
           for k, size in (("p", n * 2), ("m", blocks * 256), ("v", blocks * 256), ("m_max", blocks * 4), ("v_max", blocks * 4),
                           ("master", blocks * 1024))}
    used = {k: t.numel() - 1024 for k, t in raw.items()}
    for k, t in raw.items():
        t[512:512 + used[k]] = 0
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    import ctypes
    table = (ctypes.c_int64 * 3)(raw["p"].data_ptr() + 512, g.data_ptr(), n)
    place = lw.AdamwState(*(raw[k].data_ptr() + 512 for k in ("m", "v", "m_max", "v_max", "master")))
    options = lw.AdamwOptions(1e-2, 0.9, 0.999, 1e-8, 0.0, 1, None, None, None)
    assert lw.adamw_raw(ctypes.addressof(table), 1, 1, 1, 8, place, options, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for k, t in raw.items():
        assert (t[:512] == 0xA5).all() and (t[512 + used[k]:] == 0xA5).all(), k
    assert not raw["m"][512 + n:512 + 1024].any() and not raw["master"][512 + 4 * n:512 + 4096].any()


def test_refusals_and_versions(lw):
    run = Run(lw, [300, 40], "fp32", "fp32", 8, False)
    p, g, s = run.params, run.grads(), run.state
    flat = torch.zeros(600, device="cuda")
    for call in (lambda: lw.adamw(p, g[:1], s, lr=1), lambda: lw.adamw(p, [g[1], g[0]], s, lr=1),
                 lambda: lw.adamw([p[0], p[0]], [g[0], g[0]], s, lr=1), lambda: lw.adamw(p[:1], g[:1], s, lr=1),
                 lambda: lw.adamw([p[0], p[1].half()], g, s, lr=1), lambda: lw.adamw(p, [g[0].cpu(), g[1]], s, lr=1),
                 lambda: lw.adamw([flat[::2], p[1]], g, s, lr=1), lambda: lw.adamw(p, g, s, lr=torch.zeros(2, device="cuda")),
                 lambda: lw.adamw(p, g, {**s, "master": flat}, lr=1)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lw.adamw([t.double() for t in p], g, s, lr=1), lambda: lw.adamw(p, g, {**s, "v": s["v"].int()}, lr=1),
                 lambda: lw.adamw(p, g, s, lr=1, step=torch.ones(1, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: lw.adamw(p, g, s, lr=-1.0), lambda: lw.adamw(p, g, s, lr=1, betas=(1.0, 0.9)), lambda: lw.adamw(p, g, s, lr=1, step=0),
                 lambda: lw.adamw([flat[1:301], p[1]], g, s, lr=1)):
        with pytest.raises(lw.LowbitError):
            call()
    # parameters that require grad are updated, and a graph that saved them notices
    w = torch.ones(300, device="cuda", requires_grad=True)
    loss = (w * w).sum()
    lw.adamw([w, p[1]], g, s, lr=1e-2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
