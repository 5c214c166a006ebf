"""Adapters beside the shared projections on the GPU against the 64-bit reference: plans, the forward
pass and the gradients over shapes, ranks, types and orders, rows without an adapter, what must
not be read or written, streams, graphs and a training step of all of it together."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import adapters_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


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


def f64(t):
    return t.double().cpu().numpy()


def draw_ids(rng, T, L, order, none=0.2):
    """Adapters of T tokens: one by one, or in runs; -1 and ids past the last for some of them."""
    if order == "mixed":
        ids = rng.integers(0, L, T)
        ids[rng.random(T) < none] = -1
    else:
        cuts = np.sort(rng.integers(0, T + 1, 2 * L))
        ids = rng.integers(-1, L + 1, 2 * L + 1)[np.searchsorted(cuts, np.arange(T), side="right")]
    return ids.astype(np.int32)


class Case:
    def __init__(self, lw, T, N, K, R, L, kind, order, seed=0):
        print(f"[adapters] T {T} N {N} K {K} R {R} L {L} {kind} {order}", flush=True)
        rng = np.random.default_rng([seed, T, N, K, R, L])
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = TYPES[kind]

        def normal(*shape, by=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * by).to(t)

        self.kind, self.lw = kind, lw
        self.ids = draw_ids(rng, T, L, order)
        self.x, self.y, self.dy, self.base = normal(T, K), normal(T, N), normal(T, N, by=0.1), normal(T, K, by=0.1)
        self.a, self.b = normal(L, R, K, by=K ** -0.5), normal(L, N, R, by=0.3)
        self.scales = torch.rand(L, generator=g, device="cuda") + 0.5
        self.v = torch.randn(T, R, generator=g, device="cuda") * torch.from_numpy((self.ids >= 0) & (self.ids < L)).cuda()[:, None]
        self.dev_ids = torch.from_numpy(self.ids).cuda()
        self.plan = lw.lora_plan(self.dev_ids, L)

    def pools(self):
        return self.a, self.b, self.scales, self.plan

    def check_forward(self, out, v, y):
        arrays = [f64(t) for t in (self.x, self.a, self.b, self.scales)]
        want, want_v = ref.lora(*arrays, self.ids, None if y is None else f64(y))
        far, far_v = ref.lora_bound(*arrays, self.ids, want, self.kind)
        assert (np.abs(f64(out) - want) <= far).all()
        if v is not None:
            assert (np.abs(f64(v) - want_v) <= far_v).all()

    def check_backward(self, dx, da, db, base):
        arrays = [f64(t) for t in (self.dy, self.x, self.v, self.a, self.b, self.scales)]
        want = ref.lora_grad(*arrays, self.ids, None if base is None else f64(base))
        far = ref.lora_grad_bound(*arrays, self.ids, want[0], self.kind)
        for got, w, f in zip((dx, da, db), want, far):
            assert (np.abs(f64(got) - w) <= f).all()


# ---------------------------------------------------------------------------
# plans
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [0, 1, 63, 64, 65, 1000, 1024, 5003])
@pytest.mark.parametrize("L", [1, 3, 64, 1023, 1024])
def test_plan(lw, T, L):
    print(f"[adapters] plan T {T} L {L}", flush=True)
    rng = np.random.default_rng([T, L])
    for ids in (draw_ids(rng, T, L, "mixed"), draw_ids(rng, T, L, "runs"), np.full(T, -1), np.full(T, L - 1),
                np.full(T, L), rng.choice([-2 ** 31, 2 ** 31 - 1, 0], T)):
        got = lw.lora_plan(torch.from_numpy(np.asarray(ids, np.int32)).cuda(), L)
        order, starts = ref.plan(np.asarray(ids), L)
        assert np.array_equal(got["order"].cpu().numpy(), order)
        assert np.array_equal(got["starts"].cpu().numpy(), starts)


# ---------------------------------------------------------------------------
# shapes
# ---------------------------------------------------------------------------
SHAPES = [(1, 8, 32, 8, 1, "mixed"), (1, 4096, 4096, 16, 3, "mixed"), (2, 13, 96, 8, 2, "mixed"), (15, 64, 64, 16, 1, "runs"),
          (16, 65, 1056, 24, 2, "mixed"), (17, 301, 160, 32, 5, "runs"), (63, 127, 2048, 40, 64, "mixed"),
          (64, 1001, 544, 64, 3, "runs"), (65, 128, 992, 72, 130, "mixed"), (200, 520, 512, 128, 2, "runs"),
          (256, 257, 4096, 16, 9, "mixed"), (257, 63, 32, 8, 4, "runs"), (300, 191, 4128, 16, 1, "runs"),
          (333, 1000, 288, 104, 3, "mixed"), (700, 72, 736, 48, 1024, "mixed"), (1500, 513, 512, 32, 2, "runs"),
          (2000, 136, 1024, 128, 1, "runs"), (3100, 264, 96, 56, 20, "runs")]


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward(lw, shape, kind):
    c = Case(lw, *shape[:5], kind, shape[5])
    out, v = lw.lora(c.x, *c.pools(), y=c.y, save=True)
    c.check_forward(out, v, c.y)
    assert torch.equal(lw.lora(c.x, *c.pools(), y=c.y), out)                 # without v, and again
    c.check_forward(lw.lora(c.x, *c.pools()), None, None)                   # the adapters' part alone
    y = c.y.clone()
    assert lw.lora(c.x, *c.pools(), y=y, out=y) is y and torch.equal(y, out)  # in place
    into = torch.full_like(out, float("nan"))
    lw.lora(c.x, *c.pools(), y=c.y, out=into)
    assert torch.equal(into, out)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_backward(lw, shape, kind):
    c = Case(lw, *shape[:5], kind, shape[5], seed=1)
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    c.check_backward(dx, da, db, c.base)
    again = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, da, db)))
    alone = lw.lora_grad(c.dy, c.x, c.v, *c.pools())
    c.check_backward(*alone, None)
    base = c.base.clone()
    in_place = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=base, out=base)
    assert in_place[0] is base and torch.equal(base, dx)


def test_forward_and_backward_agree_on_v(lw):
    """What the forward pass saves is what the gradients take."""
    c = Case(lw, 200, 96, 256, 16, 3, "bf16", "mixed")
    _, c.v = lw.lora(c.x, *c.pools(), y=c.y, save=True)
    c.check_backward(*lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base), c.base)


@pytest.mark.parametrize("T", [40, 600])
def test_no_token_has_an_adapter(lw, T):
    c = Case(lw, T, 65, 64, 16, 3, "fp16", "mixed")
    c.ids[:] = -1
    c.plan = lw.lora_plan(torch.from_numpy(c.ids).cuda(), 3)
    out, v = lw.lora(c.x, *c.pools(), y=c.y, save=True)
    assert torch.equal(out, c.y) and not v.any()
    assert not lw.lora(c.x, *c.pools()).any()
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    assert torch.equal(dx, c.base) and not da.any() and not db.any()
    assert not lw.lora_grad(c.dy, c.x, c.v, *c.pools())[0].any()


def test_no_tokens(lw):
    c = Case(lw, 3, 65, 64, 16, 3, "fp16", "mixed")
    plan = lw.lora_plan(c.dev_ids[:0], 3)
    pools = (c.a, c.b, c.scales, plan)
    out, v = lw.lora(c.x[:0], *pools, y=c.y[:0], save=True)
    assert out.shape == (0, 65) and v.shape == (0, 16)
    dx, da, db = lw.lora_grad(c.dy[:0], c.x[:0], c.v[:0], *pools)
    assert dx.shape == (0, 64) and not da.any() and not db.any()


# ---------------------------------------------------------------------------
# infinities, NaN and far values
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("T", [50, 500])
def test_what_nobody_uses_reaches_nothing(lw, T, kind):
    """Bad values of tokens without an adapter, of adapters without tokens, and of ranks that tokens of
    another adapter have: results are those without them."""
    c = Case(lw, T, 77, 96, 24, 4, kind, "mixed")
    c.ids[c.ids == 2] = -1
    c.plan = lw.lora_plan(torch.from_numpy(c.ids).cuda(), 4)
    before = (*lw.lora(c.x, *c.pools(), y=c.y, save=True), *lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base))
    none = torch.from_numpy(~((c.ids >= 0) & (c.ids < 4))).cuda()
    for bad in (float("nan"), float("inf")):
        c.x[none], c.dy[none], c.v[none] = bad, bad, bad
        c.a[2], c.b[2], c.scales[2] = bad, bad, bad
        after = (*lw.lora(c.x, *c.pools(), y=c.y, save=True), *lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base))
        assert all(torch.equal(p, q) for p, q in zip(before, after))


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_bad_values_stay_where_they_belong(lw, kind):
    c = Case(lw, 300, 80, 96, 16, 2, kind, "mixed")
    t = int(np.flatnonzero(c.ids == 1)[3])
    good = lw.lora(c.x, *c.pools(), y=c.y)
    c.x[t, 5] = float("nan")
    out, v = lw.lora(c.x, *c.pools(), y=c.y, save=True)
    rest = torch.arange(300, device="cuda") != t
    assert out[t].isnan().all() and v[t].isnan().all() and torch.equal(out[rest], good[rest])
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    assert da[1, :, 5].isnan().all() and da.isnan().sum() == 16 and dx.isfinite().all() and db.isfinite().all()
    c.x[t, 5] = float("inf")
    da = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)[1]
    # u is hi + lo, and inf * hi + inf * lo is no number where lo is 0 or of the other sign: not finite, no more
    assert not da[1, :, 5].isfinite().any() and da.isfinite().sum() == da.numel() - 16
    c.x[t, 5] = 0
    c.y[t, 7] = float("inf")
    out = lw.lora(c.x, *c.pools(), y=c.y)
    assert out[t, 7].isinf() and out.isfinite().sum() == out.numel() - 1
    c.dy[t, 3] = float("nan")
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    assert dx[t].isnan().all() and dx[rest].isfinite().all()
    assert da[1].isnan().all() and da[0].isfinite().all() and db[1, 3].isnan().all() and db.isnan().sum() == 16


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("by", [2.0 ** -20, 2.0 ** 13])
def test_far_coefficients(lw, kind, by):
    """v and u far outside fp16's range on either side, from token to token and within one adapter."""
    c = Case(lw, 700, 96, 128, 16, 2, kind, "runs", seed=3)
    each = torch.exp2(torch.randint(-3, 3, (700, 1), device="cuda").float())
    c.x = (c.x.float() * each).to(TYPES[kind])
    c.a = (c.a.float() * by).to(TYPES[kind])
    c.scales *= 1.0 / by
    c.v *= by * each
    c.dy = (c.dy.float() * each * 2.0 ** -6).to(TYPES[kind])
    out, v = lw.lora(c.x, *c.pools(), y=c.y, save=True)
    c.check_forward(out, v, c.y)
    c.scales *= by
    c.check_backward(*lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base), c.base)


# ---------------------------------------------------------------------------
# memory
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,N,K,R,L", [(1, 9, 32, 8, 1), (70, 301, 96, 24, 3), (520, 75, 160, 72, 2), (300, 33, 64, 128, 40)])
def test_nothing_written_past_the_end(lw, T, N, K, R, L):
    c = Case(lw, T, N, K, R, L, "bf16", "mixed")
    st = torch.cuda.current_stream().cuda_stream
    room = {}

    def guarded(name, n, dtype, at=512):
        raw = torch.full((at + n * dtype.itemsize + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        room[name] = (raw, at, n * dtype.itemsize)
        return raw.data_ptr() + at

    p = [c.plan["order"].data_ptr(), c.plan["starts"].data_ptr(), c.a.data_ptr(), c.b.data_ptr(), c.scales.data_ptr(),
         L, R, N, K]
    need, grad = lw.lora_workspace_bytes(T, N, K, R, L), lw.lora_grad_workspace_bytes(T, N, K, R, L)
    args = [guarded("order", T, torch.int32), guarded("starts", L + 1, torch.int32)]
    assert lw.lora_plan_raw(c.dev_ids.data_ptr(), T, L, *args, st) == 0
    assert lw.lora_raw(c.x.data_ptr(), 1, T, *p, c.y.data_ptr(), guarded("out", T * N, torch.int16),
                       guarded("v", T * R, torch.float32), guarded("ws", need, torch.uint8), need, st) == 0
    assert lw.lora_grad_raw(c.dy.data_ptr(), c.x.data_ptr(), c.v.data_ptr(), 1, T, *p, c.base.data_ptr(),
                            guarded("dx", T * K, torch.int16), guarded("da", L * R * K, torch.float32),
                            guarded("db", L * N * R, torch.float32), guarded("ws2", grad, torch.uint8), grad, st) == 0
    torch.cuda.synchronize()
    for name, (raw, at, n) in room.items():
        assert (raw[:at] == 0xA5).all() and (raw[at + n:] == 0xA5).all(), name


def test_broken_plans_stay_inside(lw):
    """An order that is no permutation and starts that do not rise: unspecified results, within the buffers."""
    c = Case(lw, 300, 65, 64, 16, 5, "fp16", "mixed")
    rng = np.random.default_rng(0)
    for starts in ([0, 900, -5, 7, 2 ** 31 - 1, -2 ** 31], [300] * 6, [-1] * 6, [5, 4, 3, 2, 1, 0]):
        plan = {"order": torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, 300).astype(np.int32)).cuda(),
                "starts": torch.tensor(starts, dtype=torch.int32, device="cuda")}
        lw.lora(c.x, c.a, c.b, c.scales, plan, y=c.y, save=True)
        lw.lora_grad(c.dy, c.x, c.v, c.a, c.b, c.scales, plan, dx=c.base)
    torch.cuda.synchronize()


def test_outputs_past_32_bits(lw):
    """More outputs than 32 bits count: rows of y on either side of the border."""
    T, N, K, R = 70000, 65536, 32, 8
    c = Case(lw, 8, N, K, R, 2, "bf16", "mixed")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    ids[1::2] = 1
    rows = [0, 1, 32767, 32768, 65535, 65536, 65537, T - 1]
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    x[rows] = c.x
    y = torch.ones(T, N, dtype=torch.bfloat16, device="cuda")
    lw.lora(x, c.a, c.b, c.scales, lw.lora_plan(ids, 2), y=y, out=y)
    c.ids = ids[rows].cpu().numpy()
    c.check_forward(y[rows], None, torch.ones(8, N, dtype=torch.bfloat16, device="cuda"))
    assert (y[40000] == 1).all()


def test_inputs_past_32_bits(lw):
    T, N, K, R = 66000, 8, 65536, 8
    c = Case(lw, 8, N, K, R, 1, "fp16", "mixed")
    rows = [0, 1, 32767, 32768, 65535, 65536, 65537, T - 1]
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ids[rows] = 0
    x = torch.full((T, K), float("nan"), dtype=torch.float16, device="cuda")
    x[rows] = c.x
    dy, v = torch.zeros(T, N, dtype=torch.float16, device="cuda"), torch.zeros(T, R, device="cuda")
    dy[rows], v[rows] = c.dy, c.v
    plan = lw.lora_plan(ids, 1)
    out, vs = lw.lora(x, c.a, c.b, c.scales, plan, save=True)
    c.ids = np.zeros(8, np.int32)
    c.check_forward(out[rows], vs[rows], None)
    dx, da, db = lw.lora_grad(dy, x, v, c.a, c.b, c.scales, plan)
    c.check_backward(dx[rows], da, db, None)
    assert not dx[40000].any()


def test_pools_past_32_bits(lw):
    T, N, K, R, L = 5, 24, 65536, 128, 600
    c = Case(lw, T, N, K, R, 1, "bf16", "mixed")
    c.ids = np.zeros(T, np.int32)
    a = torch.zeros(L, R, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(L, N, R, dtype=torch.bfloat16, device="cuda")
    a[L - 1], b[L - 1] = c.a[0], c.b[0]
    plan = lw.lora_plan(torch.full((T,), L - 1, dtype=torch.int32, device="cuda"), L)
    scales = c.scales.repeat(L)
    out, v = lw.lora(c.x, a, b, scales, plan, y=c.y, save=True)
    c.check_forward(out, v, c.y)
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, a, b, scales, plan, dx=c.base)
    c.check_backward(dx, da[L - 1:], db[L - 1:], c.base)
    assert not da[:L - 1].any() and not db[:L - 1].any()


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_refusals(lw):
    c = Case(lw, 20, 64, 64, 16, 2, "fp16", "mixed")
    x, a, b, s, p, y = c.x, c.a, c.b, c.scales, c.plan, c.y
    wrong = [lambda: lw.lora(x, a, b, s, p, y=y.t()), lambda: lw.lora(x[:, ::2], a, b, s, p), lambda: lw.lora(x, a, b[:1], s, p),
             lambda: lw.lora(x, a, b, s[:1], p), lambda: lw.lora(x[:19].contiguous(), a, b, s, p), lambda: lw.lora(x.cpu(), a, b, s, p),
             lambda: lw.lora(x, a, b, s, p, y=y, out=x), lambda: lw.lora(x, a, b, s, p, y=y, out=y[:10]),
             lambda: lw.lora(x, a[0], b, s, p), lambda: lw.lora(x, a, b, s, p, out=a.view(-1)[:20 * 64].view(20, 64)),
             lambda: lw.lora_grad(c.dy, x, c.v[:, :8].contiguous(), a, b, s, p), lambda: lw.lora_grad(c.dy, x, c.v, a, b, s, p, out=x),
             lambda: lw.lora_plan(c.dev_ids, 2, out={"order": c.dev_ids})]
    for call in wrong:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lw.lora(x, a.bfloat16(), b, s, p), lambda: lw.lora(x, a, b, s.double(), p),
                 lambda: lw.lora(x, a, b, s, {k: t.long() for k, t in p.items()}),
                 lambda: lw.lora_grad(c.dy, x, c.v.half(), a, b, s, p), lambda: lw.lora_plan(c.dev_ids.long(), 2)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: lw.lora_plan(c.dev_ids, 1025), lambda: lw.lora(x, a[:, :4].contiguous(), b[:, :, :4].contiguous(), s, p),
                 lambda: lw.lora(x, a, b[:, :7].contiguous(), s, p)):
        with pytest.raises(lw.LowbitError):
            call()
    a.requires_grad_(True)
    with pytest.raises(ValueError, match="outside autograd"):
        lw.lora(x, a, b, s, p)
    with torch.no_grad():
        lw.lora(x, a, b, s, p)
    overlap = torch.zeros(21, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError), torch.no_grad():
        lw.lora(x, a, b, s, p, y=overlap[:20], out=overlap[1:])


# ---------------------------------------------------------------------------
# together: the projection, its adapters, streams and graphs, a training step
# ---------------------------------------------------------------------------
def projection(lw, g, N, K, bits, group):
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).half()
    q = lw.quantize_rtn(w, bits, group)
    return q["packed"], q["scales"], q["zeros"]


@pytest.mark.parametrize("T", [1, 12, 100])
def test_requests_beside_a_quantized_projection(lw, T):
    """4-bit projection and adapters of many requests: exactly lora on the projection's output."""
    g = torch.Generator(device="cuda").manual_seed(T)
    c = Case(lw, T, 512, 1024, 16, 8, "fp16", "mixed")
    w = projection(lw, g, 512, 1024, 4, 128)
    y = lw.qgemm(c.x, *w, 1024, 4, 128) if T > 15 else lw.qgemv(c.x, *w, 1024, 4, 128)
    c.check_forward(lw.lora(c.x, *c.pools(), y=y, out=y.clone() if T == 1 else None), None, y)
    w = projection(lw, g, 512, 1024, 8, 0)
    y = lw.linear_w8a8(c.x, *w)
    c.check_forward(lw.lora(c.x, *c.pools(), y=y), None, y)


def step(lw, ids, L, w, x, dy, a, b, scales, params, state, count):
    """Forward and backward pass of one layer with adapters, and an update of them."""
    plan = lw.lora_plan(ids, L)
    y = lw.linear_w8a8(x, *w)
    out, v = lw.lora(x, a, b, scales, plan, y=y, out=y, save=True)
    dx = lw.linear_w8a8_grad(dy, *w)
    dx, da, db = lw.lora_grad(dy, x, v, a, b, scales, plan, dx=dx, out=dx)
    lw.adamw(params, (da, db), state, lr=1e-2, weight_decay=0.01, step=count)
    return out, dx, da, db


def layer(lw, seed, kind="fp16", T=150, N=264, K=512, R=16, L=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = Case(lw, T, N, K, R, L, kind, "mixed", seed)
    w = projection(lw, g, N, K, 8, 0)
    with torch.no_grad():
        state = lw.adamw_state([c.a, c.b], bits=8, master=True)
    return c, (c.dev_ids, L, w, c.x, c.dy, c.a, c.b, c.scales, (c.a, c.b), state)


def results(c, args, outs):
    return [t.clone() for t in (*outs, c.a, c.b, *args[-1].values())]


def test_streams(lw):
    c, args = layer(lw, 0)
    want = results(c, args, step(lw, *args, 1))
    side = torch.cuda.Stream()
    c, args = layer(lw, 0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = results(c, args, step(lw, *args, 1))
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_captured_and_replayed(lw):
    """A whole step in a graph, replayed with new inputs, new ids, a new count of steps: as eager steps."""
    c, args = layer(lw, 1)
    count = torch.ones(1, dtype=torch.int32, device="cuda")
    step(lw, *args, count)  # libraries and the allocator are warm
    c, args = layer(lw, 1)
    eager, eager_args = layer(lw, 1)
    count.fill_(1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = step(lw, *args, count)
    for i in range(1, 6):
        fresh = Case(lw, 150, 264, 512, 16, 3, "fp16", "mixed" if i % 2 else "runs", seed=50 + i)
        for own in (c, eager):
            own.x.copy_(fresh.x)
            own.dy.copy_(fresh.dy)
            own.dev_ids.copy_(fresh.dev_ids)
        count.fill_(i)
        graph.replay()
        want = results(eager, eager_args, step(lw, *eager_args, i))
        torch.cuda.synchronize()
        got = results(c, args, outs)
        assert all(torch.equal(p, q) for p, q in zip(want, got)), i


def test_in_an_autograd_function(lw):
    """A layer with trained adapters in autograd: gradients of x, a and b as the reference has them."""
    c = Case(lw, 100, 96, 128, 16, 2, "bf16", "mixed")
    g = torch.Generator(device="cuda").manual_seed(0)
    w = projection(lw, g, 96, 128, 8, 0)

    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, a, b):
            y = lw.linear_w8a8(x, *w)
            out, v = lw.lora(x, a, b, c.scales, c.plan, y=y, out=y, save=True)
            ctx.save_for_backward(x, a, b, v)
            return out

        @staticmethod
        def backward(ctx, dy):
            x, a, b, v = ctx.saved_tensors
            dy = dy.contiguous()
            dx, da, db = lw.lora_grad(dy, x, v, a, b, c.scales, c.plan, dx=lw.linear_w8a8_grad(dy, *w))
            return dx, da.to(a.dtype), db.to(b.dtype)

    for t in (c.x, c.a, c.b):
        t.requires_grad_(True)
    Layer.apply(c.x, c.a, c.b).backward(c.dy)
    with torch.no_grad():
        base = lw.linear_w8a8_grad(c.dy, *w)
        _, c.v = lw.lora(c.x, *c.pools(), save=True)
        dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=base)
    x, a, b = c.x, c.a, c.b
    c.x, c.a, c.b = (t.detach().clone() for t in (x, a, b))
    c.check_backward(x.grad, da, db, base)
    assert torch.equal(a.grad, da.bfloat16()) and torch.equal(b.grad, db.bfloat16())


def test_two_calls_at_once(lw):
    """Calls on two streams at the same time, each with a workspace of its own."""
    cases = [Case(lw, 900, 513, 1024, 32, 3, "bf16", "runs", seed=i) for i in range(2)]
    want = [(*lw.lora(c.x, *c.pools(), y=c.y, save=True), *lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    got = [None, None]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i] = (*lw.lora(c.x, *c.pools(), y=c.y, save=True), *lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for w, g in zip(want, got) for p, q in zip(w, g))


def test_first_calls_captured():
    """In a new process, the very first calls go into a graph."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    print("[adapters] first calls captured", flush=True)
    code = """
import torch, sys
sys.path.insert(0, %r)
import weight_only_bit_rtn_amd as lw
g = torch.Generator(device="cuda").manual_seed(0)
sets = []
for T, R in ((1, 8), (300, 64), (300, 128)):
    n = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    sets.append((n(T, 256), n(T, 200), n(2, R, 256), n(2, 200, R), torch.ones(2, device="cuda"),
                 (torch.arange(T, device="cuda") %% 3 - 1).int()))
def run(x, y, a, b, s, ids):
    plan = lw.lora_plan(ids, 2)
    out, v = lw.lora(x, a, b, s, plan, y=y, save=True)
    return (out, v, *lw.lora_grad(y, x, v, a, b, s, plan))
p, q = (torch.ones(5000, device="cuda") for _ in range(2))
mine = {k: torch.zeros(5120 if len(k) == 1 else 20, dtype=torch.uint8 if len(k) == 1 else torch.float32, device="cuda")
        for k in ("m", "v", "m_max", "v_max")}
other = {k: t.clone() for k, t in mine.items()}
grad = torch.randn(5000, generator=g, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = [run(*s) for s in sets]
    lw.adamw([p], [grad], mine, lr=1e-2, step=5)
for _ in range(3):
    graph.replay()
    lw.adamw([q], [grad], other, lr=1e-2, step=5)
    torch.cuda.synchronize()
    for s, o in zip(sets, outs):
        assert all(torch.equal(x, y) for x, y in zip(o, run(*s)))
    assert torch.equal(p, q) and all(torch.equal(mine[k], other[k]) for k in mine)
print("captured")
""" % root
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
