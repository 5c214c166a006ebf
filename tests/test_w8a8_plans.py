"""Every kernel and tile plan that the library takes for sizes of real layers,
by the library's own planner: on the CPU, that each listed size takes the plan
it stands for, that sizes drawn from the whole range take no other, and that the
built library agrees; on the GPU, the operators at these sizes against their
definition in 64 bits.

A plan is a tile of tokens x weight rows (gradients: columns of dx) and whether
the tiles are whole, shared out along the summed index, or both; few<n> are the
kernels of up to n tokens (which quantize x themselves, or take codes), ring<n>
those of up to 16 n.  N is odd and T leaves a part of a tile throughout.
"""
from __future__ import annotations

import os
import random
import subprocess

import pytest

import w8a8_reference as ref

HERE = os.path.dirname(os.path.abspath(__file__))
CUS = 256

# of several found, the sizes of each plan with the least work
PLANS = {
    "gated": [
        ("128x128 both", (3268, 591, 4000)),
        ("128x128 shared", (599, 65, 9440)),
        ("128x128 whole", (1219, 769, 32)),
        ("192x192 both", (263, 12291, 3680)),
        ("192x192 shared", (3238, 69, 11488)),
        ("192x192 whole", (1572, 2317, 96)),
        ("256x128 both", (1010, 4121, 3936)),
        ("256x128 shared", (2727, 197, 6752)),
        ("256x128 whole", (1411, 1365, 96)),
        ("256x192 both", (1629, 3481, 8544)),
        ("256x192 shared", (3327, 261, 8832)),
        ("256x192 whole", (1543, 1219, 32)),
        ("256x256 both", (1333, 5477, 2016)),
        ("256x256 shared", (1957, 1115, 5952)),
        ("256x256 whole", (2350, 2413, 32)),
        ("256x384 both", (1876, 12371, 736)),
        ("256x384 shared", (2636, 913, 8864)),
        ("256x384 whole", (2824, 2689, 32)),
        ("64x128 both", (49, 17379, 5088)),
        ("64x128 shared", (67, 49, 2240)),
        ("64x128 whole", (65, 49, 32)),
        ("few1 codes", (1, 33, 16416)),
        ("few1 fused", (1, 17, 32)),
        ("few2 codes", (2, 17, 8256)),
        ("few2 fused", (2, 17, 32)),
        ("few4 codes", (4, 17, 4128)),
        ("few4 fused", (3, 17, 32)),
        ("ring1 whole", (5, 17, 32)),
        ("ring2 whole", (17, 17, 32)),
        ("ring3 whole", (33, 17, 32)),
        ("ring4 whole", (49, 17, 32)),
    ],
    "gated_grad": [
        ("128x128 both", (1543, 583, 2464)),
        ("128x128 shared", (67, 449, 32)),
        ("128x128 whole", (65, 49, 32)),
        ("128x256 both", (1629, 4041, 5056)),
        ("128x256 shared", (1322, 881, 928)),
        ("128x256 whole", (262, 49, 11680)),
        ("16x128 shared", (1, 705, 32)),
        ("16x128 whole", (1, 49, 32)),
        ("256x192 both", (3878, 321, 9344)),
        ("256x192 shared", (3217, 1577, 160)),
        ("256x192 whole", (523, 49, 13408)),
        ("256x256 both", (1468, 601, 10912)),
        ("256x256 shared", (2719, 2037, 992)),
        ("256x256 whole", (797, 51, 12896)),
        ("32x128 shared", (17, 705, 32)),
        ("32x128 whole", (17, 49, 32)),
        ("64x128 shared", (33, 579, 32)),
        ("64x128 whole", (33, 49, 32)),
        ("64x256 shared", (37, 1039, 6592)),
    ],
    "linear": [
        ("128x128 both", (2461, 1559, 4160)),
        ("128x128 shared", (1882, 49, 5568)),
        ("128x128 whole", (1627, 1159, 32)),
        ("192x192 both", (257, 25067, 3712)),
        ("192x192 shared", (3222, 145, 12288)),
        ("192x192 whole", (3084, 2449, 96)),
        ("256x128 both", (980, 8283, 3936)),
        ("256x128 shared", (3751, 263, 7200)),
        ("256x128 whole", (2434, 1567, 96)),
        ("256x192 both", (1309, 8067, 7840)),
        ("256x192 shared", (3558, 553, 11360)),
        ("256x192 whole", (2450, 1541, 32)),
        ("256x256 both", (554, 21833, 2016)),
        ("256x256 shared", (3533, 1157, 6496)),
        ("256x256 whole", (3329, 3471, 32)),
        ("256x384 both", (3075, 15229, 736)),
        ("256x384 shared", (969, 4133, 8864)),
        ("256x384 whole", (3130, 4895, 32)),
        ("64x128 both", (50, 34649, 2560)),
        ("64x128 shared", (71, 49, 2240)),
        ("64x128 whole", (66, 49, 32)),
        ("few1 codes", (1, 33, 16416)),
        ("few1 fused", (1, 17, 32)),
        ("few2 codes", (2, 17, 8224)),
        ("few2 fused", (2, 17, 32)),
        ("ring1 whole", (3, 17, 32)),
        ("ring2 whole", (17, 17, 32)),
        ("ring3 whole", (33, 17, 32)),
        ("ring4 whole", (49, 17, 32)),
    ],
    "linear_grad": [
        ("128x128 both", (1160, 1219, 3264)),
        ("128x128 shared", (70, 899, 32)),
        ("128x128 whole", (65, 49, 32)),
        ("128x256 both", (1594, 8161, 5024)),
        ("128x256 shared", (1293, 1765, 928)),
        ("128x256 whole", (257, 49, 11072)),
        ("16x128 shared", (1, 1409, 32)),
        ("16x128 whole", (1, 49, 32)),
        ("256x192 both", (2070, 975, 10848)),
        ("256x192 shared", (3260, 2839, 160)),
        ("256x192 whole", (663, 49, 11616)),
        ("256x256 both", (1176, 1325, 13184)),
        ("256x256 shared", (2888, 3475, 992)),
        ("256x256 whole", (844, 49, 12512)),
        ("32x128 shared", (20, 1409, 32)),
        ("32x128 whole", (17, 49, 32)),
        ("64x128 shared", (38, 1217, 32)),
        ("64x128 whole", (33, 49, 32)),
        ("64x256 shared", (33, 2067, 6656)),
    ],
}
EVERY = [(op, plan, shape) for op, plans in PLANS.items() for plan, shape in plans]


# ---------------------------------------------------------------------------
# without a GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    """[(plan, bytes of the shares)] of [(op, T, N, K)], from the header that the library is built with."""
    exe = str(tmp_path_factory.mktemp("plans") / "plans")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", os.path.join(HERE, "native", "w8a8_plans.cpp"),
                    "-o", exe], check=True)

    def ask(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        r = subprocess.run([exe, str(CUS)], input=text, capture_output=True, text=True, check=True)
        rows = [line.rsplit(" ", 1) for line in r.stdout.splitlines()]
        assert len(rows) == len(sizes)
        return [(plan, int(size)) for plan, size in rows]

    return ask


def drawn(op, count, seed):
    """Sizes of layers: weights up to the largest layer's, spread over their logarithms."""
    rng = random.Random(seed)
    two = 2 if op.startswith("gated") else 1
    out = []
    while len(out) < count:
        T, N = int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(6, 15.6))
        K = 32 * int(2 ** rng.uniform(1, 9))
        if two * N * K <= 49152 * 12288:
            out.append((op, T, N, K))
    return out


def test_listed_sizes_take_their_plans(planner):
    asked = planner([(op, *shape) for op, _, shape in EVERY])
    assert [(op, plan) for op, plan, _ in EVERY] == [(e[0], a[0]) for e, a in zip(EVERY, asked)]


@pytest.mark.parametrize("op", PLANS)
def test_no_other_plan_is_taken(planner, op):
    sizes = drawn(op, 150000, seed=len(op))
    missing = {}
    listed = {plan for plan, _ in PLANS[op]}
    for size, (plan, _) in zip(sizes, planner(sizes)):
        if plan not in listed:
            missing.setdefault(plan, size)
    assert missing == {}


def test_the_library_plans_alike(planner):
    """The room for shares is what the library asks for beside its other parts (its planner knows no GPU here and
    takes one of 256 CUs)."""
    import weight_only_bit_rtn_amd as lw
    query = {"linear": lambda *s: lw.linear_w8a8_workspace_bytes(*s, 2),
             "gated": lambda *s: lw.gated_w8a8_workspace_bytes(*s, 2),
             "linear_grad": lw.linear_w8a8_grad_workspace_bytes, "gated_grad": lw.gated_w8a8_grad_workspace_bytes}
    up256 = lambda v: (v + 255) // 256 * 256
    for op in PLANS:
        sizes = drawn(op, 2000, seed=1) + [(op, *shape) for _, shape in PLANS[op]]
        for (_, T, N, K), (plan, shares) in zip(sizes, planner(sizes)):
            if op.endswith("grad"):
                pitch = (N + 63) // 64 * 64 * (2 if op == "gated_grad" else 1)
                shares += up256(2 * T * pitch) + 2 * up256(4 * T)
            assert query[op](T, N, K) == shares, (op, T, N, K, plan)


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lw():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.get_device_properties(0).multi_processor_count != CUS:
        pytest.skip("the sizes are those of a device of 256 CUs")
    import weight_only_bit_rtn_amd as lw
    lw.load_library()
    return lw


def kind_of(i):
    import torch
    return (("fp16", torch.float16), ("bf16", torch.bfloat16))[i % 2]


def check_product(lw, g, gated, T, N, K, kind, dtype):
    import torch
    from test_w8a8_gpu import inside, integers, random_weights
    ws = [random_weights(g, N, K) for _ in range(2 if gated else 1)]
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    q = lw.quantize_act(x)

    def value(w):
        """fl32(fl32(S s) d): the integer sum d is exact in 64 bits."""
        d = q["codes"].double() @ integers(w).t()
        return q["scales"][:, None] * w[1].float().t() * d.float()

    if not gated:
        y = lw.linear_w8a8(x, *ws[0])
        assert bool((y == value(ws[0]).to(dtype)).all())
        assert bool((lw.linear_w8a8(q, *ws[0], out_dtype=dtype) == y).all())
        return
    gate, up = value(ws[0]), value(ws[1])
    h, hg, hu = lw.gated_w8a8(x, *ws[0], *ws[1], save=True)
    assert bool((hg == gate.to(dtype)).all()) and bool((hu == up.to(dtype)).all())
    v = gate.double()
    want = v * torch.sigmoid(v) * up.double()
    # sigma: an error of r in g moves it by |g| r at the most; exp, the sum, the reciprocal and three products
    r = (20 + 20 * v.abs().clamp(max=104)) * ref.U32
    inside(h, want, want.abs() * (ref.HALF_STEP[kind] * 1.001 + r) + ref.HALF_TINY[kind], "h")
    assert bool((lw.gated_w8a8(q, *ws[0], *ws[1], out_dtype=dtype) == h).all())


def check_grad(lw, g, gated, T, N, K, kind, dtype):
    import torch
    from test_w8a8_gpu import inside, integers, random_weights
    ws = [random_weights(g, N, K) for _ in range(2 if gated else 1)]
    d = (torch.randn(T, N, generator=g, device="cuda") * 0.05).to(dtype)
    if gated:
        gate, up = (torch.randn(T, N, generator=g, device="cuda").to(dtype) for _ in range(2))
        v = gate.double()
        s = torch.sigmoid(v)
        parts = [(d.double() * up.double() * (s + v * s * (1 - s)), ws[0]), (d.double() * v * s, ws[1])]
        # the slope's terms cancel: their errors are bounded by their own size, 64 half steps of d up
        extra = [(d.double() * up.double()).abs() * 64 * ref.U32, parts[1][0].abs() * 64 * ref.U32]
        call = lambda: lw.gated_w8a8_grad(d, gate, up, *ws[0], *ws[1])
    else:
        parts, extra = [(d.double(), ws[0])], [0]
        call = lambda: lw.linear_w8a8_grad(d, *ws[0])
    scale = [w[1].double().t() for w in ws]
    want = sum((p * s) @ integers(w) for (p, w), s in zip(parts, scale))
    # a factor: half a step of 11 bits and a few of 24, or half of fp16's smallest step below 2^-29 of the token's
    # largest; the sums of the terms in 32 bits; over code - 128 and 128 - z
    top = torch.stack([(p.abs() * s).amax(1) for (p, _), s in zip(parts, scale)]).amax(0)[:, None]
    terms = N * len(parts)
    bound = want.abs() * ref.HALF_STEP[kind] * 1.01 + ref.HALF_TINY[kind]
    for (p, w), s, e in zip(parts, scale, extra):
        size = (integers(w) + w[2].double() - 128).abs() + (128 - w[2].double()).abs()
        bound += ((p.abs() * (2.0 ** -11 + 8 * ref.U32 + terms * 2.0 ** -23) + e) * s + top * 2.0 ** -39) @ size * 1.01
    dx = call()
    inside(dx, want, bound, "dx")
    if N >= 512:    # sums of independent roundings: half a step each at the most, in the 2-norm
        assert float((dx.double() - want).norm()) <= float(want.norm()) * (2.0 ** -11 + ref.HALF_STEP[kind])
    assert bool((call() == dx).all())


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(EVERY)), ids=lambda i: " ".join(map(str, EVERY[i])))
def test_plan(lw, i):
    import torch
    op, plan, (T, N, K) = EVERY[i]
    print("[w8a8]", op, plan, T, N, K, flush=True)
    g = torch.Generator(device="cuda").manual_seed(i)
    check = check_grad if op.endswith("grad") else check_product
    check(lw, g, op.startswith("gated"), T, N, K, *kind_of(i))
    torch.cuda.empty_cache()
