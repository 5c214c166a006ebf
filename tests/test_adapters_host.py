"""The adapters and the AdamW step without a GPU: headers and binding agree, bad arguments are
refused on the host before anything is launched, and the 64-bit reference of the GPU tests is
what it says (hand-worked numbers, differences)."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest

import adapters_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lw():
    import weight_only_bit_rtn_amd as lw
    if not os.path.exists(lw.LIB_PATH):
        from weight_only_bit_rtn_amd import build
        build.build()
    lw.load_library()
    return lw


@pytest.mark.parametrize("name", ["lora", "adamw"])
def test_header_library_and_binding_agree(lw, name):
    text = open(os.path.join(ROOT, "include", f"lowbit_{name}.h")).read()
    declared = set(re.findall(r"LOWBIT_API\s+[\w\s\*]+?\b(lowbit_\w+)\s*\(", text))
    assert declared == set(lw.EXPORTED_LORA if name == "lora" else lw.EXPORTED_ADAMW)
    lib = ctypes.CDLL(lw.LIB_PATH)
    for entry in declared:
        assert hasattr(lib, entry), entry
    consts = {k: int(v) for k, v in re.findall(r"#define\s+(LOWBIT_\w+)\s+(\d+)", text)}
    if name == "lora":
        assert (consts["LOWBIT_LORA_MAX_R"], consts["LOWBIT_LORA_MAX_L"], consts["LOWBIT_LORA_MIN_N"]) == (
            lw.LORA_MAX_R, lw.LORA_MAX_L, lw.LORA_MIN_N)
    else:
        from weight_only_bit_rtn_amd import optimizer
        assert (consts["LOWBIT_ADAMW_BLOCK"], consts["LOWBIT_F32"]) == (lw.ADAMW_BLOCK, optimizer.F32)
        fields = re.search(r"typedef struct \{\s*double([^}]+)\}", text)[1]
        assert [f.strip(" *") for f in re.sub(r"int64_t|int32_t|float|const|\n", "", fields).replace(";", ",").split(",")
                if f.strip()] == [f for f, _ in lw.AdamwOptions._fields_]


# Addresses that are never dereferenced: each call is refused, or empty.
P = 0x7F0000000000
MIS = P + 2
BIG = 1 << 50
ARG, SHAPE, UNSUPPORTED = -1, -2, -3


def plan(lw, ids=P, T=4, L=2, order=P, starts=P):
    return lw.lora_plan_raw(ids, T, L, order, starts, None)


def lora(lw, x=P, dtype=0, T=4, order=P, starts=P, a=P, b=P, scales=P, L=2, R=8, N=16, K=64, y=P, out=P, v=None, ws=P,
         size=BIG):
    return lw.lora_raw(x, dtype, T, order, starts, a, b, scales, L, R, N, K, y, out, v, ws, size, None)


def lora_grad(lw, dy=P, x=P, v=P, dtype=0, T=4, order=P, starts=P, a=P, b=P, scales=P, L=2, R=8, N=16, K=64, base=P,
              dx=P, da=P, db=P, ws=P, size=BIG):
    return lw.lora_grad_raw(dy, x, v, dtype, T, order, starts, a, b, scales, L, R, N, K, base, dx, da, db, ws, size,
                            None)


def adamw(lw, tensors=((P, P, 10),), count=None, p=3, g=3, bits=8, m=P, v=P, m_max=P, v_max=P, master=None, lr=1e-3,
          beta1=0.9, beta2=0.999, eps=1e-8, decay=0.0, step=1, lr_at=None, step_at=None, scale_at=None, table=True,
          state=True, options=True):
    words = (ctypes.c_int64 * (3 * len(tensors) + 1))(*[w or 0 for t in tensors for w in t])
    place = lw.AdamwState(m, v, m_max, v_max, master) if state else None
    opt = lw.AdamwOptions(lr, beta1, beta2, eps, decay, step, lr_at, step_at, scale_at) if options else None
    return lw.adamw_raw(ctypes.addressof(words) if table else None, len(tensors) if count is None else count, p, g, bits,
                        place, opt, None)


def moments(lw, m=P, v=P, m_max=P, v_max=P, blocks=3, m_out=P, v_out=P):
    return lw.adamw_moments_raw(m, v, m_max, v_max, blocks, m_out, v_out, None)


BOTH = (lora, lora_grad)
NAN, INF = float("nan"), float("inf")
REFUSED = (
    [(f, dict(T=-1), ARG) for f in (plan, *BOTH)] + [(f, dict(L=-1), ARG) for f in (plan, *BOTH)]
    + [(f, dict(L=n), SHAPE) for f in (plan, *BOTH) for n in (0, 1025)]
    + [(f, dict(T=(1 << 20) + 1), SHAPE) for f in (plan, *BOTH)]
    + [(plan, {k: x}, ARG) for k in ("ids", "order", "starts") for x in (None, MIS)]
    + [(f, dict(dtype=d), UNSUPPORTED) for f in BOTH for d in (-1, 2, 3)]
    + [(f, dict(R=r), SHAPE) for f in BOTH for r in (0, 4, 12, 136)] + [(f, dict(R=-8), ARG) for f in BOTH]
    + [(f, dict(K=k), SHAPE) for f in BOTH for k in (0, 16, 65, 131072 + 32)] + [(f, dict(K=-32), ARG) for f in BOTH]
    + [(f, dict(N=n), SHAPE) for f in BOTH for n in (0, 7, (1 << 20) + 1)] + [(f, dict(N=-1), ARG) for f in BOTH]
    + [(f, dict(T=1 << 20, N=1 << 17), SHAPE) for f in BOTH] + [(f, dict(T=1 << 20, K=65536 + 32), SHAPE) for f in BOTH]
    + [(f, dict(L=1024, R=128, N=(1 << 19) + 8), SHAPE) for f in BOTH]
    + [(lora, {k: x}, ARG) for k in ("x", "order", "starts", "a", "b", "scales", "out", "ws") for x in (None, MIS)]
    + [(lora, dict(y=MIS), ARG), (lora, dict(v=MIS), ARG), (lora, dict(size=0), ARG), (lora, dict(ws=P + 16), ARG)]
    + [(lora_grad, {k: x}, ARG) for k in ("dy", "x", "v", "order", "starts", "a", "b", "scales", "dx", "da", "db", "ws")
       for x in (None, MIS)]
    + [(lora_grad, dict(base=MIS), ARG), (lora_grad, dict(size=0), ARG), (lora_grad, dict(ws=P + 16), ARG)]
    + [(adamw, dict(p=x), UNSUPPORTED) for x in (-1, 2, 4)] + [(adamw, dict(g=x), UNSUPPORTED) for x in (-1, 2, 4)]
    + [(adamw, dict(bits=x), UNSUPPORTED) for x in (0, 4, 16)]
    + [(adamw, dict(count=-1), ARG), (adamw, dict(table=False), ARG), (adamw, dict(state=False), ARG),
       (adamw, dict(options=False), ARG)]
    + [(adamw, {k: x}, ARG) for k in ("lr", "eps", "decay") for x in (-1e-3, NAN, INF)]
    + [(adamw, {k: x}, ARG) for k in ("beta1", "beta2") for x in (-0.1, 1.0, NAN)]
    + [(adamw, dict(step=0), ARG)] + [(adamw, {k: MIS + 1}, ARG) for k in ("lr_at", "step_at", "scale_at")]
    + [(adamw, {k: x}, ARG) for k in ("m", "v", "m_max", "v_max") for x in (None, MIS)]
    + [(adamw, dict(bits=32), ARG), (adamw, dict(bits=32, m_max=None), ARG), (adamw, dict(master=MIS), ARG)]
    + [(adamw, dict(tensors=((P, P, 5), t)), ARG) for t in ((None, P, 3), (P, None, 3), (MIS, P, 3), (P, MIS, 3), (P, P, -1))]
    + [(adamw, dict(tensors=((P, P, 1 << 36), (P, P, 1))), SHAPE), (adamw, dict(tensors=((P, P, 1 << 62),)), SHAPE)]
    + [(moments, dict(blocks=-1), ARG), (moments, dict(blocks=(1 << 28) + 1), SHAPE)]
    + [(moments, {k: x}, ARG) for k in ("m", "v", "m_max", "v_max", "m_out", "v_out") for x in (None, MIS)])


@pytest.mark.parametrize("f,args,status", REFUSED)
def test_refused_on_the_host(lw, f, args, status):
    assert f(lw, **args) == status


EMPTY = [(lora, dict(T=0)), (adamw, dict(tensors=())), (adamw, dict(tensors=((None, None, 0), (MIS, P, 0)))),
         (adamw, dict(count=0, table=False, state=False)), (moments, dict(blocks=0))]


@pytest.mark.parametrize("f,args", EMPTY)
def test_empty_problems_launch_nothing(lw, f, args):
    assert f(lw, **args) == 0


SIZES = [(T, N, K, R, L) for T in (1, 16, 17, 64, 255, 257, 5000, 1 << 20) for N in (8, 65, 4096) for K in (32, 4096)
         for R in (8, 72, 128) for L in (1, 7, 1024)]


def test_workspace_sizes(lw):
    for T, N, K, R, L in SIZES:
        need, grad = lw.lora_workspace_bytes(T, N, K, R, L), lw.lora_grad_workspace_bytes(T, N, K, R, L)
        # one share of every token's coefficients at the least, and no more than 64, or of N's 4
        assert 4 * T * R <= need <= 64 * 4 * T * R
        assert 4 * T * R <= grad <= 4 * 4 * T * R + 4 * R * (K + N) * (2 * T / 128 + 1)
        if need < 1 << 40:
            assert lora(lw, T=T, N=N, K=K, R=R, L=L, size=need - 1) == ARG
            assert lora_grad(lw, T=T, N=N, K=K, R=R, L=L, size=grad - 1) == ARG
    assert lw.lora_workspace_bytes(0, 8, 32, 8, 1) == 0 == lw.lora_grad_workspace_bytes(0, 8, 32, 8, 1)
    for f in (lw.lora_workspace_bytes, lw.lora_grad_workspace_bytes):
        assert f(4, 16, 65, 8, 2) == SHAPE and f(-1, 16, 64, 8, 2) == ARG and f(4, 16, 64, 12, 2) == SHAPE


def test_binding_refuses(lw):
    import torch
    h = torch.float16
    x, a, b = torch.zeros(4, 64, dtype=h), torch.zeros(2, 8, 64, dtype=h), torch.zeros(2, 16, 8, dtype=h)
    s = torch.ones(2)
    p = {"order": torch.arange(4, dtype=torch.int32), "starts": torch.zeros(3, dtype=torch.int32)}
    for call in (lambda: lw.lora_plan(torch.zeros(4, dtype=torch.int32), 2), lambda: lw.lora(x, a, b, s, p),
                 lambda: lw.lora_grad(torch.zeros(4, 16, dtype=h), x, torch.zeros(4, 8), a, b, s, p),
                 lambda: lw.adamw([x], [x], {}, lr=1e-3), lambda: lw.adamw_state([x]),
                 lambda: lw.adamw([x], [], {}, lr=1e-3), lambda: lw.adamw_state([]),
                 lambda: lw.adamw_state([x], bits=4), lambda: lw.lora_plan(torch.zeros(2, 2), 2)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: lw.lora_plan([0, 1], 2), lambda: lw.lora(x.float(), a, b, s, p), lambda: lw.adamw([3], [3], {}, lr=1)):
        with pytest.raises(TypeError):
            call()
    lw.adamw([], [], {}, lr=1e-3)


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------
def test_plan_by_hand():
    order, starts = ref.plan([2, 0, -1, 2, 0, 9, 1], 3)
    assert order.tolist() == [1, 4, 6, 0, 3, 2, 5] and starts.tolist() == [0, 2, 3, 5]


def test_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, N, K, R, L = 5, 4, 6, 2, 3
    x, a, b = rng.standard_normal((T, K)), rng.standard_normal((L, R, K)), rng.standard_normal((L, N, R))
    s, ids, y, dy = rng.standard_normal(L), np.array([1, 0, -1, 1, 7]), rng.standard_normal((T, N)), rng.standard_normal((T, N))
    out, v = ref.lora(x, a, b, s, ids, y)
    dx, da, db = ref.lora_grad(dy, x, v, a, b, s, ids)
    for of, grad in ((x, dx), (a, da), (b, db)):
        for i in np.ndindex(of.shape):
            was, ends = of[i], []
            for h in (1e-4, -1e-4):
                of[i] = was + h
                ends.append((ref.lora(x, a, b, s, ids, y)[0] * dy).sum())
            of[i] = was
            assert abs((ends[0] - ends[1]) / 2e-4 - grad[i]) < 1e-8 * (1 + abs(grad[i]))
    assert not dx[2].any() and not dx[4].any() and not da[2].any() and not db[2].any()


def test_codes_by_hand():
    n7, n8 = ref.numbers(7), ref.numbers(8)
    assert n7[127] == n8[255] == 1 and n7[0] == n8[0] == 0
    assert n7[126] == n8[254] == 0.9375 and n7[119] == n8[247] == 0.5 and n7[1] == 1.25 * 2.0 ** -16 and n8[1] == 1.25 * 2.0 ** -32
    assert (np.diff(n7) > 0).all() and (np.diff(n8) > 0).all()
    x = np.zeros(256, np.float32)
    x[:6] = [4, -2, 3.875, 3.8, 1e-9, 4 * 1.1875 * 2.0 ** -16]     # 3.875: halfway between 3.75 and 4
    m, top = ref.encode(x, 7)
    assert top[0] == 4 and m[:7].tolist() == [127, 128 + 119, 127, 126, 0, 1, 0]
    v, _ = ref.encode(np.abs(x), 8)
    # v reaches 2^-32: 1e-9 / 4 is 1.0737 * 2^-32, below its first number and not 0; 1.1875 * 2^-16 is halfway again
    assert v[:7].tolist() == [255, 247, 255, 254, 1, 129, 0]
    assert ref.encode(np.where(np.arange(256) == 1, np.float32(1e-30), x[0]).astype(np.float32), 8)[0][1] == 1
    for bad in (np.nan, np.inf, -np.inf):
        x[9] = bad
        m, top = ref.encode(x, 7)
        assert np.isnan(top[0]) and not m.any()
        assert np.isnan(ref.decode(m, m, top, top)[0]).all()
    x[:] = 1e-39
    m, top = ref.encode(x, 7)
    assert top[0] == 0 and not m.any()


def test_codes_are_the_nearest():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(256 * 20) * np.exp(rng.standard_normal(256 * 20) * 2)).astype(np.float32)
    for bits, val in ((7, x), (8, np.abs(x))):
        code, top = ref.encode(val, bits)
        back = numbers_of(code, bits) * np.repeat(top.astype(np.float64), 256)
        tab = ref.numbers(bits).astype(np.float64)
        every = np.abs(np.abs(val.reshape(-1, 1).astype(np.float64)) - tab * np.repeat(top, 256)[:, None].astype(np.float64))
        off = np.abs(np.abs(val) - np.abs(back))
        far = np.abs(val) / np.repeat(top, 256) > 2.0 ** -15
        assert (off[far] <= every.min(1)[far] + 2 * ref.U32 * np.abs(val)[far]).all()


def numbers_of(code, bits):
    n = ref.numbers(bits).astype(np.float64)
    return n[code] if bits == 8 else np.where(code > 127, -1, 1) * n[code & 127]


def test_update_by_hand():
    m, v = ref.moments(np.zeros(1, np.float32), np.zeros(1, np.float32), np.array([2.0]), 0.9, 0.999)
    p, taken = ref.update(np.array([1.0]), m, v, 0.1, 0.9, 0.999, 0.0, 0.5, 1)
    # the first step is lr in the gradient's direction, whatever its size
    assert abs(taken[0] - 0.1) < 1e-7 and abs(p[0] - (1 - 0.05 - 0.1)) < 1e-7
