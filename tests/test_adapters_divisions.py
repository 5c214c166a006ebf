"""The repeating parts of the adapter kernels: shapes whose workgroups go many times round their loops, by
the library's own division of a call.  On the CPU, that each shape is divided as it is there for; on the
GPU, results at these shapes against the definition in 64 bits.

Long chunks (gradients of a and b): many rounds of 64 tokens, several chunks to an adapter, and values of u
and v whose largest rises, falls and rises again from round to round, so that fp16's power of two follows.
Wide dx: several column ranges to a workgroup.  Long expansions, contractions and u: several steps to a wave,
in tiles of 16 and of 64 tokens.  Of the long side some columns are checked, which the definition gives one
by one."""
from __future__ import annotations

import os
import subprocess

import numpy as np
import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import adapters_reference as ref
from test_adapters_gpu import Case, f64, lw  # noqa: F401  (lw is a fixture)

HERE = os.path.dirname(os.path.abspath(__file__))

# T, N, K, R, L
LONG_SUMS_A = [(1290, 777, 65536, 8, 2), (1290, 1001, 65568, 16, 1), (1290, 1001, 65536, 24, 2), (1290, 1001, 34816, 64, 2),
               (1290, 515, 17408, 128, 1)]
LONG_SUMS_B = [(1290, 65537, 64, 16, 1), (1290, 66001, 96, 24, 2), (1290, 34817, 64, 64, 2), (1290, 17409, 64, 128, 1)]
LONG_U = [(300, 8001, 288, 8, 2), (300, 8003, 96, 24, 1), (300, 8001, 64, 64, 2), (300, 9001, 64, 128, 1), (140, 8200, 32, 40, 2)]
LONG_UP = [(250, 3001, 96, 16, 250), (250, 3003, 64, 24, 250), (200, 5001, 96, 64, 120), (200, 3001, 64, 128, 120),
           (1500, 3841, 96, 16, 100), (1500, 4099, 64, 24, 100), (1500, 3841, 64, 64, 100), (1500, 2177, 64, 104, 100)]
LONG_DOWN = [(33, 65, 12320, 16, 2), (33, 67, 12320, 64, 2), (33, 67, 12320, 128, 2), (500, 65, 16416, 24, 2),
             (500, 130, 16416, 128, 2)]


@pytest.fixture(scope="module")
def divide(tmp_path_factory):
    """Divisions of [(op, T, N, K, R, L)], from the header that the library is built with."""
    exe = str(tmp_path_factory.mktemp("divisions") / "divisions")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", os.path.join(HERE, "native", "adapter_divisions.cpp"),
                    "-o", exe], check=True)

    def ask(sizes):
        text = "\n".join(" ".join(map(str, s)) for s in sizes)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        names = {"lora": ("tile", "tiles", "splits", "k_share", "ranges", "n_share"),
                 "lora_grad": ("tiles", "splits", "n_share", "chunk", "chunks", "shares", "dx_cols", "k_cols")}
        rows = [dict(zip(names[s[0]], map(int, line.split()))) for s, line in zip(sizes, r.stdout.splitlines())]
        assert len(rows) == len(sizes)
        return rows

    return ask


def test_shapes_are_divided_as_they_are_there_for(divide):
    for shapes in (LONG_SUMS_A, LONG_SUMS_B):
        for (T, N, K, R, L), d in zip(shapes, divide([("lora_grad", *s) for s in shapes])):
            # six rounds of 64 tokens in a chunk at the least, two chunks in an adapter's at the least, a ragged last one
            assert d["chunk"] >= 6 * 64 and T // L >= d["chunk"] + 64 and T % 64 and d["shares"] > 0
            assert shapes is LONG_SUMS_B or (d["dx_cols"] >= 2 and d["k_cols"] > d["dx_cols"])
    for s, d in zip(LONG_U, divide([("lora_grad", *s) for s in LONG_U])):
        assert d["splits"] > 1 and d["n_share"] >= 4 * 512
    for (T, N, K, R, L), d in zip(LONG_UP, divide([("lora", *s) for s in LONG_UP])):
        step = 4 * (64 if R <= 64 else 32)  # outputs that a workgroup's waves take at a time
        assert d["n_share"] > 2 * step and d["tile"] == (16 if T <= 256 else 64)
    for (T, N, K, R, L), d in zip(LONG_DOWN, divide([("lora", *s) for s in LONG_DOWN])):
        step = 64 * (8 if d["tile"] == 16 and R <= 32 else 4)  # of K
        assert d["k_share"] > 3 * step and d["splits"] > 1
    # both heights of tiles, and every number of blocks of 16 ranks that kernels are made for
    assert {(s[0] <= 256, min(8, 1 << (-(-s[3] // 16) - 1).bit_length())) for s in LONG_UP} == {(t, b) for t in (True, False) for b in (1, 2, 4, 8)}


def test_the_library_divides_alike(divide):
    """The workspace that it asks for holds these shares."""
    import weight_only_bit_rtn_amd as lw
    every = LONG_SUMS_A + LONG_SUMS_B + LONG_U + LONG_UP + LONG_DOWN
    for (T, N, K, R, L), d, g in zip(every, divide([("lora", *s) for s in every]), divide([("lora_grad", *s) for s in every])):
        assert lw.lora_workspace_bytes(T, N, K, R, L) == 4 * d["splits"] * T * R
        assert lw.lora_grad_workspace_bytes(T, N, K, R, L) == 4 * (g["splits"] * T * R + g["shares"] * R * (K + N))


def columns(n):
    """Some of n columns: both ends, either side of every border of 512 and of some of 128, and others."""
    rng = np.random.default_rng(n)
    near = [np.arange(0, n + 128, 512) + d for d in (-1, 0)] + [np.arange(0, min(n, 4096), 128) + d for d in (-1, 0, 8)]
    at = np.concatenate([*near, [0, n - 1, n - 2, n - 9], rng.integers(0, n, 64)])
    return np.unique(at[(at >= 0) & (at < n)])


def some(t, at, dim):
    return f64(t.index_select(dim, torch.from_numpy(at).to(t.device)))


def far_rows(c, kind):
    """Rows of dy and v whose size changes from 64 tokens to 64 in the order of the plan: 2^-9 to 2^4, up and down."""
    size = 2.0 ** np.array([-2, -9, -5, -8, 0, -3, 4, 1, -6, 3])
    place = np.empty(len(c.ids), np.int64)
    place[c.plan["order"].cpu().numpy()] = np.arange(len(c.ids))
    by = torch.from_numpy(size[place // 64 % len(size)].astype(np.float32)).cuda()[:, None]
    c.dy = (c.dy.float() * by).to(c.dy.dtype)
    c.v = c.v * by.flip(0)


def check_gradients(c, dx, da, db, base, k_at, n_at):
    """dx and da at some columns of K from everything else, db at some outputs."""
    K, N = c.x.shape[1], c.dy.shape[1]
    dy, v, scales, ids = f64(c.dy), f64(c.v), f64(c.scales), c.ids
    x, a, b = some(c.x, k_at, 1), some(c.a, k_at, 2), f64(c.b)
    args = (dy, x, v, a, b, scales, ids)
    want = ref.lora_grad(*args, None if base is None else some(base, k_at, 1))
    far = ref.lora_grad_bound(*args, want[0], c.kind)
    got = some(dx, k_at, 1), some(da, k_at, 2), some(db, n_at, 1)
    for g, w, f in ((got[0], want[0], far[0]), (got[1], want[1], far[1]), (got[2], want[2][:, n_at], far[2][:, n_at])):
        assert np.isfinite(g).all() and (np.abs(g - w) <= f).all(), np.argwhere(~(np.abs(g - w) <= f))[:5]


def run_gradients(lw, shape, kind, order, spread, k_at, n_at):
    c = Case(lw, *shape, kind, order, seed=11)
    if spread:
        far_rows(c, kind)
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    check_gradients(c, dx, da, db, c.base, k_at, n_at)
    base = c.base.clone()
    again = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=base, out=base)
    assert again[0] is base and all(torch.equal(p, q) for p, q in zip(again, (dx, da, db)))
    check_gradients(c, *lw.lora_grad(c.dy, c.x, c.v, *c.pools()), None, k_at, n_at)


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", LONG_SUMS_A + LONG_SUMS_B, ids=str)
def test_many_rounds_of_a_chunk(lw, shape, kind, spread):  # noqa: F811
    T, N, K, R, L = shape
    if N <= 2000:
        run_gradients(lw, shape, kind, "mixed", spread, columns(K), np.arange(N))
        return
    # N is the long side: u needs all of it, db column by column not
    c = Case(lw, *shape, kind, "mixed", seed=12)
    if spread:
        far_rows(c, kind)
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    at = columns(N)
    args = [some(c.dy, at, 1), f64(c.x), f64(c.v), f64(c.a), some(c.b, at, 1), f64(c.scales), c.ids]
    want, far = ref.lora_grad(*args)[2], ref.lora_grad_bound(*args, np.zeros(c.x.shape), kind)[2]
    assert (np.abs(some(db, at, 1) - want) <= far).all()
    base = c.base.clone()
    again = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=base, out=base)
    assert again[0] is base and all(torch.equal(p, q) for p, q in zip(again, (dx, da, db)))
    assert dx.isfinite().all() and da.isfinite().all() and db.isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", LONG_U, ids=str)
def test_many_steps_of_u(lw, shape, kind):  # noqa: F811
    run_gradients(lw, shape, kind, "mixed", True, np.arange(shape[2]), columns(shape[1]))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("shape", LONG_UP + LONG_DOWN, ids=str)
def test_many_steps_of_the_forward_pass(lw, shape, kind, order):  # noqa: F811
    c = Case(lw, *shape, kind, order, seed=13)
    out, v = lw.lora(c.x, *c.pools(), y=c.y, save=True)
    at = columns(shape[1])
    args = [f64(c.x), f64(c.a), some(c.b, at, 1), f64(c.scales), c.ids]
    for y, got in ((c.y, out), (None, lw.lora(c.x, *c.pools()))):
        want, want_v = ref.lora(*args, None if y is None else some(y, at, 1))
        far, far_v = ref.lora_bound(*args, want, kind)
        assert (np.abs(some(got, at, 1) - want) <= far).all() and (np.abs(f64(v) - want_v) <= far_v).all()
    y = c.y.clone()
    assert lw.lora(c.x, *c.pools(), y=y, out=y) is y and torch.equal(y, out)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_ranks_and_tokens_far_below_the_others(lw, kind):  # noqa: F811
    """Every other rank's u 2^-12 and every third one's v 2^-20 below the rest, the largest tokens first: da and db of each
    rank are within 2^-22 of its own values and 2^-39 of the largest (fp16), or 2^-24 of its own (bf16)."""
    T, N, K, R, L = LONG_SUMS_A[3]
    c = Case(lw, T, N, K, R, 1, kind, "mixed", seed=14)
    c.b[:, :, 1::2] *= 2.0 ** -12
    c.v[:, ::3] *= 2.0 ** -20
    first = c.plan["order"][:100].long()
    c.dy[first] *= 16
    c.v[first] *= 64
    dx, da, db = lw.lora_grad(c.dy, c.x, c.v, *c.pools(), dx=c.base)
    k_at = columns(K)
    check_gradients(c, dx, da, db, c.base, k_at, np.arange(N))
    # and rank by rank: what the sums' roundings leave of that
    s, t = f64(c.scales)[0], np.flatnonzero(c.ids == 0)
    dy, x, v, b = f64(c.dy)[t], some(c.x, k_at, 1)[t], f64(c.v)[t], f64(c.b)[0]
    u, deep = dy @ b, ref.depth(N) * (np.abs(dy) @ np.abs(b))
    for got, val, rows, off in ((some(da, k_at, 2)[0], u, x, deep), (f64(db)[0].T, v, dy, 0 * v)):
        own = np.abs(val)
        floor = 2.0 ** -39 * own.max() if kind == "fp16" else 0.0
        part = np.maximum(own * (2.0 ** -22 if kind == "fp16" else 2.0 ** -24), floor)
        far = s * ((off + part + ref.depth(3 * len(t)) * own).T @ np.abs(rows)) * 1.01 + 2.0 ** -140
        assert (np.abs(got - s * (val.T @ rows)) <= far).all()
