"""8-bit moments rounded up or down by a number made of step and place (rounding="random"): the codes bit for
bit against the definition, and what it is for: second moments that follow gradients which change against
the rest of their block, where codes rounded to the nearest stay behind."""
from __future__ import annotations

import os

import numpy as np
import pytest
import torch  # before the library, which takes the HIP runtime that torch has loaded

import adapters_reference as ref
import test_adapters_host as host

BETAS = (0.9, 0.999)


@pytest.fixture(scope="module")
def lw():
    import weight_only_bit_rtn_amd as lw
    if not os.path.exists(lw.LIB_PATH):
        from weight_only_bit_rtn_amd import build
        build.build()
    lw.load_library()
    return lw


# ---------------------------------------------------------------------------
# the definition
# ---------------------------------------------------------------------------
def mix(x):
    x = np.array(x, np.uint32)
    with np.errstate(over="ignore"):
        x ^= x >> np.uint32(16)
        x *= np.uint32(0x6A09E667)
        x ^= x >> np.uint32(15)
        x *= np.uint32(0xBB67AE85)
        return x ^ x >> np.uint32(16)


def numbers_of(step, places):
    """r of m and of v at some places (int64)."""
    places = np.asarray(places, np.int64)
    with np.errstate(over="ignore"):
        key = mix(mix(step & 0xFFFFFFFF) + (places >> 32).astype(np.uint32))
    h = mix((places & 0xFFFFFFFF).astype(np.uint32) ^ key)
    return (h >> np.uint32(16)) * np.uint32(16) + np.uint32(8), (h & np.uint32(0xFFFF)) * np.uint32(16) + np.uint32(8)


def encode(x, bits, step, first=0):
    """ref.encode with codes rounded at random: x begins at place `first` of the moments."""
    nearest, top = ref.encode(x, bits)
    x = x.reshape(-1, 256)
    finite = np.isfinite(x).all(1)
    with np.errstate(all="ignore"):
        inverse = np.where(top > 0, np.float32(1) / top, np.float32(0)).astype(np.float32)
        q = (np.where(finite[:, None], np.abs(x), 0) * inverse[:, None]).astype(np.float32)
    r = numbers_of(step, first + np.arange(x.size, dtype=np.int64))[0 if bits == 7 else 1].reshape(x.shape)
    last = (1 << bits) - 1
    code = ((q.view(np.uint32) + r) >> np.uint32(20)).astype(np.int64) - (0x3F8 - last)
    code = np.clip(code, 0, None)
    if bits == 8:
        code = np.maximum(code, q > 0)
    else:
        code = np.where((code > 0) & np.signbit(x), code + 128, code)
    assert code.max(initial=0) <= 255
    return code.astype(np.uint8).reshape(-1), top


@pytest.mark.parametrize("bits", [7, 8])
def test_codes_are_neighbours_and_right_in_the_mean(bits):
    rng = np.random.default_rng(bits)
    tab = ref.numbers(bits).astype(np.float64)
    for value in (1.0, 0.99, 0.7, 0.5, 0.3001, 0.06, 3e-3, 2e-5):
        x = np.full(256 * 40, value, np.float32)
        x[::256] = 1                                   # the block's largest
        x[rng.random(x.size) < 0.5] *= 1 if bits == 8 else -1
        x[::256] = 1
        every = np.concatenate([encode(x, bits, step)[0].reshape(-1, 256)[:, 1:].reshape(-1) for step in range(1, 40)])
        got = tab[every & (127 if bits == 7 else 255)]
        q = float(np.float32(value))
        low = tab[tab <= q].max()
        high = tab[tab >= q].min()
        assert set(np.unique(got)) <= {low, high}
        # the mean of n numbers that are low or high: five times its deviation, and r's steps of 2^-16
        p = (q - low) / (high - low) if high > low else 0
        far = (high - low) * (5 * np.sqrt(max(p * (1 - p), 0) / got.size) + 2.0 ** -16)
        assert abs(got.mean() - q) <= far + 1e-7 * q


def test_the_largest_and_the_least():
    for step in range(1, 300):
        x = np.zeros(256, np.float32)
        x[:4] = [3, -3, 3 * 2.0 ** -40, 1.1 * 3 * 2.0 ** -16]
        m, top = encode(x, 7, step)
        assert top[0] == 3 and m[:4].tolist() == [127, 255, 0, 0]
        v, _ = encode(np.abs(x), 8, step)
        assert v[:3].tolist() == [255, 255, 1] and not v[4:].any() and not m[4:].any()
        # a reciprocal that rounds up gives the largest a q of 1 + 2^-23 at most
        odd = np.zeros(256, np.float32)
        odd[7] = 1.0 + step * 2.0 ** -9
        assert encode(odd, 7, step)[0][7] == 127 and encode(odd, 8, step)[0][7] == 255


def follow(encode_v, change, steps=4000, blocks=4, turn=500):
    """v of 8 bits by v of 32 after `steps`, where half of each block's gradients change by a factor at step `turn`:
    (the changed half's, the other half's)."""
    rng = np.random.default_rng(3)
    n = blocks * 256
    size = np.exp(rng.standard_normal(n)).astype(np.float32) * 1e-3
    m, v, wide_m, wide_v = (np.zeros(n, np.float32) for _ in range(4))
    half = np.arange(n) % 2 == 0
    for step in range(1, steps + 1):
        g = rng.standard_normal(n).astype(np.float32) * size
        if step > turn:
            g[half] *= np.float32(change)
        m, v = ref.moments(m, v, g, *BETAS)
        wide_m, wide_v = ref.moments(wide_m, wide_v, g, *BETAS)
        codes, top = encode_v(v, 8, step)
        v = ref.decode(np.zeros(n, np.uint8), codes, np.zeros(blocks, np.float32), top)[1]
    ratio = v / wide_v
    return ratio[half], ratio[~half]


# A step moves v by 0.001 (g^2 + v) at most and the block's largest alike: 0.004 of v in the mean, so the code is
# rounded across a gap of s <= 1/8 with probability 0.004 / s at most and a variance of 0.004 s <= 0.0005 of v^2; of
# 1 / (1 - 0.999^2) = 500 steps' memory, 0.25.  The mean of 512 values deviates by 0.5 / 512^(1/2) = 0.022.
MEAN, SPREAD = 5 * 0.022, 0.5 * 1.2


@pytest.mark.parametrize("change", [1.0, 0.1, 4.0])
def test_second_moments_follow(change):
    for ratio in follow(encode, change):
        assert abs(ratio.mean() - 1) < MEAN and np.sqrt(((ratio - 1) ** 2).mean()) < SPREAD


def test_what_the_nearest_codes_lose():
    """The reason for the other rounding, as the header has it: half of a block stays behind."""
    nearest = lambda v, bits, step: ref.encode(v, bits)  # noqa: E731
    changed, _ = follow(nearest, 0.1)
    assert np.median(changed) > 10
    _, others = follow(nearest, 4.0)
    assert np.median(others) > 3


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def test_refused_on_the_host(lw):
    random = 8 | lw.ADAMW_RANDOM
    text = open(os.path.join(host.ROOT, "include", "lowbit_adamw.h")).read()
    assert f"#define LOWBIT_ADAMW_RANDOM {lw.ADAMW_RANDOM} " in text
    for bits in (lw.ADAMW_RANDOM, 32 | lw.ADAMW_RANDOM, random + 1, random | 512):
        assert host.adamw(lw, bits=bits) == host.UNSUPPORTED
    for args in (dict(m_max=None), dict(v_max=host.MIS), dict(m=None), dict(lr=-1.0)):
        assert host.adamw(lw, bits=random, **args) == host.ARG
    assert host.adamw(lw, bits=random, tensors=()) == 0
    with pytest.raises(ValueError, match="rounding"):
        lw.adamw([], [], {}, lr=1e-3, rounding="up")


# ---------------------------------------------------------------------------
# the kernel
# ---------------------------------------------------------------------------
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def flat(tensors, blocks):
    out = np.zeros(sum(blocks) * 256, np.float32)
    at = 0
    for t, b in zip(tensors, blocks):
        out[at:at + t.numel()] = t.float().cpu().numpy()
        at += b * 256
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("kind,grads", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "bfloat16"),
                                        ("bfloat16", "float32"), ("float16", "float16"), ("float16", "float32")])
def test_codes(lw, kind, grads, master):
    gpu()
    print(f"[adamw] random {kind} {grads} master {master}", flush=True)
    rng = np.random.default_rng(5)
    sizes = [1, 3, 255, 256, 257, 1025, 4097, 70000] + [int(n) for n in rng.integers(1, 900, 150)]
    blocks = [-(-n // 256) for n in sizes]
    params = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda().to(getattr(torch, kind)) for n in sizes]
    state = lw.adamw_state(params, master=master)
    m, v = (np.zeros(sum(blocks) * 256, np.float32) for _ in range(2))
    for step in (1, 2, 1000, 123456789):
        g = [torch.from_numpy((rng.standard_normal(n) * np.exp(rng.standard_normal(n)) * 1e-2).astype(np.float32)).cuda()
             .to(getattr(torch, grads)) for n in sizes]
        m, v = ref.moments(m, v, flat(g, blocks), *BETAS)
        (cm, tm), (cv, tv) = encode(m, 7, step), encode(v, 8, step)
        lw.adamw(params, g, state, lr=1e-3, betas=BETAS, step=step, rounding="random")
        for name, want in (("m", cm), ("m_max", tm), ("v", cv), ("v_max", tv)):
            assert np.array_equal(state[name].cpu().numpy(), want), (name, step)
        m, v = ref.decode(cm, cv, tm, tv)
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(lw.adamw_moments(state), (m, v)))


@pytest.mark.gpu
def test_parameters_do_not_depend_on_the_rounding(lw):
    """Of one step: the update is made from the moments before they are rounded."""
    gpu()
    g = torch.randn(5000, device="cuda")
    p = [torch.ones(5000, device="cuda") for _ in range(2)]
    s = [lw.adamw_state([t]) for t in p]
    for t, state, rounding in zip(p, s, ("nearest", "random")):
        lw.adamw([t], [g], state, lr=0.1, rounding=rounding)
    assert torch.equal(*p) and torch.equal(s[0]["v_max"], s[1]["v_max"]) and not torch.equal(s[0]["v"], s[1]["v"])
    with pytest.raises(ValueError, match="not rounded"):
        lw.adamw(p[:1], [g], lw.adamw_state(p[:1], bits=32), lr=0.1, rounding="random")


@pytest.mark.gpu
def test_bad_gradients_and_skipped_steps(lw):
    gpu()
    p = torch.ones(600, device="cuda")
    state = lw.adamw_state([p])
    g = torch.randn(600, device="cuda")
    g[300] = float("inf")
    lw.adamw([p], [g], state, lr=0.1, rounding="random")
    assert state["m_max"].isnan().tolist() == [False, True, False] and not state["m"][256:512].any() and not state["v"][256:512].any()
    before = [t.clone() for t in state.values()]
    lw.adamw([p], [g], state, lr=0.1, step=2, rounding="random", grad_scale=torch.tensor([float("nan")], device="cuda"))
    assert all(torch.equal(a, b) or a.isnan().any() and torch.equal(a.isnan(), b.isnan()) for a, b in zip(before, state.values()))
    zero = lw.adamw_state([p])
    lw.adamw([torch.ones_like(p)], [torch.zeros_like(p)], zero, lr=0.1, rounding="random")
    assert not any(t.any() for t in zero.values())


@pytest.mark.gpu
def test_captured(lw):
    """A captured step takes its numbers from the count on the GPU: as eager steps with host counts."""
    gpu()
    shapes = (3000, 77, 130000)
    a, b = ([torch.ones(n, dtype=torch.bfloat16, device="cuda") for n in shapes] for _ in range(2))
    s, t = (lw.adamw_state(p, master=True) for p in (a, b))
    g = [torch.zeros_like(p) for p in a]
    count = torch.ones(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lw.adamw(a, g, s, lr=0.01, step=count, rounding="random")
    for step in (1, 2, 3, 70000):
        for x in g:
            x.normal_()
        count.fill_(step)
        graph.replay()
        lw.adamw(b, g, t, lr=0.01, step=step, rounding="random")
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*a, *s.values()), (*b, *t.values()))), step


@pytest.mark.gpu
def test_places_past_32_bits(lw):
    gpu()
    n = (1 << 32) + 1000
    print("[adamw] random, 2^32 values", flush=True)
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    blocks = -(-n // 256)
    state = {k: torch.zeros(blocks * 256, dtype=torch.uint8, device="cuda") for k in ("m", "v")}
    state.update({k: torch.zeros(blocks, device="cuda") for k in ("m_max", "v_max")})
    firsts = [0, (1 << 30) - 256, 1 << 30, 1 << 31, (1 << 32) - 256, 1 << 32, (1 << 32) + 512]
    x = np.full(256, 0.69921875, np.float32)    # a bf16 number between two codes' numbers
    x[5] = 1
    for at in firsts:
        g[at:at + 256] = torch.from_numpy(x).cuda()
    lw.adamw([p], [g], state, lr=0.5, step=9, rounding="random")
    m, v = ref.moments(np.zeros(256, np.float32), np.zeros(256, np.float32), x, *BETAS)
    seen = set()
    for at in firsts:
        want = encode(m, 7, 9, at)[0], encode(v, 8, 9, at)[0]
        got = [state[k][at:at + 256].cpu().numpy() for k in ("m", "v")]
        assert all(np.array_equal(a, b) for a, b in zip(got, want)), at
        seen.add(got[0].tobytes())
    assert len(seen) == len(firsts)


@pytest.mark.gpu
@pytest.mark.parametrize("change", [0.1, 4.0])
def test_a_run_follows_32_bits(lw, change):
    """Thousands of steps beside a state of 32 bits, half of every block changing its gradients' size on the way."""
    gpu()
    print(f"[adamw] a run, change {change}", flush=True)
    n, steps, turn = 8192, 4000, 500
    gen = torch.Generator(device="cuda").manual_seed(1)
    size = torch.exp(torch.randn(n, generator=gen, device="cuda")) * 1e-3
    half = torch.arange(n, device="cuda") % 2 == 0
    p, q = (torch.zeros(n, device="cuda") for _ in range(2))
    s, t = lw.adamw_state([p]), lw.adamw_state([q], bits=32)
    for step in range(1, steps + 1):
        g = torch.randn(n, generator=gen, device="cuda") * size
        if step > turn:
            g = torch.where(half, g * change, g)
        lw.adamw([p], [g], s, lr=1e-3, weight_decay=0.0, step=step, rounding="random")
        lw.adamw([q], [g], t, lr=1e-3, weight_decay=0.0, step=step)
    ratio = (lw.adamw_moments(s)[1] / t["v"]).double()
    for part in (ratio[half], ratio[~half]):    # 4096 values each: the bounds of 512 hold all the more
        assert abs(part.mean().item() - 1) < MEAN and (part - 1).square().mean().sqrt().item() < SPREAD
