"""Adapters beside the quantized projections as a user's program calls them, and the same in plain torch.

plan       the tokens of a batch sorted by their adapter
lora       out = y + scale (x A^T) B^T, each token through its own adapter; y is the shared projection's output
lora_grad  the gradients of lora: dx (added to the projection's), dA and dB
adamw      one AdamW step over many tensors, moments in 8 bits or in 32

Adapters lie in pools A[L][R][K] and B[L][N][R]; ids[T] names each token's adapter, -1 none.  Moments lie in one
buffer for all tensors, each tensor from a multiple of 256 values on; 8-bit moments have one maximum for 256 values.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 256


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decoding batch, every request with its own adapter
        dict(name="plan 64 tokens", op="plan", T=64, L=64, mixed=True, none=0.0),
        # prompts of several requests, a part of them without an adapter
        dict(name="plan 16384 tokens", op="plan", T=16384, L=16, mixed=False, none=0.2),
        # one token of one request: latency
        dict(name="lora 1x4096x4096 r16", op="lora", T=1, N=4096, K=4096, R=16, L=1, type="fp16",
             mixed=False, none=0.0, save=False),
        # a decoding batch over a pool of adapters, in the order the requests came
        dict(name="lora 64x11008x4096 r16 of 64", op="lora", T=64, N=11008, K=4096, R=16, L=64,
             type="bf16", mixed=True, none=0.1, save=False),
        # prompts of some requests, ranks padded to a pool's odd one
        dict(name="lora 1333x4096x11008 r24 of 8", op="lora", T=1333, N=4096, K=11008, R=24, L=8,
             type="fp16", mixed=False, none=0.1, save=False),
        # a training batch of the largest layer, kept for the backward pass
        dict(name="lora 8192x12288x12288 r64", op="lora", T=8192, N=12288, K=12288, R=64, L=1,
             type="bf16", mixed=False, none=0.0, save=True),
        # the backward pass of a short sequence
        dict(name="lora_grad 61x4096x4096 r8", op="lora_grad", T=61, N=4096, K=4096, R=8, L=1,
             type="fp16", mixed=False, none=0.0),
        # adapters of several tasks trained at once
        dict(name="lora_grad 2000x11008x4096 r16 of 4", op="lora_grad", T=2000, N=11008, K=4096, R=16,
             L=4, type="fp16", mixed=False, none=0.1),
        # the backward pass of a training batch of the largest layer
        dict(name="lora_grad 8192x12288x12288 r64", op="lora_grad", T=8192, N=12288, K=12288, R=64,
             L=1, type="bf16", mixed=False, none=0.0),
        # the pair of one layer
        dict(name="adamw 2 tensors, 32 bits", op="adamw", tensors=2, least=65536, most=65536, bits=32,
             type="fp32", grads="fp32", master=False, scale=False, step=1, decay=0.0),
        # all adapters of a model: 32 layers of 7 projections, clipped gradients
        dict(name="adamw 448 tensors, 8 bits", op="adamw", tensors=448, least=65536, most=176128, bits=8,
             type="fp32", grads="fp32", master=False, scale=True, step=1000, decay=0.01),
        # one large matrix with an fp32 copy
        dict(name="adamw 100 million, 8 bits", op="adamw", tensors=1, least=100663296, most=100663296,
             bits=8, type="bf16", grads="bf16", master=True, scale=False, step=100, decay=0.01),
    ]


MOST_TOKENS = 8192 * 2 * 12288      # T (K + N)
MOST_WORK = MOST_TOKENS * 64          # T (K + N) R
MOST_RANKS = 2048                   # L R
MOST_POOL = 64 * 16 * 16384         # L R (K + N)
MOST_VALUES = 100663296


def _between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "lora", "lora", "lora", "lora_grad", "lora_grad", "adamw", "adamw", "adamw"))
    none = rng.choice((0.0, 0.0, 0.1, 0.5))
    mixed = rng.random() < 0.5
    if op == "plan":
        return dict(op=op, T=_between(rng, 1, 16384), L=_between(rng, 1, 512), mixed=mixed, none=none)
    if op == "adamw":
        tensors = _between(rng, 1, 512)
        most = _between(rng, 64, min(8388608, MOST_VALUES // (2 * tensors)))
        kind = rng.choice(("fp32", "fp16", "bf16"))
        return dict(op=op, tensors=tensors, least=_between(rng, 1, most), most=most, bits=rng.choice((8, 8, 32)),
                    type=kind, grads=rng.choice(("fp32", kind)), master=kind != "fp32" and rng.random() < 0.6,
                    scale=rng.random() < 0.5, step=_between(rng, 1, 10000), decay=rng.choice((0.0, 0.01, 0.1)))
    while True:
        T = _between(rng, 1, 8192)
        K = 32 * _between(rng, 2, 384)
        N = _between(rng, 256, 12288)
        if rng.random() < 0.5:      # layers are mostly whole multiples, half of these are not
            N = N // 64 * 64
        R = 8 * _between(rng, 1, 16)
        L = _between(rng, 1, 128)
        if (T * (K + N) <= MOST_TOKENS and T * (K + N) * R <= MOST_WORK and L * R <= MOST_RANKS
                and L * R * (K + N) <= MOST_POOL):
            break
    case = dict(op=op, T=T, N=N, K=K, R=R, L=L, type=rng.choice(("fp16", "bf16")), mixed=mixed, none=none)
    if op == "lora":
        case["save"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ids(g, case):
    """An adapter for each token, -1 for a share of them: one by one, or in runs of one request's prompt."""
    T, L = case["T"], case["L"]
    if case["mixed"]:
        ids = torch.randint(0, L, (T,), generator=g, device="cuda")
        ids[torch.rand(T, generator=g, device="cuda") < case["none"]] = -1
    else:
        runs = min(T, 2 * L)
        cuts = torch.randint(0, T, (runs,), generator=g, device="cuda").sort().values
        who = torch.randint(0, L, (runs + 1,), generator=g, device="cuda")
        who[torch.rand(runs + 1, generator=g, device="cuda") < case["none"]] = -1
        at = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
        ids = who[at]
    return ids.to(torch.int32)


def _plain_plan(ids, L):
    key = torch.where((ids < 0) | (ids >= L), torch.full_like(ids, L), ids)
    order = torch.sort(key, stable=True).indices.to(torch.int32)
    count = (key[:, None] == torch.arange(L, device=ids.device)).sum(0)
    starts = torch.zeros(L + 1, dtype=torch.int32, device=ids.device)
    starts[1:] = torch.cumsum(count, 0)
    return {"order": order, "starts": starts}


def _sizes(case):
    """Sizes between the least and the most, evenly over their logarithm."""
    n, lo, hi = case["tensors"], case["least"], case["most"]
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def _rounded(values, mantissa, exponent, least):
    """Codes of values in [0, 1]: the upper bits of their fp32 form, rounded to nearest, counted down from 1's."""
    top = (1 << (mantissa + exponent)) - 1
    shift = 23 - mantissa
    raw = (values.view(torch.int32) + (1 << (shift - 1))) >> shift
    raw = (raw - ((0x3F800000 >> shift) - top)).clamp(0, top)
    return torch.maximum(raw, (least & (values > 0)).int())


def _valued(codes, mantissa, exponent):
    top = (1 << (mantissa + exponent)) - 1
    shift = 23 - mantissa
    value = ((codes.int() + ((0x3F800000 >> shift) - top)) << shift).view(torch.float32)
    return torch.where(codes == 0, torch.zeros_like(value), value)


def _packed(m, v):
    """8-bit moments: codes and a maximum for each block."""
    out = {}
    for name, x in (("m", m), ("v", v)):
        x = x.view(-1, BLOCK)
        a = x.abs()
        top = a.amax(1, keepdim=True)
        whole = (a < math.inf).all(1, keepdim=True)
        top = torch.where(whole, torch.where(top < 2.0 ** -126, torch.zeros_like(top), top),
                          torch.full_like(top, math.nan))
        inverse = torch.where(top > 0, torch.ones_like(top) / top, torch.zeros_like(top))
        q = torch.where(whole, a, torch.zeros_like(a)) * inverse
        if name == "m":
            code = _rounded(q, 3, 4, torch.tensor(False, device=x.device)) + 128 * (torch.signbit(x) & whole).int()
            code = torch.where(code == 128, torch.zeros_like(code), code)
        else:
            code = _rounded(q, 3, 5, torch.tensor(True, device=x.device))
        out[name] = code.to(torch.uint8).view(-1)
        out[name + "_max"] = top.view(-1)
    return out


def _plain_moments(state):
    """The values that 8-bit moments stand for."""
    cm = state["m"].view(-1, BLOCK)
    m = _valued(cm & 127, 3, 4) * state["m_max"][:, None]
    m = torch.where(cm > 127, -m, m)
    v = _valued(state["v"].view(-1, BLOCK), 3, 5) * state["v_max"][:, None]
    return m.view(-1), v.view(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if op == "adamw":
        sizes = _sizes(case)
        blocks = [-(-n // BLOCK) for n in sizes]
        state["sizes"], state["blocks"] = sizes, blocks
        total = sum(blocks) * BLOCK
        inside = torch.cat([torch.arange(b * BLOCK, device="cuda") < n for n, b in zip(sizes, blocks)])
        # moments in the middle of a run: their size differs from place to place, and some never had a gradient
        size = torch.exp(normal(total)) * 1e-3 * (torch.rand(total, generator=g, device="cuda") > 0.02)
        m = torch.where(inside & (case["step"] > 1), normal(total) * size * 0.3, torch.zeros((), device="cuda"))
        v = torch.where(inside & (case["step"] > 1), size * size, torch.zeros((), device="cuda"))
        state["moments"] = _packed(m, v) if case["bits"] == 8 else {"m": m, "v": v}
        p = torch.where(inside, normal(total) * 0.02, torch.zeros((), device="cuda"))
        if case["master"]:
            state["moments"]["master"] = p
        at = [0]
        for b in blocks:
            at.append(at[-1] + b * BLOCK)
        state["at"] = at[:-1]
        # one buffer holds all parameters; the tensors are its parts
        state["all"] = p.to(TYPES[case["type"]], copy=True)
        state["params"] = [state["all"][a:a + n] for a, n in zip(at, sizes)]
        grad = normal(total) * size
        state["grads"] = [grad[a:a + n].to(TYPES[case["grads"]], copy=True) for a, n in zip(at, sizes)]
        state["grad_scale"] = torch.full((1,), 0.37, device="cuda") if case["scale"] else None
        return state

    state["ids"] = _ids(g, case)
    if op == "plan":
        return state
    T, N, K, R, L, t = case["T"], case["N"], case["K"], case["R"], case["L"], TYPES[case["type"]]
    state["plan"] = _plain_plan(state["ids"], L)
    state["a"] = (normal(L, R, K) * K ** -0.5).to(t)
    state["b"] = (normal(L, N, R) * 0.05).to(t)
    state["scales"] = torch.rand(L, generator=g, device="cuda") * 2 + 0.5
    state["x"] = normal(T, K).to(t)
    if op == "lora":
        state["y"] = normal(T, N).to(t)
        return state
    state["dy"] = (normal(T, N) * 0.01).to(t)
    state["dx"] = (normal(T, K) * 0.01).to(t)
    state["v"] = torch.where((state["ids"] >= 0)[:, None], normal(T, R), torch.zeros((), device="cuda"))
    return state


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------
def _plain_mask(state):
    """[T][L R]: the adapter's scale where a column belongs to the token's adapter, 0 elsewhere."""
    L, R = state["L"], state["R"]
    mine = state["ids"][:, None] == torch.arange(L, device="cuda")
    return (mine * state["scales"]).repeat_interleave(R, 1), mine.repeat_interleave(R, 1)


def _plain_lora(state):
    T, R, L, t = state["T"], state["R"], state["L"], TYPES[state["type"]]
    scale, mine = _plain_mask(state)
    every = state["x"].float() @ state["a"].float().view(L * R, -1).t()     # through every adapter
    rows = state["b"].float().permute(0, 2, 1).reshape(L * R, -1)
    out = (state["y"].float() + (every * scale) @ rows).to(t)
    if not state["save"]:
        return out
    return out, (every * mine).view(T, L, R).sum(1)


def _plain_lora_grad(state):
    R, L, t = state["R"], state["L"], TYPES[state["type"]]
    scale, _ = _plain_mask(state)
    dy, x = state["dy"].float(), state["x"].float()
    rows = state["b"].float().permute(0, 2, 1).reshape(L * R, -1)
    u = (dy @ rows.t()) * scale
    dx = (state["dx"].float() + u @ state["a"].float().view(L * R, -1)).to(t)
    da = (u.t() @ x).view(L, R, -1)
    db = (dy.t() @ (state["v"].repeat(1, L) * scale)).view(-1, L, R).permute(1, 0, 2).contiguous()
    return dx, da, db


def _plain_adamw(state):
    b1, b2, lr, eps, t = 0.9, 0.999, 1e-3, 1e-8, state["step"]
    s = state["moments"]

    grad = torch.cat([torch.nn.functional.pad(x, (0, -n % BLOCK)) for x, n in zip(state["grads"], state["sizes"])]).float()
    if state["grad_scale"] is not None:
        grad = grad * state["grad_scale"]
    m, v = _plain_moments(s) if state["bits"] == 8 else (s["m"], s["v"])
    m = m * b1 + grad * (1 - b1)
    v = v * b2 + (grad * grad) * (1 - b2)
    p = s["master"] if state["master"] else state["all"].float()
    step = m / (v.sqrt() * (1 / math.sqrt(1 - b2 ** t)) + eps)
    p = p * (1 - lr * state["decay"]) - step * (lr / (1 - b1 ** t))
    state["all"].copy_(p)
    if state["master"]:
        s["master"].copy_(p)
    new = _packed(m, v) if state["bits"] == 8 else {"m": m, "v": v}
    torch._foreach_copy_([s[k] for k in new], list(new.values()))
    m, v = _plain_moments(s) if state["bits"] == 8 else (s["m"], s["v"])
    return state["all"], m, v, s.get("master")


def _plain(state):
    op = state["op"]
    if op == "plan":
        return _plain_plan(state["ids"], state["L"])
    return {"lora": _plain_lora, "lora_grad": _plain_lora_grad, "adamw": _plain_adamw}[op](state)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(state):
    import weight_only_bit_rtn_amd as lw
    op = state["op"]
    if op == "plan":
        return lw.lora_plan(state["ids"], state["L"])
    if op == "adamw":
        s = state["moments"]
        lw.adamw(state["params"], state["grads"], s, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=state["decay"], step=state["step"], grad_scale=state["grad_scale"])
        m, v = lw.adamw_moments(s)
        return state["all"], m, v, s.get("master")
    if op == "lora":
        return lw.lora(state["x"], state["a"], state["b"], state["scales"], state["plan"], y=state["y"],
                       save=state["save"])
    return lw.lora_grad(state["dy"], state["x"], state["v"], state["a"], state["b"], state["scales"],
                        state["plan"], dx=state["dx"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        return {"bytes": 8 * case["T"] + 4 * (case["L"] + 1), "flops": 0}
    if op == "adamw":
        n = sum(_sizes(case))
        wide = {"fp32": 4, "fp16": 2, "bf16": 2}
        # parameters and moments are read and written; 8-bit ones are written as what they stand for too
        value = 2 * wide[case["type"]] + wide[case["grads"]]
        if case["master"]:
            value += 8 - wide[case["type"]]     # the 16-bit copy is written alone
        value += 16 if case["bits"] == 32 else 4 + 4 * 4 / BLOCK + 8
        return {"bytes": int(n * value), "flops": 16 * n}
    T, N, K, R, L = case["T"], case["N"], case["K"], case["R"], case["L"]
    used = min(L, T)
    pools = used * R * (K + N) * 2 + 4 * used + 4 * (L + 1) + 4 * T
    if op == "lora":
        return {"bytes": 2 * T * K + 4 * T * N + pools + (4 * T * R if case["save"] else 0),
                "flops": 2 * T * R * (K + N)}
    return {"bytes": 2 * T * N + 6 * T * K + 4 * T * R + pools + 4 * L * R * (K + N),
            "flops": 4 * T * R * (K + N)}


def _exact_adamw(st):
    """The moments as they are defined (each operation one rounding to 32 bits, codes from those values),
    the parameters from them in 64 bits."""
    f = torch.float32
    t, s = st["step"], st["moments"]

    def once(x):
        return x.to(f).double()

    def const(x):
        return torch.tensor(x, dtype=f, device="cuda").double()

    def spread(tensors):
        out = torch.zeros(sum(st["blocks"]) * BLOCK, dtype=torch.float64, device="cuda")
        for a, n, x in zip(st["at"], st["sizes"], tensors):
            out[a:a + n] = x
        return out

    def table(bits, octaves):
        """Value of every code: (1 + i / 8) 2^(e - octaves) with the last one at 1, code 0 nothing."""
        c = torch.arange(1 << bits, device="cuda", dtype=torch.float64)
        down = (1 << bits) - 1 - c              # steps below 1, eight to an octave
        e = torch.ceil(down / 8)
        val = (1 + (8 * e - down) / 8) * torch.exp2(-e)
        val[0] = 0
        return val

    def stand(codes, top, tab):
        return once(tab[codes.view(-1, BLOCK).long()] * top.double()[:, None])

    grad = spread(st["grads"])
    if st["grad_scale"] is not None:
        grad = once(grad * st["grad_scale"].double())
    if st["bits"] == 8:
        tm, tv = table(7, 16), table(8, 32)
        m = stand(s["m"] & 127, s["m_max"], tm).view(-1)
        m = m * (1 - 2 * (s["m"] >> 7).double())
        v = stand(s["v"], s["v_max"], tv).view(-1)
        m = once(once(const(0.9) * m) + once(const(1 - 0.9) * grad))
        v = once(once(const(0.999) * v) + once(const(1 - 0.999) * once(grad * grad)))
    else:
        m = const(0.9) * s["m"].double() + const(1 - 0.9) * grad
        v = const(0.999) * s["v"].double() + const(1 - 0.999) * grad * grad
    p = s["master"].double() if st["master"] else st["all"].double()
    p = p * (1 - 1e-3 * st["decay"]) - 1e-3 / (1 - 0.9 ** t) * m / ((v / (1 - 0.999 ** t)).sqrt() + 1e-8)
    if st["bits"] == 8:
        def again(x, tab):
            x = x.view(-1, BLOCK)
            top = x.abs().amax(1, keepdim=True)
            inv = once(1 / top)
            inv[top == 0] = 0
            q = once(x.abs() * inv).clamp(max=1)
            # halfway between two neighbouring codes belongs to the upper one
            half = (tab[1:-1] + tab[2:]) / 2
            first = tab[1] - (tab[2] - tab[1]) / 2      # below it there is nothing left
            code = torch.bucketize(q, torch.cat([first[None], half]), right=True)
            if tab is tv:
                code = torch.where((q > 0) & (code == 0), torch.ones_like(code), code)
            return (once(tab[code] * top) * torch.sign(x)).view(-1)
        m, v = again(m, tm), again(v, tv)
    return p, m, v, p if st["master"] else None


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        return None
    if op == "adamw":
        return _exact_adamw(st)
    ids = st["ids"].tolist()
    of = {}
    for i, l in enumerate(ids):
        if l >= 0:
            of.setdefault(l, []).append(i)
    x, a, b = st["x"], st["a"], st["b"]
    R = case["R"]
    if op == "lora":
        out = st["y"].double()
        v = torch.zeros(case["T"], R, dtype=torch.float64, device="cuda")
        for l, rows in of.items():
            rows = torch.tensor(rows, device="cuda")
            v[rows] = torch.mm(x[rows].double(), a[l].double().t())
            out[rows] += st["scales"][l].double() * torch.mm(v[rows], b[l].double().t())
        return (out, v) if case["save"] else out
    dx, dy = st["dx"].double(), st["dy"]
    da = torch.zeros(a.shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(b.shape, dtype=torch.float64, device="cuda")
    for l, rows in of.items():
        rows = torch.tensor(rows, device="cuda")
        s, d = st["scales"][l].double(), dy[rows].double()
        u = torch.mm(d, b[l].double()) * s
        dx[rows] += torch.mm(u, a[l].double())
        da[l] = torch.mm(u.t(), x[rows].double())
        db[l] = torch.mm(d.t(), st["v"][rows].double()) * s
    return dx, da, db
