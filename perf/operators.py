"""Cases of the many-tensor optimizer operators: what is measured, on which inputs, and the operators' plain forms.

Operators (``case["op"]``):

* ``step32``: global gradient norm, clip coefficient and AdamW with 32-bit states over a list of tensors.
* ``update8``: AdamW over a list of tensors with the states in 8 bits.
* ``norm``: the global gradient norm and the step decision alone.
* ``encode8`` / ``decode8``: 32-bit states into the 8-bit form and back.

The tensors of a case are a GPT-2-style parameter list (embeddings, then per block ln, attention and MLP
weights and biases), some extra vectors and some tensors of odd sizes.  They live in flat buffers, as a
trainer's contiguous parameter buffer: "gapless" lists follow one another without a gap, so that tensors begin
at odd offsets; the others begin at multiples of ALIGN elements.  Two parameter groups: matrices with weight
decay, vectors without and at half the learning rate.

8-bit states: blocks of 32 consecutive elements of one tensor; m as E4M3 and v as E5M2 numbers, times one
power of two (E8M0) a block.  The step rounds them stochastically: a random integer below one unit of the kept
mantissa's last place is added to the bits of the scaled binary32 value before the rest is cut off.
"""
from __future__ import annotations

import math

import torch

own = False

PKG = "zero_partitioned_mixed_replica_gb300"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ALIGN = 256
BLOCK = 32
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
GROUPS = ((1e-3, 0.01), (5e-4, 0.0))      # (lr, weight decay): matrices, vectors
MAX_NORM = 1.0
SEED8 = 20                                # seed of the stochastic rounding
STEPS_BEFORE = 10                         # steps applied before the measured one
MASK32 = 0xFFFFFFFF


# -- cases -----------------------------------------------------------------------------------------------
def _case(name, op, **kw):
    c = {"name": name, "op": op, "layers": 0, "d": 1600, "ffn": 6400, "vocab": 0, "ctx": 0, "vectors": 0, "ragged": 0,
         "grad": "bf16", "out": "bf16", "scale": 1.0, "gapless": False}
    c.update(kw)
    return c


XL = dict(layers=48, d=1600, ffn=6400, vocab=50257, ctx=1024, vectors=2)
MEDIUM = dict(layers=24, d=1024, ffn=4096, vocab=50257, ctx=1024, vectors=2, ragged=9)


def listed():
    return [
        # the replicated vectors of a model whose matrices are sharded elsewhere: latency
        _case("step32 vectors", "step32", vectors=50),
        # one transformer block of the 1.5B model: one ZeRO-3 unit
        _case("step32 block", "step32", layers=1, d=1600, ffn=6400),
        # a 350M model in a gapless flat buffer with odd-sized extras, fp16 gradients under a loss scale
        _case("step32 gapless", "step32", **MEDIUM, grad="fp16", out="fp16", scale=65536.0, gapless=True),
        # the whole 1.5B model, 580 tensors
        _case("step32 xl", "step32", **XL),
        # latency of the 8-bit step
        _case("update8 vectors", "update8", vectors=50),
        # a block's reduced gradients in fp32, as a reduce-scatter leaves them
        _case("update8 block", "update8", layers=1, d=1600, ffn=6400, grad="fp32"),
        # the 350M model, gapless and odd
        _case("update8 gapless", "update8", **MEDIUM, gapless=True),
        # the whole 1.5B model, fp16 under a static loss scale
        _case("update8 xl", "update8", **XL, grad="fp16", out="fp16", scale=1024.0),
        # the norm a clipped step of one block waits for
        _case("norm block", "norm", layers=1, d=1600, ffn=6400),
        # and of the whole 1.5B model
        _case("norm xl", "norm", **XL, grad="fp16", scale=65536.0),
        # resuming a 350M run from a checkpoint with 32-bit states
        _case("encode8 medium", "encode8", **MEDIUM),
        # writing such a checkpoint
        _case("decode8 medium", "decode8", **MEDIUM),
    ]


def draw(rng):
    op = rng.choice(["step32", "step32", "update8", "update8", "norm", "encode8", "decode8"])
    while True:
        log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
        d = log(48, 2100)
        kw = dict(layers=rng.choice([0, 0, 1, log(1, 40)]), d=d, ffn=log(d, 5 * d), vocab=rng.choice([0, log(100, 50000)]),
                  vectors=log(1, 300), ragged=rng.randint(0, 12))
        kw["ctx"] = log(8, 1024) if kw["vocab"] else 0
        c = _case(None, op, **kw)
        if sum(numels(c)) <= 400_000_000:
            break
    c["grad"] = rng.choice(["bf16", "fp16", "fp32"])
    c["out"] = "fp16" if c["grad"] == "fp16" else "bf16"
    c["scale"] = 2.0 ** rng.randint(4, 16) if c["grad"] == "fp16" else 1.0
    c["gapless"] = op in ("step32", "update8", "norm") and rng.random() < 0.4
    del c["name"]
    return c


def numels(case):
    """Element counts of the case's tensors, in order."""
    d, f = case["d"], case["ffn"]
    out = [case["vocab"] * d, case["ctx"] * d] if case["vocab"] else []
    for _ in range(case["layers"]):
        out += [d, d, d * 3 * d, 3 * d, d * d, d, d, d, d * f, f, f * d, d]
    out += [d] * case["vectors"]
    out += [1 + 37 * k * k * k for k in range(case["ragged"])]      # 1, 38, 297, 1000, ...
    return out


def work(case):
    n, op = sum(numels(case)), case["op"]
    g, o = SIZE[case["grad"]], SIZE[case["out"]]
    scales = sum(2 * (-(-k // BLOCK)) for k in numels(case))
    if op == "step32":       # each array once, although the update needs the gradients again after the norm
        return {"bytes": n * (g + 12 + 12 + o), "flops": 16 * n}
    if op == "update8":
        return {"bytes": n * (g + 4 + 2 + 4 + 2 + o) + 2 * scales, "flops": 16 * n}
    if op == "norm":
        return {"bytes": n * g, "flops": 2 * n}
    return {"bytes": n * 10 + scales, "flops": 4 * n}


# -- inputs ----------------------------------------------------------------------------------------------
def _layout(case):
    """(sizes, group of each tensor, offsets in the parameter buffer, its length, offsets in the state buffer, its length)."""
    ns = numels(case)
    matrix = 4 * max(case["d"], case["ffn"])
    groups = [0 if n > matrix else 1 for n in ns]

    def offsets(align):
        at, out = 0, []
        for n in ns:
            out.append(at)
            at += -(-n // align) * align
        return out, at

    aligned, total = offsets(ALIGN)
    po, pn = offsets(1) if case["gapless"] else (aligned, total)
    so, sn = (po, pn) if case["gapless"] and case["op"] in ("step32", "norm") else (aligned, total)
    return ns, groups, po, pn, so, sn


def _inputs(case, seed, dev="cuda"):
    """The flat input tensors of a case, made from the seed alone.  What lies between tensors is zero."""
    ns, groups, po, pn, so, sn = _layout(case)
    gen = torch.Generator(dev).manual_seed(seed)
    op = case["op"]
    rand = lambda n: torch.randn(n, generator=gen, device=dev)  # noqa: E731
    gaps = [(a + n, b) for a, n, b in zip(po, ns, po[1:] + [pn]) if a + n < b]
    sgaps = [(a + n, b) for a, n, b in zip(so, ns, so[1:] + [sn]) if a + n < b]
    d = {}
    if op in ("step32", "update8", "norm"):
        g = rand(pn).mul_(1e-3 * case["scale"])
        for k, (o, n) in enumerate(zip(po, ns)):
            if k % 3 == 1:
                g[o:o + n] *= 5.0                      # gradients of other sizes in other tensors
        if case["vocab"]:                              # rows of tokens that the batch did not hold
            rows = g[po[0]:po[0] + ns[0]].view(-1, case["d"])
            rows *= (torch.rand(rows.shape[0], 1, generator=gen, device=dev) > 0.3)
        for a, b in gaps:
            g[a:b] = 0
        d["grad"] = g.to(DT[case["grad"]])
        del g
    if op in ("step32", "update8"):
        d["master"] = rand(pn).mul_(0.02)
        for a, b in gaps:
            d["master"][a:b] = 0
        d["out"] = d["master"].to(DT[case["out"]])
    if op != "norm":
        d["m"] = rand(sn).mul_(3e-4)
        d["v"] = rand(sn).square_().add_(0.05).mul_(1e-6)
        for a, b in sgaps:
            d["m"][a:b] = 0
            d["v"][a:b] = 0
    if op in ("update8", "decode8"):
        d["m8"], d["ms"], d["v8"], d["vs"] = _encode(d.pop("m"), d.pop("v"))
    elif op == "encode8":
        d["m8"] = torch.zeros(sn, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
        d["v8"] = torch.zeros(sn, dtype=torch.uint8, device=dev).view(torch.float8_e5m2)
        d["ms"] = torch.ones(sn // BLOCK, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
        d["vs"] = d["ms"].clone()
    if op == "decode8":
        d["m"], d["v"] = torch.zeros(sn, device=dev), torch.zeros(sn, device=dev)
    return d


def prepare(case, seed):
    s = _inputs(case, seed)
    ns, groups, po, pn, so, sn = _layout(case)
    dev = "cuda"
    s["case"], s["t"] = case, STEPS_BEFORE
    # the plan of the plain form: lengths of the tensors and gaps in flat order, each one's group, and the
    # place of every parameter in the state buffer where the two differ
    ends = po[1:] + [pn]
    lens = [b - a for a, b in zip(po, ends)]
    s["lens"] = torch.tensor(lens, device=dev)
    s["groups"] = torch.tensor(groups, device=dev)
    s["state_lens"] = torch.tensor([b - a for a, b in zip(so, so[1:] + [sn])], device=dev)
    s["state_offsets"] = torch.tensor(so, device=dev)
    if po != so:
        shift = torch.tensor([b - a for a, b in zip(po, so)], device=dev)
        s["place"] = torch.arange(pn, device=dev) + torch.repeat_interleave(shift, s["lens"], output_size=pn)
    if own:
        # the handle a trainer keeps: the tensors as views of the same flat buffers
        import importlib
        multi = importlib.import_module(PKG + ".multi")
        engine = importlib.import_module(PKG + ".engine")
        views = lambda t, o: [t[a:a + n] for a, n in zip(o, ns)]  # noqa: E731
        scale_views = lambda t: [t[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(so, ns)]  # noqa: E731
        if case["op"] in ("encode8", "decode8"):
            s["codec"] = multi.StateCodec8(views(s["m"], so), views(s["v"], so), views(s["m8"], so), scale_views(s["ms"]),
                                           views(s["v8"], so), scale_views(s["vs"]))
        else:
            kw = dict(groups=[engine.AdamW(lr=lr, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=wd) for lr, wd in GROUPS],
                      group_of_tensor=groups, loss_scale=case["scale"])
            if case["op"] == "norm":
                s["opt"] = multi.MultiAdamW(None, views(s["grad"], po), max_norm=MAX_NORM, **kw)
            elif case["op"] == "step32":
                s["opt"] = multi.MultiAdamW(views(s["master"], po), views(s["grad"], po), views(s["out"], po), m=views(s["m"], so),
                                            v=views(s["v"], so), max_norm=MAX_NORM, **kw)
            else:
                s["opt"] = multi.MultiAdamW(views(s["master"], po), views(s["grad"], po), views(s["out"], po), state_bits=8,
                                            m=views(s["m8"], so), v=views(s["v8"], so), m_scale=scale_views(s["ms"]),
                                            v_scale=scale_views(s["vs"]), decide=False, seed=SEED8, **kw)
            s["opt"].resume_at(STEPS_BEFORE)
            s["clip"] = s["opt"].state_fields()["clip_coef"]
    return s


# -- the operators ---------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    op = s["case"]["op"]
    if op == "norm":
        s["opt"].grad_norm()
        return {"clip": s["clip"]}
    if op == "encode8":
        s["codec"].encode()
        return {k: s[k] for k in ("m8", "ms", "v8", "vs")}
    if op == "decode8":
        s["codec"].decode()
        return {k: s[k] for k in ("m", "v")}
    s["opt"].step()
    if op == "step32":
        return {"clip": s["clip"], **{k: s[k] for k in ("master", "m", "v", "out")}}
    return {k: s[k] for k in ("master", "out", "m8", "ms", "v8", "vs")}


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "encode8":
        s["m8"], s["ms"], s["v8"], s["vs"] = _encode(s["m"], s["v"])
        return {k: s[k] for k in ("m8", "ms", "v8", "vs")}
    if op == "decode8":
        s["m"], s["v"] = _decode(s["m8"], s["ms"]), _decode(s["v8"], s["vs"])
        return {k: s[k] for k in ("m", "v")}
    s["t"] += 1
    g = s["grad"].float() * (1.0 / case["scale"])
    if op in ("step32", "norm"):
        norm = g.square().sum().sqrt()
        clip = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
        if op == "norm":
            return {"clip": clip.reshape(1)}
        g = g * clip
    lens, gr, pn = s["lens"], s["groups"], s["master"].numel()
    spread = lambda v: torch.repeat_interleave(torch.tensor(v, device=g.device)[gr], lens, output_size=pn)  # noqa: E731
    bc1, bc2 = 1.0 - BETA1 ** s["t"], 1.0 - BETA2 ** s["t"]
    if op == "step32":
        m, v = s["m"], s["v"]
    else:
        m, v = _decode(s["m8"], s["ms"]), _decode(s["v8"], s["vs"])
        if "place" in s:
            m, v = m[s["place"]], v[s["place"]]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    den = v.sqrt() / math.sqrt(bc2) + EPS
    p = s["master"] * spread([1.0 - lr * wd for lr, wd in GROUPS]) - spread([lr / bc1 for lr, _ in GROUPS]) * (m / den)
    s["master"], s["out"] = p, p.to(s["out"].dtype)
    if op == "step32":
        s["m"], s["v"] = m, v
        return {"clip": clip.reshape(1), **{k: s[k] for k in ("master", "m", "v", "out")}}
    del g, den
    if "place" in s:        # back into the blocked order of the states
        blocked = torch.zeros(2, s["m8"].numel(), device=p.device)
        blocked[0, s["place"]], blocked[1, s["place"]] = m, v
        m, v = blocked[0], blocked[1]
    rm, rv = _random(s["state_lens"], s["state_offsets"], s["m8"].numel(), s["t"])
    s["m8"], s["ms"], s["v8"], s["vs"] = _encode(m, v, rm, rv)
    return {k: s[k] for k in ("master", "out", "m8", "ms", "v8", "vs")}


# -- the 8-bit form --------------------------------------------------------------------------------------
def _encode8(x, bias, cut, dtype, floor, rnd):
    """Codes and scales of x, blocks of 32.  bias: the type's largest exponent; cut: bits a rounding cuts off; rnd: random
    integers below 2^cut that are added before the cut, or None for the nearest code."""
    top = x.view(-1, BLOCK).abs().amax(1)
    byte = ((top.view(torch.int32) + 0x1FFFFF) >> 23).sub_(bias).clamp_(min=1)
    y = x.view(-1, BLOCK) * ((254 - byte) << 23).view(torch.float32)[:, None]
    positive = y > 0 if floor else None
    if rnd is not None:
        y = ((y.view(torch.int32) + rnd.view(-1, BLOCK)) & -(1 << cut)).view(torch.float32)
    if floor:               # what is above zero stays above zero
        y = torch.where(positive, y.clamp(min=floor), y)
    bad = ~torch.isfinite(top)
    byte = torch.where(bad, 255, byte).to(torch.uint8)
    code = torch.where(bad[:, None], math.nan, y).to(dtype)
    return code.reshape(-1), byte.view(torch.float8_e8m0fnu)


def _encode(m, v, rm=None, rv=None):
    m8, ms = _encode8(m, 8, 20, torch.float8_e4m3fn, 0.0, rm)
    v8, vs = _encode8(v, 15, 21, torch.float8_e5m2, 2.0 ** -16, rv)
    return m8, ms, v8, vs


def _decode(codes, scales):
    return (codes.float().view(-1, BLOCK) * scales.float()[:, None]).view(-1)


def _mix(x):
    """32-bit integer mixing on int32 tensors (products wrap)."""
    x = x ^ ((x >> 16) & 0xFFFF)
    x = x * (0x9E3779B1 - (1 << 32))
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * (0xBB67AE85 - (1 << 32))
    return x ^ ((x >> 16) & 0xFFFF)


def _mix_int(x):
    x ^= x >> 16
    x = x * 0x9E3779B1 & MASK32
    x ^= x >> 15
    x = x * 0xBB67AE85 & MASK32
    return x ^ (x >> 16)


def _random(state_lens, state_offsets, n, t):
    """The step's random integers: below 2^20 for m and below 2^21 for v, for every place of the state buffer.  A linear
    congruential generator starts anew every 8 elements of a tensor, from a hash of the seed, the step, the tensor and the place."""
    key = _mix_int(SEED8 ^ _mix_int(t))
    dev = state_lens.device
    signed = lambda x: x - (1 << 32) if x >= 1 << 31 else x  # noqa: E731
    tensors = torch.arange(state_lens.numel(), device=dev, dtype=torch.int32)
    keys = _mix(tensors + signed(key))
    groups = torch.div(state_lens, 8, rounding_mode="floor")
    first = torch.repeat_interleave(keys, groups, output_size=n // 8)
    q = torch.arange(n // 8, device=dev) - torch.repeat_interleave(torch.div(state_offsets, 8, rounding_mode="floor"), groups, output_size=n // 8)
    x = _mix(first + q.to(torch.int32) * (0x9E3779B1 - (1 << 32)))
    rm = torch.empty(n // 8, 8, dtype=torch.int32, device=dev)
    rv = torch.empty_like(rm)
    for k in range(8):
        x = x * 1664525 + 1013904223
        rm[:, k] = (x >> 12) & 0xFFFFF
        x = x * 1664525 + 1013904223
        rv[:, k] = (x >> 11) & 0x1FFFFF
    return rm.view(-1), rv.view(-1)


# -- the definition in 64 bits ---------------------------------------------------------------------------
def _units(y, lowest, digits):
    """One unit of the last place of |y| among binary numbers with `digits` digits whose normal numbers begin at 2^lowest."""
    e = torch.frexp(y.abs())[1].double() - 1.0
    return torch.exp2(torch.clamp(e, min=float(lowest)) - (digits - 1))


def _code64(x, top_exponent, lowest, digits, floor, rnd=None, bits=0):
    """(value of the code, scale) of x (blocks of 32, binary64): the scale is the power of two that brings the largest magnitude to at most 1.75 * 2^top."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1).float().double()
    f, e = torch.frexp(top)                     # top = f * 2^e, 0.5 <= f < 1
    e = e.double() - 1 + (f > 0.875) - top_exponent
    scale = torch.exp2(torch.where(top > 0, e.clamp(min=-126), torch.full_like(e, -126.0)))
    y = x / scale[:, None]
    if rnd is not None:                         # up with the probability that the cut part has
        free = _units(y, -300, digits)          # (to the kept digits first, whatever the exponent)
        y = torch.sign(y) * torch.floor(y.abs() / free + rnd.view(-1, BLOCK).double() / 2.0 ** bits) * free
    u = _units(y, lowest, digits)
    y = torch.round(y / u) * u                  # ties to even
    if floor:
        y = torch.where(x > 0, y.clamp(min=floor), y)
    return y.reshape(-1), scale


def _random64(ns, so, sn, t):
    """_random() again, with 64-bit integers, tensor by tensor."""
    def mix(x):
        x = x ^ (x >> 16)
        x = (x * 0x9E3779B1) & MASK32
        x = x ^ (x >> 15)
        x = (x * 0xBB67AE85) & MASK32
        return x ^ (x >> 16)

    key = int(mix(torch.tensor(SEED8 ^ int(mix(torch.tensor(t))))))
    rm = torch.zeros(sn, dtype=torch.int32, device="cuda")
    rv = torch.zeros(sn, dtype=torch.int32, device="cuda")
    for k, (n, o, end) in enumerate(zip(ns, so, so[1:] + [sn])):
        if o == end:
            continue
        q = torch.arange((end - o) // 8, device="cuda")
        tensor_key = int(mix(torch.tensor((key + k) & MASK32)))
        x = mix((tensor_key + q * 0x9E3779B1) & MASK32)
        for j in range(8):
            x = (x * 1664525 + 1013904223) & MASK32
            rm[o:end].view(-1, 8)[:, j] = (x >> 12).int()
            x = (x * 1664525 + 1013904223) & MASK32
            rv[o:end].view(-1, 8)[:, j] = (x >> 11).int()
    return rm, rv


def exact(case, seed):
    d = _inputs(case, seed)
    ns, groups, po, pn, so, sn = _layout(case)
    op = case["op"]
    if op == "encode8":
        m8, ms = _code64(d["m"].double(), 8, -6, 4, 0.0)
        v8, vs = _code64(d["v"].double(), 15, -14, 3, 2.0 ** -16)
        return {"m8": m8, "ms": ms, "v8": v8, "vs": vs}
    if op in ("decode8", "update8"):
        m = (d["m8"].double().view(-1, BLOCK) * d["ms"].double()[:, None]).view(-1)
        v = (d["v8"].double().view(-1, BLOCK) * d["vs"].double()[:, None]).view(-1)
        if op == "decode8":
            return {"m": m, "v": v}
    clip = 1.0
    if op in ("step32", "norm"):
        total = 0.0
        for a in range(0, pn, 1 << 28):
            total += float((d["grad"][a:a + (1 << 28)].double() / case["scale"]).square().sum())
        clip = min(1.0, MAX_NORM / (math.sqrt(total) + 1e-6))
        if op == "norm":
            return {"clip": torch.tensor([clip], dtype=torch.float64)}
        m, v = d["m"].double(), d["v"].double()
    t = STEPS_BEFORE + 1
    p = torch.zeros(pn, dtype=torch.float64, device="cuda")
    for n, group, a, b in zip(ns, groups, po, so):
        lr, wd = GROUPS[group]
        g = d["grad"][a:a + n].double() / case["scale"] * clip
        mm = m[b:b + n].mul_(BETA1).add_(g, alpha=1.0 - BETA1)
        vv = v[b:b + n].mul_(BETA2).addcmul_(g, g, value=1.0 - BETA2)
        step = (mm / (1.0 - BETA1 ** t)) / ((vv / (1.0 - BETA2 ** t)).sqrt() + EPS)
        p[a:a + n] = d["master"][a:a + n].double() * (1.0 - lr * wd) - lr * step
    if op == "step32":
        return {"clip": torch.tensor([clip], dtype=torch.float64), "master": p, "m": m, "v": v, "out": p}
    rm, rv = _random64(ns, so, sn, t)
    out = {"master": p, "out": p, "m8": torch.empty_like(m), "v8": torch.empty_like(v), "ms": torch.empty(sn // BLOCK, dtype=torch.float64, device="cuda")}
    out["vs"] = torch.empty_like(out["ms"])
    for a in range(0, sn, 1 << 27):
        e = min(sn, a + (1 << 27))
        blocks = slice(a // BLOCK, e // BLOCK)
        out["m8"][a:e], out["ms"][blocks] = _code64(m[a:e], 8, -6, 4, 0.0, rm[a:e], 20)
        out["v8"][a:e], out["vs"][blocks] = _code64(v[a:e], 15, -14, 3, 2.0 ** -16, rv[a:e], 21)
    return out
