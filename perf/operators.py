"""Measured cases of the AdamW operators, with their plain forms.

The parameters beside the matrices that the Muon-type steps take (embeddings,
the output head, norm gains, biases), or a whole model, are stepped by AdamW:

* ``step32``   one AdamW step over many tensors, float32 moments
* ``step8``    the same with both moments in 8 bits: E4M3 codes with one
               power-of-two exponent per block of 256 entries, rounded
               stochastically with a counter-based generator
* ``norm``     the gradients' global 2-norm, the clip factor made from it and a
               flag for gradients that are not finite, all left on the device
* ``convert``  the moments from 32 to 8 bits or back

All tensors of a case live in flat buffers, each starting at a multiple of 256
entries, as a program that owns its optimizer's memory lays them out; the flat
buffers are the outputs. Entries between two tensors are zero and stay so.

Definition of a step t (every ``f32`` a rounding to float32; s the clip factor):
  g = f32(s G), m' = f32(f32(b1 m) + f32(f32(1 - b1) g)),
  v' = f32(f32(b2 v) + f32(f32(1 - b2) f32(g g))), r' = f32(sqrt v'),
  W' = W - lr (wd W + (m' / (1 - b1^t)) / (r' / sqrt(1 - b2^t) + eps)).
8 bits: of a block of x (m' or r') with largest magnitude in [2^E, 2^(E+1)) the
exponent byte is E + 120 (0 below 2^-119, 255 if not finite), y = x / 2^(byte - 127),
and the code is y with 16 random bits R added at bit 4 of its float32 pattern,
cut to three mantissa bits and put into E4M3. R of entry e (within its tensor)
is half e % 2 of word (e % 8) / 2 of Philox4x32-10 at counter (e / 8 low, e / 8
high, t, 1) and key (seed, tensor). m is a code times 2^(byte - 127), v the
square of one. ``convert`` to 8 bits rounds y to nearest instead.
"""
import math
import random

import numpy as np
import torch

own = False

LR, B1, B2, EPS, DECAY, RNG_SEED, MAX_NORM = 1e-3, 0.9, 0.999, 1e-8, 0.1, 17, 1.0
BLOCK = 256
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the final norm's gain and bias alone: a step's fixed cost
        dict(name="step32 two gains", op="step32", set="vectors", blocks=0, width=1024, w="f32", g="f32", master=False, t=0, clip=False),
        # the gains and biases beside the GPT-2-Large matrices that Muon steps: 290 short tensors
        dict(name="step32 290 vectors", op="step32", set="vectors", blocks=36, width=1280, w="f32", g="f32", master=False, t=99, clip=True),
        # ResNet-50's convolutions with their norm vectors in float32
        dict(name="step32 resnet50", op="step32", set="convs", w="f32", g="f32", master=False, t=9, clip=False),
        # a whole model of GPT-2-Large shapes, bf16 weights with a float32 master
        dict(name="step32 774M", op="step32", set="model", blocks=36, width=1280, vocab=50257, w="bf16", g="bf16", master=True, t=999, clip=True),
        # ragged tensors: lengths from one entry on, few of them whole blocks
        dict(name="step8 ragged", op="step8", set="ragged", count=61, largest=70001, mix=5, w="f32", g="f32", master=False, t=0, clip=False),
        # an embedding with its positions, bf16 weights without a master
        dict(name="step8 embedding", op="step8", set="model", blocks=0, width=1280, vocab=50257, w="bf16", g="bf16", master=False, t=99, clip=True),
        # the whole model again: 8-bit moments beside bf16 weights and their master
        dict(name="step8 774M", op="step8", set="model", blocks=36, width=1280, vocab=50257, w="bf16", g="bf16", master=True, t=999, clip=True),
        # gradient norms before those steps
        dict(name="norm 290 vectors", op="norm", set="vectors", blocks=36, width=1280, g="f32"),
        dict(name="norm resnet50", op="norm", set="convs", g="f32"),
        dict(name="norm 774M", op="norm", set="model", blocks=36, width=1280, vocab=50257, g="bf16"),
        # a 32-bit checkpoint resumed with 8-bit moments, and an 8-bit one read out
        dict(name="convert to 8 resnet50", op="convert", set="convs", to=8),
        dict(name="convert to 32 embedding", op="convert", set="model", blocks=0, width=1280, vocab=50257, to=32),
    ]


def draw(rng):
    c = dict(op=rng.choice(["step32", "step8", "norm", "convert"]))
    c["set"] = rng.choice(["ragged", "ragged", "vectors", "model"])
    if c["set"] == "ragged":
        c.update(count=rng.randint(1, 300), largest=int(10 ** rng.uniform(0.5, 7.3)), mix=rng.randrange(1 << 30))
    elif c["set"] == "vectors":
        c.update(blocks=rng.randint(0, 48), width=int(2 ** rng.uniform(5, 13)))
    else:
        c.update(blocks=rng.randint(0, 12), width=int(2 ** rng.uniform(5, 11)), vocab=int(10 ** rng.uniform(2, 4.8)))
    if c["op"] == "convert":
        c["to"] = rng.choice([8, 32])
        return c
    c["g"] = rng.choice(["f32", "bf16"])
    if c["op"] != "norm":
        c["w"] = rng.choice(["f32", "bf16"])
        c.update(master=c["w"] == "bf16" and rng.random() < 0.5, t=rng.choice([0, 1, 9, 99, 9999]), clip=rng.random() < 0.5)
    return c


def _shapes(c):
    """(rows, columns) of a case's tensors; one row: a vector."""
    if c["set"] == "convs":  # 53 convolutions as C_out x (C_in k k), each with its norm's gain and bias
        convs, c_in = [(64, 147)], 64
        for count, mid, out in ((3, 64, 256), (4, 128, 512), (6, 256, 1024), (3, 512, 2048)):
            for b in range(count):
                convs += [(mid, c_in), (mid, 9 * mid), (out, mid)] + ([(out, c_in)] if b == 0 else [])
                c_in = out
        return [s for r, k in convs for s in ((r, k), (1, r), (1, r))]
    if c["set"] == "ragged":
        rng, got, left = random.Random(c["mix"]), [], 400_000_000
        for _ in range(c["count"]):
            n = min(left, int(math.exp(rng.uniform(0, math.log(c["largest"])))))
            cols = max(1, n) if rng.random() < 0.5 else max(1, int(math.exp(rng.uniform(0, math.log(max(2, n))))))
            got.append((max(1, n // cols), cols))
            left = max(1, left - n)
        return got
    d, vectors = c["width"], [c["width"] * k for k in (1, 1, 3, 1, 1, 1, 4, 1)]
    shapes = [(1, v) for _ in range(c["blocks"]) for v in vectors] + [(1, d)] * 2
    if c["set"] == "model":
        shapes = [(c["vocab"], d), (1024, d)] + [s for _ in range(c["blocks"]) for s in ((d, 3 * d), (d, d), (d, 4 * d), (4 * d, d))] + shapes
    return shapes


def _layout(c):
    """Each tensor's (rows, columns, first entry), and the flat length."""
    got, at = [], 0
    for r, k in _shapes(c):
        got.append((r, k, at))
        at += -(-r * k // BLOCK) * BLOCK
    return got, at


def work(case):
    n = sum(r * k for r, k in _shapes(case))
    blocks = sum(-(-r * k // BLOCK) for r, k in _shapes(case))
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "norm":
        return {"bytes": n * size[case["g"]] + 12, "flops": 2 * n}
    if case["op"] == "convert":
        return {"bytes": 10 * n + 2 * blocks, "flops": 4 * n}
    weights = (8 + size[case["w"]]) if case["master"] else 2 * size[case["w"]]
    moments = 16 * n if case["op"] == "step32" else 4 * n + 4 * blocks
    return {"bytes": n * (weights + size[case["g"]]) + moments, "flops": 16 * n}


# ---------------------------------------------------------------- inputs
def _views(flat, layout):
    return [flat[at:at + r * k].view(r, k) if r > 1 else flat[at:at + k] for r, k, at in layout]


def _blank(flat, layout, total):
    """Zeroes the entries between the tensors."""
    for (r, k, at), end in zip(layout, [a for _, _, a in layout[1:]] + [total]):
        if at + r * k < end:
            flat[at + r * k:end] = 0
    return flat


def prepare(case, seed):
    layout, total = _layout(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    blocks = total // BLOCK
    # gradients differ in size from row to row; a tenth of the rows has none in this step, some never had
    size = 1e-3 * torch.exp(normal(blocks, 1))
    idle = torch.rand(blocks, 1, generator=gen, device="cuda")
    s = {"op": case["op"], "layout": layout}
    if case["op"] != "convert":
        g = _blank((normal(blocks, BLOCK) * size * (idle > 0.1)).view(-1), layout, total)
        s["g"] = g.to(BF16 if case["g"] == "bf16" else F32)
        del g
    if case["op"] == "norm":
        if own:
            import matrix_aware_sign_b200 as S
            s["norm"] = S.GradNorm(_views(s["g"], layout), MAX_NORM)
        return s
    m = _blank((normal(blocks, BLOCK) * 0.3 * size * (idle > 0.05)).view(-1), layout, total)
    v = torch.rand(blocks, BLOCK, generator=gen, device="cuda").add_(0.3).mul_(size * size * (idle > 0.05)).view(-1)
    v = _blank(v, layout, total)
    held = 8 if case["op"] == "step8" or (case["op"] == "convert" and case["to"] == 32) else 32
    s["m"], s["v"] = m, v
    if held == 8:
        s["scales"] = torch.empty(blocks, 2, dtype=torch.uint8, device="cuda")
        s["m"], s["scales"][:, 0] = _encode(m)
        s["v"], s["scales"][:, 1] = _encode(torch.sqrt(v))
    if case["op"] == "convert":
        s["to"] = case["to"]
        kind = E4M3 if case["to"] == 8 else F32
        s["m_to"], s["v_to"] = torch.zeros(total, dtype=F32, device="cuda").to(kind), torch.zeros(total, dtype=F32, device="cuda").to(kind)
        if case["to"] == 8:
            s["scales_to"] = torch.zeros(blocks, 2, dtype=torch.uint8, device="cuda")
        w = torch.zeros(total, dtype=BF16, device="cuda")
        if own:
            import matrix_aware_sign_b200 as S
            s["from_opt"] = S.AdamW(_views(w, layout), m=_views(s["m"], layout), v=_views(s["v"], layout),
                                    scales=_scale_views(s.get("scales"), layout))
            s["to_opt"] = S.AdamW(_views(w, layout), m=_views(s["m_to"], layout), v=_views(s["v_to"], layout),
                                  scales=_scale_views(s.get("scales_to"), layout))
        return s
    w = _blank((0.02 * normal(total)), layout, total)
    s["w"] = w.to(BF16 if case["w"] == "bf16" else F32)
    if case["master"]:
        s["master"] = w
    decay = [DECAY if r > 1 else 0.0 for r, _, _ in layout]
    s["t"], s["coef"] = case["t"], torch.tensor([2.0, 0.4990234375], device="cuda") if case["clip"] else None
    if own:
        import matrix_aware_sign_b200 as S
        opt = S.AdamW(_views(s["w"], layout), m=_views(s["m"], layout), v=_views(s["v"], layout),
                      scales=_scale_views(s.get("scales"), layout),
                      master=_views(s["master"], layout) if case["master"] else None,
                      weight_decay=decay, seed=RNG_SEED, t=case["t"])
        s["plan"] = S.AdamWPlan(opt, _views(s["g"], layout), B1, B2, EPS, grad_scale=s["coef"][1:] if case["clip"] else None)
    else:  # which tensor a block belongs to, its place there, and its decay
        per = torch.tensor([-(-r * k // BLOCK) for r, k, _ in layout], device="cuda")
        s["tensor"] = torch.repeat_interleave(torch.arange(len(layout), device="cuda"), per)
        s["place"] = torch.arange(blocks, device="cuda") - torch.tensor([a // BLOCK for _, _, a in layout], device="cuda")[s["tensor"]]
        s["decay"] = torch.tensor(decay, device="cuda")[s["tensor"]].view(-1, 1)
    return s


def _scale_views(scales, layout):
    return None if scales is None else [scales[at // BLOCK:at // BLOCK + -(-r * k // BLOCK)] for r, k, at in layout]


# ---------------------------------------------------------------- plain forms
def _exponent(x):
    """Exponent byte of each block of x, and the power of two that brings its values below 256."""
    field = x.abs().amax(1).view(torch.int32) >> 23
    byte = torch.where(field == 255, field, (field - 7).clamp(min=0))
    up = torch.where((byte > 0) & (byte < 255), (254 - byte) << 23, torch.zeros_like(byte)).view(F32)
    return byte.to(torch.uint8), up.view(-1, 1)


def _encode(flat, bits=None):
    """E4M3 codes and exponent bytes of a flat float32 tensor: to nearest, or with 20 random bits a value."""
    x = flat.view(-1, BLOCK)
    byte, up = _exponent(x)
    y = x * up
    if bits is not None:
        y = ((y.view(torch.int32) + bits) & -0x100000).view(F32)
    return torch.where((byte == 255).view(-1, 1), torch.zeros_like(y), y).to(E4M3).view(-1), byte


def _decode(codes, byte):
    return codes.view(-1, BLOCK).to(F32) * (byte.to(torch.int32) << 23).view(F32).view(-1, 1)


def _random_bits(s, t):
    """16 bits for each entry, at bit 4."""
    low = 0xFFFFFFFF
    e = s["place"].view(-1, 1) * (BLOCK // 8) + torch.arange(BLOCK // 8, device="cuda")
    a, b, c, d = e & low, e >> 32, torch.full_like(e, t & low), torch.ones_like(e)
    k0, k1 = RNG_SEED, s["tensor"].view(-1, 1)
    p = lambda x, y: x * y  # noqa: E731 (products mod 2^64: their halves are taken below)
    for _ in range(10):
        u, w = p(a, 0xD2511F53), p(c, 0xCD9E8D57)
        a, b, c, d = ((w >> 32) & low) ^ b ^ k0, w & low, ((u >> 32) & low) ^ d ^ k1, u & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((a, b, c, d), -1)
    return (torch.stack((words & 0xFFFF, words >> 16), -1) << 4).to(torch.int32).view(-1, BLOCK)


def _plain_step(s):
    t = s["t"] = s["t"] + 1
    g = s["g"].to(F32).view(-1, BLOCK)
    if s["coef"] is not None:
        g = g * s["coef"][1]
    eight = s["op"] == "step8"
    if eight:
        m, r = _decode(s["m"], s["scales"][:, 0]), _decode(s["v"], s["scales"][:, 1])
        v = r * r
    else:
        m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * g) * (1 - B2)
    r = torch.sqrt(v)
    source = s["master"] if "master" in s else s["w"]
    w = source.to(F32).view(-1, BLOCK)
    step = (m / (1 - B1 ** t)) / (r / math.sqrt(1 - B2 ** t) + EPS)
    w = (w - LR * (s["decay"] * w + step)).view(-1)
    if eight:
        bits = _random_bits(s, t)
        for name, x, k in (("m", m, 0), ("v", r, 1)):
            codes, byte = _encode(x.reshape(-1), bits)
            s[name].copy_(codes)
            s["scales"][:, k] = byte
    else:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
    if "master" in s:
        s["master"].copy_(w)
    s["w"].copy_(w)


def _plain_norm(s):
    total = torch.sqrt(s["g"].to(torch.float64).square().sum())
    skip = ~torch.isfinite(total)
    coef = torch.clamp(MAX_NORM / (total + 1e-6), max=1.0)
    return {"norm": total.to(F32), "coef": torch.where(skip, torch.zeros_like(coef), coef).to(F32), "skip": skip.to(torch.int32)}


def _plain_convert(s):
    if s["to"] == 8:
        for name, x, k in (("m_to", s["m"], 0), ("v_to", torch.sqrt(s["v"]), 1)):
            codes, byte = _encode(x)
            s[name].copy_(codes)
            s["scales_to"][:, k] = byte
    else:
        s["m_to"].copy_(_decode(s["m"], s["scales"][:, 0]).view(-1))
        r = _decode(s["v"], s["scales"][:, 1])
        s["v_to"].copy_((r * r).view(-1))


def run(state):
    s = state
    if s["op"] == "norm":
        if not own:
            return _plain_norm(s)
        s["norm"].run()
        return {"norm": s["norm"].norm, "coef": s["norm"].coef, "skip": s["norm"].skip}
    if s["op"] == "convert":
        if own:
            import matrix_aware_sign_b200 as S
            S.adamw_convert(s["from_opt"], s["to_opt"])
        else:
            _plain_convert(s)
        out = {"m": s["m_to"], "v": s["v_to"]}
        if s["to"] == 8:  # codes as E4M3 values, exponent bytes as the powers of two they stand for
            out["scales"] = s["scales_to"].view(torch.float8_e8m0fnu)
        return out
    if own:
        s["plan"].run(LR)
    else:
        _plain_step(s)
    out = {k: s[k] for k in ("w", "master", "m", "v") if k in s}
    if "scales" in s:
        out["scales"] = s["scales"].view(torch.float8_e8m0fnu)
    return out


# ---------------------------------------------------------------- the definition in 64 bits
def _f32(x):
    """The definition's rounding to float32 of a 64-bit result."""
    return x.to(F32).to(torch.float64)


def _blocks64(x):
    """One tensor's entries as rows of 256, short last row filled with zeros."""
    out = torch.zeros(-(-x.numel() // BLOCK) * BLOCK, dtype=torch.float64, device="cuda")
    out[:x.numel()] = x
    return out.view(-1, BLOCK)


def _held8(x, noise):
    """(values of the codes, powers of two) that 8 bits hold of one tensor's finite float32 values (given in 64 bits).
    noise: in [0, 1) for each entry (an entry goes up where its part of a code step and its noise reach 1), None: to nearest."""
    rows = _blocks64(x)
    top = rows.abs().amax(1, keepdim=True)
    exponent = torch.frexp(top)[1].to(torch.float64) - 1
    held = top >= 2.0 ** -119
    y = torch.where(held, rows * torch.exp2(7 - exponent), torch.zeros_like(rows))
    if noise is not None:  # three bits after the leading one, at every size
        step = torch.exp2(torch.frexp(y)[1].to(torch.float64) - 4)
        below = torch.floor(y.abs() / step)
        y = torch.sign(y) * step * (below + ((y.abs() / step - below) + _blocks64(noise) >= 1))
    grid = torch.exp2(torch.clamp(torch.frexp(y)[1].to(torch.float64) - 1, min=-6.0) - 3)
    power = torch.where(held, torch.exp2(exponent - 7), torch.full_like(exponent, 2.0 ** -127))
    return (torch.round(y / grid) * grid).view(-1), power.view(-1)


def _noise(n, tensor, t):
    """Random numbers of one tensor's entries, multiples of 2^-16 in [0, 1)."""
    groups = -(-n // 8)
    out = torch.empty(groups, 8, dtype=torch.float64, device="cuda")
    for first in range(0, groups, 1 << 24):
        e = torch.arange(first, min(groups, first + (1 << 24)), device="cuda", dtype=torch.int64)
        word = [e % 2 ** 32, e // 2 ** 32, torch.full_like(e, t % 2 ** 32), torch.ones_like(e)]
        key = [RNG_SEED, tensor]

        def wide(x, k):  # high and low half of a 32 x 32 bit product, by 16-bit parts
            lo, hi = x * (k & 0xFFFF), x * (k >> 16)
            mid = (lo >> 16) + (hi & 0xFFFF)
            return (hi >> 16) + (mid >> 16), ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)

        for _ in range(10):
            h0, l0 = wide(word[0], 0xD2511F53)
            h1, l1 = wide(word[2], 0xCD9E8D57)
            word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        for i, x in enumerate(word):
            out[first:first + e.numel(), 2 * i] = (x % 65536).to(torch.float64) / 65536
            out[first:first + e.numel(), 2 * i + 1] = (x // 65536).to(torch.float64) / 65536
    return out.view(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    layout, double = s["layout"], lambda x: x.to(torch.float64)  # noqa: E731
    if case["op"] == "norm":
        norm = math.sqrt(sum(float(double(g).square().sum()) for g in _views(s["g"], layout)))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "coef": torch.tensor(min(1.0, MAX_NORM / (norm + 1e-6)), dtype=torch.float64), "skip": 0}
    total = s["m"].numel()
    flat = lambda: torch.zeros(total, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {k: flat() for k in ("w", "master", "m", "v") if k in s}
    t = case.get("t", 0) + 1
    eight = case["op"] == "step8" or case.get("to") == 8
    if eight:
        out["scales"] = torch.zeros(total // BLOCK, 2, dtype=torch.float64, device="cuda")
    for i, (rows, cols, at) in enumerate(layout):
        n = rows * cols
        of = slice(at, at + n)
        blocks = slice(at // BLOCK, at // BLOCK + -(-n // BLOCK))
        m, v = double(s["m"][of]), double(s["v"][of])
        if "scales" in s:
            scale = torch.exp2(double(s["scales"][blocks]) - 127).repeat_interleave(BLOCK, 0)[:n]
            m, v = m * scale[:, 0], (v * scale[:, 1]).square()
        root = _f32(torch.sqrt(v))
        if case["op"] != "convert":
            g = double(s["g"][of])
            if eight:  # what 8 bits hold goes by the float32 moments, so their roundings belong to the definition
                g = _f32(g * double(s["coef"][1])) if case["clip"] else g
                b1, a1, b2, a2 = (float(np.float32(x)) for x in (B1, 1 - B1, B2, 1 - B2))
                m = _f32(_f32(b1 * m) + _f32(a1 * g))
                v = _f32(_f32(b2 * v) + _f32(a2 * _f32(g * g)))
                root = _f32(torch.sqrt(v))
            else:
                g = g * double(s["coef"][1]) if case["clip"] else g
                m, v = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
                root = torch.sqrt(v)
            w = double((s["master"] if case["master"] else s["w"])[of])
            w = w - LR * ((DECAY if rows > 1 else 0.0) * w + (m / -math.expm1(t * math.log(B1))) / (root / math.sqrt(-math.expm1(t * math.log(B2))) + EPS))
            for k in ("w", "master"):
                if k in out:
                    out[k][of] = w
        if eight:
            noise = _noise(n, i, t) if case["op"] == "step8" else None
            for k, (name, x) in enumerate((("m", m), ("v", root))):
                values, power = _held8(x, noise)
                out[name][of] = values[:n]
                out["scales"][blocks, k] = power
        else:
            out["m"][of], out["v"][of] = m, v
    return out
