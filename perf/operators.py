"""The measured cases of the training operators: AdamW over a list of tensors
with its states in 32 or in 8 bits, and the layer norm's forward and backward
pass.

Every case runs in two forms that take the same inputs: the plain one
(``own`` false), elementary torch operations in 32 bits, and the library's
kernels (``own`` true).  ``exact`` restates the definitions in 64 bits.

AdamW.  The tensors of a list lie in pools, one pool for each of w, g, m, v
(and the 16-bit weight copy), every tensor at the next multiple of 256
elements, the size of a scale block.  The plain form works on whole pools;
the padding holds zeros, which the update leaves at zero.

States in 8 bits.  Per block of 256 elements of one tensor, m is held as
e4m3 and v as e5m2 values times a power of two, which is chosen from the
block's largest magnitude.  Both are rounded up or down at random, with the
value as the mean; the random numbers are a hash of the seed, the step and
the element's position, so they are inputs.  A positive v does not become 0.
A stored value depends on every bit of the new moment, so the listed 8-bit
cases keep the gradient's norm below the clip threshold, as most steps of a
settled run do: the factor is then exactly 1 in every form.
"""
import math

import torch

own = False

BLOCK = 256  # elements of a scale block, and the pools' alignment
BETA1, BETA2, EPS = 0.9, 0.999, 1e-8
LR, WD, CLIP = 3e-3, 0.01, 1.0
LN_EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def adam(name, tensors, bits, g, copy, **more):
    return dict({"op": "adamw", "name": name, "tensors": tensors, "bits": bits, "g": g,
                 "copy": copy, "clipped": False, "zero": False}, **more)


def norm(name, op, rows, cols, x, w, **more):
    return dict({"op": op, "name": name, "rows": rows, "cols": cols, "x": x, "w": w, "bias": True,
                 "pad": 0, "accumulate": False}, **more)


def listed():
    return [
        # the gains and shifts of the 25 layer norms of the 110M model: many tiny tensors,
        # where launches and latency are all the time
        adam("adamw32_gains", "gains", 32, "f32", False, clipped=True),
        # sizes of every kind from one element up, no multiples of anything, gradients
        # of 16 bits, zeroed for the next accumulation
        adam("adamw32_ragged", "ragged:240:40000000:5", 32, "f16", False, clipped=True, zero=True),
        # the 110M model's 196 tensors in mixed precision: 16-bit gradients and the 16-bit
        # copy of the weights that the next forward pass reads
        adam("adamw32_110m", "gpt110m", 32, "bf16", True, clipped=True),
        # the smallest list in 8 bits: a few adapter matrices
        adam("adamw8_adapters", "ragged:24:400000:9", 8, "f32", False),
        # the 110M model with its moments in 8 bits
        adam("adamw8_110m", "gpt110m", 8, "bf16", True),
        # a 570M model (width 2048, 10 blocks, a vocabulary of 32000) in 8 bits: the largest
        adam("adamw8_570m", "decoder:2048:10:32000", 8, "bf16", True),
        # one token's vector: the latency of a call
        norm("ln_fwd_token", "ln_fwd", 1, 768, "bf16", "f32"),
        # one norm of the 110M model's step: 8 sequences of 1024 tokens
        norm("ln_fwd_8192x768", "ln_fwd", 8192, 768, "bf16", "f32"),
        # a wide model's long batch
        norm("ln_fwd_65536x4096", "ln_fwd", 65536, 4096, "bf16", "bf16"),
        # its backward twin, added into the 32-bit gradient that the optimizer reads
        norm("ln_bwd_8192x768", "ln_bwd", 8192, 768, "bf16", "f32", accumulate=True),
        # a width that divides by nothing, in 32 bits
        norm("ln_bwd_5003x1021", "ln_bwd", 5003, 1021, "f32", "f32"),
        # the wide model's backward pass
        norm("ln_bwd_65536x4096", "ln_bwd", 65536, 4096, "bf16", "bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.5:
        count, total = spread(1, 400), spread(2000, 3e8)
        case = adam("", "ragged:%d:%d:%d" % (count, total, rng.randrange(1 << 20)),
                    rng.choice((8, 32)), rng.choice(("f32", "bf16", "f16")), rng.random() < 0.5,
                    zero=rng.random() < 0.25)
        case["clipped"] = case["bits"] == 32 and rng.random() < 0.5
    else:
        cols = spread(16, 16384)
        if rng.random() < 0.6:
            cols = max(8, cols // 8 * 8)
        rows = spread(1, min(1 << 17, (1 << 28) // cols))
        x = rng.choice(("f32", "bf16", "f16"))
        case = norm("", rng.choice(("ln_fwd", "ln_bwd")), rows, cols, x, rng.choice(("f32", x)),
                    bias=rng.random() < 0.8, pad=rng.choice((0, 0, 0, 8, 40, 13)))
        case["accumulate"] = case["op"] == "ln_bwd" and rng.random() < 0.5
    del case["name"]
    return case


def numels(spec):
    """The tensors of a list by its name: their numbers of elements."""
    kind, *args = spec.split(":")
    args = [int(a) for a in args]
    if kind == "gains":
        return [768] * 50
    if kind == "gpt110m":  # embeddings; q, k, v, o, two MLP matrices, biases, norms; last norm
        d, ff = 768, 3072
        block = [d * d, d] * 4 + [d * ff, ff, ff * d, d] + [d] * 4
        return [32000 * d, 1024 * d] + block * 12 + [d, d]
    if kind == "decoder":
        d, layers, vocab = args
        return [vocab * d] + [d * d] * 4 * layers + [4 * d * d] * 2 * layers + [d] * (2 * layers + 1)
    count, total, seed = args  # ragged: sizes spread over their logarithm, scaled to the total
    r = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.rand(count, generator=r, dtype=torch.float64) * 9.0)
    return [max(1, int(s)) for s in size * (total / float(size.sum()))]


def work(case):
    if case["op"] == "adamw":
        n = sum(numels(case["tensors"]))
        state = 8 if case["bits"] == 32 else 2 + 8 / BLOCK
        each = SIZE[case["g"]] + 2 * (4 + state) + 2 * case["copy"] + SIZE[case["g"]] * case["zero"]
        return {"bytes": each * n, "flops": 20 * n}
    n, c = case["rows"] * case["cols"], case["cols"]
    s, sw = SIZE[case["x"]], SIZE[case["w"]]
    if case["op"] == "ln_fwd":
        return {"bytes": 2 * s * n + 8 * case["rows"] + sw * c * (1 + case["bias"]), "flops": 8 * n}
    grads = (1 + case["bias"]) * (4 if case["accumulate"] else sw) * (1 + case["accumulate"])
    return {"bytes": 3 * s * n + 8 * case["rows"] + (sw + grads) * c, "flops": 16 * n}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def prepare(case, seed):
    r = torch.Generator(device="cuda").manual_seed(seed)
    make = prepare_adamw if case["op"] == "adamw" else prepare_norm
    return make(case, seed, r)


def normal(r, n, sigma=1.0, mean=0.0):
    return torch.empty(n, device="cuda").normal_(mean, sigma, generator=r)


def prepare_adamw(case, seed, r):
    sizes = torch.tensor(numels(case["tensors"]))
    blocks = (sizes + BLOCK - 1) // BLOCK
    starts = (blocks.cumsum(0) - blocks) * BLOCK
    total = int(blocks.sum()) * BLOCK
    # which places of the pools belong to a tensor, and which decay: matrices, not vectors
    place = torch.arange(total, device="cuda", dtype=torch.int32)
    first = torch.repeat_interleave(starts.cuda(), blocks.cuda()).int().repeat_interleave(BLOCK)
    length = torch.repeat_interleave(sizes.cuda(), blocks.cuda()).int().repeat_interleave(BLOCK)
    real = place - first < length
    decays = sizes > 4096
    count = int(sizes.sum())
    # gradients of one scale with a tail of large ones; the norm above or below the threshold
    g = normal(r, total) * torch.exp(normal(r, total, 0.7)) * real
    g *= (4.0 if case["clipped"] else 0.5) * CLIP / math.sqrt(2.7 * count)
    typical = float((g * g).sum().sqrt()) / math.sqrt(count)
    w = normal(r, total, 0.02) * real
    m = (0.3 * typical * normal(r, total) + 0.05 * g) * real
    v = (typical * typical * torch.exp(normal(r, total, 1.0, -0.5)) * 0.1) * real
    s = {"case": case, "w": w, "g": g.to(TYPES[case["g"]]), "t": 100, "seed": seed & 0x7FFFFFFF}
    if case["bits"] == 8:
        key = mix(torch.tensor([seed & 0x7FFFFFFF], device="cuda", dtype=torch.int32))
        h = mix(place ^ key)
        s["m"], s["m_scale"] = squeeze(m, h >> 16, *E4M3)
        s["v"], s["v_scale"] = squeeze(v, h, *E5M2)
        del h
    else:
        s["m"], s["v"] = m, v
    if case["copy"]:
        s["w_lp"] = w.to(torch.bfloat16)
    if not own:
        s["decay"] = torch.repeat_interleave(decays.cuda(), blocks.cuda())
        s["blocks"] = total // BLOCK
        return s
    import optimizer_step_resumable_gb300 as osr

    def parts(pool):
        return [pool[a:a + n] for a, n in zip(starts.tolist(), sizes.tolist())]

    def scales(pool):
        return [pool[a // BLOCK:a // BLOCK + b] for a, b in zip(starts.tolist(), blocks.tolist())]

    s["list"] = osr.adamw_list_create(
        parts(s["w"]), parts(s["g"]), parts(s["m"]), parts(s["v"]),
        m_scale=scales(s["m_scale"]) if case["bits"] == 8 else None,
        v_scale=scales(s["v_scale"]) if case["bits"] == 8 else None,
        w_lp=parts(s["w_lp"]) if case["copy"] else None, decay=decays.tolist())
    return s


def prepare_norm(case, seed, r):
    rows, cols, kind = case["rows"], case["cols"], TYPES[case["x"]]

    def matrix(sigma, wander):
        # rows of their own mean and scale, in a buffer whose rows are `pad` apart
        x = normal(r, rows * (cols + case["pad"]), sigma).view(rows, -1)
        x *= 0.5 + torch.rand(rows, 1, device="cuda", generator=r)
        if wander:
            x += normal(r, rows, wander).view(rows, 1)
        return x.to(kind)[:, :cols]

    s = {"case": case, "x": matrix(1.5, 1.0)}
    s["weight"] = normal(r, cols, 0.2, 1.0).to(TYPES[case["w"]])
    if case["op"] == "ln_fwd":
        s["bias"] = normal(r, cols, 0.2).to(TYPES[case["w"]]) if case["bias"] else None
        s["y"] = torch.empty(rows, cols, device="cuda", dtype=kind)
        s["mean"], s["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
    else:
        s["dy"] = matrix(1e-3, 0)
        s["mean"], s["rstd"] = statistics(s["x"].float())
        grad = torch.float32 if case["accumulate"] else TYPES[case["w"]]
        s["dx"] = torch.empty(rows, cols, device="cuda", dtype=kind)
        s["dweight"] = normal(r, cols, 0.01).to(grad)
        s["dbias"] = normal(r, cols, 0.01).to(grad) if case["bias"] else None
    if own:
        import optimizer_step_resumable_gb300 as osr
        s["norm"] = osr.layernorm_create(cols)
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if op == "adamw":
        (own_adamw if own else plain_adamw)(state)
        return {k: state[k] for k in ("w", "g", "m", "v", "m_scale", "v_scale", "w_lp")
                if k in state and (k != "g" or state["case"]["zero"])}
    if op == "ln_fwd":
        (own_forward if own else plain_forward)(state)
        return state["y"], state["mean"], state["rstd"]
    (own_backward if own else plain_backward)(state)
    return [state["dx"], state["dweight"]] + ([state["dbias"]] if state["case"]["bias"] else [])


def own_adamw(s):
    import optimizer_step_resumable_gb300 as osr
    osr.adamw_list_step(s["list"], s["t"], LR, WD, CLIP, seed=s["seed"], zero_grad=s["case"]["zero"])


def own_forward(s):
    import optimizer_step_resumable_gb300 as osr
    osr.layernorm_forward(s["norm"], s["x"], s["weight"], s["bias"], eps=LN_EPS, y=s["y"],
                          mean=s["mean"], rstd=s["rstd"])


def own_backward(s):
    import optimizer_step_resumable_gb300 as osr
    osr.layernorm_backward(s["norm"], s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                           dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"],
                           accumulate=s["case"]["accumulate"])


# ---- AdamW, plain --------------------------------------------------------
def mix(x):
    """A hash of 32 bits: xor-shifts and odd multipliers (int32, wrapping)."""
    x = (x ^ ((x >> 16) & 0xFFFF)) * -1640531535
    x = (x ^ ((x >> 15) & 0x1FFFF)) * -2048144777
    return x ^ ((x >> 16) & 0xFFFF)


# (significand bits, exponent bias, exponent of a block's largest value, type)
E4M3 = (3, 7, 7, torch.float8_e4m3fn)
E5M2 = (2, 15, 14, torch.float8_e5m2)


def squeeze(x, random, bits, bias, top, kind):
    """8-bit values and block scales of x, rounded by the low 16 bits of `random`."""
    b = x.view(-1, BLOCK)
    exponent = ((b.abs().amax(1).view(torch.int32) >> 23) - top).clamp(min=1)
    scale = (exponent << 23).view(torch.float32)
    inverse = ((254 - exponent) << 23).view(torch.float32)
    # moved down so that the format's subnormals are binary32's: then all that is below a
    # kept bit is the low 23 - bits of the word
    low = (b.abs() * inverse[:, None] * 2.0 ** (bias - 127)).view(-1).view(torch.int32)
    code = (low + ((random & 0xFFFF) << (7 - bits))) >> (23 - bits)
    if kind == torch.float8_e5m2:
        code = torch.where(x > 0, code.clamp(min=1), code)
    code = code | ((x.view(torch.int32) >> 24) & 0x80)
    return code.to(torch.uint8).view(kind), scale


def spread_out(x, scale):
    return (x.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def plain_adamw(s):
    case, t = s["case"], s["t"]
    g = s["g"].float()
    total = (g * g).sum().sqrt()
    g = g * torch.where(total > CLIP, CLIP / total, torch.ones_like(total))
    if case["bits"] == 8:
        m, v = spread_out(s["m"], s["m_scale"]), spread_out(s["v"], s["v_scale"])
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + ((1 - BETA2) * g) * g
    update = (LR / (1 - BETA1 ** t)) * (m / (v.sqrt() * (1 / math.sqrt(1 - BETA2 ** t)) + EPS))
    decay = torch.where(s["decay"], 1 - LR * WD, 1.0).float()
    s["w"].copy_((s["w"].view(-1, BLOCK) * decay[:, None]).view(-1) - update)
    if case["bits"] == 8:
        key = mix(torch.tensor(t, dtype=torch.int32))
        key = int(mix(key ^ s["seed"]))
        random = mix(torch.arange(m.numel(), device="cuda", dtype=torch.int32) ^ key)
        for name, x, bits_, form in (("m", m, random >> 16, E4M3), ("v", v, random, E5M2)):
            code, scale = squeeze(x, bits_, *form)
            s[name].copy_(code)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if case["copy"]:
        s["w_lp"].copy_(s["w"])
    if case["zero"]:
        s["g"].zero_()


# ---- layer norm, plain ---------------------------------------------------
def statistics(x):
    mean = x.mean(1)
    d = x - mean[:, None]
    return mean, 1 / ((d * d).mean(1) + LN_EPS).sqrt()


def plain_forward(s):
    x = s["x"].float()
    mean, rstd = statistics(x)
    y = (x - mean[:, None]) * rstd[:, None] * s["weight"].float()
    s["y"].copy_(y if s["bias"] is None else y + s["bias"].float())
    s["mean"].copy_(mean)
    s["rstd"].copy_(rstd)


def plain_backward(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    a = dy * s["weight"].float()
    s["dx"].copy_(rstd * (a - a.mean(1)[:, None] - xhat * (a * xhat).mean(1)[:, None]))
    dweight, dbias = (dy * xhat).sum(0), dy.sum(0)
    add = s["case"]["accumulate"]
    s["dweight"].copy_(s["dweight"] + dweight if add else dweight)
    if s["dbias"] is not None:
        s["dbias"].copy_(s["dbias"] + dbias if add else dbias)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "adamw" and sum(numels(case["tensors"])) > 1.5e8:
        return None
    s = prepare(case, seed)
    wide = {k: x.double() for k, x in s.items()
            if isinstance(x, torch.Tensor) and x.is_floating_point()}
    if case["op"] == "adamw":
        return exact_adamw(case, s, wide)
    x = wide["x"]
    if case["op"] == "ln_fwd":
        mean, var = x.mean(1, keepdim=True), x.var(1, correction=0, keepdim=True)
        rstd = (var + LN_EPS).rsqrt()
        y = (x - mean) * rstd * wide["weight"] + (wide["bias"] if case["bias"] else 0.0)
        return y, mean[:, 0], rstd[:, 0]
    dy, n = wide["dy"], case["cols"]
    rstd = wide["rstd"][:, None]
    xhat = (x - wide["mean"][:, None]) * rstd
    a = dy * wide["weight"]
    dx = rstd / n * (n * a - a.sum(1, keepdim=True) - xhat * (a * xhat).sum(1, keepdim=True))
    add = 1.0 if case["accumulate"] else 0.0
    out = [dx, torch.einsum("rc,rc->c", dy, xhat) + add * wide["dweight"]]
    return out + ([dy.sum(0) + add * wide["dbias"]] if case["bias"] else [])


def exact_adamw(case, s, wide):
    t, g = s["t"], wide["g"]
    g = g * min(1.0, CLIP / float(torch.linalg.vector_norm(g)))
    if case["bits"] == 8:
        for k in ("m", "v"):
            wide[k] = wide[k] * wide[k + "_scale"].repeat_interleave(BLOCK)
    m = torch.lerp(g, wide["m"], BETA1)
    v = torch.lerp(g.square(), wide["v"], BETA2)
    step = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
    w = wide["w"] * (1 - LR * WD * s["decay"].repeat_interleave(BLOCK)) - LR * step
    out = {"w": w, "m": m, "v": v}
    if case["bits"] == 8:
        key = mix_exact(mix_exact(t) ^ s["seed"])
        h = mix_exact(torch.arange(m.numel(), device="cuda", dtype=torch.int64) ^ key)
        for k, u, lowest, digits, top in (("m", h >> 16, -6, 3, 7), ("v", h & 0xFFFF, -14, 2, 14)):
            x = out[k].abs().view(-1, BLOCK)
            most = x.amax(1)
            power = (torch.frexp(most).exponent - 1 - top).clamp(min=-126)
            power = torch.where(most > 0, power, -126)  # a block of zeros
            scale = torch.ldexp(torch.ones_like(most), power)
            x = x / scale[:, None]
            # the neighbours of x in the format are multiples of `unit`
            binade = (torch.frexp(x).exponent - 1).clamp(min=lowest)
            unit = torch.ldexp(torch.ones_like(x), binade - digits)
            value = unit * torch.floor(x / unit + u.view(-1, BLOCK) / 65536)
            if k == "v":
                value = torch.where(x > 0, value.clamp(min=2.0 ** -16), value)
            out[k] = torch.copysign(value.view(-1), out[k])
            out[k + "_scale"] = scale
        if case["g"] != "f32":
            # 0.9 m + 0.1 g of so few significand bits often is a power of two, or a stored
            # value, to the last bit: which side of it m lies on no arithmetic says
            out["m"] = out["m_scale"] = None
    if case["copy"]:
        out["w_lp"] = w
    if case["zero"]:
        out["g"] = torch.zeros_like(g)
    return out


def mix_exact(x):
    """mix() on whole numbers that are not negative, below 2 ** 32."""
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x85EBCA77) & 0xFFFFFFFF
    return x ^ (x >> 16)
