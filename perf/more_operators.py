"""The measured cases of the operators between the layer norm and the
optimizer: the matrix product with bias, activation and residual and its
backward pass, the cross entropy over a vocabulary whose logits are never
kept and its gradient, and the distillation from a teacher's top logits and
its gradient.

Every case runs in two forms that take the same inputs: the plain one
(``own`` false), elementary torch operations in 32 bits, and the library's
kernels (``own`` true).  ``exact`` restates the definitions in 64 bits, the
gradients by automatic differentiation.

Matrix product: y = act(x W^T + b) + residual, z = x W^T + b the
pre-activation that the backward pass reads; dz = dy act'(z), dx = dz W,
dW = dz^T x, db = sum of dz over the rows.

Cross entropy: logits l = x W^T; lse = log sum exp l; loss = lse - l[target] +
z_loss lse^2, one a row, 0 where the target is negative (padding).  The
gradient of sum(scale loss): dl = scale ((1 + 2 z_loss lse) exp(l - lse) -
[target]), dx = dl W, dW = dl^T x.

Distillation: q = softmax of the teacher's k logits over T, p = softmax of the
student's over T; loss = T^2 sum_k q_k (log q_k - log p[id_k]), one a row;
entries with a negative id are absent, a row without entries has loss 0.  The
gradient of sum(scale loss): scale T (p - q) at the student's logits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def linear(name, op, rows, cin, cout, x, act, **more):
    return dict({"op": op, "name": name, "rows": rows, "in": cin, "out": cout, "x": x, "act": act,
                 "bias": True, "residual": False, "keep": False, "in_out": False,
                 "accumulate": False}, **more)


def ce(name, op, rows, dim, vocab, x, **more):
    return dict({"op": op, "name": name, "rows": rows, "dim": dim, "vocab": vocab, "x": x,
                 "ignored": 0.05, "z_loss": 0.0}, **more)


def distill(name, op, rows, vocab, k, x, **more):
    return dict({"op": op, "name": name, "rows": rows, "vocab": vocab, "k": k, "x": x,
                 "temperature": 1.0}, **more)


def listed():
    return [
        # one token through a wide model's MLP, as generation does it: the weights' bytes
        linear("linear_fwd_token", "linear_fwd", 1, 2048, 8192, "bf16", "gelu"),
        # the output projection of the 110M model's attention, with its residual: 8 sequences
        # of 1024 tokens
        linear("linear_fwd_8192x768", "linear_fwd", 8192, 768, 768, "bf16", "none",
               residual=True),
        # the first half of a wide model's MLP in a training step: the largest
        linear("linear_fwd_16384x4096", "linear_fwd", 16384, 4096, 16384, "bf16", "gelu_tanh",
               keep=True),
        # the 110M projection's backward pass, its weight stored (in, out) and its gradients
        # added into the 32-bit ones that the optimizer reads
        linear("linear_bwd_8192x768", "linear_bwd", 8192, 768, 768, "bf16", "none", in_out=True,
               accumulate=True),
        # a wide MLP's first half, backward through its activation
        linear("linear_bwd_8192x4096", "linear_bwd", 8192, 4096, 8192, "bf16", "gelu"),
        # sizes that divide by nothing
        linear("linear_bwd_5003x1021", "linear_bwd", 5003, 1021, 1531, "f16", "gelu"),
        # the loss of the 110M model's step, and its gradient: the tied embedding is the head
        ce("ce_fwd_8192x768", "ce_fwd", 8192, 768, 32000, "bf16"),
        ce("ce_bwd_8192x768", "ce_bwd", 8192, 768, 32000, "bf16"),
        # an odd vocabulary and a ragged batch, with the penalty on the logits' scale
        ce("ce_bwd_1001x509", "ce_bwd", 1001, 509, 10007, "f16", ignored=0.3, z_loss=1e-4),
        # a student of the 110M model's vocabulary and the 32 best logits of its teacher
        distill("distill_fwd_8192x32000", "distill_fwd", 8192, 32000, 32, "bf16"),
        distill("distill_bwd_8192x32000", "distill_bwd", 8192, 32000, 32, "bf16",
                temperature=2.0),
        # an odd vocabulary, whose rows start anywhere, in 32 bits
        distill("distill_bwd_2003x50021", "distill_bwd", 2003, 50021, 50, "f32"),
    ]


MOST = 2 * 16384 * 4096 * 16384  # the largest listed case's multiplications and additions


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        n = spread(lo, hi)
        return max(8, n // 8 * 8) if rng.random() < 0.6 else n

    kind = rng.choice(("linear", "linear", "ce", "ce", "distill"))
    x = rng.choice(("bf16", "f16"))
    back = rng.random() < 0.5
    if kind == "linear":
        cin, cout = width(64, 8192), width(64, 16384)
        act = rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu"))
        rows = min(spread(1, 16384), max(1, MOST // ((4 if back else 2) * cin * cout)))
        case = linear("", "linear_bwd" if back else "linear_fwd", rows, cin, cout, x, act,
                      bias=rng.random() < 0.7, in_out=rng.random() < 0.4)
        if back:
            case["accumulate"] = act == "none" and rng.random() < 0.5
        else:
            case["residual"] = rng.random() < 0.4
            case["keep"] = act != "none" and rng.random() < 0.5
    elif kind == "ce":
        dim = width(64, 4096)
        vocab = width(1000, min(130000, 280_000_000 // dim))
        rows = min(spread(1, 16384), max(1, MOST // ((6 if back else 2) * dim * vocab)),
                   (1 << 29) // vocab)
        case = ce("", "ce_bwd" if back else "ce_fwd", rows, dim, vocab, x,
                  ignored=rng.choice((0.0, 0.05, 0.5)), z_loss=rng.choice((0.0, 1e-4)))
    else:
        vocab = width(1000, 130000)
        case = distill("", "distill_bwd" if back else "distill_fwd",
                       min(spread(1, 8192), (1 << 27) // vocab), vocab, spread(1, 128),
                       rng.choice(("f32", x)), temperature=rng.choice((1.0, 2.0)))
    del case["name"]
    return case


def work(case):
    rows, s = case["rows"], SIZE[case["x"]]
    if case["op"].startswith("linear"):
        a, b, back = case["in"], case["out"], case["op"] == "linear_bwd"
        if not back:
            values = rows * a + a * b + rows * b * (1 + case["residual"] + case["keep"])
            return {"bytes": s * (values + b * case["bias"]), "flops": 2 * rows * a * b}
        values = 2 * rows * a + a * b + rows * b * (1 + (case["act"] != "none"))
        grads = (a * b + b * case["bias"]) * (8 if case["accumulate"] else s)
        return {"bytes": s * values + grads, "flops": 4 * rows * a * b}
    if case["op"].startswith("ce"):
        n, d, back = case["vocab"], case["dim"], case["op"] == "ce_bwd"
        return {"bytes": s * (1 + back) * (rows * d + n * d) + rows * (12 if back else 16),
                "flops": (6 if back else 2) * rows * n * d}
    back = case["op"] == "distill_bwd"
    return {"bytes": s * rows * case["vocab"] * (1 + back) + rows * (12 * case["k"] + 8),
            "flops": (4 + 2 * back) * rows * case["vocab"]}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def normal(r, shape, sigma=1.0):
    return torch.empty(shape, device="cuda").normal_(0.0, sigma, generator=r)


def prepare(case, seed):
    r = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    kind = TYPES[case["x"]]
    if case["op"].startswith("linear"):
        prepare_linear(case, s, r, kind)
    elif case["op"].startswith("ce"):
        prepare_ce(case, s, r, kind)
    else:
        prepare_distill(case, s, r, kind)
    return s


def prepare_linear(case, s, r, kind):
    rows, a, b = case["rows"], case["in"], case["out"]
    # rows as a layer norm leaves them; weights that keep their scale
    s["x"] = normal(r, (rows, a)).to(kind)
    w = normal(r, (a, b) if case["in_out"] else (b, a), a ** -0.5).to(kind)
    s["weight"] = w.T if case["in_out"] else w
    s["bias"] = normal(r, b, 0.2).to(kind) if case["bias"] else None
    if case["op"] == "linear_fwd":
        s["residual"] = normal(r, (rows, b), 2.0).to(kind) if case["residual"] else None
        s["y"] = torch.empty(rows, b, device="cuda", dtype=kind)
        s["z"] = torch.empty(rows, b, device="cuda", dtype=kind) if case["keep"] else None
    else:
        s["dy"] = normal(r, (rows, b), 1e-2).to(kind)
        s["z"] = normal(r, (rows, b)).to(kind) if case["act"] != "none" else None
        grad = torch.float32 if case["accumulate"] else kind
        s["dx"] = torch.empty(rows, a, device="cuda", dtype=kind)
        dw = normal(r, w.shape, 0.01).to(grad)
        s["dweight"] = dw.T if case["in_out"] else dw
        s["dbias"] = normal(r, b, 0.01).to(grad) if case["bias"] else None
    if own:
        import optimizer_step_resumable_gb300 as osr
        s["linear"] = osr.linear_create(a, b)


def prepare_ce(case, s, r, kind):
    rows, d, n = case["rows"], case["dim"], case["vocab"]
    s["x"] = normal(r, (rows, d)).to(kind)
    s["weight"] = normal(r, (n, d), 1.5 * d ** -0.5).to(kind)
    # frequent tokens come first, as a vocabulary is sorted; some places are padding
    u = torch.rand(rows, device="cuda", generator=r)
    target = (torch.exp(u * math.log(n)) - 1).long().clamp(0, n - 1)
    padding = torch.rand(rows, device="cuda", generator=r) < case["ignored"]
    s["target"] = torch.where(padding, -100, target)
    s["scale"] = 1.0 / rows if case["x"] == "bf16" else 64.0 / rows  # loss scaling in f16
    if case["op"] == "ce_fwd":
        s["loss"], s["lse"] = (torch.empty(rows, device="cuda") for _ in range(2))
    else:
        s["lse"] = (s["x"].float() @ s["weight"].float().T).logsumexp(1)
        s["dx"], s["dweight"] = torch.empty_like(s["x"]), torch.empty_like(s["weight"])
    if own:
        import optimizer_step_resumable_gb300 as osr
        s["ce"] = osr.linear_cross_entropy_create(d, n)


def prepare_distill(case, s, r, kind):
    rows, n, k = case["rows"], case["vocab"], case["k"]
    s["logits"] = normal(r, (rows, n), 2.0).to(kind)
    # the teacher's best: the student's logits with a say of its own, some entries absent
    places = torch.randint(0, n, (rows, 4 * k), device="cuda", generator=r)
    value = s["logits"].gather(1, places).float() + normal(r, (rows, 4 * k), 1.5)
    best = value.topk(k, dim=1)
    ids = places.gather(1, best.indices)
    absent = torch.rand(rows, k, device="cuda", generator=r) < 0.05
    s["ids"] = torch.where(absent, -1, ids)
    s["values"] = best.values
    if case["op"] == "distill_fwd":
        s["loss"], s["lse"] = (torch.empty(rows, device="cuda") for _ in range(2))
    else:
        s["lse"] = (s["logits"].float() / case["temperature"]).logsumexp(1)
        s["dlogits"] = torch.empty_like(s["logits"])
        s["scale"] = 1.0 / rows if case["x"] != "f16" else 64.0 / rows
    if own:
        import optimizer_step_resumable_gb300 as osr
        s["distill"] = osr.distill_create(n, k)


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    (own_pass if own else PLAIN[op])(state)
    keys = {"linear_fwd": ("y", "z"), "linear_bwd": ("dx", "dweight", "dbias"),
            "ce_fwd": ("loss", "lse"), "ce_bwd": ("dx", "dweight"),
            "distill_fwd": ("loss", "lse"), "distill_bwd": ("dlogits",)}[op]
    return {k: state[k] for k in keys if state[k] is not None}


def own_pass(s):
    import optimizer_step_resumable_gb300 as osr
    case = s["case"]
    op = case["op"]
    if op == "linear_fwd":
        osr.linear_forward(s["linear"], s["x"], s["weight"], s["bias"], residual=s["residual"],
                           activation=case["act"], y=s["y"], z=s["z"])
    elif op == "linear_bwd":
        osr.linear_backward(s["linear"], s["dy"], s["x"], s["weight"], z=s["z"],
                            activation=case["act"], dx=s["dx"], dweight=s["dweight"],
                            dbias=s["dbias"], accumulate=case["accumulate"])
    elif op == "ce_fwd":
        osr.linear_cross_entropy_forward(s["ce"], s["x"], s["weight"], s["target"],
                                         z_loss=case["z_loss"], loss=s["loss"], lse=s["lse"])
    elif op == "ce_bwd":
        osr.linear_cross_entropy_backward(s["ce"], s["x"], s["weight"], s["target"], s["lse"],
                                          scale=s["scale"], z_loss=case["z_loss"], dx=s["dx"],
                                          dweight=s["dweight"])
    elif op == "distill_fwd":
        osr.distill_forward(s["distill"], s["logits"], s["ids"], s["values"],
                            temperature=case["temperature"], loss=s["loss"], lse=s["lse"])
    else:
        osr.distill_backward(s["distill"], s["logits"], s["ids"], s["values"], s["lse"],
                             temperature=case["temperature"], scale=s["scale"],
                             dlogits=s["dlogits"])


# ---- matrix product, plain -----------------------------------------------
def activate(z, act):
    """act(z)."""
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
    return 0.5 * z * (1 + torch.tanh(u))


def slope(z, act):
    """act'(z)."""
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        g = 1 / (1 + torch.exp(-z))
        return g * (1 + z * (1 - g))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)


def plain_linear_fwd(s):
    z = s["x"].float() @ s["weight"].float().T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if s["z"] is not None:
        s["z"].copy_(z)
    y = activate(z, s["case"]["act"])
    s["y"].copy_(y if s["residual"] is None else y + s["residual"].float())


def plain_linear_bwd(s):
    case = s["case"]
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * slope(s["z"].float(), case["act"])
    s["dx"].copy_(dz @ s["weight"].float())
    dw, db = dz.T @ s["x"].float(), dz.sum(0)
    s["dweight"].copy_(s["dweight"] + dw if case["accumulate"] else dw)
    if s["dbias"] is not None:
        s["dbias"].copy_(s["dbias"] + db if case["accumulate"] else db)


# ---- cross entropy, plain ------------------------------------------------
def plain_ce_fwd(s):
    target, z_loss = s["target"], s["case"]["z_loss"]
    logits = s["x"].float() @ s["weight"].float().T
    most = logits.amax(1)
    lse = most + torch.exp(logits - most[:, None]).sum(1).log()
    at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    s["loss"].copy_(torch.where(target >= 0, lse - at + z_loss * lse * lse, 0.0))
    s["lse"].copy_(lse)


def plain_ce_bwd(s):
    target, z_loss, lse = s["target"], s["case"]["z_loss"], s["lse"]
    x, weight = s["x"].float(), s["weight"].float()
    scale = torch.where(target >= 0, s["scale"], 0.0)
    dl = torch.exp(x @ weight.T - lse[:, None])
    dl *= (scale * (1 + 2 * z_loss * lse))[:, None]
    place = target.clamp(min=0)[:, None]
    dl.scatter_add_(1, place, -scale[:, None])
    s["dx"].copy_(dl @ weight)
    s["dweight"].copy_(dl.T @ x)


# ---- distillation, plain -------------------------------------------------
def teacher(s):
    """The teacher's probabilities and their logarithms; 0 where absent."""
    there = s["ids"] >= 0
    v = torch.where(there, s["values"].float() / s["case"]["temperature"], -torch.inf)
    v = v - v.amax(1, keepdim=True)
    e = torch.where(there, torch.exp(v), 0.0)
    total = e.sum(1, keepdim=True)
    q = torch.where(there, e / total, 0.0)
    return q, torch.where(there, v - total.log(), 0.0)


def plain_distill_fwd(s):
    t = s["case"]["temperature"]
    q, log_q = teacher(s)
    l = s["logits"].float() / t
    most = l.amax(1, keepdim=True)
    lse = most[:, 0] + torch.exp(l - most).sum(1).log()
    log_p = l.gather(1, s["ids"].clamp(min=0)) - lse[:, None]
    s["loss"].copy_(t * t * (q * (log_q - log_p)).sum(1))
    s["lse"].copy_(lse)


def plain_distill_bwd(s):
    t = s["case"]["temperature"]
    q, _ = teacher(s)
    some = (s["ids"] >= 0).any(1, keepdim=True)
    d = torch.where(some, torch.exp(s["logits"].float() / t - s["lse"][:, None]), 0.0)
    d.scatter_add_(1, s["ids"].clamp(min=0), -q)
    s["dlogits"].copy_(d * (t * s["scale"]))


PLAIN = {"linear_fwd": plain_linear_fwd, "linear_bwd": plain_linear_bwd, "ce_fwd": plain_ce_fwd,
         "ce_bwd": plain_ce_bwd, "distill_fwd": plain_distill_fwd,
         "distill_bwd": plain_distill_bwd}


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"].startswith("linear") and work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    wide = {k: x.double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x
            for k, x in s.items()}
    if case["op"].startswith("linear"):
        return exact_linear(case, wide)
    if case["op"].startswith("ce"):
        return exact_ce(case, wide)
    return exact_distill(case, wide)


def exact_linear(case, s):
    f = torch.nn.functional
    act = {"none": lambda z: z, "relu": f.relu, "silu": f.silu, "gelu": f.gelu,
           "gelu_tanh": lambda z: f.gelu(z, approximate="tanh")}[case["act"]]
    if case["op"] == "linear_fwd":
        z = f.linear(s["x"], s["weight"], s["bias"])
        y = act(z) + (s["residual"] if case["residual"] else 0.0)
        return {"y": y, "z": z} if case["keep"] else {"y": y}
    if case["act"] == "none":
        dz = s["dy"]
    else:
        z = s["z"].requires_grad_()
        dz, = torch.autograd.grad(act(z), z, s["dy"])
    add = 1.0 if case["accumulate"] else 0.0
    out = {"dx": torch.mm(dz, s["weight"]),
           "dweight": add * s["dweight"] + torch.einsum("ro,ri->oi", dz, s["x"])}
    if case["bias"]:
        out["dbias"] = add * s["dbias"] + torch.einsum("ro->o", dz)
    return out


def exact_ce(case, s):
    x, w, target = s["x"], s["weight"], s["target"]
    back = case["op"] == "ce_bwd"
    x.requires_grad_(back), w.requires_grad_(back)
    with torch.set_grad_enabled(back):
        logits = x @ w.mT
        lse = logits.logsumexp(1)
        nll = torch.nn.functional.cross_entropy(logits, target, reduction="none",
                                                ignore_index=-100)
        loss = nll + torch.where(target == -100, 0.0, case["z_loss"] * lse.square())
        if back:
            dx, dw = torch.autograd.grad(loss.sum() * s["scale"], (x, w))
            return {"dx": dx, "dweight": dw}
    return {"loss": loss, "lse": lse}


def exact_distill(case, s):
    t, ids, logits = case["temperature"], s["ids"], s["logits"]
    back = case["op"] == "distill_bwd"
    logits.requires_grad_(back)
    absent = ids == -1
    with torch.set_grad_enabled(back):
        log_p = torch.log_softmax(logits / t, 1)
        log_q = torch.log_softmax((s["values"] / t).masked_fill(absent, -1e300), 1)
        terms = log_q.exp() * (log_q - log_p.take_along_dim(ids.clamp(min=0), 1))
        loss = t ** 2 * terms.masked_fill(absent, 0.0).sum(1)
        if back:
            return {"dlogits": torch.autograd.grad(loss.sum() * s["scale"], logits)[0]}
    return {"loss": loss, "lse": (logits / t).logsumexp(1)}
