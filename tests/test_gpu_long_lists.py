"""Lists so long that a block of the update takes many units: those whose
units follow a plain stride (about 4000 of a kind, where a block takes seven),
and those of 2^24 elements and more, whose units are handed out by a counter
that the last block resets.  Several steps follow one another without a wait,
a non-finite one among them.

32-bit states: the flat step's bits (the clip is off, so the formula is the
same in the same roundings).  8-bit states: the bytes of the formulas in torch
float32, one operation a rounding, after which each value goes to one of its
neighbours as its random number says.  Weights of 8-bit states: within 1e-6 of
their largest term, as for short lists.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

LR, WD = 3e-3, 0.01
B1, B2, EPS = 0.9, 0.999, 1e-8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def ragged(total, seed):
    """Sizes from 1 to some 200,000 that add up to `total`."""
    rng = np.random.default_rng(seed)
    sizes = []
    while total > 0:
        n = min(total, int(np.exp(rng.uniform(0, 12.2))))
        sizes.append(n)
        total -= n
    return sizes


# (sizes of tensors with 32-bit states, of those with 8-bit ones).  Four
# blocks of an SM and 152 SMs are 608 blocks: 4000 units are seven a block.
MIDDLE, LONG = 4000 * 2048 + 77, (1 << 25) + 12_345
LISTS = {"middle": ([MIDDLE], []), "middle8": ([], [MIDDLE]),
         "middle both": (ragged(MIDDLE, 1), ragged(MIDDLE, 2)),
         "one": ([LONG], []), "many": (ragged(LONG, 3), []),
         "one8": ([], [LONG]), "many8": ([], ragged(LONG, 4)),
         "both": ([LONG, 7], [3, LONG]), "many both": (ragged(LONG, 5), ragged(LONG, 6))}


class Arrays:
    """Two pools, one a kind of state, whose tensors lie one behind the other
    (32 bits) or start at multiples of 256 elements (8 bits); the list's order
    takes them in turn."""

    def __init__(self, plain, eight, g, seed):
        r = torch.Generator(device="cuda").manual_seed(seed)
        self.plain, self.eight = plain, eight
        n = sum(plain)
        self.starts8 = [256 * int(b) for b in np.cumsum([0] + [-(-k // 256) for k in eight])]
        n8 = self.starts8[-1]

        def normal(n, s):
            return torch.empty(n, device="cuda").normal_(0, s, generator=r)

        self.w, self.g = normal(n, 0.02), normal(n, 1e-3).to(TYPES[g])
        self.m, self.v = normal(n, 3e-4), normal(n, 1e-3).square_()
        self.w8, self.g8 = normal(n8, 0.02), normal(n8, 1e-3).to(TYPES[g])
        self.real = torch.zeros(n8, dtype=torch.bool, device="cuda")
        for a, k in zip(self.starts8, eight):
            self.real[a:a + k] = True
        for x in (self.w8, self.g8):
            x.masked_fill_(~self.real, 0.0)
        self.m8, self.v8 = (torch.zeros(n8, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ms, self.vs = (torch.zeros(n8 // 256, device="cuda") for _ in range(2))

    def make(self):
        cut = np.cumsum([0] + self.plain).tolist()
        f8 = (torch.float8_e4m3fn, torch.float8_e5m2)
        a = [[x[i:j] for x in (self.w, self.g, self.m, self.v)] + [None, None]
             for i, j in zip(cut, cut[1:])]
        b = [[x[i:i + k] for x in (self.w8, self.g8, self.m8.view(f8[0]), self.v8.view(f8[1]))]
             + [x[i // 256:i // 256 + -(-k // 256)] for x in (self.ms, self.vs)]
             for i, k in zip(self.starts8, self.eight)]
        order, block0, blocks = [], [], 0  # in turn; blocks before each 8-bit tensor
        for k in range(max(len(a), len(b))):
            if k < len(a):
                order.append(a[k])
                blocks += -(-self.plain[k] // 256)
            if k < len(b):
                order.append(b[k])
                block0.append(blocks)
                blocks += -(-self.eight[k] // 256)
        # the position of every element of the 8-bit pool in the list's blocks
        self.position = torch.zeros(self.w8.numel(), dtype=torch.int64, device="cuda")
        for i, j, p in zip(self.starts8, self.starts8[1:], block0):
            self.position[i:j] = 256 * p + torch.arange(j - i, device="cuda")
        return osr.adamw_list_create(*[[t[i] for t in order] for i in range(6)])


# ---- 8-bit states in torch -------------------------------------------------
def mix(x):
    """The hash of 32-bit words, in int64."""
    x = ((x ^ (x >> 16)) * 0x9E3779B1) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x85EBCA77) & 0xFFFFFFFF
    return x ^ (x >> 16)


def widen(codes, scale, kind):
    return codes.view(kind).float() * scale.repeat_interleave(256)


def power_of_two(e):
    """2^e in float64, from its bits (torch.ldexp goes through float32's pow)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def narrow(x, u, digits, lowest, top, positive):
    """(values' codes, scales) of float32 x in blocks of 256, each value taken
    to the lower neighbour or, as u of 2^16 says, to the upper one."""
    b = x.abs().double().view(-1, 256)
    most = b.amax(1)
    power = torch.where(most > 0, (torch.frexp(most).exponent - 1 - top).clamp(min=-126), -126)
    scale = power_of_two(power)
    y = b / scale[:, None]
    # the neighbours are multiples of a unit; lowest: the smallest normal exponent
    binade = (torch.frexp(y).exponent - 1).clamp(min=lowest)
    binade = torch.where(y > 0, binade, lowest)
    y = y * power_of_two(digits - binade)  # in units
    low = y.floor()
    # as far above the lower neighbour as the float32 word's low bits say
    bits = 23 - digits
    up = torch.floor((y - low) * 2.0 ** bits) + u.view(-1, 256).double() * 2.0 ** (bits - 16) >= 2.0 ** bits
    whole = (low + up).long()
    # a whole number of units is the code: normal numbers' first bit joins the exponent
    code = ((binade - lowest).long() << digits) + whole
    if positive:
        code = torch.where((code == 0) & (b > 0), 1, code)
    code = code.view(-1) | torch.where(torch.signbit(x), 0x80, 0)
    return code.to(torch.uint8), scale.float()


def model_step(a, t, seed):
    """The new bytes and scales of the 8-bit pool, and its moments before them."""
    one = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    g = a.g8.float()
    m = widen(a.m8, a.ms, torch.float8_e4m3fn)
    v = widen(a.v8, a.vs, torch.float8_e5m2)
    m = one(B1) * m + one(1 - B1) * g
    v = one(B2) * v + (one(1 - B2) * g) * g
    key = int(mix(torch.tensor(int(mix(torch.tensor(t))) ^ seed)))
    h = mix((a.position & 0xFFFFFFFF) ^ key)
    m8, ms = narrow(m, h >> 16, 3, -6, 7, False)
    v8, vs = narrow(v, h & 0xFFFF, 2, -14, 14, True)
    return (m8, ms, v8, vs), m, v


def test_the_model_s_codes_are_the_formats():
    """Every finite code, widened, is taken back to itself."""
    for kind, digits, lowest, top, count in ((torch.float8_e4m3fn, 3, -6, 7, 0x78),
                                             (torch.float8_e5m2, 2, -14, 14, 0x78)):
        codes = torch.zeros(256, dtype=torch.uint8, device="cuda")
        codes[:count] = torch.arange(count, device="cuda")
        x = codes.view(kind).float()
        assert bool(x.isfinite().all())
        got, scale = narrow(x, torch.zeros(256, device="cuda"), digits, lowest, top, False)
        assert float(scale[0]) == 1.0 and torch.equal(got, codes)


@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("which", list(LISTS))
def test_steps_of_long_lists(which, g):
    plain, eight = LISTS[which]
    a = Arrays(plain, eight, g, 7)
    flat = [x.clone() for x in (a.w, a.g.float(), a.m, a.v)]
    n = flat[0].numel()
    seed = 21
    with a.make() as lst, osr.adamw_create(max(n, 1)) as ctx:
        want8, w8 = None, a.w8.double()
        big = torch.zeros_like(w8)
        for t in (1, 2, 3):  # what the list has to come to
            if n:
                osr.adamw_clip_step(ctx, *flat, t, LR, WD, float("inf"))
            if eight:
                kept = [x.clone() for x in (a.m8, a.ms, a.v8, a.vs)]
                if want8:
                    for x, y in zip((a.m8, a.ms, a.v8, a.vs), want8):
                        x.copy_(y)
                want8, m, v = model_step(a, t, seed)
                for x, y in zip((a.m8, a.ms, a.v8, a.vs), kept):
                    x.copy_(y)
                den = (v.double() / (1 - B2 ** t)).sqrt() + EPS
                u = LR / (1 - B1 ** t) * m.double() / den
                # m's and v's roundings one by one: a few 2^-24 of the larger addend
                big = torch.maximum(big, torch.maximum(w8.abs(), LR / (1 - B1 ** t) * (
                    m.abs().double() + 2 * (1 - B1) * a.g8.double().abs()) / den))
                w8 = w8 * (1 - LR * WD) - u
        bad = a.g8 if eight else a.g
        last = bad.numel() - 1 if not eight else int(a.real.nonzero()[-1])
        keep = bad[last].clone()
        torch.cuda.synchronize()
        # two steps, one that a gradient spoils and that must leave all as it
        # is, one more; nothing waits in between
        osr.adamw_list_step(lst, 1, LR, WD, float("inf"), seed=seed)
        osr.adamw_list_step(lst, 2, LR, WD, float("inf"), seed=seed)
        bad[last] = float("inf")
        osr.adamw_list_step(lst, 3, LR, WD, float("inf"), seed=seed, zero_grad=True)
        bad[last:last + 1].copy_(keep)
        osr.adamw_list_step(lst, 3, LR, WD, float("inf"), seed=seed)
        norm, factor = osr.adamw_list_last_norm(lst)
    exact = float((a.g.double().square().sum() + a.g8.double().square().sum()).sqrt())
    assert norm == pytest.approx(exact, rel=1e-6) and factor == 1.0
    for name, x, y in zip("wgmv", (a.w, a.g.float(), a.m, a.v), flat):
        assert torch.equal(x, y), (name, int((x != y).sum()))
    if eight:
        for name, x, y in zip(("m", "m_scale", "v", "v_scale"), (a.m8, a.ms, a.v8, a.vs), want8):
            where = a.real if x.numel() == a.real.numel() else slice(None)
            diff = (x != y)[where]
            assert not bool(diff.any()), (name, int(diff.sum()))
        err = (a.w8.double() - w8).abs()
        assert bool((err <= 3e-6 * big + 2.0 ** -148)[a.real].all()), float((err / big.clamp(min=1e-30))[a.real].max())


@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_norm_of_long_lists(g):
    """Blocks of the norm with many rounds of loads within a tensor and across
    tensors, clipped: the factor reaches every element."""
    for plain in ([LONG], ragged(LONG, 8), [1 << 27]):
        a = Arrays(plain, [], g, 9)
        exact = float(a.g.double().square().sum().sqrt())
        m, v = a.m.double(), a.v.double()
        grad = a.g.double() * (0.5 / exact)
        with a.make() as lst:
            osr.adamw_list_step(lst, 1, LR, WD, 0.5)
            norm, factor = osr.adamw_list_last_norm(lst)
        assert norm == pytest.approx(exact, rel=1e-6) and factor == pytest.approx(0.5 / exact, rel=1e-6)
        big = torch.maximum(B1 * m.abs(), (1 - B1) * grad.abs())
        assert bool(((a.m.double() - (B1 * m + (1 - B1) * grad)).abs() <= 1e-6 * big + 2.0 ** -148).all())
        v1 = B2 * v + (1 - B2) * grad * grad
        assert bool(((a.v.double() - v1).abs() <= 1e-6 * v1 + 2.0 ** -148).all())
        del m, v, grad, big, v1
