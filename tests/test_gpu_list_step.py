"""The step over a list of tensors against plain references.

32-bit states: the flat step's bits (same formula, factor 1), and the update
in 64 bits within the bars of parity.py (1e-6 of the largest term; the list
step's longest chain of roundings is the flat step's, plus two for 8-bit
states, whose moments round each product and sum on its own: 10 x 2^-24 and
the norm's 3.6e-7 through the factor stay below it).

8-bit states: the stored bytes equal those of the same formulas in numpy
float32 (one IEEE rounding per operation) wherever the clip factor is 1; with
a factor that differs in its last bit a value may round to the other
neighbour, so there the bar is one spacing of the 8-bit format.
"""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

LR, WD = 3e-3, 0.01
B1, B2, EPS = 0.9, 0.999, 1e-8
SIZES = [1, 0, 3, 255, 256, 257, 1023, 1024, 1025, 70_001, 4096]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.manual_seed(0)


def blocks(n):
    return -(-n // 256)


class State:
    """A list's arrays, each tensor in memory of its own at `shift` elements
    past an allocation's start; `eight`: which tensors have 8-bit states."""

    def __init__(self, sizes, seed, g="f32", eight=(), shift=0, copy=None, sigma=1e-3):
        rng = np.random.default_rng(seed)
        self.sizes, self.eight = sizes, [bool(e) for e in (eight or [0] * len(sizes))]

        def put(a, dtype):
            t = torch.zeros(a.size + shift, dtype=dtype, device="cuda")
            t[shift:] = torch.from_numpy(a).to("cuda").to(dtype)
            return t[shift:]

        def normal(n, s):
            return (rng.standard_normal(n) * s).astype(np.float32)

        self.w = [put(normal(n, 0.02), torch.float32) for n in sizes]
        self.g = [put(normal(n, sigma), TYPES[g]) for n in sizes]
        self.m, self.v, self.ms, self.vs = [], [], [], []
        for n, e in zip(sizes, self.eight):
            if e:
                self.m.append(torch.zeros(n + shift, dtype=torch.uint8, device="cuda")[shift:]
                              .view(torch.float8_e4m3fn))
                self.v.append(torch.zeros(n + shift, dtype=torch.uint8, device="cuda")[shift:]
                              .view(torch.float8_e5m2))
                self.ms.append(torch.zeros(blocks(n), device="cuda"))
                self.vs.append(torch.zeros(blocks(n), device="cuda"))
            else:
                self.m.append(put(normal(n, sigma / 3), torch.float32))
                self.v.append(put(normal(n, sigma) ** 2, torch.float32))
                self.ms.append(None)
                self.vs.append(None)
        self.lp = [put(np.zeros(n, np.float32), TYPES[copy]) for n in sizes] if copy else None

    def make(self, **kw):
        return osr.adamw_list_create(self.w, self.g, self.m, self.v, self.ms, self.vs, self.lp,
                                     **kw)

    def host(self):
        """Float64 copies of w, g, m, v."""
        out = []
        for k in range(len(self.sizes)):
            wide = [self.w[k].double(), self.g[k].double(), self.m[k].float().double(),
                    self.v[k].float().double()]
            if self.eight[k]:
                for i, s in ((2, self.ms[k]), (3, self.vs[k])):
                    wide[i] = wide[i] * s.double().repeat_interleave(256)[:wide[i].numel()]
            out.append([t.cpu().numpy() for t in wide])
        return out

    def bytes(self):
        parts = list(itertools.chain(self.w, self.g, self.m, self.v, self.ms, self.vs,
                                     self.lp or ()))
        return b"".join(t.view(torch.uint8).cpu().numpy().tobytes() for t in parts
                        if t is not None and t.numel())


def reference(host, t, clip, scale=1.0, decay=None, lr=LR, wd=WD):
    """(w, m, v, term magnitudes of w, m) of every tensor, in 64 bits."""
    norm = scale * np.sqrt(sum(float(np.sum(h[1] ** 2)) for h in host))
    s = scale * (clip / norm if norm > clip else 1.0)
    out = []
    for k, (w, g, m, v) in enumerate(host):
        d = 1 - lr * wd if decay is None or decay[k] else 1.0
        gh = s * g
        m1, v1 = B1 * m + (1 - B1) * gh, B2 * v + (1 - B2) * gh * gh
        den = np.sqrt(v1 / (1 - B2 ** t)) + EPS
        upd = lr * (m1 / (1 - B1 ** t)) / den
        big = np.maximum.reduce([np.abs(m1), B1 * np.abs(m), (1 - B1) * np.abs(gh)])
        u = lr / (1 - B1 ** t) * big / den
        w1 = w * d - upd
        out.append((w1, m1, v1, np.maximum.reduce([np.abs(w1), np.abs(w * d), u]), big))
    return out, norm, s


def close(got, want, mag, rtol=1e-6, label=""):
    err = np.abs(got - want)
    bad = np.nonzero(~(err <= rtol * mag + 2.0 ** -148))[0]
    assert not bad.size, (label, bad.size, int(bad[0]), got[bad[0]], want[bad[0]])


def check(state, before, t, clip, scale=1.0, decay=None, wd=WD):
    want, norm, s = reference(before, t, clip, scale, decay, wd=wd)
    after = state.host()
    for k, (w1, m1, v1, wmag, mmag) in enumerate(want):
        close(after[k][0], w1, wmag, label=("w", k))
        if state.eight[k]:
            # one spacing: 1/8 of m's value, 1/4 of v's, or the smallest value times the scale
            ms = state.ms[k].double().repeat_interleave(256)[:m1.size].cpu().numpy()
            vs = state.vs[k].double().repeat_interleave(256)[:v1.size].cpu().numpy()
            assert np.all(np.abs(after[k][2] - m1) <= 0.126 * np.abs(m1) + ms * 2.0 ** -9), k
            assert np.all(np.abs(after[k][3] - v1) <= 0.251 * v1 + vs * 2.0 ** -16), k
            assert np.all(after[k][3][v1 > 0] > 0), k
        else:
            close(after[k][2], m1, mmag, label=("m", k))
            close(after[k][3], v1, v1, label=("v", k))
        if state.lp:
            lp = state.w[k].to(state.lp[k].dtype)
            assert torch.equal(lp, state.lp[k])
    return norm, s


@pytest.mark.parametrize("g", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("eight", [0, 1])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_steps_against_64_bits(g, eight, shift):
    st = State(SIZES, 3, g, [eight] * len(SIZES), shift, copy="bf16" if shift != 4 else None)
    with st.make() as lst:
        for t in (1, 2, 3):
            before = st.host()
            osr.adamw_list_step(lst, t, LR, WD, 0.1, seed=5)
            norm, s = check(st, before, t, 0.1)
            got = osr.adamw_list_last_norm(lst)
            assert got[0] == pytest.approx(norm, rel=1e-6) and got[1] == pytest.approx(s, rel=1e-6)
            assert s < 1  # clipped


def test_both_kinds_of_state_in_one_list():
    eight = [k % 2 for k in range(len(SIZES))]
    decay = [k % 3 != 0 for k in range(len(SIZES))]
    st = State(SIZES, 4, "bf16", eight, copy="f16")
    with st.make(decay=decay) as lst:
        for t in (1, 2):
            before = st.host()
            osr.adamw_list_step(lst, t, LR, 0.5, 1.0, grad_scale=0.25, seed=t)
            check(st, before, t, 1.0, 0.25, decay, wd=0.5)
        osr.adamw_list_set_decay(lst, None)
        before = st.host()
        osr.adamw_list_step(lst, 3, LR, 0.5, 1.0)
        check(st, before, 3, 1.0, wd=0.5)


def test_32_bit_states_equal_the_flat_step():
    """With factor 1 on both sides the update is the same formula, element by
    element, so the same bits, wherever the tensors start."""
    sizes = [769, 3, 4096, 257, 2048]
    n = sum(sizes)
    rng = np.random.default_rng(0)
    base = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda() for _ in range(4)]
    base[3].square_()
    flat, listed = ([x.clone() for x in base] for _ in range(2))
    cut = np.cumsum([0] + sizes)
    w, g, m, v = ([x[a:b] for a, b in zip(cut, cut[1:])] for x in listed)
    with osr.adamw_create(n) as ctx, osr.adamw_list_create(w, g, m, v) as lst:
        for t in (1, 2, 7):
            osr.adamw_clip_step(ctx, *flat, t, LR, WD, float("inf"))
            osr.adamw_list_step(lst, t, LR, WD, float("inf"))
    for a, b in zip(flat, listed):
        assert torch.equal(a, b)


# ---- 8-bit states, byte for byte ------------------------------------------
def mix(x):
    x = np.uint32(x) if np.isscalar(x) else x.astype(np.uint32)
    with np.errstate(over="ignore"):
        x = (x ^ (x >> np.uint32(16))) * np.uint32(0x9E3779B1)
        x = (x ^ (x >> np.uint32(15))) * np.uint32(0x85EBCA77)
        return x ^ (x >> np.uint32(16))


def decode(code, bits, bias):
    """The values of 8-bit codes (bits: of the significand), from the format."""
    c = code.astype(np.int64)
    e, f = (c & 0x7F) >> bits, c & ((1 << bits) - 1)
    v = np.where(e > 0, (1 + f / 2.0 ** bits) * 2.0 ** (e - bias), f / 2.0 ** bits * 2.0 ** (1 - bias))
    return np.where(c & 0x80, -v, v)


def encode(x, u, bits, bias, top, positive):
    """Codes and scales of float32 x (in blocks of 256): neighbours in the
    format by search in its table of values, chosen by u of 2^16."""
    table = decode(np.arange(0x7F if bits == 3 else 0x7C), bits, bias)
    code = np.zeros(x.size, np.uint8)
    scales = np.zeros(blocks(x.size), np.float32)
    for b in range(blocks(x.size)):
        at = slice(256 * b, min(x.size, 256 * b + 256))
        a = np.abs(x[at].astype(np.float64))
        most = a.max()
        e = int(np.floor(np.log2(most))) - top if most > 0 else -126
        scales[b] = 2.0 ** max(e, -126)
        y = a / float(scales[b])
        lo = np.searchsorted(table, y, side="right") - 1
        frac = (y - table[lo]) / (table[lo + 1] - table[lo])
        c = lo + (np.floor(frac * 2.0 ** (20 if bits == 3 else 21))
                  + u[at].astype(np.float64) * (16 if bits == 3 else 32)
                  >= 2.0 ** (20 if bits == 3 else 21))
        if positive:
            c = np.where((c == 0) & (a > 0), 1, c)
        code[at] = c.astype(np.uint8) | np.where(np.signbit(x[at]), 0x80, 0).astype(np.uint8)
    return code, scales


def model_step(code, g, t, seed, block0):
    """One update of the moments in numpy float32, one rounding an operation."""
    (mc, ms), (vc, vs) = code
    n = g.size
    f = np.float32
    m = decode(mc, 3, 7).astype(f) * np.repeat(ms, 256)[:n]
    v = decode(vc, 2, 15).astype(f) * np.repeat(vs, 256)[:n]
    m = f(B1) * m + f(1 - B1) * g
    v = f(B2) * v + (f(1 - B2) * g) * g
    key = mix(int(mix(t)) ^ seed)
    h = mix((np.arange(n, dtype=np.uint64) + 256 * block0).astype(np.uint32) ^ key)
    return encode(m, h >> np.uint32(16), 3, 7, 7, False), encode(v, h & np.uint32(0xFFFF), 2, 15, 14, True)


def test_float8_tables_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    for bits, bias, kind, bad in ((3, 7, torch.float8_e4m3fn, {0x7F, 0xFF}),
                                  (2, 15, torch.float8_e5m2, set(range(0x7C, 0x80)) | set(range(0xFC, 0x100)))):
        want = torch.from_numpy(codes).view(kind).float().numpy()
        keep = [c for c in codes if int(c) not in bad]
        assert np.array_equal(decode(codes, bits, bias)[keep].astype(np.float32), want[keep])


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_8_bit_states_byte_for_byte(shift, g):
    sizes = [300, 1, 0, 2049, 256]
    st = State(sizes, 8, g, [1] * len(sizes), shift)
    # gradients over many magnitudes, exact zeros, a block of zeros, subnormal ones
    rng = np.random.default_rng(1)
    for k, n in enumerate(sizes):
        if n:
            x = rng.standard_normal(n) * 10.0 ** rng.uniform(-9, 1, n)
            x[rng.random(n) < 0.1] = 0
            if n > 1000:
                x[256:512] = 0
                x[512:768] = 1e-30
            st.g[k].copy_(torch.from_numpy(x.astype(np.float32)))
    model = [((np.zeros(n, np.uint8), np.zeros(blocks(n), np.float32)),) * 2 for n in sizes]
    starts = np.cumsum([0] + [blocks(n) for n in sizes])
    with st.make() as lst:
        for t in (1, 2, 3, 10):
            osr.adamw_list_step(lst, t, LR, WD, float("inf"), seed=77)
            for k, n in enumerate(sizes):
                if not n:
                    continue
                grad = st.g[k].float().cpu().numpy()
                model[k] = model_step(model[k], grad, t, 77, int(starts[k]))
                for name, c, s, (want, scale) in zip("mv", (st.m[k], st.v[k]), (st.ms[k], st.vs[k]), model[k]):
                    got = c.view(torch.uint8).cpu().numpy()
                    assert np.array_equal(s.cpu().numpy(), scale), (t, k, name)
                    bad = np.nonzero(got != want)[0]
                    assert not bad.size, (t, k, name, bad.size, int(bad[0]), got[bad[0]], want[bad[0]])


def test_8_bit_states_of_16_bit_gradients_byte_for_byte():
    """beta1 m + (1 - beta1) g of operands with few bits is often a power of
    two or a stored value to the last bit (about one block in a thousand), and
    there a fused multiply-add would round to the other side."""
    n = 300_000
    st = State([n], 12, "bf16", [1])
    grad = st.g[0].float().cpu().numpy()
    model = ((np.zeros(n, np.uint8), np.zeros(blocks(n), np.float32)),) * 2
    with st.make() as lst:
        for t in (1, 2, 3):
            osr.adamw_list_step(lst, t, LR, WD, float("inf"), seed=5)
            model = model_step(model, grad, t, 5, 0)
            for c, s, (want, scale) in zip((st.m[0], st.v[0]), (st.ms[0], st.vs[0]), model):
                assert np.array_equal(s.cpu().numpy(), scale)
                assert np.array_equal(c.view(torch.uint8).cpu().numpy(), want)


@pytest.mark.parametrize("sizes", [[7, 2048, 5000, 300], [3_000_000, 1, 70_000]])
def test_norm_of_numbers_of_all_sizes(sizes):
    """Squares that float32 holds, beside some that it does not (above and
    below), in one warp, one block and one list.  A run of up to 32 squares is
    summed in float32, each rounded once and added in at most 7 roundings, so
    the sum is within 8 x 2^-24 and its root within 2.4e-7; the rest adds 2^-40."""
    for k in range(6):
        st = State(sizes, k, "f32", [0] * len(sizes))
        if k == 1:
            st.g[0][::3] = 1e21
        if k == 2:
            st.g[-1][-1] = -3e22
        if k == 3:
            for g in st.g:
                g.mul_(1e-25)
        if k == 4:
            for g in st.g[1:]:
                g.zero_()
        if k == 5:
            for g in st.g:
                g.fill_(2.0 ** 39)
        want = np.sqrt(sum(float((g.double() ** 2).sum()) for g in st.g))
        with st.make() as lst:
            osr.adamw_list_step(lst, 1, LR, WD, 1.0)
            norm, factor = osr.adamw_list_last_norm(lst)
            assert norm == pytest.approx(want, rel=1e-6)
            assert factor == pytest.approx(min(1.0, 1.0 / want), rel=1.1e-6)


def test_8_bit_moments_that_are_not_finite_spoil_only_themselves():
    """A NaN or infinite stored moment, away from its block's largest, leaves
    every other element's bytes and its block's scale as they were (weights:
    the root and the quotient may come from the other form, 1e-6 of the update)."""
    n = 1000
    a, b = State([n], 6, "f32", [1]), State([n], 6, "f32", [1])
    with a.make() as la, b.make() as lb:
        for st, lst in ((a, la), (b, lb)):
            st.g[0][[5, 300, 600]] = 1e-4
            osr.adamw_list_step(lst, 1, LR, WD, float("inf"), seed=2)
        b.m[0].view(torch.uint8)[5] = 0x7F  # nan
        b.v[0].view(torch.uint8)[300] = 0x7D  # nan
        b.v[0].view(torch.uint8)[600] = 0x7C  # inf
        for st, lst in ((a, la), (b, lb)):
            osr.adamw_list_step(lst, 2, LR, WD, float("inf"), seed=2)
    am, av, bm, bv = (t.view(torch.uint8).cpu().numpy() for t in (a.m[0], a.v[0], b.m[0], b.v[0]))
    assert torch.equal(a.ms[0], b.ms[0]) and torch.equal(a.vs[0], b.vs[0])
    assert np.isnan(b.m[0].float().cpu().numpy()[5])
    assert np.isnan(b.v[0].float().cpu().numpy()[300])
    assert np.isinf(b.v[0].float().cpu().numpy()[600])
    assert np.array_equal(np.nonzero(am != bm)[0], [5])
    assert np.array_equal(np.nonzero(av != bv)[0], [300, 600])
    aw, bw = a.w[0].cpu().numpy(), b.w[0].cpu().numpy()
    assert np.isnan(bw[[5, 300]]).all() and np.isfinite(np.delete(bw, [5, 300])).all()
    rest = np.delete(np.arange(n), [5, 300, 600])
    # both are within U |w| + 1e-6 of the update, at most 3.2 lr, of the formula
    assert np.all(np.abs(aw - bw)[rest] <= 2 * (2.0 ** -24 * np.abs(aw)[rest] + 3.2e-6 * LR))


def test_rounding_has_the_value_as_its_mean():
    """65,536 equal moments between two neighbours: the stored ones' mean is
    within 6 standard deviations (spacing / 2 / sqrt(n) at most) of it, and a
    v that a step moves by 0.1% of its spacing follows the formula on average."""
    n = 1 << 16
    st = State([n], 0, "f32", [1])
    st.g[0].fill_(1.1)
    with st.make() as lst:
        for t in range(1, 41):
            osr.adamw_list_step(lst, t, LR, WD, float("inf"), seed=3)
    m, v = st.host()[0][2:]
    # every step keeps the mean, so the mean's error is a sum of t steps' errors
    want_m, want_v = 1.1 * (1 - B1 ** 40), 1.1 ** 2 * (1 - B2 ** 40)
    assert abs(m.mean() - want_m) <= 6 * np.sqrt(40) * (want_m / 8) / 2 / np.sqrt(n) + 1e-6
    assert abs(v.mean() - want_v) <= 6 * np.sqrt(40) * (want_v / 4) / 2 / np.sqrt(n) + 1e-6
    assert len(np.unique(v)) > 1


def test_random_numbers_depend_on_seed_and_step():
    def run(seed, t):
        st = State([5000], 2, "f32", [1])
        with st.make() as lst:
            osr.adamw_list_step(lst, t, LR, WD, float("inf"), seed=seed)
        return st.m[0].view(torch.uint8).cpu().numpy()
    a = run(1, 1)
    assert np.array_equal(a, run(1, 1))
    assert (a != run(2, 1)).mean() > 0.2 and (a != run(1, 2)).mean() > 0.2


# ---- the rest of the contract ----------------------------------------------
def test_same_inputs_same_bytes_and_resume():
    """Two runs agree byte for byte, and so does one resumed from copies."""
    def fresh():
        return State(SIZES, 9, "f16", [k % 2 for k in range(len(SIZES))], copy="bf16")

    a, b = fresh(), fresh()
    with a.make() as lst:
        for t in range(1, 7):
            osr.adamw_list_step(lst, t, LR, WD, 0.5, seed=11)
    with b.make() as lst:
        for t in range(1, 4):
            osr.adamw_list_step(lst, t, LR, WD, 0.5, seed=11)
    c = fresh()
    for name in ("w", "m", "v", "ms", "vs", "lp"):
        for x, y in zip(getattr(c, name), getattr(b, name)):
            if x is not None and x.numel():
                x.view(torch.uint8).copy_(y.view(torch.uint8))
    with c.make() as lst:
        for t in range(4, 7):
            osr.adamw_list_step(lst, t, LR, WD, 0.5, seed=11)
    assert a.bytes() == c.bytes()


@pytest.mark.parametrize("eight", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_non_finite_gradient_changes_nothing(eight, bad):
    st = State([100, 3000], 1, "f32", [eight] * 2, copy="bf16")
    with st.make() as lst:
        osr.adamw_list_step(lst, 1, LR, WD, 1.0)
        st.g[1][2999] = bad
        before = st.bytes()
        osr.adamw_list_step(lst, 2, LR, WD, 1.0, zero_grad=True)
        with pytest.raises(osr.NonFiniteGradient):
            osr.adamw_list_last_norm(lst)
        assert st.bytes() == before
        st.g[1][2999] = 0.0
        osr.adamw_list_step(lst, 2, LR, WD, 1.0)
        assert osr.adamw_list_last_norm(lst)[0] > 0


def test_norm_of_extreme_gradients():
    """Squares beyond float32's range at either end."""
    for big in (1e25, 1e-30):
        st = State([5000, 17], 1)
        for g in st.g:
            g.copy_((g * (big / 1e-3)))
        want = np.sqrt(sum(float((g.double() ** 2).sum()) for g in st.g))
        with st.make() as lst:
            osr.adamw_list_step(lst, 1, LR, WD, 1.0)
            assert osr.adamw_list_last_norm(lst)[0] == pytest.approx(want, rel=1e-6)


def test_zero_grad_and_rebinding():
    st = State([1000, 5], 6, "bf16", [1, 0])
    with st.make() as lst:
        before = st.host()
        osr.adamw_list_step(lst, 1, LR, WD, 1.0, zero_grad=True)
        check(st, before, 1, 1.0)
        assert not any(bool(g.any()) for g in st.g)
        # gradients of another type in new memory
        new = [torch.randn(n, device="cuda") for n in st.sizes]
        osr.adamw_list_bind(lst, st.w, new, st.m, st.v, st.ms, st.vs)
        st.g = new
        before = st.host()
        osr.adamw_list_step(lst, 2, LR, WD, 1.0)
        check(st, before, 2, 1.0)


def test_hyperparameters():
    st = State([700], 5)
    with st.make() as lst:
        osr.adamw_list_set_hparams(lst, 0.0, 0.0, 0.0)
        w, g = st.w[0].double(), st.g[0].double()
        osr.adamw_list_step(lst, 1, LR, 0.0, float("inf"))
        # m = g, v = g^2: a step of lr against the sign
        want = w - LR * g.sign()
        assert float((st.w[0].double() - want).abs().max()) <= 1e-6 * LR + 2.0 ** -24 * 0.2


@pytest.mark.parametrize("eps", [1e-45, 1e-42, 1e-39, 1.1e-38, 2e-38])
@pytest.mark.parametrize("eight", [0, 1])
def test_eps_below_the_normal_numbers(eight, eps):
    """An element that never had a gradient has m = v = 0 and keeps its decayed
    weight, as 0 / eps is 0 for any eps above 0."""
    n = 600
    st = State([n], 5, eight=[eight])
    st.g[0][::2] = 0.0
    if not eight:
        st.m[0].zero_()
        st.v[0].zero_()
    w = st.w[0].clone()
    with st.make() as lst:
        osr.adamw_list_set_hparams(lst, B1, B2, eps)
        osr.adamw_list_step(lst, 1, LR, WD, float("inf"))
    assert torch.equal(st.w[0][::2], w[::2] * float(np.float32(1 - LR * WD)))
    step = (st.w[0][1::2].double() - w[1::2].double() * (1 - LR * WD)).abs()
    assert float((step - LR).abs().max()) <= 1e-6 * LR + 2.0 ** -24 * 0.2


@pytest.mark.parametrize("sizes", [[], [0], [0, 0, 0]])
def test_lists_without_elements(sizes):
    st = State(sizes, 1)
    with st.make() as lst:
        osr.adamw_list_step(lst, 1, LR, WD, 1.0)
        assert osr.adamw_list_last_norm(lst) == (0.0, 1.0)


def test_many_tensors():
    sizes = [1 + (k * 7919) % 613 for k in range(3000)]
    st = State(sizes, 2, "bf16", [k % 2 for k in range(3000)])
    with st.make() as lst:
        before = st.host()
        osr.adamw_list_step(lst, 1, LR, WD, 0.5)
        check(st, before, 1, 0.5)


def test_on_another_stream_and_in_a_graph():
    a, b = State(SIZES, 9, eight=[1] * len(SIZES)), State(SIZES, 9, eight=[1] * len(SIZES))
    with a.make() as la, b.make() as lb:
        for t in (1, 2):
            osr.adamw_list_step(la, t, LR, WD, 0.5)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        osr.adamw_list_step(lb, 1, LR, WD, 0.5, stream=s)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            osr.adamw_list_step(lb, 2, LR, WD, 0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert a.bytes() == b.bytes()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("eight", [(0, 0, 0, 0), (1, 1, 1, 1), (0, 1, 0, 1)])
def test_steps_in_a_row_wait_for_one_another(eight, g, shift):
    """Every step reads what the one before and the kernel between them wrote,
    in every block's first unit and in the later ones: the bytes of a run with
    the device idle between any two calls."""
    sizes = [5_000_000, 70_001, 3, 5_000_003]

    def steps(rest):
        st = State(sizes, 13, g, eight, shift, copy="bf16")
        with st.make() as lst:
            for t in range(1, 7):
                rest()
                osr.adamw_list_step(lst, t, LR, WD, 0.5, seed=t)
                rest()
                if t % 2:
                    for x in st.g:
                        x.mul_(-0.75)
        return st.bytes()

    want = steps(torch.cuda.synchronize)
    for _ in range(2):
        assert steps(lambda: None) == want


def test_nothing_outside_the_tensors_is_written():
    """Sentinels before and after every array of odd-sized tensors."""
    n, pad = 1283, 64
    for eight in (0, 1):
        pools = {}

        def guarded(dtype, count):
            size = torch.empty(0, dtype=dtype).element_size()
            t = torch.full((count + 2 * pad,), 1, dtype=torch.uint8 if size == 1 else dtype,
                           device="cuda")
            pools[len(pools)] = (t, count)
            inner = t[pad:pad + count]
            inner.zero_()
            return inner.view(dtype) if size == 1 else inner

        f8 = (torch.float8_e4m3fn, torch.float8_e5m2) if eight else (torch.float32,) * 2
        w, g = guarded(torch.float32, n), guarded(torch.bfloat16, n)
        m, v = (guarded(d, n) for d in f8)
        ms, vs = (guarded(torch.float32, blocks(n)) for _ in range(2))
        lp = guarded(torch.float16, n)
        g.fill_(0.25)
        with osr.adamw_list_create([w], [g], [m], [v], [ms], [vs], [lp]) as lst:
            osr.adamw_list_step(lst, 1, LR, WD, 1.0, zero_grad=True)
        for t, count in pools.values():
            assert bool((t[:pad] == 1).all()) and bool((t[pad + count:] == 1).all())
        assert bool((w != 0).all()) and not bool(g.any())


# ---- refusals ----------------------------------------------------------------
def test_refusals():
    st = State([300, 20], 1, eight=[1, 0])
    args = [st.w, st.g, st.m, st.v, st.ms, st.vs]

    def refused(exc, **change):
        a = list(args)
        for i, x in change.items():
            a[int(i[1:])] = x
        with pytest.raises(exc):
            osr.adamw_list_create(*a)

    half = [x.bfloat16() for x in st.w]
    refused(TypeError, _0=half)
    refused(TypeError, _1=[st.g[0], half[1]])
    refused(TypeError, _1=[x.double() for x in st.g])
    refused(TypeError, _0=[x.cpu() for x in st.w])
    refused(TypeError, _0=[torch.zeros(600, device="cuda")[::2], st.w[1]])
    refused(TypeError, _3=[st.v[0].view(torch.uint8), st.v[1]])
    refused(ValueError, _1=[st.g[0][:-1], st.g[1]])
    refused(ValueError, _2=[st.m[0]])
    refused(TypeError, _4=None)
    refused(ValueError, _4=[st.ms[0][:1], None])
    refused(osr.AdamWError, _1=[st.w[0], st.g[1]])  # g on w: the arrays overlap
    refused(osr.AdamWError, _5=[st.ms[0], None])  # both scales in one place
    both = torch.zeros(320, device="cuda")
    refused(osr.AdamWError, _0=[both[:300], both[299:319]])
    with pytest.raises(TypeError):
        osr.adamw_list_create(*args, w_lp=st.w)
    with pytest.raises(osr.AdamWError):
        osr.adamw_list_create(*args, decay=[1])
    with osr.adamw_list_create(*args) as lst:
        with pytest.raises(osr.AdamWError) as e:
            osr.adamw_list_last_norm(lst)
        assert e.value.status == osr.ESTATE
        for bad in (dict(t=0), dict(lr=-1.0), dict(wd=float("nan")), dict(clip=0.0),
                    dict(grad_scale=0.0), dict(lr=float("inf"))):
            kw = dict(t=1, lr=LR, wd=WD, clip=1.0)
            kw.update(bad)
            with pytest.raises(osr.AdamWError) as e:
                osr.adamw_list_step(lst, **kw)
            assert e.value.status == osr.EINVAL
        with pytest.raises(osr.AdamWError):
            osr.adamw_list_set_hparams(lst, 1.0, 0.9, 1e-8)


def test_a_step_needs_bound_arrays():
    import ctypes
    h = ctypes.c_void_p()
    n = (ctypes.c_int64 * 1)(10)
    assert osr.library().adamw_list_create(1, n, None, ctypes.byref(h)) == osr.OK
    st = osr.library().adamw_list_step(h, 1, LR, WD, 1.0, 1.0, 0, 0, None)
    assert st == osr.ESTATE
    # misaligned and missing arrays
    w = torch.zeros(64, device="cuda")
    row = (ctypes.c_void_p * 1)
    ok = [row(w[16 * k:].data_ptr()) for k in range(4)]
    odd = row(w.data_ptr() + 2)
    for args in ([odd, ok[1], ok[2], ok[3]], [ok[0], odd, ok[2], ok[3]], [ok[0], ok[1], row(None), ok[3]]):
        st = osr.library().adamw_list_bind(h, args[0], args[1], osr.DTYPE_F32, args[2], args[3],
                                           None, None, None, osr.DTYPE_BF16)
        assert st == osr.EINVAL
    assert osr.library().adamw_list_bind(h, ok[0], ok[1], 9, ok[2], ok[3], None, None, None,
                                         osr.DTYPE_BF16) == osr.EINVAL
    assert osr.library().adamw_list_destroy(h) == osr.OK
