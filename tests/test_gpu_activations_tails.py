"""The activations and their slopes far from 0, where the result is small: off by
their type's rounding and a few units of float32, relative to themselves.

U = 2^-8 or 2^-11.  Off the rounding: the arguments of the powers of two have a
rounding each, which counts |argument| fold (z^2 / 2 log2 e, at most 130 in
binary32's range: 2^-16), and the formulas' own errors are below 2^-20.  A sum of
two terms (a slope) errs by that much of both terms.  Results below the type's
smallest normal number may be 0, and so may those that are a factor times a power of
two below 2^-126: the factor is |z| <= 13 in a value, and at most 13 x 1.6 (1 +
0.135 x 13^2), below 500, in a slope.
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALL = {"bf16": 2.0 ** -126, "f16": 2.0 ** -14}  # normal from there on
FEW = 2.0 ** -16
N = 1024


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def phi(z):
    return torch.exp(-0.5 * z * z) * 0.3989422804014327


def tail(z):
    """The normal distribution at z, in 64 bits also far below 0."""
    far = 0.5 * torch.special.erfcx(z.abs() * 0.5 ** 0.5) * torch.exp(-0.5 * z * z)
    return torch.where(z < 0, far, 1 - far)


def parts(act, z):
    """(value, slope, the sizes of the slope's terms)."""
    if act == "gelu":
        a, b = tail(z), z * phi(z)
        return z * a, a + b, a + b.abs()
    if act == "gelu_tanh":
        k = (2 / torch.pi) ** 0.5
        g = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
        inner = 2 * k * (1 + 3 * 0.044715 * z * z)
        return z * g, g + z * g * (1 - g) * inner, g + (z * g * (1 - g) * inner).abs()
    g = torch.sigmoid(z)
    return z * g, g * (1 + z * (1 - g)), g * (1 + z.abs() * (1 - g))


def check(got, want, size, kind, factor):
    off = (got.double() - want).abs()
    small = max(SMALL[kind], factor * 2.0 ** -126)
    bad = ~(off <= U[kind] * want.abs() * (1 + FEW) + FEW * size)
    bad &= (want.abs() >= small) | (got.double().abs() > 2 * small)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


# few rows, divided sums and whole tiles finish their sums in kernels of their own
@pytest.mark.parametrize("rows,cin", [(1, 64), (5, 64), (40, 64), (40, 4096), (300, 64)])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_values(act, kind, rows, cin):
    # the pre-activation is the bias alone, in float32
    z = torch.linspace(-13.0, 13.0, N, device="cuda")
    x = torch.zeros(rows, cin, device="cuda", dtype=TYPES[kind])
    w = torch.zeros(N, cin, device="cuda", dtype=TYPES[kind])
    with osr.linear_create(cin, N) as lin:
        y = osr.linear_forward(lin, x, w, bias=z, activation=act)
    value, _, _ = parts(act, z.double())
    check(y, value.expand(rows, N), value.abs(), kind, 13)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 3])
def test_slopes(act, kind, pad):
    # dz through the unit matrix, and its column sums
    rows = 33
    z = torch.linspace(-13.0, 13.0, N, device="cuda").to(TYPES[kind]).expand(rows, N)
    z = torch.cat([z, z[:, :pad]], 1)[:, :N]  # rows on vectors, and anywhere
    dy = torch.ones(rows, N, device="cuda", dtype=TYPES[kind])
    w = torch.eye(N, device="cuda", dtype=TYPES[kind])
    x = torch.zeros(rows, N, device="cuda", dtype=TYPES[kind])
    db = torch.empty(N, device="cuda")
    dw = torch.empty(N, N, device="cuda")
    with osr.linear_create(N, N) as lin:
        dx, _, _ = osr.linear_backward(lin, dy, x, w, z=z, activation=act, dweight=dw, dbias=db)
    _, slope, size = parts(act, z.double())
    check(dx, slope, size, kind, 500)
    off = (db.double() - slope.sum(0)).abs()
    assert bool((off <= FEW * size.sum(0) + rows * 500 * 2.0 ** -126).all())


INF, NAN = float("inf"), float("nan")


# z through the bias: infinities and NaN beside ordinary values, in each of the kernels
# that finish sums
@pytest.mark.parametrize("rows,cin", [(1, 64), (5, 64), (40, 64), (40, 4096), (300, 64)])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("residual", [False, True])
def test_values_at_infinity_and_nan(act, rows, cin, residual):
    z = torch.zeros(264, device="cuda")
    z[::4], z[1::4], z[2::4] = INF, -INF, NAN
    x = torch.zeros(rows, cin, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(264, cin, device="cuda", dtype=torch.bfloat16)
    res = torch.full((rows, 264), 3.0, device="cuda", dtype=torch.bfloat16) if residual else None
    with osr.linear_create(cin, 264) as lin:
        y = osr.linear_forward(lin, x, w, bias=z, residual=res, activation=act).float()
    more = 3.0 if residual else 0.0
    assert bool((y[:, ::4] == INF).all()) and bool((y[:, 1::4] == more).all())
    assert bool(y[:, 2::4].isnan().all()) and bool((y[:, 3::4] == more).all())


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("cols", [264, 261])
def test_slopes_at_infinity_and_nan(act, cols):
    rows = 33
    z = torch.zeros(rows, cols, device="cuda", dtype=torch.float16)
    z[:, ::4], z[:, 1::4], z[5, 2::4] = INF, -INF, NAN
    dy = torch.full((rows, cols), 2.0, device="cuda", dtype=torch.float16)
    w = torch.eye(cols, device="cuda", dtype=torch.float16)
    db = torch.empty(cols, device="cuda")
    with osr.linear_create(cols, cols) as lin:
        dx, _, _ = osr.linear_backward(lin, dy, dy, w, z=z, activation=act, dbias=db)
    at_zero = 0.0 if act == "relu" else 1.0  # 2 act'(0)
    want = torch.full((cols,), at_zero, device="cuda")
    want[::4], want[1::4] = 2.0, 0.0
    assert bool(((dx.float() - want).abs() <= 2.0 ** -10)[torch.arange(rows) != 5].all())
    assert bool(dx[5].isnan().all())  # a factor of all sums of its row
    want = (rows * want)
    want[2::4] = NAN
    assert bool(db[2::4].isnan().all())
    assert bool(((db - want).abs() <= rows * 2.0 ** -10)[~want.isnan()].all())
