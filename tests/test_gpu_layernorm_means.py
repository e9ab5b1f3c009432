"""The layer norm of rows whose mean is far larger than their spread, against
the formulas in 64 bits, with bars that do not grow with the width.

u = 2^-24, N = 128 additions in a row at most (rows of up to 50,001 elements).
The first mean errs by at most c = (N + 2) u mean|x|.  The differences from it
are exact where x is within a factor 2 of it; their sum, e, then corrects it:

* mean: u |mean| from its last rounding, (N + 3) u mean|d| from e;
* variance: (2 N + 8) u (var + c^2), half of which, relative, is rstd's, plus 4 u;
* y: (N + 6) u mean|d| rstd |w| from the mean, 4 u more of c rstd |w| from its
  correction, and rstd's error; with |d| <= |x - mean| + c.
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

U, N = 2.0 ** -24, 128
EPS = 1e-5
WIDTHS = [40, 96, 768, 1021, 3000, 4096, 16_384, 50_001]
TYPES = {"f32": (torch.float32, U), "bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11)}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def check(x, w, b, y, mean, rstd):
    X = x.double()
    mu = X.mean(1, keepdim=True)
    var = ((X - mu) ** 2).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + EPS)
    c = (N + 2) * U * X.abs().mean(1, keepdim=True)
    d = (X - mu).abs().mean(1, keepdim=True) + c
    off = (N + 6) * U * d
    assert bool(((mean.double()[:, None] - mu).abs() <= U * mu.abs() + off).all())
    share = 0.5 * (2 * N + 8) * U * (var + c * c) / (var + EPS) + 4 * U
    share = share / (1 - 2 * share).clamp(min=0.25)  # from the first order to a bound
    assert float(share.max()) < 0.3
    assert bool(((rstd.double()[:, None] - r).abs() <= share * r).all())
    W, B = (1.0, 0.0) if w is None else (w.double(), b.double())
    xh = (X - mu) * r
    want = xh * W + B
    scale = abs(W) if w is None else W.abs()
    bar = (off + 4 * U * c) * r * (1 + share) * scale + (share + 4 * U) * (xh * W).abs() + 2 * U * want.abs()
    u = TYPES[{torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[x.dtype]][1]
    bar = bar + u * (want.abs() + bar) + 2.0 ** -25
    bad = ~((y.double() - want).abs() <= bar)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist(), float(y.double().abs().max()))


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,value", [("f32", 3.0), ("f32", 1000.1), ("f32", -12345.67),
                                        ("f32", 1e-3), ("bf16", 1000.0), ("f16", -1001.0)])
@pytest.mark.parametrize("shift", [0, 1])
def test_constant_rows(cols, kind, value, shift):
    """y is the bias, and the mean is the value itself."""
    dtype, u = TYPES[kind]
    pool = torch.full((5 * (cols + shift) + shift,), value, device="cuda", dtype=dtype)
    x = pool[shift:].view(5, cols + shift)[:, :cols]
    b = torch.full((cols,), 0.25, device="cuda")
    w = torch.full((cols,), 2.0, device="cuda")
    with osr.layernorm_create(cols) as ln:
        y, mean, rstd = osr.layernorm_forward(ln, x, w, b, eps=EPS)
    check(x, w, b, y, mean, rstd)
    assert bool((mean == x[:, 0].float()).all())


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("value", [100_000.1, -3e6])
def test_constant_rows_of_large_values(cols, value):
    """Where the bars of the variance say nothing any more: the differences'
    mean takes them to (N + 6) u c, with rstd at most 1 / sqrt(eps)."""
    x = torch.full((3, cols), value, device="cuda")
    with osr.layernorm_create(cols) as ln:
        y, mean, rstd = osr.layernorm_forward(ln, x, eps=EPS)
    c = (N + 2) * U * abs(value)
    assert float(y.abs().max()) <= (N + 10) * U * c * EPS ** -0.5
    assert bool((mean == x[:, 0]).all()) and bool((rstd > 0).all())


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("mean,spread", [(1000.1, 1e-3), (-12345.67, 0.1), (1e6, 1.0), (0.0, 1.0)])
@pytest.mark.parametrize("pad,at", [(0, 0), (3, 1)])
def test_rows_far_from_zero(cols, mean, spread, pad, at):
    r = torch.Generator(device="cuda").manual_seed(cols)
    pool = torch.empty(7 * (cols + pad) + at, device="cuda").normal_(0, spread, generator=r) + mean
    x = pool[at:].view(7, cols + pad)[:, :cols]
    w = torch.empty(cols, device="cuda").normal_(1.0, 0.3, generator=r)
    b = torch.empty(cols, device="cuda").normal_(0.0, 0.3, generator=r)
    with osr.layernorm_create(cols) as ln:
        check(x, w, b, *osr.layernorm_forward(ln, x, w, b, eps=EPS))


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,at", [(0, 0), (3, 1)])
def test_means_of_exact_sums(cols, kind, pad, at):
    """Multiples of 2^-6 below 4, whose sums float32 holds in any order: the
    mean is the sum times 1 / cols in two roundings, however close to 0."""
    dtype, _ = TYPES[kind]
    r = torch.Generator(device="cuda").manual_seed(cols)
    rows = 33
    whole = torch.randint(-255, 256, (rows, cols + pad), generator=r, device="cuda")
    for k in range(rows):  # the sum: -16 to 16
        left = int(whole[k, :cols].sum()) - (k - 16)
        # taken from as many elements as it needs, without leaving the range
        change = torch.where(whole[k, :cols] * left > 0, whole[k, :cols], 0)
        take = change.abs().cumsum(0)
        part = (abs(left) - (take - change.abs())).clamp(min=0).minimum(change.abs())
        whole[k, :cols] -= change.sign() * part
        assert int(whole[k, :cols].sum()) == k - 16
    pool = torch.zeros(rows * (cols + pad) + at, device="cuda", dtype=dtype)
    pool[at:] = (whole.float() / 64).flatten().to(dtype)
    x = pool[at:].view(rows, cols + pad)[:, :cols]
    with osr.layernorm_create(cols) as ln:
        y, mean, rstd = osr.layernorm_forward(ln, x, eps=EPS)
    mu = x.double().mean(1)
    assert bool(((mean.double() - mu).abs() <= 2.01 * U * mu.abs()).all()), float(
        ((mean.double() - mu).abs() / mu.abs().clamp(min=1e-30)).max())
    check(x, None, None, y, mean, rstd)


def test_means_that_are_not_numbers():
    """The mean of a row with an infinity is that infinity; of a row whose sum
    leaves float32's range, an infinity; of a row with a NaN, NaN."""
    for cols in (64, 768, 1021, 3000, 20_000):
        x = torch.randn(6, cols, device="cuda")
        x[1, 3], x[2, 5], x[3, 7] = float("inf"), -float("inf"), float("nan")
        x[4] = 3e38
        with osr.layernorm_create(cols) as ln:
            y, mean, rstd = osr.layernorm_forward(ln, x)
        assert mean[1] == float("inf") and mean[2] == -float("inf") and mean[4] == float("inf")
        assert bool(mean[3].isnan()) and bool(y[1:5].isnan().all())
        assert bool(y[[0, 5]].isfinite().all())
