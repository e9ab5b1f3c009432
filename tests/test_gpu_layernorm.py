"""The layer norm's forward and backward pass against the formulas in 64 bits.

u = 2^-24.  Error bars, from the order of the operations:

* mean: a sum of float32 in at most 64 additions in a row (32 in a thread, 5
  in the warp, 16 over warps, the rest slack) errs by at most 64 u mean|x|; the
  product with 1/cols, itself rounded, adds 2 u.  Rows wider than 16384 go in
  512 chains of cols / 512 additions.
* rstd: the variance's sum errs by the same count of u relative; the mean's
  error d enters as d^2 / var.  Half of it, plus 4 u.
* y = (x - mean) rstd w + b: the mean's error times |rstd w|, (rstd's bar + 4
  u) |xhat w|, u |b|, then the rounding to the type.
* dx: with a = dy w, N additions in each of the two sums:
  rstd (8 u |a| + (N + 8) u (mean|a| + |xhat| mean|a xhat|)).
* dweight, dbias: every term rounded a few times, at most `rows` + 80 additions
  in a row: (rows + 90) u sum|terms|, then the rounding to the type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# unit roundoff, and half the smallest spacing
ROUND = {torch.float32: (U, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.manual_seed(0)


def inputs(rows, cols, kind, wkind, seed, pad=(0, 0, 0), at=(0, 0, 0), mean=1.0):
    """x, dy and a place for the output, rows `pad` apart, starting `at`."""
    r = torch.Generator(device="cuda").manual_seed(seed)

    def matrix(p, a):
        t = torch.empty(rows * (cols + p) + a + 16, device="cuda").normal_(0, 1.5, generator=r)
        t = t.to(TYPES[kind])[a:a + rows * (cols + p)].view(rows, cols + p)[:, :cols]
        t += (torch.randn(rows, 1, device="cuda", generator=r) * mean).to(t.dtype)
        return t

    x, dy, out = (matrix(p, a) for p, a in zip(pad, at))
    w = torch.empty(cols, device="cuda").normal_(1.0, 0.3, generator=r).to(TYPES[wkind])
    b = torch.empty(cols, device="cuda").normal_(0.0, 0.3, generator=r).to(TYPES[wkind])
    return x, dy, out, w, b


def chain(cols):
    return 64 + (0 if cols <= 16384 else cols // 512 + 16)


def check_forward(x, w, b, eps, y, mean, rstd):
    n = chain(x.shape[1])
    X = x.double()
    mu = X.mean(1, keepdim=True)
    var = ((X - mu) ** 2).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    mean_bar = (n + 2) * U * X.abs().mean(1, keepdim=True)
    rstd_bar = (n + 4) * U + mean_bar ** 2 / (var + eps)  # relative
    assert bool(((mean.double()[:, None] - mu).abs() <= mean_bar + 2.0 ** -149).all())
    assert bool(((rstd.double()[:, None] - r).abs() <= rstd_bar * r).all())
    W = torch.ones_like(X[0]) if w is None else w.double()
    B = torch.zeros_like(X[0]) if b is None else b.double()
    xh = (X - mu) * r
    want = xh * W + B
    u, tiny = ROUND[x.dtype]
    bar = (mean_bar * r * W.abs() + (rstd_bar + 4 * U) * (xh * W).abs() + U * B.abs()) * 1.01
    bar = bar + u * (want.abs() + bar) + tiny
    bad = ~((y.double() - want).abs() <= bar)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist())


def check_backward(dy, x, w, mean, rstd, dx, dw, db, before=None):
    rows, cols = x.shape
    n = chain(cols)
    X, G = x.double(), dy.double()
    r = rstd.double()[:, None]
    xh = (X - mean.double()[:, None]) * r
    a = G * (1.0 if w is None else w.double())
    m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    want = r * (a - m1 - xh * m2)
    bar = r * (8 * U * a.abs() + (n + 8) * U * (a.abs().mean(1, keepdim=True)
                                                + xh.abs() * (a * xh).abs().mean(1, keepdim=True)))
    u, tiny = ROUND[x.dtype]
    bad = ~((dx.double() - want).abs() <= bar + u * (want.abs() + bar) + tiny)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:3].tolist())
    for k, (got, terms) in enumerate(((dw, G * xh), (db, G))):
        if got is None:
            continue
        total = terms.sum(0)
        bar = (rows + 90) * U * terms.abs().sum(0)
        if before is not None:
            total = total + before[k].double()
            bar = bar + U * total.abs()
        u, tiny = ROUND[got.dtype]
        bad = ~((got.double() - total).abs() <= bar + u * (total.abs() + bar) + tiny)
        assert not bool(bad.any()), (k, int(bad.sum()), bad.nonzero()[:3].tolist())


def run(rows, cols, kind, wkind="f32", seed=0, eps=1e-5, affine="wb", grad=None,
        pad=(0, 0, 0), at=(0, 0, 0), mean=1.0, accumulate=False):
    x, dy, out, w, b = inputs(rows, cols, kind, wkind, seed, pad, at, mean)
    w, b = (w if "w" in affine else None), (b if "b" in affine else None)
    with osr.layernorm_create(cols) as ln:
        y, mu, rstd = osr.layernorm_forward(ln, x, w, b, eps=eps, y=out)
        check_forward(x, w, b, eps, y, mu, rstd)
        gt = TYPES[grad or wkind]
        dw, db = (torch.full((cols,), 0.5, device="cuda", dtype=gt) for _ in range(2))
        before = (dw.clone(), db.clone()) if accumulate else None
        dx = torch.full_like(out, 7.0) if out.is_contiguous() else out
        osr.layernorm_backward(ln, dy, x, w, mu, rstd, dx=dx, dweight=dw, dbias=db,
                               accumulate=accumulate)
        check_backward(dy, x, w, mu, rstd, dx, dw, db, before)


# every layout of rows over threads, both sides of each border, widths that
# divide by nothing
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 31, 57, 58, 64, 65, 121, 128, 250, 256, 257, 505,
                                  512, 600, 761, 762, 768, 1000, 1017, 1018, 1021, 1024, 1025,
                                  2041, 2048, 2049, 4089, 4090, 4096, 5001, 8185, 8186, 8192])
def test_widths(kind, cols):
    run(37, cols, kind, "f32" if cols % 2 else kind, seed=cols)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cols", [10_000, 16_377, 16_378, 16_384, 16_385, 20_480, 50_001])
def test_wide_rows(kind, cols):
    run(9, cols, kind, "f32", seed=cols)


# both sides of the forward pass's own borders between layouts
@pytest.mark.parametrize("kind,cols", [("f32", 2816), ("f32", 2820), ("f32", 2823), ("f32", 4092),
                                       ("f32", 4100), ("f32", 6144), ("f32", 6148), ("f32", 8188),
                                       ("bf16", 1026), ("bf16", 1499), ("f16", 1999), ("bf16", 2047),
                                       ("bf16", 2050)])
def test_forward_layouts(kind, cols):
    run(45, cols, kind, "f32", seed=cols)
    run(45, cols, kind, "f32", seed=cols, pad=(13, 13, 0))


@pytest.mark.parametrize("cols", [2980, 3000, 3004, 3006, 7424, 7500, 7504, 7506])
def test_forward_layouts_of_float32_rows(cols):
    run(45, cols, "f32", "f32", seed=cols)
    run(45, cols, "f32", "f32", seed=cols, pad=(4, 0, 8))


# rows that are looked at several times
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [24_576, 24_577, 65_528, 65_536, 65_537, 81_920, 131_071, 131_072,
                                  131_073])
def test_rows_wider_than_a_block(kind, cols):
    run(5, cols, kind, kind, seed=cols, accumulate=True)


@pytest.mark.parametrize("pad,at", [((8, 8, 8), (0, 0, 0)), ((3, 3, 3), (1, 1, 1)),
                                    ((1, 5, 2), (0, 3, 6)), ((13, 13, 0), (0, 0, 0))])
@pytest.mark.parametrize("cols", [16_400, 17_011])
def test_rows_wider_than_a_block_at_strides_and_places(cols, pad, at):
    run(301, cols, "bf16", "f32", seed=cols, pad=pad, at=at)
    run(19, cols, "f32", "f32", seed=cols, pad=pad, at=at)


def test_widest_rows():
    run(2, 1 << 18, "bf16")


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 9, 63, 64, 65, 1000, 4865, 20_001])
@pytest.mark.parametrize("cols", [40, 129, 768, 1025])
def test_row_counts(rows, cols):
    run(rows, cols, "bf16", "f32", seed=rows)


def test_many_rows():
    run(300_001, 96, "bf16", "bf16", seed=2)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [24, 200, 768, 1021, 2000, 6000])
@pytest.mark.parametrize("pad,at", [((8, 8, 8), (0, 0, 0)), ((3, 3, 3), (1, 1, 1)),
                                    ((1, 5, 2), (0, 3, 6)), ((0, 0, 0), (5, 0, 0)),
                                    ((0, 16, 8), (4, 4, 4))])
def test_strides_and_places(kind, cols, pad, at):
    run(21, cols, kind, "f32", seed=cols, pad=pad, at=at)


@pytest.mark.parametrize("affine", ["", "w", "b", "wb"])
@pytest.mark.parametrize("wkind", ["f32", "f16"])
@pytest.mark.parametrize("grad", ["f32", "bf16", "f16"])
def test_weights_and_gradient_types(affine, wkind, grad):
    run(50, 320, "f16", wkind, affine=affine, grad=grad)
    run(50, 321, "f16", wkind, affine=affine, grad=grad, accumulate=True)


@pytest.mark.parametrize("mean", [0.0, 1e3, 1e6])
def test_rows_far_from_zero(mean):
    """The variance is of the differences, so a mean 10^6 spreads away costs
    the differences' bits only, not the variance's sign."""
    run(16, 768, "f32", mean=mean)


def test_constant_rows_and_eps():
    for eps in (1e-5, 0.0, 1.0):
        x = torch.full((4, 256), 3.0, device="cuda")
        if eps == 0.0:
            x[:, ::2] = -3.0
        with osr.layernorm_create(256) as ln:
            y, mu, rstd = osr.layernorm_forward(ln, x, eps=eps)
            check_forward(x, None, None, eps, y, mu, rstd)
            if eps:
                assert not bool(y.any())


@pytest.mark.parametrize("kind,cols", [("f32", 40), ("bf16", 41), ("bf16", 600), ("f32", 1021),
                                       ("f32", 3000)])
def test_backward_of_large_means_and_factors(kind, cols):
    """mean x rstd past float32 must not reach the lanes that the row does not fill."""
    x = torch.full((5, cols), 2.0 ** 80, device="cuda", dtype=TYPES[kind])
    dy = torch.randn(5, cols, device="cuda").to(TYPES[kind])
    mean, rstd = torch.full((5,), 2.0 ** 80, device="cuda"), torch.full((5,), 2.0 ** 50, device="cuda")
    dw, db = (torch.empty(cols, device="cuda") for _ in range(2))
    with osr.layernorm_create(cols) as ln:
        dx, _, _ = osr.layernorm_backward(ln, dy, x, None, mean, rstd, dweight=dw, dbias=db)
    check_backward(dy, x, None, mean, rstd, dx, dw, db)


def test_non_finite_rows_stay_rows():
    """A row with inf or nan gives a row of nan and leaves the others alone;
    its columns' gradient sums are nan where the formula's are."""
    for cols in (64, 768, 1021, 3000):
        x = torch.randn(12, cols, device="cuda").bfloat16()
        x[3, 5], x[7, 0] = float("inf"), float("nan")
        keep = [r for r in range(12) if r not in (3, 7)]
        with osr.layernorm_create(cols) as ln:
            y, mu, rstd = osr.layernorm_forward(ln, x)
            assert bool(y[[3, 7]].isnan().all())
            check_forward(x[keep], None, None, 1e-5, y[keep], mu[keep], rstd[keep])
            dy = torch.randn(12, cols, device="cuda").bfloat16()
            db = torch.zeros(cols, device="cuda")
            dx, _, _ = osr.layernorm_backward(ln, dy, x, None, mu, rstd, dbias=db)
            assert bool(dx[[3, 7]].isnan().all()) and bool(db.isfinite().all())
            check_backward(dy[keep], x[keep], None, mu[keep], rstd[keep], dx[keep], None, None)


@pytest.mark.parametrize("cols", [5, 96, 1000])
def test_gradients_are_the_differences(cols):
    """The directional derivative of sum(dy y) in x, weight and bias, by
    central differences in 64 bits."""
    x, dy, _, w, b = inputs(6, cols, "f32", "f32", cols)
    with osr.layernorm_create(cols) as ln:
        _, mu, rstd = osr.layernorm_forward(ln, x, w, b)
        dw, db = (torch.empty(cols, device="cuda") for _ in range(2))
        dx, _, _ = osr.layernorm_backward(ln, dy, x, w, mu, rstd, dweight=dw, dbias=db)

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return float((dy.double() * (d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * w + b)).sum())

    at = [t.double() for t in (x, w, b)]
    for k, grad in enumerate((dx, dw, db)):
        step = torch.randn_like(at[k])
        h = 1e-5
        up, down = (list(at) for _ in range(2))
        up[k], down[k] = at[k] + h * step, at[k] - h * step
        slope = (loss(*up) - loss(*down)) / (2 * h)
        got = float((grad.double() * step).sum())
        # float32 gradients; the differences' own error: h^2 and 2^-53 |loss| / h
        scale = float((grad.double() * step).abs().sum()) + abs(slope)
        assert abs(got - slope) <= 1e-5 * scale + 1e-6


def test_same_bits_every_time():
    x, dy, _, w, _ = inputs(5000, 768, "bf16", "f32", 1)
    with osr.layernorm_create(768) as ln:
        first = None
        for _ in range(3):
            _, mu, rstd = osr.layernorm_forward(ln, x, w)
            dw, db = (torch.empty(768, device="cuda") for _ in range(2))
            dx, _, _ = osr.layernorm_backward(ln, dy, x, w, mu, rstd, dweight=dw, dbias=db)
            now = [t.clone() for t in (mu, rstd, dx, dw, db)]
            first = first or now
            assert all(torch.equal(a, b) for a, b in zip(first, now))


def chained(wait, steps=6, rows=300, cols=768):
    """Forward, backward and list step in a chain where each reads what the one
    before wrote; `wait`: with the device idle between any two."""
    torch.manual_seed(3)
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    dw, db = torch.zeros(cols, device="cuda"), torch.zeros(cols, device="cuda")
    state = [[torch.zeros(cols, device="cuda") for _ in range(2)] for _ in range(2)]
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    rest = torch.cuda.synchronize if wait else lambda: None
    with osr.layernorm_create(cols) as ln, osr.adamw_list_create([w, b], [dw, db], *state) as lst:
        rest()
        for t in range(1, steps + 1):
            osr.layernorm_forward(ln, x, w, b, y=y, mean=mean, rstd=rstd)
            rest()
            osr.layernorm_forward(ln, y, w, b, y=x, mean=mean, rstd=rstd)
            rest()
            osr.layernorm_backward(ln, x, y, w, mean, rstd, dx=dx, dweight=dw, dbias=db,
                                   accumulate=True)
            rest()
            osr.layernorm_backward(ln, dx, y, w, mean, rstd, dx=x, dweight=dw, dbias=db,
                                   accumulate=True)
            rest()
            osr.adamw_list_step(lst, t, 1e-2, 0.1, 1.0, zero_grad=t % 2 == 0)
            rest()
    return [x, y, dx, w, b, dw, db, mean, rstd] + state[0] + state[1]


def test_kernels_in_a_row_wait_for_one_another():
    """A kernel is set up while the one before it still runs."""
    want = chained(True)
    for _ in range(5):
        for got, ref in zip(chained(False), want):
            assert torch.equal(got, ref)


def test_captured_calls():
    want = chained(True, steps=1)
    x, w, b = (t.clone() for t in (want[0], want[3], want[4]))
    y, mean, rstd = torch.empty_like(x), *(torch.empty(300, device="cuda") for _ in range(2))
    dx, dw, db = torch.empty_like(x), torch.zeros_like(w), torch.zeros_like(b)

    def passes(ln):
        osr.layernorm_forward(ln, x, w, b, y=y, mean=mean, rstd=rstd)
        osr.layernorm_backward(ln, y, x, w, mean, rstd, dx=dx, dweight=dw, dbias=db)

    with osr.layernorm_create(768) as ln:
        passes(ln)
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, mean, rstd, dx, dw, db)]
        for t in (y, mean, rstd, dx, dw, db):
            t.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            passes(ln)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((y, mean, rstd, dx, dw, db), want):
            assert torch.equal(got, ref)


def test_no_rows():
    for cols in (768, 20_000):
        x = torch.empty(0, cols, device="cuda")
        st = torch.empty(0, device="cuda")
        w = torch.ones(cols, device="cuda")
        with osr.layernorm_create(cols) as ln:
            y, mu, rstd = osr.layernorm_forward(ln, x, w)
            assert y.shape == (0, cols) and mu.numel() == 0
            dw = torch.ones(cols, device="cuda")
            osr.layernorm_backward(ln, x, x, w, st, st, dweight=dw, accumulate=True)
            assert bool((dw == 1).all())
            osr.layernorm_backward(ln, x, x, w, st, st, dweight=dw)
            assert not bool(dw.any())


def test_shapes_streams_and_optional_outputs():
    x = torch.randn(3, 5, 96, device="cuda")
    with osr.layernorm_create(96) as ln:
        y, mu, rstd = osr.layernorm_forward(ln, x)
        assert y.shape == x.shape and mu.shape == (3, 5)
        check_forward(x.view(15, 96), None, None, 1e-5, y.view(15, 96), mu.view(-1), rstd.view(-1))
        one, _, _ = osr.layernorm_forward(ln, x[0, 0])  # a single vector
        assert torch.equal(one, y[0, 0])
        part, _, _ = osr.layernorm_forward(ln, x[:, 1])  # rows 5 x 96 apart
        assert torch.equal(part, y[:, 1])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = torch.empty_like(y)
        osr.layernorm_forward(ln, x, y=other, stream=s)
        dx0, _, _ = osr.layernorm_backward(ln, x, x, None, mu, rstd)
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(other, y)
        graph = torch.cuda.CUDAGraph()
        dx, dw = torch.empty_like(x), torch.zeros(96, device="cuda")
        with torch.cuda.graph(graph):
            osr.layernorm_backward(ln, x, x, None, mu, rstd, dx=dx, dweight=dw)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, dx0) and bool(dw.any())


@pytest.mark.parametrize("cols", [61, 768, 1021, 17_000])
def test_nothing_outside_the_rows_is_written(cols):
    """Sentinels around and between the rows of y and dx, around the
    statistics and the weights' gradients."""
    rows, pad = 11, 9
    x = torch.randn(rows, cols, device="cuda").bfloat16()

    guard = -(2.0 ** 100)  # no result of these inputs

    def guarded(shape, dtype=torch.float32):
        return torch.full(shape, guard, device="cuda", dtype=dtype)

    y, dx = (guarded((rows + 2, cols + pad), torch.bfloat16) for _ in range(2))
    mu, rstd = (guarded((rows + 8,)) for _ in range(2))
    dw, db = (guarded((cols + 8,)) for _ in range(2))
    with osr.layernorm_create(cols) as ln:
        osr.layernorm_forward(ln, x, y=y[1:-1, :cols], mean=mu[4:-4], rstd=rstd[4:-4])
        osr.layernorm_backward(ln, x, x, None, mu[4:-4], rstd[4:-4], dx=dx[1:-1, :cols],
                               dweight=dw[4:-4], dbias=db[4:-4])
    for t in (y, dx):
        assert bool((t[0] == guard).all()) and bool((t[-1] == guard).all()) and bool((t[:, cols:] == guard).all())
        assert not bool((t[1:-1, :cols] == guard).all())
    for t in (mu, rstd, dw, db):
        assert bool((t[:4] == guard).all()) and bool((t[-4:] == guard).all())
        assert not bool((t[4:-4] == guard).any())


def test_offsets_past_32_bits():
    """A matrix of more than 2^32 elements (rows far apart): the last rows."""
    cols, stride, rows = 64, 1 << 20, 4100
    pool = torch.zeros(rows * stride, device="cuda", dtype=torch.bfloat16)
    x = pool.view(rows, stride)[:, :cols]
    x.copy_(torch.randn(rows, cols, device="cuda"))
    with osr.layernorm_create(cols) as ln:
        y, mu, rstd = osr.layernorm_forward(ln, x)
        check_forward(x, None, None, 1e-5, y, mu, rstd)
        dw = torch.zeros(cols, device="cuda")
        dx, _, _ = osr.layernorm_backward(ln, y, x, None, mu, rstd, dweight=dw)
        check_backward(y, x, None, mu, rstd, dx, dw, None)


def test_refusals():
    with osr.layernorm_create(64) as ln:
        x = torch.randn(4, 64, device="cuda")
        w = torch.ones(64, device="cuda")
        _, mu, rstd = osr.layernorm_forward(ln, x, w)
        for kw, exc in ((dict(x=x.cpu()), TypeError), (dict(x=x.double()), TypeError),
                        (dict(x=x[:, :63]), TypeError), (dict(x=x.t().contiguous().t()), TypeError),
                        (dict(weight=w[:63]), ValueError), (dict(weight=w.double()), TypeError),
                        (dict(weight=w.bfloat16()), osr.AdamWError),
                        (dict(bias=w.bfloat16()), TypeError), (dict(y=x.bfloat16()), TypeError),
                        (dict(y=x[:3]), TypeError), (dict(mean=mu[:3]), ValueError),
                        (dict(rstd=rstd.double()), TypeError), (dict(eps=-1.0), osr.AdamWError),
                        (dict(eps=float("nan")), osr.AdamWError)):
            args = dict(x=x, weight=w)
            args.update(kw)
            with pytest.raises(exc):
                osr.layernorm_forward(ln, **args)
        for kw, exc in ((dict(dy=x.bfloat16()), TypeError), (dict(dy=x[:3]), TypeError),
                        (dict(mean=mu[:3]), ValueError), (dict(dweight=w[:63]), ValueError),
                        (dict(dweight=w.double()), TypeError), (dict(dx=x[:3]), TypeError),
                        (dict(dweight=w, dbias=w.bfloat16()), TypeError)):
            args = dict(dy=x, x=x, weight=w, mean=mu, rstd=rstd)
            args.update(kw)
            with pytest.raises(exc):
                osr.layernorm_backward(ln, **args)
        import ctypes  # noqa: F401
        L = osr.library()
        p, odd = x.data_ptr(), x.data_ptr() + 2
        base = [ln.handle, p, 64, 0, None, None, 0, p, 64, None, None, 4, 1e-5, None]
        for i, bad in ((1, None), (1, odd), (2, 63), (3, 5), (6, 1), (8, 10), (11, -1)):
            args = list(base)
            args[i] = bad
            assert L.layernorm_forward(*args) == osr.EINVAL, i
        assert L.layernorm_backward(ln.handle, p, 64, p, 64, 0, None, 0, mu.data_ptr(),
                                    rstd.data_ptr(), p, 64, None, None, 0, 4, 2, None) == osr.EINVAL
