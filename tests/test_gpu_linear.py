"""The linear layer's forward and backward pass against the formulas in 64
bits.

u = 2^-24 (float32); U = 2^-8 or 2^-11, the rounding of the 16-bit types.

* A sum of n products on the tensor cores: products of 16-bit values are exact,
  each addition may cut instead of round, so it errs by 2 u of its result: at
  most (n + 64) 2 u sum|terms|, in whatever order.
* act(z): the error of z times the slope's bound, 1.13, and the function's own:
  e^x in the fast form has 2 + 1.2 |x| units of 2^-23, the quotient 2, the
  argument a few u of itself, which count |x| fold: (12 + 8 |x|) 2 u |act(z)|;
  erf is within 2 units of 1: 8 u |z|.
* dz = dy act'(z): the same count relative to |dy| (1 + |z|); rounded to its
  type when there is an activation: U |dz|.
* Each output is rounded once more.
* Over many elements the roundings are independent, and one of them has the
  root mean square U / sqrt(3) at most: with two of them, 0.82 U of the
  output's norm, of the coarser type's U; the bound is that U, and the norm of
  the float32 parts' bars.
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# unit roundoff, and half the smallest spacing
ROUND = {torch.float32: (u, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}
F = torch.nn.functional
ACT = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
       "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def argument(z, act):
    """|x| of the e^x that an activation takes, 0 where it takes none."""
    if act == "silu":
        return z.abs()
    if act == "gelu_tanh":
        return (1.5957691 * (z + 0.044715 * z ** 3)).abs()
    return torch.zeros_like(z)


def matrix(r, rows, cols, kind, pad=0, at=0, sigma=1.0):
    """rows x cols in a buffer whose rows are `pad` apart, starting at `at`."""
    t = torch.empty(rows * (cols + pad) + at + 16, device="cuda").normal_(0, sigma, generator=r)
    return t.to(TYPES[kind])[at:at + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def near(got, want, bar, name, small=None, factor=0.0):
    """bar: all errors before the last rounding; small: float32's share of them;
    factor: U of the other rounding's type."""
    U, tiny = ROUND[got.dtype]
    off = (got.double() - want).abs()
    bad = ~(off <= bar + U * (want.abs() + bar) + tiny)
    assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:3].tolist(),
                                 got[bad][:3].tolist(), want[bad][:3].tolist())
    if got.numel() >= 4096 and got.dtype is not torch.float32:
        most = max(U, factor) * want.norm() + (bar if small is None else small).norm()
        assert float(off.norm()) <= float(most) + tiny * got.numel() ** 0.5, name


def run(rows, cin, cout, kind="bf16", act="none", in_out=False, bias="x", residual=False,
        grad=None, grad_in_out=False, accumulate=False, pad=0, at=0, seed=0, dx=True):
    r = torch.Generator(device="cuda").manual_seed(seed)
    x = matrix(r, rows, cin, kind, pad, at)
    w = matrix(r, cin if in_out else cout, cout if in_out else cin, kind, pad, at,
               cin ** -0.5)
    w = w.T if in_out else w
    b = None if bias is None else matrix(r, 1, cout, kind if bias == "x" else bias)[0].contiguous()
    res = matrix(r, rows, cout, kind, pad, at) if residual else None
    z = matrix(r, rows, cout, kind, pad, at)
    y = matrix(r, rows, cout, kind, pad, at)
    with osr.linear_create(cin, cout) as lin:
        osr.linear_forward(lin, x, w, b, residual=res, activation=act, y=y, z=z)
        X, W = x.double(), w.double()
        Z = X @ W.T + (0.0 if b is None else b.double())
        bar = (cin + 64) * 2 * u * (X.abs() @ W.abs().T) + 2 * u * Z.abs()
        near(z, Z, bar, "z")
        Y = ACT[act](Z)
        if act != "none":
            bar = 1.13 * bar + (12 + 8 * argument(Z, act)) * 2 * u * Y.abs() + 8 * u * Z.abs()
        if residual:
            Y = Y + res.double()
            bar = bar + u * Y.abs()
        near(y, Y, bar, "y")

        dy = matrix(r, rows, cout, kind, pad, at, 0.1)
        gt = TYPES[grad or kind]
        dw = matrix(r, cin if grad_in_out else cout, cout if grad_in_out else cin,
                    "f32", pad, at).to(gt)
        dw = dw.T if grad_in_out else dw
        db = torch.ones(cout, device="cuda", dtype=gt)
        before = (dw.double(), db.double()) if accumulate else (0.0, 0.0)
        out = matrix(r, rows, cin, kind, pad, at) if dx else False
        osr.linear_backward(lin, dy, x, w, z=z if act != "none" else None, activation=act, dx=out,
                            dweight=dw, dbias=db, accumulate=accumulate)
        D = dy.double()
        dz, dz_bar, U = D, torch.zeros_like(D), 0.0
        if act != "none":
            zz = z.double().requires_grad_()
            dz, = torch.autograd.grad(ACT[act](zz), zz, D)
            zz = zz.detach()
            dz_bar = (12 + 8 * argument(zz, act)) * 2 * u * D.abs() * (1 + zz.abs())
            U = ROUND[x.dtype][0]
        rounded = dz_bar + U * (dz.abs() + dz_bar) + (ROUND[x.dtype][1] if U else 0.0)
        size = dz.abs() + rounded
        if dx:
            sums = (cout + 64) * 2 * u * (size @ W.abs())
            near(out, dz @ W, rounded @ W.abs() + sums, "dx", dz_bar @ W.abs() + sums)
        want = dz.T @ X + before[0]
        sums = (rows + 64) * 2 * u * (size.T @ X.abs()) + u * want.abs()
        near(dw, want, rounded.T @ X.abs() + sums, "dweight", dz_bar.T @ X.abs() + sums, U)
        want = dz.sum(0) + before[1]
        near(db, want, dz_bar.sum(0) + (rows + 64) * u * dz.abs().sum(0) + u * want.abs(), "dbias")


# one row to some tiles, both sides of the borders between the tile's forms
@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rows(rows, kind):
    run(rows, 136, 520, kind, "gelu" if rows % 2 else "none", residual=rows % 3 == 0, seed=rows)


# widths on both sides of vectors, blocks of the inner dimension and tiles
@pytest.mark.parametrize("cin,cout", [(1, 1), (1, 300), (300, 1), (7, 9), (8, 16), (63, 65),
                                      (64, 64), (65, 127), (72, 128), (200, 129), (333, 255),
                                      (520, 257), (1021, 511), (2048, 768)])
@pytest.mark.parametrize("in_out", [False, True])
def test_widths(cin, cout, in_out):
    run(150, cin, cout, "bf16", "silu", in_out=in_out, grad_in_out=not in_out, seed=cin)
    run(40, cin, cout, "f16", "none", in_out=in_out, grad_in_out=in_out, grad="f32",
        accumulate=True, seed=cout)


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_activations(act, kind):
    run(300, 264, 392, kind, act, residual=True, bias="f32")
    run(20, 264, 392, kind, act, bias=None)


# rows that start anywhere: copies of the matrices that are read, elements one by one
@pytest.mark.parametrize("pad,at", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 7), (16, 16)])
def test_strides_and_addresses(pad, at):
    run(270, 256, 320, "bf16", "gelu_tanh", residual=True, pad=pad, at=at)
    run(70, 256, 320, "f16", "none", in_out=True, grad_in_out=True, residual=True, pad=pad, at=at)


@pytest.mark.parametrize("rows", [3000, 20000])
@pytest.mark.parametrize("grad", ["f32", None])
def test_long_sums(rows, grad):
    run(rows, 256, 264, "bf16", "none", grad=grad, accumulate=grad == "f32")
    run(rows, 96, 40, "f16", "relu", grad=grad, dx=False)


# tiles of 192 columns, whose half a block has is no whole number of copies
@pytest.mark.parametrize("cin,cout", [(72, 768), (200, 760)])
@pytest.mark.parametrize("in_out", [False, True])
def test_tiles_of_192_columns(cin, cout, in_out):
    run(8100, cin, cout, "bf16", "relu", in_out=in_out, residual=True)


def test_chains_of_sums():
    # so many rows, and so many tiles, that one pair of blocks sums a tile of the
    # weight's gradient in several chains, added up in its place
    run(13000, 2048, 4100, "bf16", "none", grad="f32", accumulate=True)
    run(13000, 2049, 4096, "f16", "silu", grad="f32", grad_in_out=True)


def test_long_chains_lose_little_of_a_sum_of_equal_signs():
    # 1024 products are 64 steps of 16; each cuts the sum so far by less than a unit
    # of its last place, 2^-23 of it, and the sum so far is half of the last one in
    # the mean: 64 x 2^-24, then 13 roundings of the chains' sums
    rows, cin, cout = 13000, 2056, 4104
    r = torch.Generator(device="cuda").manual_seed(5)
    x = (torch.rand(rows, cin, device="cuda", generator=r) + 0.5).bfloat16()
    dy = (torch.rand(rows, cout, device="cuda", generator=r) + 0.5).bfloat16()
    w = torch.zeros(cout, cin, device="cuda", dtype=torch.bfloat16)
    lin = osr.linear_create(cin, cout)
    want = dy.double().T @ x.double()
    first = None
    for _ in range(2):
        dw = torch.zeros(cout, cin, device="cuda")
        osr.linear_backward(lin, dy, x, w, dx=False, dweight=dw, accumulate=True)
        off = ((dw.double() - want).abs() / want).max().item()
        assert off < 64 * 2.0 ** -24 + 13 * 2.0 ** -24, off
        assert first is None or torch.equal(first, dw)
        first = dw


@pytest.mark.parametrize("cin,cout,grad_in_out", [(2048, 100, False), (100, 2048, True),
                                                  (2050, 33, False)])
def test_chains_of_sums_of_a_narrow_gradient(cin, cout, grad_in_out):
    # more chains than parts: the tile's long side along the gradient's columns
    run(40000, cin, cout, "bf16", "none", grad="f32", grad_in_out=grad_in_out, accumulate=True)


# gradients of a third type, and few rows whose weight is small or large
@pytest.mark.parametrize("rows", [2, 3, 7, 8, 9, 300])
def test_types_and_few_rows(rows):
    run(rows, 200, 312, "bf16", "gelu", grad="f16", in_out=rows % 2 == 0)
    run(rows, 2056, 4104, "f16", "none", grad="bf16", in_out=rows % 2 == 1, residual=True)


@pytest.mark.parametrize("rows,cin,cout", [(1, 768, 96), (5, 4096, 1000), (130, 640, 384),
                                           (600, 1200, 900), (2048, 64, 512)])
@pytest.mark.parametrize("in_out", [False, True])
def test_whole_numbers_are_exact(rows, cin, cout, in_out):
    # small integers: every sum is a whole number below 2^24, so nothing is rounded
    r = torch.Generator(device="cuda").manual_seed(rows)

    def whole(*shape):
        return torch.randint(-3, 4, shape, device="cuda", generator=r).bfloat16()

    x, dy, b = whole(rows, cin), whole(rows, cout), whole(cout)
    w = whole(cin, cout).T if in_out else whole(cout, cin)
    dw = torch.empty((cin, cout) if in_out else (cout, cin), device="cuda")
    dw = dw.T if in_out else dw
    db = torch.empty(cout, device="cuda")
    with osr.linear_create(cin, cout) as lin:
        y = osr.linear_forward(lin, x, w, b)
        dx, _, _ = osr.linear_backward(lin, dy, x, w, dweight=dw, dbias=db)
    assert torch.equal(y, (x.double() @ w.double().T + b.double()).bfloat16())
    assert torch.equal(dx, (dy.double() @ w.double()).bfloat16())
    assert torch.equal(dw.double(), dy.double().T @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))


def test_gradients_against_differences():
    # the loss sum(y dy) along random directions, by central differences of the
    # float64 forward formula at the kernel's own inputs
    r = torch.Generator(device="cuda").manual_seed(3)
    x, dy = matrix(r, 33, 48, "f16"), matrix(r, 33, 40, "f16")
    w, b = matrix(r, 40, 48, "f16", sigma=0.2), matrix(r, 1, 40, "f16")[0].contiguous()
    for act in ACT:
        with osr.linear_create(48, 40) as lin:
            z = torch.empty(33, 40, device="cuda", dtype=torch.float16)
            osr.linear_forward(lin, x, w, b, activation=act, z=z)
            dw, db = torch.empty(40, 48, device="cuda"), torch.empty(40, device="cuda")
            dx, _, _ = osr.linear_backward(lin, dy, x, w, z=z, activation=act, dweight=dw, dbias=db)

        def loss(x, w, b):
            return float((ACT[act](x @ w.T + b) * dy.double()).sum())

        at = [x.double(), w.double(), b.double()]
        for i, g in enumerate((dx, dw, db)):
            way = torch.randn(at[i].shape, device="cuda", generator=r, dtype=torch.float64)
            h = 1e-4
            p, m = ([a + s * h * way if j == i else a for j, a in enumerate(at)] for s in (1, -1))
            slope = (loss(*p) - loss(*m)) / (2 * h)
            terms = float((g.double() * way).abs().sum())
            # roundings of z, dz and g: 2^-11 each of the terms, z's times a
            # slope's slope of about 1 (relu: a z near 0 may change sides)
            assert abs(float((g.double() * way).sum()) - slope) <= 4 * 2.0 ** -11 * terms + 0.02, act


def test_not_a_number_and_infinity_stay_in_their_rows():
    x = torch.ones(300, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(256, 64, device="cuda", dtype=torch.bfloat16)
    x[7, 3], x[150, 60] = float("nan"), float("inf")
    with osr.linear_create(64, 256) as lin:
        y = osr.linear_forward(lin, x, w, activation="relu")
    assert bool(y[7].isnan().all()) and bool((y[150] == float("inf")).all())
    y[7] = y[150] = 64.0
    assert bool((y == 64.0).all())


def test_residual_in_place_and_rows_left_alone():
    r = torch.Generator(device="cuda").manual_seed(1)
    x, w = matrix(r, 200, 64, "bf16"), matrix(r, 48, 64, "bf16")
    big = torch.full((260, 64), 3.0, device="cuda", dtype=torch.bfloat16)
    y = big[20:220, 8:56]
    with osr.linear_create(64, 48) as lin:
        osr.linear_forward(lin, x, w, residual=y, y=y)
    want = x.double() @ w.double().T + 3.0
    assert float((y.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) * 1.01
    big[20:220, 8:56] = 3.0
    assert bool((big == 3.0).all())


def test_no_rows():
    x = torch.empty(0, 24, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(40, 24, device="cuda", dtype=torch.bfloat16)
    with osr.linear_create(24, 40) as lin:
        assert osr.linear_forward(lin, x, w).shape == (0, 40)
        dy = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16)
        dw, db = torch.ones(40, 24, device="cuda"), torch.ones(40, device="cuda")
        osr.linear_backward(lin, dy, x, w, dweight=dw, dbias=db, accumulate=True)
        assert bool((dw == 1).all()) and bool((db == 1).all())
        osr.linear_backward(lin, dy, x, w, dweight=dw, dbias=db)
        assert bool((dw == 0).all()) and bool((db == 0).all())


def test_the_same_bits_every_time_on_streams_and_in_graphs():
    r = torch.Generator(device="cuda").manual_seed(5)
    x, w, dy = matrix(r, 999, 776, "bf16"), matrix(r, 520, 776, "bf16"), matrix(r, 999, 520, "bf16")
    z = matrix(r, 999, 520, "bf16")
    with osr.linear_create(776, 520) as lin:
        def step(stream=None):
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            y = osr.linear_forward(lin, x, w, activation="gelu", stream=stream)
            dw, db = (torch.zeros(s, device="cuda") for s in ((520, 776), 520))
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            dx, _, _ = osr.linear_backward(lin, dy, x, w, z=z, activation="gelu", dweight=dw,
                                           dbias=db, stream=stream)
            return y, dx, dw, db

        first = step()
        side = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        both = [step(s) for s in side]  # one context, two calls at a time
        torch.cuda.synchronize()
        for got in both:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for _ in range(2):
            for t in captured:
                t.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, captured))


def test_refusals():
    def t(*shape, dtype=torch.bfloat16):
        return torch.ones(shape, device="cuda", dtype=dtype)

    with osr.linear_create(64, 48) as lin:
        x, w, dy = t(10, 64), t(48, 64), t(10, 48)
        for bad in (dict(x=t(10, 63)), dict(weight=t(64, 48)), dict(x=t(10, 64).float()),
                    dict(weight=t(48, 64).half()), dict(bias=t(47)), dict(y=t(10, 47)),
                    dict(z=t(9, 48)), dict(residual=t(10, 48).half()),
                    dict(activation="tanh"), dict(y=t(20, 96)[::2, ::2]), dict(x=x.cpu()),
                    dict(bias=t(48, dtype=torch.float16))):
            with pytest.raises((TypeError, ValueError, osr.AdamWError)):
                osr.linear_forward(lin, **{**dict(x=x, weight=w), **bad})
        whole = t(10, 64 + 48)
        for bad in (dict(x=whole[:, :64], y=whole[:, 40:88]), dict(y=whole[:, :48], z=whole[:, 8:56]),
                    dict(y=whole[:, :48], residual=whole[:, 8:56])):
            with pytest.raises(osr.AdamWError, match="overlaps"):
                osr.linear_forward(lin, **{**dict(x=x, weight=w), **bad})
        for bad in (dict(dy=t(10, 47)), dict(dx=t(9, 64)), dict(dweight=t(48, 63)),
                    dict(dbias=t(64)), dict(activation="gelu"), dict(dx=t(10, 64).half()),
                    dict(dx=x, dweight=t(48, 64)),
                    dict(dweight=t(48, 64), dbias=t(48, dtype=torch.float32))):
            with pytest.raises((TypeError, ValueError, osr.AdamWError)):
                osr.linear_backward(lin, **{**dict(dy=dy, x=x, weight=w), **bad})
        # a workspace that is too small, or not on its boundary
        need = osr.linear_workspace(lin, 10, osr.LINEAR_FOR_BACKWARD)
        mem = torch.empty(need + 256, device="cuda", dtype=torch.uint8)
        dw, db = t(48, 64), t(48)
        with pytest.raises(osr.AdamWError, match="needs"):
            osr.linear_backward(lin, dy, x, w, z=dy, activation="relu", dweight=dw, dbias=db,
                                workspace=mem[:256])
        with pytest.raises(osr.AdamWError, match="256-byte"):
            osr.linear_backward(lin, dy, x, w, z=dy, activation="relu", dweight=dw, dbias=db,
                                workspace=mem[8:])
        osr.linear_backward(lin, dy, x, w, z=dy, activation="relu", dweight=dw, dbias=db,
                            workspace=mem[:need])
