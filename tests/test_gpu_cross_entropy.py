"""The cross entropy without kept logits against the formulas in 64 bits.

u = 2^-24 (float32); U = 2^-8 or 2^-11, the rounding of the 16-bit types.

* A logit: (dim + 64) 2 u sum|x w|, as the tensor cores may cut instead of
  round; e is the largest of a row's.
* lse: e, the sum's chain (at most 32 / 4 + 4 + vocab / 128 / 8 + 8 additions and a
  rescaling at each, 2^-22 for each power of two) and a few u of the value:
  e + (2 vocab / 1024 + 60) 2^-22 + 4 u |lse|.  loss: twice that, and
  z_loss lse^2 with twice the error of lse times |z_loss lse|.
* dl: p's error is p (e + 2^-22 (2 + |l - lse|)), with lse as given; the
  factors and their product and difference count 4 u; rounded to its type:
  U |dl|, and for binary16 half the smallest spacing, 2^-25, in units in which
  the largest factor is at least 2^14.
* dx, dweight: those through the product, the product's own
  (n + 64) 2 u sum|terms|, the roundings of the pieces' sum and the output.
* Norms: two independent roundings have 0.82 U of the output's norm, as each has
  the root mean square U / sqrt(3) at most; the bound is U, and the norm of the
  float32 parts' bars (a gradient whose terms cancel has nothing else).
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: (u, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def matrix(r, rows, cols, kind, pad=0, at=0, sigma=1.0):
    t = torch.empty(rows * (cols + pad) + at + 16, device="cuda").normal_(0, sigma, generator=r)
    return t.to(TYPES[kind])[at:at + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def near(got, want, bar, name, small=None):
    """bar: all errors before the last rounding; small: float32's share of them."""
    U, tiny = ROUND[got.dtype]
    off = (got.double() - want).abs()
    bad = ~(off <= bar + U * (want.abs() + bar) + tiny)
    assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:3].tolist(),
                                 got[bad][:3].tolist(), want[bad][:3].tolist())
    if got.numel() >= 4096 and got.dtype is not torch.float32:
        most = U * want.norm() + (bar if small is None else small).norm()
        assert float(off.norm()) <= float(most) + tiny * got.numel() ** 0.5, name


def inputs(rows, dim, vocab, kind, in_out=False, pad=0, at=0, seed=0, ignored=0.2, spread=2.0):
    r = torch.Generator(device="cuda").manual_seed(seed)
    x = matrix(r, rows, dim, kind, pad, at)
    w = matrix(r, dim if in_out else vocab, vocab if in_out else dim, kind, pad, at,
               spread * dim ** -0.5)
    w = w.T if in_out else w
    target = torch.randint(0, vocab, (rows,), device="cuda", generator=r)
    target[torch.rand(rows, device="cuda", generator=r) < ignored] = -100
    return r, x, w, target


def check_forward(x, w, target, z_loss, loss, lse):
    X, W = x.double(), w.double()
    logits = X @ W.T
    e = ((x.shape[1] + 64) * 2 * u * (X.abs() @ W.abs().T)).amax(1)
    want = logits.logsumexp(1)
    bar = e + (2 * w.shape[0] / 1024 + 60) * 2.0 ** -22 + 4 * u * want.abs()
    near(lse, want, bar, "lse")
    at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    full = torch.where(target >= 0, want - at + z_loss * want * want, 0.0)
    near(loss, full, 2 * bar + 3 * abs(z_loss) * want.abs() * bar + 4 * u * at.abs(), "loss")
    assert bool((loss[target < 0] == 0).all())
    return e


def run(rows, dim, vocab, kind="bf16", in_out=False, grad=None, grad_in_out=False,
        accumulate=False, z_loss=0.0, dloss=False, scale=1.0, pad=0, at=0, seed=0, ignored=0.2,
        dx=True):
    r, x, w, target = inputs(rows, dim, vocab, kind, in_out, pad, at, seed, ignored)
    with osr.linear_cross_entropy_create(dim, vocab) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target, z_loss=z_loss)
        e = check_forward(x, w, target, z_loss, loss, lse)
        gt = TYPES[grad or kind]
        dw = matrix(r, dim if grad_in_out else vocab, vocab if grad_in_out else dim, "f32", pad,
                    at, 0.01).to(gt)
        dw = dw.T if grad_in_out else dw
        before = dw.double() if accumulate else 0.0
        g = torch.randn(rows, device="cuda", generator=r) if dloss else None
        out = matrix(r, rows, dim, kind, pad, at) if dx else False
        osr.linear_cross_entropy_backward(ce, x, w, target, lse, dloss=g, scale=scale,
                                          z_loss=z_loss, dx=out, dweight=dw,
                                          accumulate=accumulate)
    X, W, L = x.double(), w.double(), lse.double()[:, None]
    logits = X @ W.T
    factor = scale * (1.0 if g is None else g.double()) * (target >= 0).double()
    f = (factor * (1 + 2 * z_loss * lse.double()))[:, None]
    p = torch.exp(logits - L)
    dl = f * p
    there = torch.zeros_like(dl)
    there.scatter_(1, target.clamp(min=0)[:, None], factor[:, None])
    dl = dl - there
    U = ROUND[x.dtype][0]
    most = torch.maximum(f.abs().max(), factor.abs().max())
    bar = (f.abs() * p * (e[:, None] + 2.0 ** -22 * (2 + (logits - L).abs()))
           + 4 * u * (f.abs() * p + there.abs()))
    small = bar + (2.0 ** -39 * most if kind == "f16" else 0.0)
    bar = small + U * (dl.abs() + small)
    size = dl.abs() + bar
    if dx:
        sums = (vocab + 64) * 2 * u * (size @ W.abs())
        near(out, dl @ W, bar @ W.abs() + sums, "dx", small @ W.abs() + sums)
    want = dl.T @ X + before
    sums = (rows + 64) * 2 * u * (size.T @ X.abs()) + u * want.abs()
    near(dw, want, bar.T @ X.abs() + sums, "dweight", small.T @ X.abs() + sums)


@pytest.mark.parametrize("rows", [1, 2, 31, 128, 129, 256, 257, 600])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rows(rows, kind):
    run(rows, 136, 1000, kind, seed=rows, z_loss=1e-3 if rows % 2 else 0.0, dloss=rows % 3 == 0,
        ignored=0.0 if rows == 1 else 0.2)


# vocabularies on both sides of threads' chunks, halves of tiles and tiles
@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 127, 128, 129, 160, 255, 256, 257, 400, 512,
                                   1021, 5000])
@pytest.mark.parametrize("in_out", [False, True])
def test_vocabularies(vocab, in_out):
    run(90, 72, vocab, "bf16", in_out=in_out, grad_in_out=not in_out, seed=vocab)
    run(90, 67, vocab, "f16", in_out=in_out, grad_in_out=in_out, grad="f32", accumulate=True,
        seed=vocab, scale=64.0)


@pytest.mark.parametrize("dim", [1, 8, 63, 64, 65, 200, 509, 1024])
def test_dims(dim):
    run(140, dim, 777, "bf16", seed=dim, dloss=True)


@pytest.mark.parametrize("pad,at", [(8, 8), (3, 0), (0, 1), (5, 7)])
def test_strides_and_addresses(pad, at):
    run(130, 96, 640, "bf16", pad=pad, at=at)
    run(130, 96, 640, "f16", in_out=True, grad_in_out=True, pad=pad, at=at)


def test_several_pieces():
    # 256 MiB hold 8192 columns for 16384 rows: three pieces, the last shorter
    run(16384, 40, 20000, "bf16", grad="f32", accumulate=True)
    run(16384, 40, 20000, "f16", in_out=True, grad_in_out=True, scale=1.0 / 16384)


@pytest.mark.parametrize("scale", [1e-20, 1e-6, 1.0, 1e6, 1e20])
def test_factors_of_any_size(scale):
    # gradients of the logits keep their bits whatever the scale
    r, x, w, target = inputs(200, 64, 300, "bf16")
    with osr.linear_cross_entropy_create(64, 300) as ce:
        _, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        dw1, dw2 = (torch.empty(300, 64, device="cuda") for _ in range(2))
        dx1, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, scale=scale, dweight=dw1)
        dx2, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, dweight=dw2)
        # two roundings each to bfloat16 of the weights' terms, three of x's
        for a, b, most in ((dw1, dw2, 2.0 ** -8), (dx1, dx2, 2.0 ** -7)):
            a, b = a.double(), scale * b.double()
            assert float((a - b).norm()) <= most * float(b.norm())
        h, hw = x.half(), w.half()
        _, lse = osr.linear_cross_entropy_forward(ce, h, hw, target)
        osr.linear_cross_entropy_backward(ce, h, hw, target, lse, scale=scale, dx=False, dweight=dw1)
        osr.linear_cross_entropy_backward(ce, h, hw, target, lse, dx=False, dweight=dw2)
        a, b = dw1.double(), scale * dw2.double()
        assert float((a - b).norm()) <= 2.0 ** -10 * float(b.norm())


def test_rows_without_a_target():
    # all of a batch, and garbage behind the last sequence
    r, x, w, target = inputs(300, 64, 1000, "bf16")
    target[:] = -1
    with osr.linear_cross_entropy_create(64, 1000) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target, z_loss=1.0)
        dw = torch.ones(1000, 64, device="cuda")
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, z_loss=1.0, dweight=dw)
        assert bool((loss == 0).all()) and bool((dx == 0).all()) and bool((dw == 0).all())
        x[250:] = float("nan")
        target[:250] = 5
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse)
        assert bool((loss[250:] == 0).all()) and bool((dx[250:] == 0).all())
        assert bool(loss[:250].isfinite().all()) and bool(dx[:250].isfinite().all())
        assert bool(lse[250:].isnan().all())


def test_a_target_past_the_vocabulary_shows():
    r, x, w, target = inputs(40, 64, 300, "bf16", ignored=0.0)
    target[7], target[9] = 300, 1 << 40
    with osr.linear_cross_entropy_create(64, 300) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse)
    bad = loss.isnan()
    assert bad.nonzero()[:, 0].tolist() == [7, 9]
    assert torch.equal(dx.isnan().all(1), bad) and torch.equal(dx.isnan().any(1), bad)


def test_large_logits():
    # logits up to about a thousand: no overflow, the largest wins
    r, x, w, target = inputs(100, 256, 2000, "bf16", spread=300.0)
    with osr.linear_cross_entropy_create(256, 2000) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
    check_forward(x, w, target, 0.0, loss, lse)


@pytest.mark.parametrize("vocab", [1, 40, 2000])
def test_logits_far_below_zero(vocab):
    # all of a row's logits near -600 or below: nothing to compare them with but one another
    r, x, w, target = inputs(100, 64, vocab, "bf16", spread=0.5)
    x, w = x.abs() + 1, w - 8
    with osr.linear_cross_entropy_create(64, vocab) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse)
    assert float(lse.max()) < -400 and bool(dx.isfinite().all())
    check_forward(x, w, target, 0.0, loss, lse)


def test_gradients_against_differences():
    r, x, w, target = inputs(50, 32, 200, "f16")
    g = torch.rand(50, device="cuda", generator=r)
    z_loss = 0.05
    with osr.linear_cross_entropy_create(32, 200) as ce:
        _, lse = osr.linear_cross_entropy_forward(ce, x, w, target, z_loss=z_loss)
        dw = torch.empty(200, 32, device="cuda")
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, dloss=g, scale=0.5,
                                                  z_loss=z_loss, dweight=dw)

    def loss(x, w):
        logits = x @ w.T
        lse = logits.logsumexp(1)
        at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
        return float((0.5 * g * (target >= 0) * (lse - at + z_loss * lse * lse)).sum())

    at = [x.double(), w.double()]
    for i, d in enumerate((dx, dw)):
        way = torch.randn(at[i].shape, device="cuda", generator=r, dtype=torch.float64)
        h = 1e-5
        p, m = ([a + s * h * way if j == i else a for j, a in enumerate(at)] for s in (1, -1))
        slope = (loss(*p) - loss(*m)) / (2 * h)
        # the roundings of dl and of the gradient, of all terms
        terms = float((d.double() * way).abs().sum())
        assert abs(float((d.double() * way).sum()) - slope) <= 2.0 ** -9 * terms


def test_the_same_bits_every_time_on_streams_and_in_graphs():
    r, x, w, target = inputs(700, 200, 3001, "bf16")
    with osr.linear_cross_entropy_create(200, 3001) as ce:
        def step(stream=None):
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target, stream=stream)
            dw = torch.zeros(3001, 200, device="cuda")
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, dweight=dw,
                                                      stream=stream)
            return loss, lse, dx, dw

        first = step()
        side = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        both = [step(s) for s in side]
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


def test_no_rows():
    w = torch.ones(40, 24, device="cuda", dtype=torch.bfloat16)
    x = torch.empty(0, 24, device="cuda", dtype=torch.bfloat16)
    target = torch.empty(0, device="cuda", dtype=torch.int64)
    with osr.linear_cross_entropy_create(24, 40) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        assert loss.shape == (0,)
        dw = torch.ones(40, 24, device="cuda")
        osr.linear_cross_entropy_backward(ce, x, w, target, lse, dweight=dw, accumulate=True)
        assert bool((dw == 1).all())
        osr.linear_cross_entropy_backward(ce, x, w, target, lse, dweight=dw)
        assert bool((dw == 0).all())


def test_refusals():
    r, x, w, target = inputs(20, 64, 96, "bf16")
    with osr.linear_cross_entropy_create(64, 96) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        for bad in (dict(x=x[:, :63]), dict(weight=w[:95]), dict(target=target.int()),
                    dict(target=target[:19]), dict(weight=w.half()), dict(x=x.float()),
                    dict(loss=torch.empty(19, device="cuda")), dict(z_loss=float("inf")),
                    dict(lse=torch.empty(20, device="cuda", dtype=torch.float64)),
                    dict(target=target.cpu())):
            with pytest.raises((TypeError, ValueError, osr.AdamWError)):
                osr.linear_cross_entropy_forward(ce, **{**dict(x=x, weight=w, target=target), **bad})
        for bad in (dict(lse=lse[:19]), dict(dx=x), dict(dx=x.half()), dict(dweight=w),
                    dict(dloss=lse.double()), dict(scale=float("nan")), dict(dweight=w[:, :63])):
            with pytest.raises((TypeError, ValueError, osr.AdamWError)):
                osr.linear_cross_entropy_backward(ce, **{**dict(x=x, weight=w, target=target,
                                                                lse=lse), **bad})
