"""Sums over many rows: 16-bit gradients over hundreds of thousands, float32 ones
in chains of 1024.

The tensor cores cut their float32 sums: of equal signs, each 16 products lose up to
1.7 x 2^-24 of the sum.  Chains of 2^14 products (binary16) and 2^17 (bfloat16)
lose less than 2^-13 and 2^-10, a quarter of the type's rounding U = 2^-11 or 2^-8,
and each further chain one rounding, 2^-24.
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
CHAIN = {"bf16": 1 << 17, "f16": 1 << 14}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def positive(r, rows, cols, kind, sigma=1.0):
    return ((torch.rand(rows, cols, device="cuda", generator=r) + 0.5) * sigma).to(TYPES[kind])


def check(got, want, rows, kind):
    off = got.double() / want - 1
    chains = -(-rows // CHAIN[kind])
    cut = U[kind] / 4 + chains * 2.0 ** -24
    assert float(off.abs().max()) <= (U[kind] + cut) * (1 + U[kind])
    # roundings to 16 bits have no mean, cuts do; 5 standard deviations of a mean
    # of roundings, U / sqrt(3) each
    assert abs(float(off.mean())) <= cut + 5 * U[kind] / (3 * off.numel()) ** 0.5


# tiles enough for all pairs of blocks (no division of the rows), few, and narrow ones
@pytest.mark.parametrize("cin,cout,grad_in_out", [(2304, 4352, False), (768, 520, False),
                                                  (520, 96, False), (96, 520, True)])
@pytest.mark.parametrize("kind,grad,dx", [("f16", "f16", False), ("f16", "f16", True),
                                          ("bf16", "bf16", True), ("bf16", "f16", False)])
def test_gradient_of_a_weight(cin, cout, grad_in_out, kind, grad, dx):
    block, times = 8192, 128  # rows that come again, so that 64 bits are quick
    rows = block * times + 17
    r = torch.Generator(device="cuda").manual_seed(5)
    scale = 2.0 ** torch.rand(cout, device="cuda", generator=r)  # mantissas of all sizes
    x, dy = positive(r, block, cin, kind), positive(r, block, cout, kind, scale / 128)
    want = dy.double().T @ x.double() * times + dy[:17].double().T @ x[:17].double()
    x, dy = (torch.cat([t.repeat(times, 1), t[:17]]) for t in (x, dy))
    w = torch.zeros(cout, cin, device="cuda", dtype=TYPES[kind])
    dw = torch.empty((cin, cout) if grad_in_out else (cout, cin), device="cuda", dtype=TYPES[grad])
    dw = dw.T if grad_in_out else dw
    with osr.linear_create(cin, cout) as lin:
        osr.linear_backward(lin, dy, x, w, dx=None if dx else False, dweight=dw)
        check(dw, want, rows, grad)
        # added to what is there, and the same bits
        again = dw.clone()
        dw.fill_(1.0)
        osr.linear_backward(lin, dy, x, w, dx=False, dweight=dw, accumulate=True)
        check(dw, want + 1.0, rows, grad)
        osr.linear_backward(lin, dy, x, w, dx=None if dx else False, dweight=dw)
        assert torch.equal(dw, again)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_outputs_over_many_inputs(kind):
    # bias, activation, residual and z behind a sum in chains
    cin, cout, rows = (1 << 19) + 24, 328, 260
    r = torch.Generator(device="cuda").manual_seed(7)
    x, w = positive(r, rows, cin, kind), positive(r, cout, cin, kind, 2.0 ** -14)
    b = positive(r, 1, cout, kind)[0].contiguous()
    res = positive(r, rows, cout, kind)
    z = torch.empty(rows, cout, device="cuda", dtype=TYPES[kind])
    with osr.linear_create(cin, cout) as lin:
        y = osr.linear_forward(lin, x, w, b, residual=res, activation="relu", z=z)
        dy = torch.empty(rows, cout, device="cuda", dtype=TYPES[kind]).copy_(res)
    want = sum(x[:, i:i + 65536].double() @ w[:, i:i + 65536].double().T
               for i in range(0, cin, 65536)) + b.double()
    check(z, want, cin, kind)
    check(y, want + res.double(), cin, kind)
    with osr.linear_create(cout, cin) as lin:  # the other way round: dx over many outputs
        dx, _, _ = osr.linear_backward(lin, x, dy, w.T)
    check(dx, want - b.double(), cin, kind)


def test_cross_entropy():
    # all logits alike: dl is (1 / vocab - [target]), so the rows of dweight without a
    # target sum equal terms
    rows, dim, vocab = 1 << 18, 256, 300
    r = torch.Generator(device="cuda").manual_seed(9)
    x = positive(r, rows, dim, "f16", 2.0 ** -4)
    w = torch.zeros(vocab, dim, device="cuda", dtype=torch.float16)
    target = torch.randint(0, 8, (rows,), device="cuda", generator=r)
    dw = torch.empty_like(w)
    with osr.linear_cross_entropy_create(dim, vocab) as ce:
        _, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        osr.linear_cross_entropy_backward(ce, x, w, target, lse, dx=False, dweight=dw, scale=64.0)
    p = float(torch.tensor(1 / vocab * 2 ** 14).half()) * 2.0 ** -14  # dl's rounding to 16 bits
    want = 64.0 * p * x.double().sum(0)
    off = dw[8:].double() / want - 1
    # 2^14 / 300 lies 0.13 of a spacing, 7e-5 of itself, from where it would round the
    # other way, and errs by 2^-20: so dl is p
    assert float(off.abs().max()) <= 1.25 * U["f16"] + 2.0 ** -19
    assert bool((dw[8:] == dw[8]).all())


# a float32 gradient: chains of 1024 products, 64 steps of 16, lose less than 2^-23 of
# the sum for each; wide ones and narrow ones, whose tiles lie the other way round
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cin,cout,grad_in_out", [
    (13000, 2056, 4104, False), (40000, 2048, 100, False), (40000, 100, 2048, True),
    (40000, 2050, 33, False), (5000, 768, 768, True)])
def test_float32_gradients_keep_their_bits(kind, rows, cin, cout, grad_in_out):
    r = torch.Generator(device="cuda").manual_seed(11)
    w = torch.zeros(cout, cin, device="cuda", dtype=TYPES[kind])
    cut, roundings = 64 * 2.0 ** -23, (-(-rows // 1024) + 1) * 2.0 ** -24
    with osr.linear_create(cin, cout) as lin:
        def gradient(x, dy):
            dw = torch.zeros((cin, cout) if grad_in_out else (cout, cin), device="cuda")
            dw = dw.T if grad_in_out else dw
            osr.linear_backward(lin, dy, x, w, dx=False, dweight=dw, accumulate=True)
            return dw

        x, dy = positive(r, rows, cin, kind), positive(r, rows, cout, kind)
        want = dy.double().T @ x.double()
        dw = gradient(x, dy)
        assert float((dw.double() / want - 1).abs().max()) <= cut + roundings
        assert torch.equal(dw, gradient(x, dy))
        # of either sign: a chain's partial sums are no larger than its terms' norm in
        # the mean, so the cuts' norm is no larger than that share of the gradient's
        x, dy = (torch.randn(rows, n, device="cuda", generator=r).to(TYPES[kind])
                 for n in (cin, cout))
        want = dy.double().T @ x.double()
        assert float((gradient(x, dy).double() - want).norm()) <= (cut + roundings) * float(want.norm())


def test_chains_through_the_workspace_in_a_graph_and_on_streams():
    # a binary16 gradient over more rows than one chain takes, beside dx: captured and
    # replayed over garbage, and two calls at a time with one context
    rows, cin, cout = 40000, 600, 520
    r = torch.Generator(device="cuda").manual_seed(13)
    x, dy = positive(r, rows, cin, "f16"), positive(r, rows, cout, "f16", 2.0 ** -8)
    w = positive(r, cout, cin, "f16")
    with osr.linear_create(cin, cout) as lin:
        def step(stream=None):
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            dw = torch.empty(cout, cin, device="cuda", dtype=torch.float16)
            db = torch.empty(cout, device="cuda", dtype=torch.float16)
            dx, _, _ = osr.linear_backward(lin, dy, x, w, dweight=dw, dbias=db, stream=stream)
            return dx, dw, db

        first = step()
        check(first[1], dy.double().T @ x.double(), rows, "f16")
        torch.cuda.synchronize()
        both = [step(torch.cuda.Stream()) for _ in range(2)]
        torch.cuda.synchronize()
        for got in both:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for _ in range(3):
            for t in captured:
                t.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, captured))
        # asks whether a replayed kernel gave up: no rows, no launch
        osr.linear_forward(lin, x[:0], w)
