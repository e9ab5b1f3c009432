"""Arrays of one allocation: columns of one matrix are apart, and an output on
an input is refused at every width."""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.manual_seed(0)


@pytest.mark.parametrize("cols", [8, 61, 768, 1021, 17_001])
def test_columns_of_one_matrix(cols):
    """x, y, dy and dx side by side: the results of arrays of their own."""
    rows = 37
    pool = torch.randn(rows, 4 * cols, device="cuda").bfloat16()
    x, y, dy, dx = (pool[:, k * cols:(k + 1) * cols] for k in range(4))
    xo, dyo = x.clone(), dy.clone()
    w = torch.rand(cols, device="cuda") + 0.5
    with osr.layernorm_create(cols) as ln:
        _, mean, rstd = osr.layernorm_forward(ln, x, w, y=y)
        dw = torch.empty(cols, device="cuda")
        osr.layernorm_backward(ln, dy, x, w, mean, rstd, dx=dx, dweight=dw)
        assert torch.equal(x, xo) and torch.equal(dy, dyo)
        X = xo.double()
        want = (X - X.mean(1, keepdim=True)) / (X.var(1, keepdim=True, correction=0) + 1e-5).sqrt() * w
        # rounded once to bfloat16 from float32
        assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all())
        dx1, dw1, _ = osr.layernorm_backward(ln, dyo, xo, w, mean, rstd, dx=torch.empty_like(xo),
                                             dweight=torch.empty_like(dw))
        # other places, other orders of the sums
        assert bool(((dx.double() - dx1.double()).abs() <= 2.0 ** -7 * dx1.abs().double() + 1e-4).all())
        assert bool(((dw - dw1).abs() <= 1e-5 * dw1.abs() + 1e-3).all())


@pytest.mark.parametrize("cols", [64, 1021, 17_001])
def test_outputs_on_inputs_are_refused(cols):
    x = torch.randn(9, cols, device="cuda")
    dy, w = torch.randn_like(x), torch.ones(cols, device="cuda")
    with osr.layernorm_create(cols) as ln:
        y, mean, rstd = osr.layernorm_forward(ln, x, w)
        kept = x.clone()
        for kw in (dict(y=x), dict(y=x.view(-1)[:9 * cols].view(9, cols)), dict(mean=rstd, rstd=rstd),
                   dict(mean=x.view(-1)[3:12])):
            with pytest.raises(osr.AdamWError) as e:
                osr.layernorm_forward(ln, x, w, **kw)
            assert e.value.status == osr.EINVAL and "overlaps" in str(e.value)
        both = torch.empty(cols, device="cuda")
        for kw in (dict(dx=x), dict(dx=dy), dict(dweight=w), dict(dweight=both, dbias=both)):
            with pytest.raises(osr.AdamWError) as e:
                osr.layernorm_backward(ln, dy, x, w, mean, rstd, **kw)
            assert e.value.status == osr.EINVAL
        assert torch.equal(x, kept)
