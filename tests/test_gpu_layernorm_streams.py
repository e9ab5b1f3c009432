"""Outputs that the layer norm's calls allocate, on a stream that is not the
current one."""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("by_handle", [False, True])
def test_allocated_outputs_belong_to_the_call_s_stream(by_handle):
    """Memory that was freed while kernels of the current stream may still use
    it must not become an output of another stream: nothing orders the two."""
    rows, cols = 4096, 768
    x = torch.randn(rows, cols, device="cuda").bfloat16()
    w = torch.ones(cols, device="cuda")
    with osr.layernorm_create(cols) as ln:
        want, mean, rstd = osr.layernorm_forward(ln, x, w)
        dx_want, _, _ = osr.layernorm_backward(ln, x, x, w, mean, rstd)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        stream = s.cuda_stream if by_handle else s

        def freed():
            """Addresses that the allocator gives the current stream's next tensors."""
            ts = [torch.empty_like(x) for _ in range(3)] + [torch.empty(rows, device="cuda") for _ in range(6)]
            return {t.data_ptr() for t in ts}

        was = freed()
        y, mu, rs = osr.layernorm_forward(ln, x, w, stream=stream)
        assert not was & {y.data_ptr(), mu.data_ptr(), rs.data_ptr()}
        was = freed()
        dx, _, _ = osr.layernorm_backward(ln, x, x, w, mean, rstd, stream=stream)
        assert not was & {dx.data_ptr()}
        s.synchronize()
        assert torch.equal(y, want) and torch.equal(mu, mean) and torch.equal(rs, rstd)
        assert torch.equal(dx, dx_want)
