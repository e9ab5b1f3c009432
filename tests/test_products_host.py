"""Host-side checks of the linear layer's, the cross entropy's and the
distillation's entry points: the arguments that are refused before any CUDA
call."""
import ctypes

import pytest

import optimizer_step_resumable_gb300 as osr


@pytest.mark.parametrize("name,sizes,word", [
    ("linear_create", (0, 8), "in_features"), ("linear_create", ((1 << 24) + 1, 8), "in_features"),
    ("linear_create", (8, -3), "out_features"), ("linear_create", (1 << 24, 1 << 17), "2^40"),
    ("linear_cross_entropy_create", (0, 8), "dim"),
    ("linear_cross_entropy_create", ((1 << 20) + 1, 8), "dim"),
    ("linear_cross_entropy_create", (8, (1 << 24) + 1), "vocab"),
    ("distill_create", (0, 4), "vocab"), ("distill_create", ((1 << 30) + 1, 4), "vocab"),
    ("distill_create", (100, 0), "k="), ("distill_create", (100, 1025), "k=")])
def test_create_refuses(lib, name, sizes, word):
    out = ctypes.c_void_p(1)
    assert getattr(lib, name)(*sizes, ctypes.byref(out)) == osr.EINVAL
    assert out.value is None and word in osr.adamw_last_error()


def test_null_handles(lib):
    n = ctypes.c_int64()
    for name in ("linear", "linear_cross_entropy", "distill"):
        assert getattr(lib, name + "_create")(8, 8, None) == osr.EINVAL
        assert getattr(lib, name + "_destroy")(None) == osr.OK
    assert lib.linear_workspace(None, 1, 0, ctypes.byref(n)) == osr.EINVAL
    assert lib.linear_cross_entropy_workspace(None, 1, 0, ctypes.byref(n)) == osr.EINVAL
    assert lib.linear_forward(None, None, 0, None, 0, 1, None, 0, None, 0, 0, None, 0, None, 0, 0, 0,
                              None, 0, None) == osr.EINVAL
    assert lib.linear_backward(None, None, 0, None, 0, None, 0, 1, None, 0, 0, None, 0, None, 0, None,
                               0, 0, 0, None, 0, None) == osr.EINVAL
    assert lib.linear_cross_entropy_forward(None, None, 0, None, 0, 1, None, 0.0, None, None, 0, 0,
                                            None, 0, None) == osr.EINVAL
    assert lib.linear_cross_entropy_backward(None, None, 0, None, 0, 1, None, None, None, 1.0, 0.0,
                                             None, 0, None, 0, 0, 0, 0, None, 0, None) == osr.EINVAL
    assert lib.distill_forward(None, None, 0, 0, None, None, 0, 1.0, None, None, 0, None) == osr.EINVAL
    assert lib.distill_backward(None, None, 0, 0, None, None, 0, 1.0, None, None, 1.0, None, 0, 0,
                                None) == osr.EINVAL


def test_create_without_gpu_fails_cleanly(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    out = ctypes.c_void_p()
    for name in ("linear_create", "linear_cross_entropy_create", "distill_create"):
        assert getattr(lib, name)(64, 64, ctypes.byref(out)) == osr.ECUDA
        assert out.value is None


def test_the_binding_knows_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "adamw_ckpt.h")) as f:
        defined = dict(re.findall(r"#define (LINEAR_\w+) (\d+)", f.read()))
    for name in ("IN_OUT", "GRAD_IN_OUT", "ACCUMULATE", "FOR_BACKWARD", "FOR_ANY_ADDRESS"):
        assert int(defined["LINEAR_" + name]) == getattr(osr, "LINEAR_" + name)
    for name, code in osr.ACTIVATIONS.items():
        assert int(defined["LINEAR_" + name.upper()]) == code
