"""Host-side checks of the list step's and the layer norm's entry points: the
arguments that are refused before any CUDA call."""
import ctypes

import pytest

import optimizer_step_resumable_gb300 as osr


@pytest.mark.parametrize("cols", [0, -1, (1 << 18) + 1])
def test_layernorm_create_refuses(lib, cols):
    out = ctypes.c_void_p(1)
    assert lib.layernorm_create(cols, ctypes.byref(out)) == osr.EINVAL
    assert out.value is None and "cols" in osr.adamw_last_error()


@pytest.mark.parametrize("numels", [[-1], [5, 1 << 31], [3, -7, 2]])
def test_list_create_refuses(lib, numels):
    out = ctypes.c_void_p(1)
    table = (ctypes.c_int64 * len(numels))(*numels)
    assert lib.adamw_list_create(len(numels), table, None, ctypes.byref(out)) == osr.EINVAL
    assert out.value is None and "numel" in osr.adamw_last_error()


def test_null_handles_and_tables(lib):
    out = ctypes.c_void_p()
    assert lib.adamw_list_create(-1, None, None, ctypes.byref(out)) == osr.EINVAL
    assert lib.adamw_list_create(2, None, None, ctypes.byref(out)) == osr.EINVAL
    assert lib.adamw_list_create(0, None, None, None) == osr.EINVAL
    assert lib.layernorm_create(8, None) == osr.EINVAL
    assert lib.adamw_list_step(None, 1, 0.1, 0.0, 1.0, 1.0, 0, 0, None) == osr.EINVAL
    assert lib.adamw_list_last_norm(None, None, None) == osr.EINVAL
    assert lib.adamw_list_set_decay(None, None, 0) == osr.EINVAL
    assert lib.adamw_list_set_hparams(None, 0.9, 0.999, 1e-8) == osr.EINVAL
    assert lib.layernorm_forward(None, None, 0, 0, None, None, 0, None, 0, None, None, 0, 1e-5,
                                 None) == osr.EINVAL
    assert lib.adamw_list_destroy(None) == osr.OK and lib.layernorm_destroy(None) == osr.OK


def test_create_without_gpu_fails_cleanly(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    out = ctypes.c_void_p()
    assert lib.layernorm_create(768, ctypes.byref(out)) == osr.ECUDA
    table = (ctypes.c_int64 * 1)(10)
    assert lib.adamw_list_create(1, table, None, ctypes.byref(out)) == osr.ECUDA


def test_the_binding_knows_the_block_size():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "adamw_ckpt.h")) as f:
        assert int(re.search(r"#define ADAMW_STATE_BLOCK (\d+)", f.read()).group(1)) == osr.STATE_BLOCK
