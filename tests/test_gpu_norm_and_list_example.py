"""examples/norm_and_list_step.py runs as written, at a small size: it
learns, and the run resumed from its file ends in the same bits."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns_and_resumes(lib, tmp_path):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location(
        "norm_and_list_step", os.path.join(ROOT, "examples", "norm_and_list_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses, same = mod.main(steps=60, dim=96, path=str(tmp_path / "state.pt"))
    assert same
    assert losses[-1] < 0.7 * losses[0]
