"""Temperatures that the distillation takes: those whose square and inverse float32
holds.  Checked before any CUDA call."""
import pytest

import optimizer_step_resumable_gb300 as osr
from test_products_devices_host import create, fake, fake_path, place  # noqa: F401


@pytest.mark.parametrize("t,good", [
    (1.0, True), (2.0 ** -60, True), (2.0 ** 60, True), (20.0, True), (0.01, True),
    (2.0 ** -61, False), (2.0 ** 61, False), (1e-30, False), (3.5e-39, False), (1e25, False),
    (1e300, False), (0.0, False), (-1.0, False), (float("inf"), False), (float("nan"), False)])
def test_temperatures(fake, t, good):  # noqa: F811
    ds = create(fake, "distill", 1000, 8)
    calls = (
        lambda: fake.distill_forward(ds, place(1), 1000, osr.DTYPE_F32, place(2), place(3),
                                     osr.DTYPE_F32, t, place(4), place(5), 10, None),
        lambda: fake.distill_backward(ds, place(1), 1000, osr.DTYPE_F32, place(2), place(3),
                                      osr.DTYPE_F32, t, place(4), None, 1.0, place(6), 1000, 10,
                                      None))
    for call in calls:
        before = fake.fake_launches()
        assert call() == (osr.OK if good else osr.EINVAL)
        assert fake.fake_launches() == before + good
        assert good or b"temperature" in fake.adamw_last_error()
    assert fake.distill_destroy(ds) == osr.OK
