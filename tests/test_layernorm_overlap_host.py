"""Which arrays of a layer norm's call may not overlap, on a runtime that runs
nothing: against a byte by byte count."""
import ctypes

import numpy as np
import pytest

import optimizer_step_resumable_gb300 as osr
from test_devices_host import context, fake, fake_path  # noqa: F401 - fixtures

BASE = 1 << 40
FAR = [(k + 2) << 40 for k in range(8)]


def covered(begin, stride, rows, cols, size):
    """The bytes that an array's rows take."""
    at = begin + size * (stride * np.arange(rows)[:, None] * (rows > 1))
    return set((at + np.arange(cols * size)).ravel().tolist())


def test_rows_against_rows(fake):  # noqa: F811
    """y beside x: the same and other strides, every kind of offset."""
    rng = np.random.default_rng(0)
    for _ in range(4000):
        cols, rows = int(rng.integers(1, 9)), int(rng.integers(1, 12))
        xs, ys = (cols + int(rng.choice([0, 1, cols, rng.integers(0, 40)])) for _ in range(2))
        ys = xs if rng.random() < 0.5 else ys
        dtype = int(rng.choice([osr.DTYPE_F32, osr.DTYPE_BF16]))
        size = 4 if dtype == osr.DTYPE_F32 else 2
        shift = int(rng.integers(-12 * 40, 12 * 40)) if rng.random() < 0.3 else int(rng.integers(-20, 20))
        y = BASE + size * shift
        ln = context(fake, cols)
        got = fake.layernorm_forward(ln, BASE, xs, dtype, None, None, 0, y, ys, FAR[0], FAR[1], rows,
                                     1e-5, None)
        both = covered(BASE, xs, rows, cols, size) & covered(y, ys, rows, cols, size)
        assert got == (osr.EINVAL if both else osr.OK), (cols, rows, xs, ys, size, shift)
        fake.layernorm_destroy(ln)


def test_vectors_against_rows(fake):  # noqa: F811
    """mean between and on the rows of y."""
    cols, rows, stride = 4, 5, 24
    ln = context(fake, cols)
    for shift in range(-8, 24 * 5 + 8):
        got = fake.layernorm_forward(ln, FAR[0], cols, 0, None, None, 0, BASE, stride,
                                     BASE + 4 * shift, None, rows, 1e-5, None)
        both = covered(BASE, stride, rows, cols, 4) & covered(BASE + 4 * shift, 0, 1, rows, 4)
        assert got == (osr.EINVAL if both else osr.OK), shift
    fake.layernorm_destroy(ln)


COLS, ROWS = 64, 10


def test_every_pair_of_the_forward_pass(fake):  # noqa: F811
    names = ["x", "weight", "bias", "y", "mean", "rstd"]
    outputs = {"y", "mean", "rstd"}
    for cols in (COLS, 20_000):
        ln = context(fake, cols)
        for a in names:
            for b in names:
                at = dict(zip(names, FAR))
                if a != b:
                    at[b] = at[a]
                got = fake.layernorm_forward(ln, at["x"], cols, 0, at["weight"], at["bias"], 0,
                                             at["y"], cols, at["mean"], at["rstd"], ROWS, 1e-5, None)
                wrong = a != b and {a, b} & outputs
                assert got == (osr.EINVAL if wrong else osr.OK), (a, b)
                if wrong:
                    assert "overlaps" in fake.adamw_last_error().decode()
        fake.layernorm_destroy(ln)


def test_every_pair_of_the_backward_pass(fake):  # noqa: F811
    names = ["dy", "x", "weight", "mean", "rstd", "dx", "dweight", "dbias"]
    outputs = {"dx", "dweight", "dbias"}
    for cols in (COLS, 20_000):
        ln = context(fake, cols)
        for a in names:
            for b in names:
                at = dict(zip(names, FAR))
                if a != b:
                    at[b] = at[a]
                got = fake.layernorm_backward(ln, at["dy"], cols, at["x"], cols, 0, at["weight"], 0,
                                              at["mean"], at["rstd"], at["dx"], cols, at["dweight"],
                                              at["dbias"], 0, ROWS, 0, None)
                wrong = a != b and {a, b} & outputs
                assert got == (osr.EINVAL if wrong else osr.OK), (a, b)
        fake.layernorm_destroy(ln)


def test_arrays_that_are_not_there_overlap_nothing(fake):  # noqa: F811
    ln = context(fake, COLS)
    assert fake.layernorm_forward(ln, BASE, COLS, 0, None, None, 0, FAR[0], COLS, None, None, ROWS,
                                  1e-5, None) == osr.OK
    assert fake.layernorm_forward(ln, BASE, COLS, 0, None, None, 0, BASE, COLS, BASE, BASE, 0, 1e-5,
                                  None) == osr.OK  # no rows
    assert fake.layernorm_backward(ln, BASE, COLS, BASE, COLS, 0, None, 0, FAR[1], FAR[1], FAR[0],
                                   COLS, None, None, 0, ROWS, 0, None) == osr.OK


@pytest.mark.parametrize("rows", [1 << 20, 1 << 28])
def test_columns_of_one_matrix(fake, rows):  # noqa: F811
    """x and y side by side in rows of one matrix."""
    ln = context(fake, 16)
    for at, want in ((16, osr.OK), (15, osr.EINVAL), (-1, osr.EINVAL), (-16, osr.OK),
                     (32 * (rows - 1) + 15, osr.EINVAL), (32 * (rows - 1) + 16, osr.OK)):
        assert fake.layernorm_forward(ln, BASE, 32, 0, None, None, 0, BASE + 4 * at, 32, None, None,
                                      rows, 1e-5, None) == want, at
    fake.layernorm_destroy(ln)
