"""The list step with 32-bit states against the flat step, bit for bit, over
the whole range of float32: moments that have died away, gradients far below
eps, weights of 0, subnormal numbers.  Clip is off, so the factor is 1 on both
sides and the two are the same formula in the same roundings."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

LR, WD = 3e-3, 0.01
N = 40_961


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def steps_of_both(w, g, m, v, hparams, steps, lr=LR, wd=WD, decay=None):
    """(flat, listed): the arrays after the steps; the list is cut in three."""
    base = [torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda() for x in (w, g, m, v)]
    n = base[0].numel()
    flat, listed = ([x.clone() for x in base] for _ in range(2))
    cut = [0, n // 4 // 8 * 8, n // 2 + 3, n]
    parts = [[x[a:b] for a, b in zip(cut, cut[1:])] for x in listed]
    with osr.adamw_create(n) as ctx, osr.adamw_list_create(*parts) as lst:
        osr.adamw_set_hparams(ctx, *hparams)
        osr.adamw_list_set_hparams(lst, *hparams)
        for t in steps:
            osr.adamw_clip_step(ctx, *flat, t, lr, wd, float("inf"))
            osr.adamw_list_step(lst, t, lr, wd, float("inf"))
    return flat, listed


def same_bits(flat, listed):
    for name, a, b in zip("wgmv", flat, listed):
        a, b = (x.view(torch.int32).cpu().numpy() for x in (a, b))
        bad = np.nonzero(a != b)[0]
        assert not bad.size, (name, bad.size, int(bad[0]), hex(a[bad[0]]), hex(b[bad[0]]))


def magnitudes(rng, low, high, n=N, zeros=0.1):
    """Values of both signs, spread over their exponent of two."""
    x = np.ldexp(rng.uniform(1, 2, n), rng.integers(low, high, n)) * rng.choice([-1.0, 1.0], n)
    x[rng.random(n) < zeros] = 0.0
    return x.astype(np.float32)


HPARAMS = [(0.9, 0.999, 1e-8), (0.9, 0.999, 1e-15), (0.9, 0.999, 1e-30), (0.9, 0.5, 1e-8),
           (0.5, 0.9, 1e-12), (0.0, 0.0, 1e-8), (0.9, 0.999, 1.0), (0.9, 0.999, 0.0)]


@pytest.mark.parametrize("hparams", HPARAMS)
@pytest.mark.parametrize("lr,wd", [(LR, WD), (1e-10, 0.0), (1e3, 0.1), (0.0, 0.01)])
def test_every_magnitude(hparams, lr, wd):
    """Gradients from 2^-100 (their norm stays a number), moments down to the
    smallest subnormal number, weights from 0 to ordinary ones."""
    rng = np.random.default_rng(1)
    w = magnitudes(rng, -149, 2, zeros=0.2)
    w[:100] = -0.0
    g = magnitudes(rng, -100, 1, zeros=0.3)
    m = magnitudes(rng, -149, 1)
    v = np.abs(magnitudes(rng, -149, 1))
    same_bits(*steps_of_both(w, g, m, v, hparams, (1, 2, 7), lr, wd))


@pytest.mark.parametrize("hparams", HPARAMS)
@pytest.mark.parametrize("size", [1e-14, 1e-16, 1e-18, 1e-20])
def test_tiny_gradients_from_the_zero_state(hparams, size):
    """v = (1 - beta2) g^2 far below 2^-96 while m is an ordinary number: the
    update is a share of lr, whatever g's size."""
    rng = np.random.default_rng(2)
    g = rng.standard_normal(N) * size
    w = np.where(rng.random(N) < 0.5, 0.0, rng.standard_normal(N) * 0.02)
    same_bits(*steps_of_both(w, g, np.zeros(N), np.zeros(N), hparams, (1, 2, 3)))


@pytest.mark.parametrize("beta1", [0.9, 0.5])
def test_rows_that_no_gradient_reaches_any_more(beta1):
    """m dies away to a few units of the smallest subnormal number; v follows
    a hundred times slower; w only decays, or stays 0."""
    rng = np.random.default_rng(3)
    w = np.where(rng.random(N) < 0.2, 0.0, rng.standard_normal(N) * 0.02)
    m = rng.standard_normal(N) * 2.0 ** -rng.uniform(90, 140, N)
    v = rng.standard_normal(N) ** 2 * 2.0 ** -rng.uniform(0, 140, N)
    same_bits(*steps_of_both(w, np.zeros(N), m, v, (beta1, 0.999, 1e-8), range(300, 360)))


def test_weights_whose_decay_ends_between_two_floats():
    """w (1 - lr wd) exactly half-way between two floats: there the sign of
    even the smallest update decides.  The factor 1 - 2^-10 takes 10 bits, so
    one w in 2^10 of those with 24 random bits is such a tie."""
    rng = np.random.default_rng(4)
    w = np.ldexp(rng.integers(1 << 23, 1 << 24, N).astype(np.float64), -24)
    w[::2] = np.ldexp((rng.integers(1 << 13, 1 << 14, w[::2].size) * 1024 + 512), -24)
    m = magnitudes(rng, -149, -99)
    v = np.abs(magnitudes(rng, -149, 1))
    same_bits(*steps_of_both(w, np.zeros(N), m, v, (0.9, 0.999, 1e-8), (5,), lr=2.0 ** -7,
                             wd=2.0 ** -3))


def test_moments_that_are_not_numbers():
    """Infinite, NaN and negative second moments: the flat step's results."""
    rng = np.random.default_rng(5)
    w, m = rng.standard_normal(N) * 0.02, magnitudes(rng, -149, 1, zeros=0.4)
    v = np.abs(magnitudes(rng, -149, 1))
    v[::5], v[1::5], v[2::5] = np.inf, np.nan, -v[2::5]
    m[::7] = np.nan
    flat, listed = steps_of_both(w, np.zeros(N), m, v, (0.9, 0.999, 1e-8), (3,))
    for a, b in zip(flat, listed):
        assert torch.equal(a.isnan(), b.isnan())
        a.nan_to_num_(nan=0.0, posinf=float("inf"), neginf=-float("inf"))
        b.nan_to_num_(nan=0.0, posinf=float("inf"), neginf=-float("inf"))
    same_bits(flat, listed)
