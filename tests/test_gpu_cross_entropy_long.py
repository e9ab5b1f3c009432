"""The cross entropy of wide inputs: what the logits' sums may lose, gradients of
several pieces of the vocabulary, and the largest that binary16 has to hold.

A logit is cut by up to 2^-23 of the sum of its terms' sizes for each 16 inputs;
loss and lse err by as much as the logits, and by a few units of the logits'
conversions and of the sum of exponentials, 2^-20 of 1 and 2^-22 of themselves.
U = 2^-8 or 2^-11 is the rounding of the 16-bit types.
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def inputs(rows, dim, vocab, kind, signs, seed=0):
    r = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, dim, device="cuda", generator=r)
    w = torch.randn(vocab, dim, device="cuda", generator=r) * dim ** -0.5
    if not signs:
        x, w = x.abs(), w.abs()
    target = torch.randint(0, vocab, (rows,), device="cuda", generator=r)
    target[::7] = -1
    return x.to(TYPES[kind]), w.to(TYPES[kind]), target


@pytest.mark.parametrize("dim", [768, 2048, 4104, 20000])
@pytest.mark.parametrize("kind,signs", [("f16", True), ("f16", False), ("bf16", False)])
def test_losses_of_wide_inputs(dim, kind, signs):
    x, w, target = inputs(300, dim, 1500, kind, signs)
    with osr.linear_cross_entropy_create(dim, 1500) as ce:
        loss, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
    X, W = x.double(), w.double()
    logits = X @ W.T
    cut = dim * 2.0 ** -27 * (X.abs() @ W.abs().T).amax(1)
    want = logits.logsumexp(1)
    at = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    few = 2.0 ** -20 + 2.0 ** -22 * (want.abs() + logits.abs().amax(1))
    assert bool(((lse.double() - want).abs() <= cut + few).all())
    there = target >= 0
    off = (loss.double() - (want - at)).abs()[there]
    assert bool((off <= (2 * cut + 2 * few)[there]).all())
    assert bool((loss[~there] == 0).all())


# the third type of a gradient (neither float32 nor the others'), and float32, over
# pieces: 256 MiB hold 32768 columns for 4096 rows, so three
@pytest.mark.parametrize("kind,grad", [("bf16", "f16"), ("f16", "bf16"), ("bf16", "f32"),
                                       ("f16", "f16")])
@pytest.mark.parametrize("grad_in_out", [False, True])
def test_gradients_over_pieces(kind, grad, grad_in_out):
    rows, dim, vocab = 4096, 520, 70001
    x, w, target = inputs(rows, dim, vocab, kind, True, seed=3)
    scale = 64.0
    dw = torch.full((dim, vocab) if grad_in_out else (vocab, dim), 0.25, device="cuda").to(TYPES[grad])
    dw = dw.T if grad_in_out else dw
    with osr.linear_cross_entropy_create(dim, vocab) as ce:
        _, lse = osr.linear_cross_entropy_forward(ce, x, w, target)
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, scale=scale, dweight=dw,
                                                  accumulate=True)
    want_dx = torch.zeros(rows, dim, device="cuda", dtype=torch.float64)
    X = x.double()
    rounded = fine = total = 0.0
    for first in range(0, vocab, 8192):
        W = w[first:first + 8192].double()
        dl = torch.exp(X @ W.T - lse.double()[:, None])
        here = (target >= first) & (target < first + len(W))
        dl[here.nonzero()[:, 0], target[here] - first] -= 1.0
        dl = dl * scale * (target >= 0)[:, None]
        want_dx += dl @ W
        want = dl.T @ X
        off = dw[first:first + 8192].double() - 0.25 - want
        rounded += float(off.square().sum())
        total += float(want.square().sum())
        fine += float((want + 0.25).square().sum())
    # dl's roundings and cuts are independent of one another; logits, lse and the
    # products' sums err by 2^-17 at most; then the output's own rounding
    most = (U[kind] + 2.0 ** -17) * total ** 0.5 + U[grad] * fine ** 0.5
    assert rounded ** 0.5 <= most
    off = (dx.double() - want_dx).norm()
    assert float(off) <= (2 * U[kind] + 2.0 ** -17) * float(want_dx.norm())


@pytest.mark.parametrize("g", [1.0, 1.9999, 3.9, 6e-5, 1.9999 * 2.0 ** 100])
@pytest.mark.parametrize("factor", [-1.0, -0.5, -3.0, 1.0])
def test_factors_of_opposite_signs_stay_in_range(g, factor):
    # a penalty that turns the sign of p's factor: the target's place gets p factor g - g,
    # up to twice the larger of both
    rows, dim, vocab = 40, 64, 300
    x = torch.ones(rows, dim, device="cuda", dtype=torch.float16)
    w = torch.zeros(vocab, dim, device="cuda", dtype=torch.float16)
    w[7] = 0.5  # its logit is 32, the others 0: p is 1 to 300 e^-32
    target = torch.full((rows,), 7, device="cuda")
    dloss = torch.full((rows,), g, device="cuda")
    scale = 1.0 / g
    z_loss = (factor - 1) / (2 * 32.0)
    dw = torch.empty(vocab, dim, device="cuda")
    with osr.linear_cross_entropy_create(dim, vocab) as ce:
        _, lse = osr.linear_cross_entropy_forward(ce, x, w, target, z_loss=z_loss)
        dx, _ = osr.linear_cross_entropy_backward(ce, x, w, target, lse, dloss=dloss, scale=scale,
                                                  z_loss=z_loss, dweight=dw)
    # dl = factor - 1 in units of g.  It errs by its rounding, U of itself, and by p's
    # error: the exponent is a difference of numbers near 46 (32 in powers of two),
    # each rounded, 46 x 2^-24 twice, times log 2: below 2^-17 of |factor|, also where
    # dl is 0.  Then the output's rounding.
    want = factor - 1.0
    off = U["f16"] * abs(want) + 2.0 ** -17 * (abs(factor) + 1)
    assert bool(((dx.double() - want * 0.5).abs() <= off + 2.0 ** -12 * abs(want)).all())
    assert bool(((dw[7].double() - want * rows).abs() <= off * rows).all())
