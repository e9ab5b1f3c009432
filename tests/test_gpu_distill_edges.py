"""The distillation at the edges of its inputs: entries that are none, and the
temperatures it takes."""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def inputs(rows, vocab, k, kind=torch.float32, seed=0):
    r = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(rows, vocab, device="cuda", generator=r).to(kind)
    ids = torch.randint(0, vocab, (rows, k), device="cuda", generator=r)
    return logits, ids, torch.randn(rows, k, device="cuda", generator=r)


def both(logits, ids, values, **more):
    with osr.distill_create(logits.shape[1], ids.shape[1]) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values, **more)
        return loss, lse, osr.distill_backward(ds, logits, ids, values, lse, **more)


# the first entries (read beside the row), later ones, and whole rows
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [8, 70])
def test_masked_entries_past_the_vocabulary_are_none(kind, k):
    logits, ids, values = inputs(8, 1000, k, kind)
    values[:, 3] = values[:, k - 1] = -INF
    values[6] = -INF
    clean = both(logits, ids, values)
    ids[1, 3], ids[2, k - 1], ids[3, 3] = 1000, 1 << 40, 2 ** 31 + 5
    ids[6] = 1000
    got = both(logits, ids, values)
    for a, b in zip(clean[:2], got[:2]):
        assert torch.equal(a, b)
    # a place that such an entry named before holds the same probability, rounded anew
    assert torch.allclose(clean[2].float(), got[2].float(),
                          rtol=2.0 ** -7 if kind is torch.bfloat16 else 2.0 ** -18, atol=1e-12)
    assert got[0][6] == 0 and not bool(got[2][6].any())
    # with a value, it shows
    values[1, 3], values[2, k - 1] = 0.5, NAN
    loss, _, dl = both(logits, ids, values)
    assert loss.isnan().tolist() == dl.isnan().all(1).tolist() == [i in (1, 2) for i in range(8)]


@pytest.mark.parametrize("t", [2.0 ** -60, 2.0 ** -30, 2.0 ** -8, 2.0 ** 8])
def test_temperatures_of_any_size(t):
    # logits and values in units of t: T^2 times the loss and T times the gradient of T = 1
    logits, ids, values = inputs(20, 1000, 8)
    loss, lse, dl = both(logits, ids, values)
    got = both(logits * t, ids, values * t, temperature=t)
    assert torch.allclose(got[1], lse, rtol=2.0 ** -20)
    assert torch.allclose(got[0] / t ** 2, loss, rtol=2.0 ** -18, atol=2.0 ** -18)
    assert torch.allclose(got[2] / t, dl, rtol=2.0 ** -18, atol=2.0 ** -22)
    assert bool((got[0] > 0).all())
