"""The distillation from top logits against the formulas in 64 bits.

u = 2^-24.  Powers of two in the fast form err by 2^-22 of their value and by
u |argument|, the argument's own rounding; logarithms and sums of at most n
additions in a row by a few u.

* lse: (2^-22 + u (|lse| + max|l / T|) 4 + n u), n = vocab / 2048 + 64 additions.
* loss: T^2 sum of q times (the errors of log q and log p: 8 u of each
  magnitude, lse's, 2^-21), and q's own relative error 2^-20 + 8 u max|v / T|
  times |log q - log p|.
* dl: factor (p (2^-21 + 4 u (|l / T| + |lse|)) + q's error), then 4 u of p and
  q, and the rounding to the type.  The fast power of two gives 0 where its value
  is below 2^-126, so p and q each may miss that much: 2^-125 factor.
"""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu

u = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {torch.float32: (u, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def near(got, want, bar, name):
    U, tiny = ROUND[got.dtype]
    off = (got.double() - want).abs()
    bad = ~(off <= bar + U * (want.abs() + bar) + tiny)
    assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[:3].tolist(),
                                 got[bad][:3].tolist(), want[bad][:3].tolist())


def matrix(r, rows, cols, kind, pad=0, at=0, sigma=1.0):
    t = torch.empty(rows * (cols + pad) + at + 16, device="cuda").normal_(0, sigma, generator=r)
    return t.to(TYPES[kind])[at:at + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def inputs(rows, vocab, k, kind, vkind="f32", pad=0, at=0, seed=0, absent=0.1, spread=3.0):
    r = torch.Generator(device="cuda").manual_seed(seed)
    logits = matrix(r, rows, vocab, kind, pad, at, spread)
    ids = torch.randint(0, vocab, (rows, k), device="cuda", generator=r)
    ids[torch.rand(rows, k, device="cuda", generator=r) < absent] = -1
    values = torch.empty(rows, k, device="cuda").normal_(0, spread, generator=r).to(TYPES[vkind])
    return r, logits, ids, values


def teacher(ids, values, t):
    there = (ids >= 0) & (values != -float("inf"))
    v = torch.where(there, values.double() / t, -1e300)
    some = there.any(1, keepdim=True)
    log_q = torch.where(there & some, v - v.logsumexp(1, keepdim=True), 0.0)
    return torch.where(there & some, log_q.exp(), 0.0), log_q, some


def check(logits, ids, values, t, loss, lse, dl=None, g=None):
    rows, vocab = logits.shape
    L = logits.double() / t
    n = vocab / 2048 + 64
    want = L.logsumexp(1)
    lse_bar = 2.0 ** -22 + 4 * u * (want.abs() + L.abs().amax(1)) + n * u
    near(lse, want, lse_bar, "lse")
    q, log_q, some = teacher(ids, values, t)
    at = L.gather(1, ids.clamp(min=0))
    log_p = at - want[:, None]
    full = torch.where(q > 0, q * (log_q - log_p), 0.0)
    biggest = torch.where(q > 0, values.double().abs() / t, 0.0).amax(1, keepdim=True)
    q_bar = q * (2.0 ** -20 + 8 * u * biggest + 8 * u * log_q.abs())
    bar = (q * (8 * u * (log_q.abs() + at.abs() + biggest) + lse_bar[:, None] + 2.0 ** -21)
           + q_bar * (log_q - log_p).abs()) * 1.01
    near(loss, t * t * full.sum(1), t * t * bar.sum(1) + 64 * u * t * t * full.abs().sum(1), "loss")
    if dl is None:
        return
    given = lse.double()[:, None]
    factor = (g * t)[:, None]
    p = torch.where(some, torch.exp(L - given), 0.0)
    sums = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), q)
    sums_bar = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), q_bar)
    bar = factor.abs() * (p * (2.0 ** -21 + 4 * u * (L.abs() + given.abs())) + sums_bar
                          + (4 + ids.shape[1]) * u * (p + sums) + 2.0 ** -125)
    near(dl, factor * (p - sums), bar, "dlogits")


def run(rows, vocab, k, kind="f32", vkind="f32", t=1.0, pad=0, at=0, out_at=None, seed=0,
        in_place=False, dloss=True, absent=0.1):
    r, logits, ids, values = inputs(rows, vocab, k, kind, vkind, pad, at, seed, absent)
    g = torch.randn(rows, device="cuda", generator=r) if dloss else None
    with osr.distill_create(vocab, k) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values, temperature=t)
        kept = logits.clone()
        out = logits if in_place else matrix(r, rows, vocab, kind, pad,
                                             at if out_at is None else out_at)
        osr.distill_backward(ds, logits, ids, values, lse, temperature=t, dloss=g, scale=0.5,
                             dlogits=out)
    g = 0.5 * (torch.ones(rows, device="cuda") if g is None else g).double()
    check(kept, ids, values, t, loss, lse, out, g)


@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 100, 511, 512, 513, 4096, 16384, 16391, 32000,
                                   50021, 130001])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_vocabularies(vocab, kind):
    run(5, vocab, 16, kind, t=2.0, seed=vocab)
    run(3, vocab, 33, kind, kind, seed=vocab, in_place=True)


@pytest.mark.parametrize("rows", [1, 2, 300, 5000])
def test_rows(rows):
    run(rows, 777, 8, "bf16", seed=rows, dloss=rows % 2 == 0)


# more entries than threads, and than the vocabulary: ids that occur often
@pytest.mark.parametrize("k", [1, 2, 31, 32, 64, 127, 511, 512, 513, 1024])
@pytest.mark.parametrize("vocab", [40, 5000])
def test_entries(k, vocab):
    run(20, vocab, k, "f32", t=0.7, seed=k)


@pytest.mark.parametrize("pad,at,out_at", [(8, 0, 0), (3, 1, 1), (0, 5, 5), (1, 0, 3), (8, 8, 4)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_strides_and_addresses(pad, at, out_at, kind):
    run(20, 1000, 10, kind, pad=pad, at=at, out_at=out_at)


def test_rows_without_entries():
    r, logits, ids, values = inputs(6, 1000, 8, "f32", absent=0.0)
    ids[0] = -1
    values[1] = -float("inf")       # entries of no weight are none
    values[2, :7] = -float("inf")   # one of weight 1
    values[3, 3] = -float("inf")
    ids[4, 1:] = -7
    logits[0, 5] = float("nan")
    with osr.distill_create(1000, 8) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values)
        dl = osr.distill_backward(ds, logits, ids, values, lse)
    assert loss[:2].tolist() == [0.0, 0.0] and not bool(dl[:2].any())
    one = torch.ones(5, device="cuda", dtype=torch.float64)
    check(logits[1:], ids[1:], values[1:], 1.0, loss[1:], lse[1:], dl[1:], one)


def test_an_id_past_the_vocabulary_shows():
    r, logits, ids, values = inputs(6, 1000, 8, "bf16")
    ids[2, 3], ids[4, 0] = 1000, 1 << 40
    with osr.distill_create(1000, 8) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values)
        dl = osr.distill_backward(ds, logits, ids, values, lse)
    assert loss.isnan().tolist() == dl.isnan().all(1).tolist() == [False, False, True, False, True,
                                                                   False]
    assert not bool(dl[[0, 1, 3, 5]].isnan().any())


def test_masked_logits_and_large_ones():
    # logits of -infinity have no share; values up to thousands do not overflow
    r, logits, ids, values = inputs(40, 3000, 20, "f32", spread=500.0)
    ids = ids.clamp(max=1499)
    logits[:, 1500:] = -float("inf")
    with osr.distill_create(3000, 20) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values)
        dl = osr.distill_backward(ds, logits, ids, values, lse)
    assert not bool(dl[:, 1500:].any())
    one = torch.ones(40, device="cuda", dtype=torch.float64)
    check(logits[:, :1500], ids, values, 1.0, loss, lse, dl[:, :1500], one)


def test_logits_far_below_zero():
    r, logits, ids, values = inputs(40, 3000, 20, "f32")
    logits -= 1000
    values -= 5000
    with osr.distill_create(3000, 20) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values)
        dl = osr.distill_backward(ds, logits, ids, values, lse)
    one = torch.ones(40, device="cuda", dtype=torch.float64)
    check(logits, ids, values, 1.0, loss, lse, dl, one)


def test_gradient_against_differences():
    r, logits, ids, values = inputs(20, 50, 6, "f32", spread=1.0)
    t = 1.5
    with osr.distill_create(50, 6) as ds:
        _, lse = osr.distill_forward(ds, logits, ids, values, temperature=t)
        dl = osr.distill_backward(ds, logits, ids, values, lse, temperature=t)
    q, log_q, _ = teacher(ids, values, t)

    def loss(x):
        log_p = torch.log_softmax(x / t, 1).gather(1, ids.clamp(min=0))
        return float(t * t * (q * (log_q - log_p)).sum())

    way = torch.randn(20, 50, device="cuda", generator=r, dtype=torch.float64)
    h = 1e-4
    slope = (loss(logits.double() + h * way) - loss(logits.double() - h * way)) / (2 * h)
    terms = float((dl.double() * way).abs().sum())
    # float32 of the gradient, and h^2 times a third derivative of about 1 a row
    assert abs(float((dl.double() * way).sum()) - slope) <= 2.0 ** -18 * terms + 1e-5


def test_the_same_bits_on_streams_and_in_graphs():
    r, logits, ids, values = inputs(100, 5003, 12, "bf16")
    with osr.distill_create(5003, 12) as ds:
        def step(stream=None):
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            loss, lse = osr.distill_forward(ds, logits, ids, values, stream=stream)
            return loss, lse, osr.distill_backward(ds, logits, ids, values, lse, stream=stream)

        first = step()
        torch.cuda.synchronize()
        both = [step(torch.cuda.Stream()) for _ in range(2)]
        torch.cuda.synchronize()
        for got in both:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for t in captured:
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, captured))


def test_no_rows_and_refusals():
    r, logits, ids, values = inputs(4, 64, 8, "bf16")
    with osr.distill_create(64, 8) as ds:
        loss, lse = osr.distill_forward(ds, logits[:0], ids[:0], values[:0])
        assert loss.shape == (0,)
        assert osr.distill_backward(ds, logits[:0], ids[:0], values[:0], lse).shape == (0, 64)
        loss, lse = osr.distill_forward(ds, logits, ids, values)
        for bad in (dict(logits=logits[:, :63]), dict(ids=ids.int()), dict(ids=ids[:, :7]),
                    dict(values=values[:3]), dict(values=values.double()), dict(temperature=0.0),
                    dict(temperature=-1.0), dict(temperature=float("nan")),
                    dict(temperature=1e-45), dict(loss=torch.empty(3, device="cuda")),
                    dict(ids=ids.cpu()), dict(loss=lse, lse=lse)):
            with pytest.raises((TypeError, ValueError, osr.AdamWError)):
                osr.distill_forward(ds, **{**dict(logits=logits, ids=ids, values=values), **bad})
        wide = torch.empty(4, 128, device="cuda", dtype=torch.bfloat16)
        for bad in (dict(lse=lse[:3]), dict(dlogits=logits.float()), dict(dloss=lse.double()),
                    dict(scale=float("inf")), dict(logits=wide[:, :64], dlogits=wide[:, 8:72])):
            with pytest.raises((TypeError, ValueError, osr.AdamWError)):
                osr.distill_backward(ds, **{**dict(logits=logits, ids=ids, values=values, lse=lse),
                                            **bad})
