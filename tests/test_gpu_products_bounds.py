"""What the linear layer, the cross entropy and the distillation write: their
outputs and nothing else, within the workspace they ask for; and places more than
2^31 elements into an array."""
import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(autouse=True)
def _lib(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class Guarded:
    """Matrices within buffers of a pattern, which has to survive around them."""

    def __init__(self):
        self.held = []

    def matrix(self, rows, cols, kind, pad=0, at=0):
        size = 2 if kind != "f32" else 4
        lead = 64 + at
        n = lead + rows * (cols + pad) + 64
        raw = torch.full((n * size,), 0x5A, device="cuda", dtype=torch.uint8)
        flat = raw.view(TYPES[kind])
        view = flat[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        self.held.append((raw, view))
        return view

    def memory(self, need):
        raw = torch.full((need + 4096,), 0x5A, device="cuda", dtype=torch.uint8)
        self.held.append((raw, raw[:need]))
        return raw[:need]

    def check(self):
        for raw, view in self.held:
            # what is not the matrix is still the pattern
            if view.dtype is torch.uint8:
                view.fill_(0x5A)
            else:
                bits = torch.int16 if view.element_size() == 2 else torch.int32
                view.view(bits).fill_(0x5A5A if bits is torch.int16 else 0x5A5A5A5A)
            assert bool((raw == 0x5A).all())


SHAPES = [(1, 64, 64), (2, 768, 96), (3, 65, 33), (9, 128, 200), (40, 72, 520), (130, 67, 131),
          (257, 200, 777), (300, 1021, 509), (700, 136, 768), (1500, 64, 40)]


@pytest.mark.parametrize("rows,cin,cout", SHAPES)
@pytest.mark.parametrize("pad,at,kind", [(0, 0, "bf16"), (8, 16, "f16"), (3, 5, "bf16")])
@pytest.mark.parametrize("in_out", [False, True])
def test_linear_writes_its_outputs_only(rows, cin, cout, pad, at, kind, in_out):
    g = Guarded()
    x, dy = (torch.randn(rows, n, device="cuda").to(TYPES[kind]) for n in (cin, cout))
    w = torch.randn(cin, cout, device="cuda").to(TYPES[kind]).T if in_out else \
        torch.randn(cout, cin, device="cuda").to(TYPES[kind])
    y, z = g.matrix(rows, cout, kind, pad, at), g.matrix(rows, cout, kind, pad, at)
    dx = g.matrix(rows, cin, kind, pad, at)
    dw = g.matrix(cin, cout, "f32", pad, at).T if in_out else g.matrix(cout, cin, "f32", pad, at)
    db = g.matrix(1, cout, "f32")[0]
    any_address = osr.LINEAR_FOR_ANY_ADDRESS
    with osr.linear_create(cin, cout) as lin:
        osr.linear_forward(lin, x, w, activation="gelu", y=y, z=z,
                           workspace=g.memory(osr.linear_workspace(lin, rows, any_address)))
        osr.linear_backward(lin, dy, x, w, z=dy, activation="gelu", dx=dx, dweight=dw, dbias=db,
                            workspace=g.memory(osr.linear_workspace(
                                lin, rows, any_address | osr.LINEAR_FOR_BACKWARD)))
    torch.cuda.synchronize()
    g.check()


@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
@pytest.mark.parametrize("pad,at,kind", [(0, 0, "bf16"), (3, 5, "f16")])
def test_losses_write_their_outputs_only(rows, dim, vocab, pad, at, kind):
    g = Guarded()
    x = torch.randn(rows, dim, device="cuda").to(TYPES[kind])
    w = torch.randn(vocab, dim, device="cuda").to(TYPES[kind])
    target = torch.randint(0, vocab, (rows,), device="cuda")
    loss, lse = g.matrix(1, rows, "f32")[0], g.matrix(1, rows, "f32")[0]
    dx, dw = g.matrix(rows, dim, kind, pad, at), g.matrix(vocab, dim, kind, pad, at)
    any_address = osr.LINEAR_FOR_ANY_ADDRESS
    with osr.linear_cross_entropy_create(dim, vocab) as ce:
        osr.linear_cross_entropy_forward(
            ce, x, w, target, loss=loss, lse=lse,
            workspace=g.memory(osr.linear_cross_entropy_workspace(ce, rows, any_address)))
        osr.linear_cross_entropy_backward(
            ce, x, w, target, lse, dx=dx, dweight=dw,
            workspace=g.memory(osr.linear_cross_entropy_workspace(
                ce, rows, any_address | osr.LINEAR_FOR_BACKWARD)))
    logits = torch.randn(rows, vocab, device="cuda").to(TYPES[kind])
    ids = torch.randint(-1, vocab, (rows, 7), device="cuda")
    values = torch.randn(rows, 7, device="cuda")
    dl = g.matrix(rows, vocab, kind, pad, at)
    loss2, lse2 = g.matrix(1, rows, "f32")[0], g.matrix(1, rows, "f32")[0]
    with osr.distill_create(vocab, 7) as ds:
        osr.distill_forward(ds, logits, ids, values, loss=loss2, lse=lse2)
        osr.distill_backward(ds, logits, ids, values, lse2, dlogits=dl)
    torch.cuda.synchronize()
    g.check()


def test_places_beyond_32_bits():
    # 280,000 x 8192 outputs and 70,000 x 32,000 logits: the last rows, and some
    # before them, against small calls on the same inputs, bit for bit where tiles
    # meet the same rows
    rows, cin, cout = 280_000, 64, 8192
    x = torch.randn(rows, cin, device="cuda").bfloat16()
    w = torch.randn(cout, cin, device="cuda").bfloat16()
    with osr.linear_create(cin, cout) as lin:
        y = osr.linear_forward(lin, x, w)
        for first in (0, 262_143, rows - 4096):
            assert torch.equal(y[first:first + 4096], osr.linear_forward(lin, x[first:first + 4096], w))
        dx, _, _ = osr.linear_backward(lin, y, x, w)
        want = y[-300:].double() @ w.double()
        # bfloat16 outputs; float32 sums of 8192 terms are 2^-11 of that apart
        assert float((dx[-300:].double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
        del dx
    del y
    rows, vocab, k = 70_000, 32_000, 4
    logits = torch.randn(rows, vocab, device="cuda", dtype=torch.bfloat16)
    ids = torch.randint(0, vocab, (rows, k), device="cuda")
    values = torch.randn(rows, k, device="cuda")
    with osr.distill_create(vocab, k) as ds:
        loss, lse = osr.distill_forward(ds, logits, ids, values)
        dl = osr.distill_backward(ds, logits, ids, values, lse)
        for first in (0, 67_108, rows - 50):
            part = slice(first, first + 50)
            l2, s2 = osr.distill_forward(ds, logits[part], ids[part], values[part])
            d2 = osr.distill_backward(ds, logits[part], ids[part], values[part], s2)
            assert torch.equal(loss[part], l2) and torch.equal(lse[part], s2)
            assert torch.equal(dl[part], d2)
