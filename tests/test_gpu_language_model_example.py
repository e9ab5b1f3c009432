"""examples/language_model.py: it runs as written, and the gradients that its
passes add up, layer norm, linear layers, loss and distillation together, are
those of the same model by automatic differentiation in 64 bits."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
import optimizer_step_resumable_gb300 as osr  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = torch.nn.functional


@pytest.fixture(scope="module")
def example(lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location(
        "language_model", os.path.join(ROOT, "examples", "language_model.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_it_runs(example):
    told, heard = example.main(steps=4, dim=64, vocab=200, rows=256, k=8)
    assert all(0.0 <= x < float("inf") for x in told + heard)


def in_64_bits(model, tokens):
    """The weights as leaves, and the last norm's output."""
    w = [c.double().requires_grad_() for c in model.copy]
    x = w[0][tokens]
    for k in range(model.blocks):
        gain, shift, w1, b1, w2, b2 = w[1 + 6 * k:7 + 6 * k]
        y = F.layer_norm(x, (model.dim,), gain, shift)
        x = x + F.gelu(y @ w1 + b1) @ w2 + b2
    return w, F.layer_norm(x, (model.dim,), *w[-2:])


def compare(model, want):
    # bfloat16 between the layers: a value passes some 6 roundings a block and 4 at
    # the head, forward and backward, each 2^-8 of it at most and independent, and
    # the gradient's every factor errs by them: sqrt(2 * (6 * 2 + 4)) 2^-8 / sqrt(3)
    # = 1.3e-2 of the norm, taken twice for the slopes' own dependence on them
    for k, (got, w) in enumerate(zip(model.g, want)):
        off = float((got.double() - w).norm())
        assert off <= 2.6e-2 * float(w.norm()) + 1e-12, (k, off, float(w.norm()))


@pytest.mark.parametrize("rows", [77, 512])
def test_gradients_of_the_loss(example, rows):
    model = example.Model(300, 64, 2, seed=3)
    tokens, target = example.batch(300, rows, 1, 0)
    loss = model.learn(tokens, target)
    w, y = in_64_bits(model, tokens)
    full = F.cross_entropy(y @ w[0].T, target, reduction="none", ignore_index=-100)
    assert float((loss.double() - full.detach()).norm()) <= 2.6e-2 * float(full.detach().norm())
    compare(model, torch.autograd.grad(full.sum() / rows, w))
    model.close()


def test_gradients_of_the_distillation(example):
    model = example.Model(300, 64, 1, seed=4)
    tokens, _ = example.batch(300, 200, 2, 0)
    r = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.rand(200, 300, device="cuda", generator=r).topk(10, dim=1).indices
    ids[::7, 4:] = -1
    values = torch.randn(200, 10, device="cuda", generator=r)
    model.learn_from(tokens, ids, values, 2.0)
    w, y = in_64_bits(model, tokens)
    log_p = torch.log_softmax(y @ w[0].T / 2.0, 1).gather(1, ids.clamp(min=0))
    log_q = torch.log_softmax((values.double() / 2.0).masked_fill(ids < 0, -1e300), 1)
    loss = 4.0 * (log_q.exp() * (log_q - log_p)).masked_fill(ids < 0, 0.0).sum()
    compare(model, torch.autograd.grad(loss / 200, w))
    model.close()


def test_a_step_captured_and_replayed(example):
    # forward, loss, backward and the update in a graph, replayed: the same bits as
    # the steps one by one.  No token comes twice, as the order in which index_add_
    # would add its rows is not fixed
    tokens = torch.randperm(256, device="cuda")[:240]
    _, target = example.batch(256, 240, 1, 0)
    ran = []
    for captured in (False, True):
        model = example.Model(256, 64, 1, seed=6)

        def step():
            model.learn(tokens, target)
            osr.adamw_list_step(model.list, 1, lr=1e-3, wd=0.01, clip=1.0, zero_grad=True)

        if captured:
            start = [[x.clone() for x in model.w], [x.clone() for x in model.copy]]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):  # once outside the graph, then the weights back
                model.learn(tokens, target)
            torch.cuda.current_stream().wait_stream(side)
            for g in model.g:
                g.zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for now, was in zip((model.w, model.copy), start):
                for a, b in zip(now, was):
                    a.copy_(b)
            for _ in range(3):
                graph.replay()
        else:
            for _ in range(3):
                step()
        torch.cuda.synchronize()
        ran.append([x.clone() for x in model.w])
        model.close()
    for k, (a, b) in enumerate(zip(*ran)):
        assert torch.equal(a, b), k
