"""The example model trains and decodes on the library's layers.  Needs an
MI355X; marked ``gpu``."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_lm.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("recurrent_lm", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_lowers_the_loss(example, dev, dtype):
    """The sequences repeat after four tokens, so that most of the loss of a
    uniform guess can be learned."""
    torch.manual_seed(0)
    model = example.RecurrentLM(17, 64, 96, 2, dtype).to(dev)
    losses = example.train(model, 200, 8, 64, 17, dev)
    assert losses[-1] < 0.6 * losses[0], (losses[0], losses[-1])


def test_steps_equal_the_whole_sequence(example, dev):
    """Token by token on the recurrent states against all tokens at once: in
    float32 the two differ by the order of sums of at most a few hundred terms,
    far below 1e-4 of values near one."""
    torch.manual_seed(1)
    model = example.RecurrentLM(31, 48, 80, 2, torch.float32).to(dev)
    tokens = torch.randint(0, 31, (3, 40), device=dev)
    with torch.no_grad():
        whole = model.hidden(tokens)
    states = model.states(3)
    for t in range(tokens.shape[1]):
        got = model.step(tokens[:, t], states)
        assert (got - whole[:, t]).abs().max() < 1e-4, t
    assert model.generate(tokens, 5).shape == (3, 5)


def test_loss_gradient_is_the_difference_quotient(example, dev):
    """Through embedding, norms, recurrences and loss: the derivative along a
    direction against a central difference at step 1e-2, whose error is the
    float32 loss's 1e-6 over the step and the third derivative times 1e-4."""
    torch.manual_seed(2)
    model = example.RecurrentLM(23, 40, 64, 2, torch.float32).to(dev)
    tokens = torch.randint(0, 23, (4, 30), device=dev)
    params = list(model.parameters())
    direction = [torch.randn_like(p) * p.detach().abs().mean() for p in params]
    size = sum(d.square().sum() for d in direction).sqrt()
    direction = [d / size for d in direction]
    loss = model.loss(tokens)
    grads = torch.autograd.grad(loss, params)
    slope = sum((g * d).sum() for g, d in zip(grads, direction)).item()

    def at(step):
        with torch.no_grad():
            for p, d in zip(params, direction):
                p.add_(d, alpha=step)
            value = model.loss(tokens).item()
            for p, d in zip(params, direction):
                p.sub_(d, alpha=step)
        return value

    quotient = (at(1e-2) - at(-1e-2)) / 2e-2
    norm = sum(g.square().sum() for g in grads).sqrt().item()
    assert abs(slope - quotient) < 1e-3 * norm + 1e-3 * abs(slope), (slope, quotient, norm)
