"""GPU: the training step of examples/train_step.py, every operator in its place."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "train_step.py")


def load():
    spec = importlib.util.spec_from_file_location("train_step", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("states", [8, 32])
def test_loss_falls(lib, states):
    """The goal vectors have unit variance, so the loss starts above 0.5 (its value for a zero
    output) and learning the commonest tokens takes it well below."""
    run = load().Training(states=states)
    losses = [float(run.step()) for _ in range(60)]
    assert all(torch.isfinite(torch.tensor(losses)))
    assert sum(losses[-5:]) / 5 < 0.5 * sum(losses[:5]) / 5


def test_own_experts_gradient(lib):
    """The block's dx against the double-precision derivative along one direction: bf16 rows,
    sums and products keep the two within a few percent."""
    m = load()
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, d, f, E, R = 128, 64, 64, 4, 2
    block = m.OwnExperts(T, d, f, E, R, gen)
    x = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    c = torch.randn(T, d, generator=gen, device="cuda").bfloat16()
    block.forward(x)
    dx = block.backward(c).double()
    slot_row, idx = block.slot_row.clone(), block.idx.long()

    def loss(z):        # the same routing, in 64 bits
        logits = z @ block.wg.double()
        w = torch.softmax(torch.gather(logits, 1, idx), 1)
        out = z.clone()
        for r in range(R):
            e = idx[:, r]
            h = torch.relu(torch.einsum("td,tdf->tf", z, block.A[e].double())) ** 2
            y = torch.einsum("tf,tfd->td", h, block.B[e].double())
            out = out + torch.where(slot_row[:, r, None] >= 0, w[:, r, None] * y, 0.0)
        return (out * c.double()).sum()

    z = x.double().requires_grad_(True)
    loss(z).backward()
    err = (dx - z.grad).norm() / z.grad.norm()
    assert float(err) < 0.03
