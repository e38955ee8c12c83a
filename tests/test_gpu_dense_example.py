"""The example training program: its gradients against autograd, and that it learns with either form of AdamW's states."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")


def load():
    spec = importlib.util.spec_from_file_location("train_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_of_a_step_are_autograds():
    """The dense gradients that a step leaves, against autograd in 64 bits over the same pooled rows.  Each is a product in
    fp32 of at most 1024 rows or 256 columns of values that carry fp32 rounding: 1e-4 of the gradient's largest value
    is above 1024 * 2^-24 of the sums' sizes."""
    m = load()
    model = m.Model()
    ids, clicks = model.batch()
    pooled = model.tbe.forward(model.tables, ids, model.offsets).double()
    params = [p.double().requires_grad_() for p in model.params]
    w1, w2, gain, shift, b1, b2 = params
    parts = []
    at = 0
    for d in m.D:
        parts.append(torch.nn.functional.layer_norm(pooled[:, at:at + d], (d,), gain[at:at + d], shift[at:at + d], 1e-5))
        at += d
    logit = (torch.relu(torch.cat(parts, 1) @ w1 + b1) @ w2 + b2).squeeze(1)
    loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, clicks.double())
    loss.backward()
    got = model.step(ids, clicks, 1e-3)
    assert abs(float(got) - float(loss)) <= 1e-5 * float(loss)
    for g, p in zip(model.grads, params):
        assert float((g.double() - p.grad).abs().max()) <= 1e-4 * float(p.grad.abs().max())


@pytest.mark.parametrize("states", ["f32", "q8"])
def test_it_learns(states):
    m = load()
    model = m.Model(states)
    losses = torch.stack([model.step(*model.batch(), lr=3e-3) for _ in range(200)])
    assert float(losses[-20:].mean()) < 0.9 * float(losses[:20].mean())
