"""The new operators together: a training step of a small FP8 language model
against torch's autograd in float32, and a few steps of training."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ts():
    from fp8_block_scaled_05_amd import train_step
    return train_step


def reference(cfg, p, tokens, target):
    p = {k: v.detach().clone().requires_grad_(True) for k, v in p.items()}
    x = p["embedding"][tokens]
    for i in range(cfg.layers):
        h = torch.nn.functional.gelu(x @ p[f"up{i}"].t() + p[f"up_bias{i}"], approximate="tanh")
        x = x + h @ p[f"down{i}"].t() + p[f"down_bias{i}"]
    loss = torch.nn.functional.cross_entropy(x @ p["head"].t(), target)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p.items()}


def test_gradients_follow_autograd(ts):
    """E4M3 operands keep three mantissa bits: an element is off by at most
    2^-4, by 2^-4 / sqrt(3) in the root mean square over a binade's worst half,
    and a product's two operands and the layer's chain of four products and z
    make at most five such independent relative errors: 5^(1/2) 2^-4 / 3^(1/2)
    = 0.081 of the gradient's norm, so the angle's cosine is above 1 - 0.081^2.
    The head's, with bf16 operands, sees the hidden states' two products."""
    cfg = ts.Config()
    p = ts.init(cfg)
    tokens, target = ts.batch(cfg, 700, 3)
    loss, grads = ts.loss_and_grads(cfg, p, tokens, target)
    want, ref = reference(cfg, p, tokens, target)
    assert abs(loss.item() - want) < 0.081 * want
    assert set(grads) == set(ref)
    for k in ref:
        a, b = grads[k].double().flatten(), ref[k].double().flatten()
        cos = float(a @ b / (a.norm() * b.norm()))
        assert cos > 1 - 0.081 ** 2, (k, cos)
        assert abs(float(a.norm() / b.norm()) - 1) < 0.081, k


def test_training_lowers_the_loss(ts):
    """From about log(vocab) + the logits' spread to a tenth of it: the task is
    a lookup."""
    cfg = ts.Config(vocab=200, layers=1)
    p, state = ts.init(cfg), {}
    losses = []
    for step in range(40):
        loss, grads = ts.loss_and_grads(cfg, p, *ts.batch(cfg, 500, step))
        ts.update(p, grads, state, 0.01)
        losses.append(loss.item())
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < losses[0] / 10
