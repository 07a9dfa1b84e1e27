"""A training step of the language model of pre-norm gated blocks: the norm, the
gated product, their backward passes and the head together, against torch's
autograd in float32."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ts():
    from fp8_block_scaled_05_amd import train_step
    return train_step


def norm(x, g):
    return x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + 1e-6) * g


def reference(cfg, p, tokens, target):
    p = {k: v.detach().clone().requires_grad_(True) for k, v in p.items()}
    act = torch.nn.functional.silu
    if cfg.act == "gelu":
        act = lambda v: torch.nn.functional.gelu(v, approximate="tanh")
    x = p["embedding"][tokens]
    for i in range(cfg.layers):
        gate, up = (norm(x, p[f"norm{i}"]) @ p[f"up{i}"].t()).split(cfg.inner, dim=1)
        x = x + (act(gate) * up) @ p[f"down{i}"].t()
    loss = torch.nn.functional.cross_entropy(norm(x, p["norm"]) @ p["head"].t(), target)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,layers", [(700, 2), (50, 1)])
def test_gradients_follow_autograd(ts, act, rows, layers):
    """An E4M3 operand's element is off by at most 2^-4, by 2^-4 / sqrt(3) in the
    root mean square over a binade's worst half.  A gradient's chain holds at most
    eight such independent relative errors (two operands of its own product, two
    of each of gate and up, and two of the products behind): 8^(1/2) 2^-4 /
    3^(1/2) = 0.102 of its norm, so the angle's cosine is above 1 - 0.102^2."""
    cfg = ts.Config(block="gated", act=act, layers=layers)
    p = ts.init(cfg)
    for k in p:
        if k.startswith("norm"):
            p[k] += 0.1 * torch.randn_like(p[k])
    tokens, target = ts.batch(cfg, rows, 3)
    loss, grads = ts.loss_and_grads(cfg, p, tokens, target)
    want, ref = reference(cfg, p, tokens, target)
    assert abs(loss.item() - want) < 0.102 * want
    assert set(grads) == set(ref)
    for k in ref:
        a, b = grads[k].double().flatten(), ref[k].double().flatten()
        cos = float(a @ b / (a.norm() * b.norm()))
        assert cos > 1 - 0.102 ** 2, (k, cos)
        assert abs(float(a.norm() / b.norm()) - 1) < 0.102, k


def test_training_steps_run(ts):
    cfg = ts.Config(vocab=200, layers=1, block="gated", act="silu")
    p, state = ts.init(cfg), {}
    for step in range(3):
        loss, grads = ts.loss_and_grads(cfg, p, *ts.batch(cfg, 300, step))
        ts.update(p, grads, state, 0.01)
        assert math.isfinite(loss.item())
        assert all(bool(torch.isfinite(v).all()) for v in p.values())


def test_unknown_block(ts):
    with pytest.raises(ValueError, match="block must be"):
        ts.init(ts.Config(block="moe"))
