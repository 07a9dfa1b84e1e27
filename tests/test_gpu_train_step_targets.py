"""The training step's mean loss over targets that carry one."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_targets_outside_the_vocabulary():
    """A position without a loss is one whatever its target says: ignore_index,
    negative, or past the vocabulary."""
    from fp8_block_scaled_05_amd import train_step as ts
    cfg = ts.Config()
    p = ts.init(cfg)
    tokens, target = ts.batch(cfg, 300, 5)
    other = target.clone()
    none = torch.nonzero(target == -100)[:, 0]
    other[none[::2]] = cfg.vocab
    other[none[1::3]] = -7
    loss, grads = ts.loss_and_grads(cfg, p, tokens, target)
    loss2, grads2 = ts.loss_and_grads(cfg, p, tokens, other)
    assert torch.equal(loss, loss2)
    for k in grads:
        assert torch.equal(grads[k], grads2[k]) or k == "embedding", k
    # index_add_ on the GPU adds in any order: FP32 sums of at most 300 rows
    a, b = grads["embedding"], grads2["embedding"]
    assert torch.all((a - b).abs() <= 300 * 2.0 ** -23 * a.abs().max())
