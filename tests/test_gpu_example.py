"""The example's training step: the loss falls, and a step with a gradient
that is not finite leaves every weight and state alone."""
import math
import os
import sys

import pytest
import torch

from gpu_common import need_gpu, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_loss_falls():
    need_gpu()
    import train_step
    say("example: 60 steps")
    losses, norms = train_step.train(60, log=say)
    assert torch.isfinite(losses).all() and torch.isfinite(norms).all()
    # from guessing among 256 tokens to well below
    assert float(losses[:3].mean()) > 0.9 * math.log(256)
    assert float(losses[-5:].mean()) < 0.75 * float(losses[:3].mean())


def test_step_with_nan_changes_nothing():
    need_gpu()
    import train_step
    model = train_step.Model(torch.Generator().manual_seed(1)).cuda()
    trainer = train_step.Trainer(model)
    trainer.G.normal_(0, 1e-3)
    trainer.flat_rest.normal_(0, 1e-3)
    say("example: one step, then one with a NaN")
    trainer.step()
    held = [trainer.W, trainer.M, trainer.v] + [t for a in trainer.adamw.tensors[1:] for t in a] + trainer.matrices
    before = [t.detach().clone() for t in held]
    trainer.G[3, 7, 11] = math.nan
    got = trainer.step()
    assert math.isnan(float(got.norm)) and math.isnan(float(got.clip))
    for a, b in zip(held, before):
        assert torch.equal(a.detach(), b)
