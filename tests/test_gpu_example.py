"""The example that runs the operators together: graph replays of the serving stack equal the
eager step bit for bit, and the training steps lower the loss."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    from examples import decoder_block


def test_serving_stack_replays_like_the_eager_step():
    replayed, eager = decoder_block.serve(tokens=5, hidden=512, inter=256, experts=6, top_k=2, layers=2, steps=4)
    assert torch.equal(replayed, eager) and bool(torch.isfinite(eager).all())


def test_training_steps_lower_the_loss():
    losses = decoder_block.train(tokens=256, hidden=512, out=256, steps=12)
    assert losses[-1] < 0.9 * losses[0], losses
