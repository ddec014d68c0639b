"""The adapter example: trainer, patch and sampler together."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss_and_the_sampler_follows():
    from examples import adapter_step

    losses, shares, same = adapter_step.run(steps=12)
    assert same
    assert losses[-1] < 0.9 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
    assert all(0 < s <= 1 for s in shares)
    torch.cuda.synchronize()
