"""The example's reinforcement-learning step on the GPU: the rollout over the
paged FP8 cache agrees with the training forward, the gradients reach the
last layer's norms, and the step repeats bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def step(torch_cuda):
    from examples import rl_step
    return rl_step, rl_step.rl_step()


def test_rollout_and_training_agree(step):
    """The two passes differ by the FP8 keys and values alone (3-bit mantissas:
    2^-4 at most an entry); a wrong slot, position or token gives unrelated
    logits, whose metric over 2048 tokens is far above 1.5."""
    mod, r = step
    assert 1.0 <= r["metric"] < 1.5
    assert all(s.numel() <= mod.WIDTH * mod.BLOCK for s in r["sequences"])
    assert torch.isfinite(r["logp_rollout"]).all() and (r["logp_rollout"] <= 0).all()
    gap = (r["logp_train"] - r["logp_rollout"].flatten()).abs()
    assert float(gap.median()) < 0.25


def test_gradients_are_finite_and_reach_every_token(step):
    mod, r = step
    for n, t in r["grads"].items():
        assert torch.isfinite(t).all() and float(t.float().norm()) > 0, n
    assert r["grads"]["norm1"].shape == (mod.HIDDEN,)


def test_repeatable(step):
    mod, r = step
    again = mod.rl_step()
    assert again["metric"] == r["metric"]
    assert all(torch.equal(a, b) for a, b in zip(again["sequences"], r["sequences"]))
    assert torch.equal(again["grads"]["norm2"], r["grads"]["norm2"])
