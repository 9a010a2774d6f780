"""examples/policy_step.py on the GPU: the rollout's log-probabilities are the trainer's, bit
for bit, so no token is cut off and the policy loss is minus the mean advantage; every gradient
is finite, not zero, and the same on every run."""

import importlib.util
import os

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def step():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "policy_step.py")
    spec = importlib.util.spec_from_file_location("policy_step", path)
    module = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["policy_step"] = module
    spec.loader.exec_module(module)
    return module


def test_rollout_and_trainer_agree(step):
    policy = step.Policy.random(0, DEV)
    tokens, old = step.rollout(policy, 5, 40, 1, DEV)
    adv = torch.tensor([1.0, -0.5, 2.0, 0.25, -1.5], device=DEV)
    stats, logp, grads = step.train_step(policy, tokens, old, adv, prompt=3)
    torch.cuda.synchronize()
    assert torch.equal(logp.view(torch.int32), old.view(torch.int32))
    assert float(stats[4]) == 0.0
    # ratios of exactly 1, sequences of equal weight: minus the mean advantage, rounded once
    assert abs(float(stats[1]) + float(adv.double().mean())) <= 2.0 ** -24
    assert set(grads) == {"dq", "dk", "dv", "da", "db", "dS0", "norm_weight", "norm_bias"}
    for name, g in grads.items():
        assert bool(torch.isfinite(g).all()) and float(g.abs().max()) > 0.0, name
    again = step.train_step(policy, tokens, old, adv, prompt=3)[2]
    for name, g in grads.items():
        assert torch.equal(g, again[name]), name


def test_main_prints_agreement(step, capsys):
    step.main()
    out = capsys.readouterr().out
    assert "the same bits" in out and "DIFFER" not in out
