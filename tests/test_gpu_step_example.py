"""examples/policy_update.py on the GPU: rollout and trainer agree on every log-probability bit for
bit, before and after an update; the projection's gradient is the product of the logits' gradient
and the norm's outputs up to their rounding to 8 bits; an update moves every weight as its states
say, the same on every run."""

import os
import sys

import pytest
import torch

from bitwise_consistent_linear_amd import api
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples")
    sys.path.insert(0, path)
    try:
        import policy_update
    finally:
        sys.path.remove(path)
    return policy_update


def one_step(example, policy, optimiser, seed):
    policy.ready()
    tokens, old = example.rollout(policy, 5, 33, seed, DEV)
    adv = torch.tensor([1.0, -0.5, 2.0, 0.25, -1.5], device=DEV)
    _, logp, grads = example.train_step(policy, tokens, old, adv, prompt=3)
    assert torch.equal(logp.view(torch.int32), old.view(torch.int32))
    norm = optimiser.step([[policy.d_w], [grads["norm_weight"], grads["norm_bias"]]])
    return tokens, grads, norm


def test_steps(example):
    runs = []
    for _ in range(2):
        policy = example.Projection.random(0, DEV)
        before = [policy.w.clone(), policy.norm_weight.clone(), policy.norm_bias.clone()]
        optimiser = example.Optimiser([policy.w, policy.norm_weight, policy.norm_bias])
        for seed in (1, 2):
            tokens, grads, norm = one_step(example, policy, optimiser, seed)
            assert bool(((tokens >= 0) & (tokens < example.VOCAB)).all())
            assert float(norm) > 0
            for g in (policy.d_w, grads["norm_weight"], grads["norm_bias"]):
                assert bool(torch.isfinite(g).all()) and float(g.abs().max()) > 0
        after = [policy.w, policy.norm_weight, policy.norm_bias]
        for a, b in zip(after, before):
            assert not torch.equal(a, b) and bool(torch.isfinite(a).all())
        runs.append([t.clone() for t in after] + [tokens, norm])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_projection_gradient(example):
    """d_w against binary64: an e4m3 value is within 2^-4 of the norm's output, an e5m2 value
    within 2^-3 of the logits' gradient, or half a step of the lowest of its block (2^-10 / 448 and
    2^-17 / 57344 of the block's largest), which adds less than 0.01 of the largest products."""
    policy = example.Projection.random(3, DEV)
    policy.ready()
    g = torch.Generator(device=DEV).manual_seed(4)
    o = torch.randn(200, example.HV, example.D_HEAD, generator=g, device=DEV)
    logits, saved = policy.head(o)
    d = torch.randn(logits.shape, generator=g, device=DEV).bfloat16()
    d_h, d_gamma, d_beta = policy.head_bwd(d, saved)
    y = api.layer_norm_fwd(saved[0], policy.norm_weight, policy.norm_bias)[0].double().cpu()
    dd = d.double().cpu()
    want, size = dd.t() @ y, dd.abs().t() @ y.abs()
    bound = (2.0 ** -4 + 2.0 ** -3 + 2.0 ** -7) * size + 0.01 * float(dd.abs().max() * y.abs().max())
    assert bool(((policy.d_w.double().cpu() - want).abs() <= bound).all())
    for t in (d_h, d_gamma, d_beta):
        assert bool(torch.isfinite(t).all())


def test_main(example, capsys):
    example.main(2)
    out = capsys.readouterr().out
    assert out.count("the same bits") == 2 and "DIFFER" not in out
