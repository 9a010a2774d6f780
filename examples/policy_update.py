"""On-policy training steps that move weights: what policy_step.py does, with tokens drawn by the
library, a vocabulary projection in 8-bit floating point whose gradients are 8-bit products too, and
an AdamW update with 8-bit states behind a clipped gradient norm.

Each step rolls out tokens with the weights of the moment (temperature and top-p), recomputes
their log-probabilities in the trainer's packed batch, which agree bit for bit, forms the clipped
loss and updates the projection and the norm. Nothing of a step waits for the host.

    python examples/policy_update.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from policy_step import CHUNK, D_HEAD, HV, SCALE, VOCAB, WIDTH, Policy, train_step  # noqa: E402
from bitwise_consistent_linear_amd import api  # noqa: E402

TOP_P = 0.95


class Projection(Policy):
    """The policy with its projection held in bfloat16 and used in 8-bit floating point."""

    def ready(self):
        """What a step needs of the weights in 8 bits: by rows forward, by columns backward."""
        self.wq, self.w_scale, self.wtq, self.wt_scale = api.quantize_f8(self.w, layout="both")

    def head(self, o):
        h = o.reshape(-1, WIDTH)
        y, mean, rstd = api.layer_norm_fwd(h, self.norm_weight, self.norm_bias)
        xq, x_scale, xtq, xt_scale = api.quantize_f8(y, layout="both")
        logits = api.linear_f8_fwd(xq, x_scale, self.wq, self.w_scale, out_dtype=torch.bfloat16)
        return logits, (h, mean, rstd, xtq, xt_scale)

    def head_bwd(self, d_logits, saved):
        h, mean, rstd, xtq, xt_scale = saved
        d_y, self.d_w = api.linear_f8_bwd(d_logits, self.wtq, self.wt_scale, xtq, xt_scale,
                                          fmt="e5m2", dx_dtype=torch.float32)
        return api.layer_norm_bwd(d_y, h, self.norm_weight, mean, rstd)


class Optimiser:
    """AdamW over bfloat16 and float32 parameters, states in 8 bits: a list for each type."""

    def __init__(self, params, lr=1e-2, max_norm=1.0):
        self.lists = [[p for p in params if p.dtype is t] for t in (torch.bfloat16, torch.float32)]
        self.states = [self.zeros(ps) for ps in self.lists]
        self.lr, self.max_norm, self.t = lr, max_norm, 0

    @staticmethod
    def zeros(params):
        def codes(dtype):
            return [torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(dtype)
                    for p in params]

        def scales():
            return [torch.zeros(-(-p.numel() // api.ADAMW_BLOCK), device=p.device) for p in params]

        return codes(torch.float8_e4m3fn), codes(torch.uint8), scales(), scales()

    def step(self, grads):
        """grads: float32, in the order of the parameters' lists. Returns their norm [1]."""
        self.t += 1
        norm, factor = api.grad_norm([g for gs in grads for g in gs], max_norm=self.max_norm)
        for ps, gs, (m, v, m_scale, v_scale) in zip(self.lists, grads, self.states):
            api.adamw_step(ps, gs, m, v, self.t, m_scale=m_scale, v_scale=v_scale, lr=self.lr,
                           weight_decay=0.0, grad_scale=factor)
        return norm


def rollout(policy, n, steps, seed, device):
    """As policy_step.rollout, tokens drawn by the library: tokens [n, steps + 1] and the
    log-probabilities [n, steps] of all but the first."""
    gen = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (n, 1), generator=gen, device=device)
    u = torch.rand((steps, n), generator=gen, device=device)
    state = torch.zeros((n, HV, D_HEAD, D_HEAD), device=device)
    logps = []
    for t in range(steps):
        q, k, v, a, b = policy.inputs(tokens[:, -1])
        pos = torch.full((n,), t, dtype=torch.int32, device=device)
        logits, _ = policy.head(api.decode_step(pos, q, k, v, a, b, state, chunk=CHUNK))
        token, _ = api.sample_tokens(logits, u[t], temperature=1 / SCALE, top_p=TOP_P)
        logp, _, _ = api.token_logprob_fwd(logits, token, scale=SCALE)
        logps.append(logp)
        tokens = torch.cat([tokens, token[:, None]], 1)
    return tokens, torch.stack(logps, 1)


def main(steps=3):
    dev = torch.device("cuda:0")
    policy = Projection.random(0, dev)
    optimiser = Optimiser([policy.w, policy.norm_weight, policy.norm_bias])
    for i in range(steps):
        policy.ready()
        tokens, old_logp = rollout(policy, 8, 48, i, dev)
        advantages = torch.randn(8, generator=torch.Generator().manual_seed(i)).to(dev)
        stats, logp, grads = train_step(policy, tokens, old_logp, advantages)
        norm = optimiser.step([[policy.d_w], [grads["norm_weight"], grads["norm_bias"]]])
        same = torch.equal(logp.view(torch.int32), old_logp.view(torch.int32))
        print(f"step {i}: log-probabilities {'the same bits' if same else 'DIFFER'}, loss "
              f"{stats[0].item():.4f}, entropy {stats[3].item():.4f}, |gradient| {norm.item():.4g}")


if __name__ == "__main__":
    main()
