"""One step of on-policy training with a gated delta rule layer and its policy head.

A rollout samples tokens one at a time (engine_decode, then the head), a trainer recomputes
their log-probabilities over the packed batch (trainer_fwd, then the same head), forms the
clipped policy loss and takes its gradient back to the layer's inputs. Rollout and trainer
agree bit for bit on every token's log-probability: the layer by its contract, the head since
each of its rows depends on that row alone. So the first step's ratios are exactly 1.

The head: norm of the layer's output, 8-bit vocabulary projection, log-probability of the
chosen token. Its projection's gradient passes straight through the quantisation, with the
weights as the 8-bit product sees them.

    python examples/policy_step.py
"""

import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bitwise_consistent_linear_amd import api  # noqa: E402

HK, HV, D_HEAD, CHUNK = 2, 4, 64, 16
VOCAB, WIDTH = 1024, HV * D_HEAD
SCALE = 1.25  # inverse sampling temperature


@dataclass
class Policy:
    """Tables that give a token's q, k, v, decay and write strength, and the head's weights."""

    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    a: torch.Tensor
    b: torch.Tensor
    norm_weight: torch.Tensor
    norm_bias: torch.Tensor
    wq: torch.Tensor        # int8 [VOCAB, WIDTH], laid out once
    w_scale: torch.Tensor
    w: torch.Tensor         # the same weights in bfloat16, for the gradient

    @classmethod
    def random(cls, seed, device):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=gen, device=device)

        def uniform(*shape):
            return torch.rand(shape, generator=gen, device=device)

        k = normal(VOCAB, HK, D_HEAD)
        wq, w_scale = api.quantize_rows(normal(VOCAB, WIDTH) * (1.5 / WIDTH ** 0.5))
        return cls(normal(VOCAB, HK, D_HEAD).bfloat16(),
                   (k / k.norm(dim=2, keepdim=True)).bfloat16(),
                   normal(VOCAB, HV, D_HEAD).bfloat16(), 0.9 + 0.1 * uniform(VOCAB, HV),
                   uniform(VOCAB, HV), 1.0 + 0.1 * normal(WIDTH), 0.1 * normal(WIDTH), wq,
                   w_scale, (wq[:, :WIDTH].float() * w_scale[:, None]).bfloat16())

    def inputs(self, tokens):
        return [t[tokens].contiguous() for t in (self.q, self.k, self.v, self.a, self.b)]

    def head(self, o):
        """Logits of layer outputs o [M, HV, D_HEAD], and what the gradient needs."""
        h = o.reshape(-1, WIDTH)
        y, mean, rstd = api.layer_norm_fwd(h, self.norm_weight, self.norm_bias)
        xq, x_scale = api.quantize_rows(y)
        logits = api.linear_i8_fwd(xq, x_scale, self.wq, self.w_scale, out_dtype=torch.bfloat16)
        return logits, (h, mean, rstd)

    def head_bwd(self, d_logits, saved):
        h, mean, rstd = saved
        d_y = api.linear_fwd(d_logits, self.w)
        return api.layer_norm_bwd(d_y, h, self.norm_weight, mean, rstd)


def rollout(policy, n, steps, seed, device):
    """Samples `steps` tokens for each of n sequences. Returns tokens [n, steps + 1] and the
    log-probabilities [n, steps] of all but the first."""
    gen = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (n, 1), generator=gen, device=device)
    state = torch.zeros((n, HV, D_HEAD, D_HEAD), device=device)
    logps = []
    for t in range(steps):
        q, k, v, a, b = policy.inputs(tokens[:, -1])
        pos = torch.full((n,), t, dtype=torch.int32, device=device)
        logits, _ = policy.head(api.decode_step(pos, q, k, v, a, b, state, chunk=CHUNK))
        u = torch.rand((n, VOCAB), generator=gen, device=device).clamp_(1e-30, 1.0 - 1e-7)
        token = (SCALE * logits.float() - torch.log(-torch.log(u))).argmax(1)
        logp, _, _ = api.token_logprob_fwd(logits, token, scale=SCALE)
        logps.append(logp)
        tokens = torch.cat([tokens, token[:, None]], 1)
    return tokens, torch.stack(logps, 1)


def train_step(policy, tokens, old_logp, advantages, prompt=4, clip=0.2, entropy_coef=0.001):
    """The loss of sampled tokens [n, steps + 1] and its gradient with respect to the layer's
    inputs and the norm's parameters; the first `prompt` tokens are not scored. Returns
    (stats [5], log-probabilities [n, steps], gradients)."""
    n, steps = old_logp.shape
    dev = tokens.device
    cu = torch.arange(0, (n + 1) * steps, steps, dtype=torch.int32, device=dev)
    q, k, v, a, b = policy.inputs(tokens[:, :-1].reshape(-1))
    target = tokens[:, 1:].reshape(-1).contiguous()
    o, chunk_states = api.trainer_fwd(cu, q, k, v, a, b, chunk=CHUNK,
                                      total_chunks=n * (steps // CHUNK))
    logits, saved = policy.head(o)
    logp, lse, entropy = api.token_logprob_fwd(logits, target, scale=SCALE, entropy=True)

    mask = (torch.arange(steps, device=dev) >= prompt).repeat(n)
    loss = dict(entropy=entropy, mask=mask, cu_seqlens=cu, clip_low=clip, clip_high=clip,
                entropy_coef=entropy_coef, reduction="sequence")
    args = (logp, old_logp.reshape(-1), advantages.repeat_interleave(steps))
    stats, weight = api.policy_loss_fwd(*args, **loss)

    d_logp, d_entropy = api.policy_loss_bwd(*args, weight, **loss)
    d_logits = api.token_logprob_bwd(logits, target, lse, d_logp, scale=SCALE, entropy=entropy,
                                     d_entropy=d_entropy, d_logits=logits)
    d_h, d_weight, d_bias = policy.head_bwd(d_logits, saved)
    grads = api.trainer_bwd(cu, q, k, v, a, b, chunk_states, d_h.view_as(o), chunk=CHUNK,
                            total_chunks=n * (steps // CHUNK))
    return stats, logp.view(n, steps), {**grads, "norm_weight": d_weight, "norm_bias": d_bias}


def main():
    dev = torch.device("cuda:0")
    policy = Policy.random(0, dev)
    tokens, old_logp = rollout(policy, 8, 48, 1, dev)
    advantages = torch.randn(8, generator=torch.Generator().manual_seed(2)).to(dev)
    stats, logp, grads = train_step(policy, tokens, old_logp, advantages)
    torch.cuda.synchronize()
    same = torch.equal(logp.view(torch.int32), old_logp.view(torch.int32))
    names = ("loss", "policy loss", "KL", "entropy", "share cut off")
    print("trainer and rollout log-probabilities:", "the same bits" if same else "DIFFER")
    print(", ".join(f"{n} {v:.4f}" for n, v in zip(names, stats.tolist())))
    print(", ".join(f"|{n}| {g.norm().item():.4g}" for n, g in grads.items()))


if __name__ == "__main__":
    main()
