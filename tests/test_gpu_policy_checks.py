"""The policy head where a look at shapes or at the result itself would not do: rows with
infinities in bfloat16, patterns around every output of calls with bad offsets, gradients at
half a loss, and every call on a stream of its own."""

import numpy as np
import pytest
import torch

import policy_ref as R
from bitwise_consistent_linear_amd import api
from gpu_util import DEV
from test_gpu_policy import BF16, F32, head_state, policy_inputs, rand, gen, same_bits

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dt,top", [(F32, 0), (BF16, 127)], ids=["f32", "bf16"])
def test_quantized_infinities(dt, top):
    """3.4e38 is finite in binary32 and rounds to infinity in bfloat16 (its largest value is
    3.39e38): 0 beside the infinities, or one of them."""
    x = torch.zeros(2, 300)
    x[0, :7] = torch.tensor([1.0, -2.0, INF, -INF, 3.4e38, 0.0, -1.0])
    x[1, 299] = -INF
    q, s = api.quantize_rows(x.to(dt).to(DEV))
    want = torch.zeros(2, 384, dtype=torch.int8)
    want[0, :5] = torch.tensor([0, 0, 127, -127, top])
    want[1, 299] = -127
    assert torch.equal(q.cpu(), want) and s.tolist() == [INF, INF]


class Guarded:
    """A buffer inside a larger one that holds a pattern."""

    def __init__(self, n, dtype, before=1024, value=85):
        self.value, self.before, self.n = value, before, n
        self.all = torch.full((before + n + 4096,), value, dtype=dtype, device=DEV)
        self.inner = self.all[before:before + n]

    def check(self, label):
        assert bool((self.all[:self.before] == self.value).all()), f"{label}: before"
        assert bool((self.all[self.before + self.n:] == self.value).all()), f"{label}: after"


BAD = [[0, 900, 100, 2**31 - 1], [-5, -7, 400, 1000], [1000, 0, 1000, 0], [10**6] * 4, [-1] * 4,
       [700, 300, 300, 900]]
MANY = [[int(v) for v in np.random.default_rng(s).integers(-3000, 9000, 700)] for s in (1, 2)]


@pytest.mark.parametrize("T", [1000, 5000, 70000])
@pytest.mark.parametrize("cu", BAD + MANY, ids=lambda c: f"{len(c) - 1}_{c[0]}")
def test_bad_offsets_write_their_outputs_alone(cu, T):
    """Starts are clamped to [0, T] and a slot is span + sequence, below the slots' number."""
    N = len(cu) - 1
    z, c = torch.zeros(T, device=DEV), torch.tensor(cu, dtype=torch.int32, device=DEV)
    need = api.policy_loss_workspace_bytes(api.GdnPolicyShape(T, N, 1, 0, 0.2, 0.2, 0, 0.1, 0.1))
    room = Guarded(need, torch.uint8)
    stats, weight = Guarded(5, F32), Guarded(N, F32)
    dl, de = Guarded(T, F32), Guarded(T, F32)
    kw = dict(ref_logp=z, entropy=z, cu_seqlens=c, kl_coef=0.1, entropy_coef=0.1,
              reduction="sequence")
    api.policy_loss_fwd(z, z, z, stats=stats.inner, weight=weight.inner, workspace=room.inner, **kw)
    api.policy_loss_bwd(z, z, z, weight.inner, d_logp=dl.inner, d_entropy=de.inner, **kw)
    torch.cuda.synchronize()
    for g, label in ((room, "workspace"), (stats, "stats"), (weight, "weight"), (dl, "d_logp"),
                     (de, "d_entropy")):
        g.check(label)
    assert bool((dl.inner != dl.value).all()) and bool((de.inner != de.value).all())


@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_gradient_at_half_a_loss(reduction):
    """The bounds are halved with the gradient."""
    lengths = [0, 3, 1000, 17, 2, 2, 2, 2500, 0] + [40] * 60
    cu, logp, old, adv, ref, ent, mask = policy_inputs("x", lengths, 5)
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    kw = dict(ref_logp=up(ref), entropy=up(ent), mask=up(mask), cu_seqlens=up(cu), clip_low=0.2,
              clip_high=0.28, dual_clip=3.0, kl_coef=0.05, entropy_coef=0.01, reduction=reduction)
    _, weight = api.policy_loss_fwd(up(logp), up(old), up(adv), **kw)
    dl, de = api.policy_loss_bwd(up(logp), up(old), up(adv), weight, d_loss=0.5, **kw)
    _, _, wl, we = R.policy(logp, old, adv, ref, ent, mask, cu, 0.2, 0.28, 3.0, 0.05, 0.01,
                            reduction)
    wl, we = 0.5 * wl, 0.5 * we
    R.check(dl, wl, torch.from_numpy(np.abs(wl) * R.POLICY_REL + R.POLICY_ABS * 1e-3), "d_logp")
    R.check(de, we, torch.from_numpy(np.abs(we) * R.POLICY_REL), "d_entropy")


def test_every_call_on_a_stream_of_its_own():
    """The eight calls with stream=, the side stream behind the current one's work, against the
    same calls without; workspaces and outputs belong to the side stream."""
    s = head_state(45)
    ref = (s["old"] + rand(gen(46), 300, scale=0.1).to(DEV)).contiguous()
    kw = dict(entropy_coef=0.01, kl_coef=0.05, mask=s["mask"], cu_seqlens=s["cu"], ref_logp=ref)

    def step(**on):
        y, mean, rstd = api.layer_norm_fwd(s["x"], s["w"], s["b"], **on)
        xq, xs = api.quantize_rows(y, **on)
        z = api.linear_i8_fwd(xq, xs, s["wq"], s["ws"], out_dtype=BF16, **on)
        logp, lse, ent = api.token_logprob_fwd(z, s["ids"], scale=0.8, entropy=True, **on)
        stats, weight = api.policy_loss_fwd(logp, s["old"], s["adv"], entropy=ent, **kw, **on)
        dl, de = api.policy_loss_bwd(logp, s["old"], s["adv"], weight, entropy=ent, **kw, **on)
        d = api.token_logprob_bwd(z, s["ids"], lse, dl, scale=0.8, entropy=ent, d_entropy=de, **on)
        dx, dw, db = api.layer_norm_bwd(s["dy"], s["x"], s["w"], mean, rstd, **on)
        return [y, mean, rstd, xq, xs, z, logp, lse, ent, stats, weight, dl, de, d, dx, dw, db]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = step(stream=side)
        side.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            same_bits(a, b, f"output {i}")
