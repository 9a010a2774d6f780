"""The logits gradient on rows of any magnitude: rows shifted far from zero, masked with the
type's lowest value, or of it alone. What it is held to is the 64-bit gradient of the
log-probability and entropy themselves, not of a log-sum-exp that was rounded to binary32."""

import pytest
import torch

import policy_ref as R
from bitwise_consistent_linear_amd import api
from gpu_util import DEV, log
from test_gpu_policy import BF16, DTYPES, F32, gen, rand, same_bits

pytestmark = pytest.mark.gpu

NEAR = 64.0  # rows whose |lse| is smaller take it as the forward rounded it


def far_rows(V, dt, seed):
    """(logits [M, V], ids [M]): each row another place, mask or end."""
    g = gen(seed)
    low, top, inf = torch.finfo(dt).min, torch.finfo(dt).max, float("inf")
    shifts = [0.0, 30.0, -58.0, 62.0, 70.0, -70.0, 1e3, 1e4, -1e4, 1e6, -1e9, 1e30]
    z = rand(g, len(shifts) + 8, V, scale=2.5)
    ids = torch.randint(0, V, (z.shape[0],), generator=g)
    for i, s in enumerate(shifts):
        z[i] += s
    z = z.to(dt)
    n = len(shifts)
    z[n] = low                      # nothing but the lowest value: uniform
    z[n + 1] = -1e9
    z[n + 2] = low                  # one finite maximum, chosen, and not chosen
    z[n + 2, ids[n + 2]] = 5.0
    z[n + 3] = low
    z[n + 3, V // 2] = 2.5
    ids[n + 3] = V - 1
    z[n + 4] = low                  # the largest value against the lowest
    z[n + 4, V // 2] = top
    z[n + 5] = (z[n + 5].float() + 1e4).to(dt)
    z[n + 5, V // 3 + 1:] = -inf    # a shifted row with masked columns
    ids[n + 5] = 0
    z[n + 6] = -inf                 # nothing admissible
    z[n + 7] = (z[n + 7].float() - 1e6).to(dt)
    ids[n + 7] = -1                 # not scored
    return z, ids


def gradient(z, ids, dlp, de, scale, dtype):
    """(gradient, bound, log-sum-exp) in binary64. Distances from a row's maximum keep what its
    place would cost; with them the bounds of policy_ref hold, whose lse is then the logarithm
    of the sum alone. Its error, and that of the entropy given to the gradient, multiply p; a
    row near zero adds its lse's own rounding; the gradient's own sums add at most 6 u for each
    of V / 2048 changes of a maximum."""
    s = float(torch.tensor(scale, dtype=F32))
    M, V = z.shape
    x = z.to(R.F64)
    m = x.amax(1, keepdim=True)
    use = (ids >= 0) & (m[:, 0] > -float("inf"))
    x = x - torch.where(m == -float("inf"), 0.0, m)
    x[~use] = 0.0
    at = ids.clamp(0, V - 1)
    (_, _), (ls, e_ls), (H, e_H) = R.logprob_bounds(x, at, scale)
    logq = s * x - ls[:, None]
    p = logq.exp()
    dist = torch.where(p > 0, logq.abs(), 0.0)
    g, h = dlp.to(R.F64)[:, None], (torch.zeros_like(dlp) if de is None else de).to(R.F64)[:, None]
    d = -p * g - torch.where(p > 0, h * p * (logq + H[:, None]), 0.0)
    d[torch.arange(M), at] += g[:, 0]
    lse = (s * torch.where(m == -float("inf"), 0.0, m)[:, 0] + ls)
    e_c = e_ls + R.U * (6 * V / 2048 + ls + torch.where(lse.abs() < NEAR, lse.abs(), 0.0))
    e_c, e_H = e_c[:, None], e_H[:, None]
    k = g.abs() + h.abs() * (dist + H.abs()[:, None])
    e = s * p * (k * (R.U * (4 * dist + 12) + e_c) + h.abs() * (e_c + e_H)) * 1.01
    e[torch.arange(M), at] += 4 * R.U * s * g[:, 0].abs()
    e = e + s * k * 2.0 ** -125
    want = torch.where(use[:, None], s * d, 0.0)
    return want, e + (R.half_step(dtype) if dtype != F32 else R.U) * (want.abs() + e)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.8, 1.0, 1.5])
@pytest.mark.parametrize("V", [1, 7, 300, 3000, 4099, 70001])
def test_gradient_of_far_rows(V, scale, dt):
    log(f"far rows V={V} scale={scale} {dt}")
    dt = DTYPES[dt]
    z, ids = far_rows(V, dt, V)
    M = z.shape[0]
    g = gen(V + 1)
    dlp, de = rand(g, M), rand(g, M, scale=0.3)
    zd, idd = z.to(DEV), ids.to(DEV)
    _, lse, ent = api.token_logprob_fwd(zd, idd, scale=scale, entropy=True)
    kw = dict(scale=scale, entropy=ent, d_entropy=de.to(DEV))
    both = api.token_logprob_bwd(zd, idd, lse, dlp.to(DEV), **kw)
    want, bound = gradient(z, ids, dlp, de, scale, dt)
    R.check(both, want, bound, "d_logits with entropy")
    d = api.token_logprob_bwd(zd, idd, lse, dlp.to(DEV), scale=scale)
    want, bound = gradient(z, ids, dlp, None, scale, dt)
    R.check(d, want, bound, "d_logits")
    # the same bits for a row alone, in a wider buffer and in the logits' place
    wide = torch.full((M, V + 13), float("nan"), dtype=dt, device=DEV)
    wide[:, 5:5 + V] = zd
    same_bits(api.token_logprob_bwd(wide[:, 5:5 + V], idd, lse, dlp.to(DEV), **kw), both, "strided")
    for i in (7, 12, 16):
        one = api.token_logprob_bwd(zd[i:i + 1], idd[i:i + 1], lse[i:i + 1], dlp[i:i + 1].to(DEV),
                                    scale=scale)
        same_bits(one, d[i:i + 1], f"row {i} alone")
    api.token_logprob_bwd(zd, idd, lse, dlp.to(DEV), d_logits=zd, **kw)
    same_bits(zd, both, "in the logits' place")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_far_rows_with_nan_or_infinity_are_nan(dt):
    """A NaN or +infinity among a far row's logits: NaN for that row, the others as they are."""
    dt = DTYPES[dt]
    z = (rand(gen(5), 4, 5000, scale=2.5) + 1e4).to(dt)
    ids, dlp = torch.tensor([1, 2, 3, 4]), torch.ones(4, device=DEV)
    clean = z.clone()
    z[1, 4990], z[2, 0] = float("nan"), float("inf")
    out = []
    for t in (z, clean):
        _, lse, ent = api.token_logprob_fwd(t.to(DEV), ids.to(DEV), entropy=True)
        out.append(api.token_logprob_bwd(t.to(DEV), ids.to(DEV), lse, dlp, entropy=ent,
                                         d_entropy=dlp))
    assert bool(out[0][1].isnan().all()) and bool(out[0][2].isnan().all())
    for i in (0, 3):
        same_bits(out[0][i], out[1][i], "rows beside")


def test_far_rows_in_a_graph():
    """Replays with rows near and far in turn, against eager calls."""
    z, ids = far_rows(3000, BF16, 9)
    zd, idd, dlp = z.to(DEV), ids.to(DEV), torch.ones(z.shape[0], device=DEV)

    def step():
        _, lse, _ = api.token_logprob_fwd(zd, idd)
        return api.token_logprob_bwd(zd, idd, lse, dlp)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    near = rand(gen(10), *z.shape, scale=2.5, dtype=BF16).to(DEV)
    for new in (near, z.to(DEV), near, z.to(DEV)):
        zd.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got, want = out.clone(), step()
        torch.cuda.synchronize()
        same_bits(got, want, "replay")
