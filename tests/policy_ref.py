"""Plain 64-bit forms of the policy-head operators (torch float64 on the CPU), written from
their formulas, with error bounds for a binary32 computation of each output.

A bound counts roundings: u = 2^-24 is half a step of binary32, a sum of terms whose longest
chain of additions is `depth` long is off by at most depth u sum|terms|, and a value that is
rounded to bfloat16 at the end is off by 2^-8 of itself more (torch.finfo().eps / 2)."""

import numpy as np
import torch

U = 2.0 ** -24
F64 = torch.float64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------------------------ norm

# A lane adds at most 32 values of a row, 64 lanes and 16 waves are added after it.
NORM_DEPTH = 32 + 6 + 16


def norm_fwd(x, weight, bias, eps, kind):
    x, w = x.to(F64), weight.to(F64)
    b = torch.zeros_like(w) if bias is None else bias.to(F64)
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], dtype=F64)
    xc = x - mean[:, None]
    rstd = (xc.square().mean(1) + eps).rsqrt()
    return xc * rstd[:, None] * w + b, mean, rstd


def norm_fwd_bounds(x, weight, bias, eps, kind, dtype):
    """Bounds of y, mean and rstd. The mean is off by DEPTH u mean|x|; with it every distance,
    whose squares' sum has the same depth; 1 / sqrt halves the variance's error."""
    y, mean, rstd = norm_fwd(x, weight, bias, eps, kind)
    x, w = x.to(F64), weight.to(F64).abs()
    b = torch.zeros_like(w) if bias is None else bias.to(F64).abs()
    e_mean = (NORM_DEPTH + 2) * U * x.abs().mean(1) if kind == "layer" else torch.zeros_like(rstd)
    xc = (x - mean[:, None]).abs()
    # var: sum of (xc + e)^2, with e_mean in first order cancelled by the sum of xc being 0
    # (e^2 is left) but for the roundings of xc, u |xc| each
    rel_var = (NORM_DEPTH + 6) * U + e_mean.square() * rstd.square()
    rel = rel_var / 2 + 3 * U
    e_y = w * rstd[:, None] * (e_mean[:, None] + xc * (rel[:, None] + 4 * U)) + U * (y.abs() + b)
    e_y = e_y + (half_step(dtype) * (y.abs() + e_y) if dtype != torch.float32 else 0)
    return (y, e_y + 1e-38), (mean, e_mean + 1e-38), (rstd, rel * rstd)


def norm_bwd(dy, x, weight, mean, rstd, kind):
    dy, x, w = dy.to(F64), x.to(F64), weight.to(F64)
    rstd = rstd.to(F64)[:, None]
    xh = (x - mean.to(F64)[:, None]) * rstd if kind == "layer" else x * rstd
    g = dy * w
    c1 = (g * xh).mean(1, keepdim=True)
    c2 = g.mean(1, keepdim=True) if kind == "layer" else 0.0
    return rstd * (g - c2 - xh * c1), (dy * xh).sum(0), dy.sum(0)


# Rows that one block adds, its groups of rows, the blocks that one wave adds and the waves:
# under 128 one after the other for up to 8192 rows.
ROWS_DEPTH = 128


def norm_bwd_bounds(dy, x, weight, mean, rstd, kind, dtype):
    dx, dw, db = norm_bwd(dy, x, weight, mean, rstd, kind)
    dy, x, w = dy.to(F64).abs(), x.to(F64), weight.to(F64).abs()
    rs = rstd.to(F64)[:, None]
    # a distance from the mean is one rounding of the distance; times rstd another
    xh = ((x - mean.to(F64)[:, None]) * rs if kind == "layer" else x * rs).abs()
    g = dy * w
    c1 = (g * xh).mean(1, keepdim=True)
    c2 = g.mean(1, keepdim=True) if kind == "layer" else 0.0
    e = rs * U * (4 * g + (NORM_DEPTH + 8) * (c2 + xh * c1))
    e = e + (half_step(dtype) * (dx.abs() + e) if dtype != torch.float32 else U * dx.abs())
    return ((dx, e + 1e-38), (dw, (ROWS_DEPTH + 4) * U * (dy * xh).sum(0) + 1e-38),
            (db, ROWS_DEPTH * U * dy.sum(0) + 1e-38))


# --------------------------------------------------------------------------- 8-bit product

def quantize(x, k_pad):
    """(q int64 [M, k_pad], scale float32 [M]) of finite rows. The quotient of values of 24
    bits in binary64 decides a tie, which is exact in it, and no other value is within
    binary64's half step of one."""
    x = x.to(F64)
    a = x.abs().amax(1)
    q = torch.round(127.0 * x / torch.where(a > 0, a, 1.0)[:, None]).to(torch.int64)
    full = torch.zeros((x.shape[0], k_pad), dtype=torch.int64)
    full[:, :x.shape[1]] = q
    scale = a.numpy().astype(np.float32) / np.float32(127.0)
    return full, torch.from_numpy(scale)


def linear_i8(xq, x_scale, wq, w_scale, dtype):
    """Bit for bit: integer sums (exact in binary64, below 2^53), then three roundings."""
    acc = torch.matmul(xq.to(F64), wq.to(F64).t()).numpy().astype(np.int64)
    y = acc.astype(np.float32) * x_scale.numpy()[:, None]
    return torch.from_numpy(y * w_scale.numpy()[None, :]).to(dtype)


# ------------------------------------------------------------------------- log-probability

def scaled(logits, scale):
    return logits.to(F64) * float(np.float32(scale))


def logprob(logits, ids, scale):
    z = scaled(logits, scale)
    V = z.shape[1]
    use = (ids >= 0) & (ids < V)
    lse = torch.logsumexp(z, 1)
    none = lse == -np.inf
    at = ids.clamp(0, V - 1).to(torch.int64)[:, None]
    logq = z - torch.where(none, 0.0, lse)[:, None]
    logp = torch.where(none, -np.inf, logq.gather(1, at)[:, 0])
    p = logq.exp()
    ent = -torch.where(p > 0, p * logq, 0.0).sum(1)
    zero = torch.zeros((), dtype=F64)
    return (torch.where(use, logp, zero), torch.where(use, lse, zero),
            torch.where(use, ent, zero))


def logprob_bounds(logits, ids, scale):
    """A thread adds at most V / 256 exponentials after one another (and V < 256 of them at
    most 8), lanes and waves under 32 more. A difference from the maximum, times the constant
    scale / ln 2, is off by 4 u of itself, which is the exponential's relative error, with 2 u
    of its own; in the sum's logarithm that counts by the probabilities."""
    logp, lse, ent = logprob(logits, ids, scale)
    z = scaled(logits, scale)
    V = z.shape[1]
    at = ids.clamp(0, V - 1).to(torch.int64)[:, None]
    top = z.amax(1, keepdim=True)
    top = torch.where(top == -np.inf, 0.0, top)
    d = torch.where(z == -np.inf, 0.0, (z - top).abs())
    p = (z - torch.where(lse == -np.inf, 0.0, lse)[:, None]).exp()
    mean_d = (p * d).sum(1)
    mean_d2 = (p * d * d).sum(1)
    depth = V / 256 + 8 + 32
    ls = (lse - top[:, 0]).abs()
    ls = torch.where(torch.isfinite(ls), ls, 0.0)
    # a merge rescales by an exponential: at most 32 + V / 4096 of them, 6 u each and 4 u of
    # the distance between maxima, which is at most the largest distance that counts
    merges = (32 + V / 4096) * 6
    e_s = U * (depth + merges + 6 + 8 * mean_d)
    e_ls = e_s + 2 * U * ls
    e_logp = e_ls + 4 * U * d.gather(1, at)[:, 0]
    e_lse = e_ls + 2 * U * (top[:, 0].abs() + ls)
    e_ent = 2 * e_ls + U * ((depth + merges + 10) * 2 * mean_d + 8 * mean_d2)
    return (logp, e_logp), (lse, e_lse), (ent, e_ent)


def logprob_bwd(logits, ids, lse, d_logp, scale, entropy=None, d_entropy=None):
    s = float(np.float32(scale))
    z = scaled(logits, scale)
    M, V = z.shape
    use = (ids >= 0) & (ids < V) & (lse != -np.inf)
    lse = torch.where(use, lse.to(F64), 0.0)
    g = torch.where(use, d_logp.to(F64), 0.0)[:, None]
    logq = z - lse[:, None]
    p = torch.where(use[:, None], logq.exp(), 0.0)
    d = -p * g
    if d_entropy is not None:
        h = torch.where(use, d_entropy.to(F64), 0.0)[:, None]
        H = torch.where(use, entropy.to(F64), 0.0)[:, None]
        d = d - torch.where(p > 0, h * p * (logq + H), 0.0)
    rows = torch.arange(M)
    d[rows, ids.clamp(0, V - 1).to(torch.int64)] += g[:, 0]
    return torch.where(use[:, None], s * d, 0.0)


def logprob_bwd_bounds(logits, ids, lse, d_logp, scale, entropy, d_entropy, dtype):
    """p is off by 4 u of |z - lse| and 4 u; what multiplies it by three roundings of its
    parts; the row's g stands beside it at the chosen token."""
    s = float(np.float32(scale))
    want = logprob_bwd(logits, ids, lse, d_logp, scale, entropy, d_entropy)
    z = scaled(logits, scale)
    M, V = z.shape
    use = (ids >= 0) & (ids < V) & (lse != -np.inf)
    logq = z - torch.where(use, lse.to(F64), 0.0)[:, None]
    p = torch.where(use[:, None], logq.exp(), 0.0)
    dist = torch.where(p > 0, logq.abs(), 0.0)
    k = torch.where(use, d_logp.to(F64).abs(), 0.0)[:, None].expand(M, V).clone()
    if d_entropy is not None:
        k = k + torch.where(use, d_entropy.to(F64).abs(), 0.0)[:, None] * (
            dist + torch.where(use, entropy.to(F64).abs(), 0.0)[:, None])
    e = s * p * k * U * (4 * dist + 12)
    rows = torch.arange(M)
    e[rows, ids.clamp(0, V - 1).to(torch.int64)] += 4 * U * s * torch.where(
        use, d_logp.to(F64).abs(), 0.0)
    # an exponential that underflows binary32 (denormals not kept by the instruction) is 0
    e = e + s * k * 2.0 ** -125
    return want, e + (half_step(dtype) if dtype != torch.float32 else U) * (want.abs() + e)


# ----------------------------------------------------------------------------- policy loss

def policy(logp, old, adv, ref, ent, mask, cu, clip_low, clip_high, dual, kl_coef, ent_coef,
           reduction):
    """(stats [5], weight [N], d_logp [T], d_entropy [T]) in binary64, token by token."""
    T, N = len(logp), len(cu) - 1
    f = lambda v: None if v is None else np.asarray(v, dtype=np.float64)  # noqa: E731
    logp, old, adv, ref, ent = map(f, (logp, old, adv, ref, ent))
    mask = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    spans = [[t for t in range(cu[n], cu[n + 1]) if mask[t]] for n in range(N)]
    total, live = sum(map(len, spans)), sum(1 for s in spans if s)
    weight, stats = np.zeros(N), np.zeros(5)
    d_logp, d_ent = np.zeros(T), np.zeros(T)
    for n, span in enumerate(spans):
        if not span:
            continue
        w = 1.0 / (len(span) * live) if reduction == "sequence" else 1.0 / total
        weight[n] = w
        for t in span:
            r = np.exp(logp[t] - old[t])
            a, b = r * adv[t], min(max(r, 1.0 - clip_low), 1.0 + clip_high) * adv[t]
            gain, cut = min(a, b), a > b
            if dual and adv[t] < 0 and gain < dual * adv[t]:
                gain, cut = dual * adv[t], True
            kl = slope = 0.0
            if ref is not None:
                u = ref[t] - logp[t]
                kl, slope = np.expm1(u) - u, -np.expm1(u)
            stats[1:] += w * np.array([-gain, kl, 0.0 if ent is None else ent[t], float(cut)])
            d_logp[t] = w * ((kl_coef if ref is not None else 0.0) * slope
                             - (0.0 if cut else a))
            d_ent[t] = -w * ent_coef
    stats[0] = (stats[1] + (kl_coef * stats[2] if ref is not None else 0.0)
                - (ent_coef * stats[3] if ent is not None else 0.0))
    return stats, weight, d_logp, d_ent


# binary64 terms and sums: what is left is the rounding of the outputs to binary32 and of the
# weight before it multiplies (u each), and binary64's own 2^-52 over up to 2^20 terms.
POLICY_REL, POLICY_ABS = 2.5 * U, 1e-9


def check(got, want, bound, label):
    """|got - want| <= bound everywhere; NaN and infinities where `want` has them."""
    got = got.detach().to("cpu").to(F64)
    want, bound = (torch.as_tensor(v, dtype=F64) for v in (want, bound))
    assert got.shape == want.shape, f"{label}: {tuple(got.shape)} vs {tuple(want.shape)}"
    special = ~torch.isfinite(want)
    same = torch.where(torch.isnan(want), torch.isnan(got), got == want)
    assert bool(same[special].all()), f"{label}: non-finite values differ"
    off = torch.where(special, 0.0, (got - want).abs())
    over = ~(off <= torch.where(special, 0.0, bound.expand_as(want)))
    if bool(over.any()):
        i = tuple(int(v) for v in torch.nonzero(over)[0])
        raise AssertionError(f"{label}: {int(over.sum())} of {want.numel()} over their bound; "
                             f"first at {i}: {float(got[i])!r} vs {float(want[i])!r}, bound "
                             f"{float(bound.expand_as(want)[i]):.3g}")
