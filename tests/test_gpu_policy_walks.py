"""Loops over rows and sequences past their first iteration. Sizes follow the launch rules: more rows
than a launch has groups of threads for (forward norm 2048 workgroups, 256 of rows wider than
8192; backward 256; quantisation 2048, or 262144 threads of rows longer than 16384; sums of
sequences 65536 workgroups of 64), in every variant of a kernel. The same bits as in batches
small enough for one iteration, and the last rows against the 64-bit form."""

import numpy as np
import pytest
import torch

import policy_ref as R
from bitwise_consistent_linear_amd import api
from gpu_util import DEV, log
from test_gpu_policy import DTYPES, norm_inputs, gen, same_bits

pytestmark = pytest.mark.gpu


def pieces(M, step):
    return [(lo, min(lo + step, M)) for lo in range(0, M, step)]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("M,D,dt", [(2100, 4096, "bf16"), (2100, 4096, "f32"), (4500, 2500, "bf16"),
                                    (2100, 5000, "bf16"), (4200, 5000, "f32"), (300, 8200, "f32"),
                                    (600, 8200, "bf16"), (600, 16384, "bf16"), (600, 16384, "f32"),
                                    (70000, 72, "bf16"), (40000, 72, "f32"), (9000, 300, "f32")])
def test_norm_forward(M, D, dt, kind):
    log(f"norm forward walk {kind} {M}x{D} {dt}")
    x, w, b, _ = norm_inputs(M, D, DTYPES[dt], DTYPES[dt], M + D)
    b = b if kind == "layer" else None
    xd, wd, bd = x.to(DEV), w.to(DEV), None if b is None else b.to(DEV)
    y, mean, rstd = api.layer_norm_fwd(xd, wd, bd, kind=kind)
    for lo, hi in pieces(M, 250 if D > 128 else 20000):
        y1, m1, r1 = api.layer_norm_fwd(xd[lo:hi], wd, bd, kind=kind)
        same_bits(y1, y[lo:hi], f"y {lo}")
        same_bits(r1, rstd[lo:hi], f"rstd {lo}")
        if kind == "layer":
            same_bits(m1, mean[lo:hi], f"mean {lo}")
    (wy, ey), (wm, em), (wr, er) = R.norm_fwd_bounds(x[-60:], w, b, 1e-5, kind, x.dtype)
    R.check(y[-60:], wy, ey, "y")
    R.check(rstd[-60:], wr, er, "rstd")
    if kind == "layer":
        R.check(mean[-60:], wm, em, "mean")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("M,D,dt", [(600, 8200, "bf16"), (600, 16384, "f32"), (700, 16381, "bf16"),
                                    (600, 4096, "f32"), (70000, 72, "bf16"), (5000, 300, "f32")])
def test_norm_backward(M, D, dt, kind):
    log(f"norm backward walk {kind} {M}x{D} {dt}")
    x, w, _, dy = norm_inputs(M, D, DTYPES[dt], DTYPES[dt], M + D)
    xd, wd, dyd = x.to(DEV), w.to(DEV), dy.to(DEV)
    _, mean, rstd = api.layer_norm_fwd(xd, wd, kind=kind)
    dx, dw, db = api.layer_norm_bwd(dyd, xd, wd, mean, rstd, kind=kind, bias=True)
    for lo, hi in pieces(M, 250 if D > 128 else 16000):
        m = None if mean is None else mean[lo:hi]
        d1, _, _ = api.layer_norm_bwd(dyd[lo:hi], xd[lo:hi], wd, m, rstd[lo:hi], kind=kind)
        same_bits(d1, dx[lo:hi], f"dx {lo}")
    hm = None if mean is None else mean.cpu()
    (wx, ex), (ww, ew), (wb, eb) = R.norm_bwd_bounds(dy, x, w, hm, rstd.cpu(), kind, x.dtype)
    R.check(dx, wx, ex, "dx")
    R.check(dw, ww, ew, "d_weight")
    R.check(db, wb, eb, "d_bias")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(40000, 100), (9000, 500), (2100, 4000), (2100, 8200),
                                 (1000, 33000)])
def test_quantize(M, K, dt):
    log(f"quantize walk {M}x{K} {dt}")
    x = (torch.randn(M, K, generator=gen(M)) * 3).to(DTYPES[dt])
    x[-3] = 0.0
    xd = x.to(DEV)
    q, s = api.quantize_rows(xd)
    for lo, hi in pieces(M, 250 if K > 128 else 20000):
        q1, s1 = api.quantize_rows(xd[lo:hi])
        same_bits(q1, q[lo:hi], f"q {lo}")
        same_bits(s1, s[lo:hi], f"scale {lo}")
    wq, ws = R.quantize(x[-60:], -(-K // 128) * 128)
    assert torch.equal(q[-60:].cpu().to(torch.int64), wq)
    same_bits(s[-60:].cpu(), ws, "scale")


def policy(logp, old, adv, ref, ent, mask, cu, clip, kl_coef, ent_coef, reduction):
    """The loss of many sequences in binary64, whole arrays at a time; clip_low = clip_high."""
    logp, old, adv, ref, ent = (v.astype(np.float64) for v in (logp, old, adv, ref, ent))
    N, T = len(cu) - 1, len(logp)
    seq = np.repeat(np.arange(N), np.diff(cu))
    count = np.bincount(seq[mask], minlength=N).astype(np.float64)
    live = count > 0
    weight = np.zeros(N)
    weight[live] = 1.0 / (count[live] * live.sum()) if reduction == "sequence" else 1.0 / count.sum()
    r = np.exp(logp - old)
    a, b = r * adv, np.clip(r, 1.0 - clip, 1.0 + clip) * adv
    u = ref - logp
    terms = np.stack([-np.minimum(a, b), np.expm1(u) - u, ent, (a > b).astype(np.float64)])
    wt = np.where(mask, weight[seq], 0.0)
    means = (terms * wt).sum(1)
    stats = np.concatenate([[means[0] + kl_coef * means[1] - ent_coef * means[2]], means])
    d_logp = wt * (-kl_coef * np.expm1(u) - np.where(a > b, 0.0, a))
    assert d_logp.shape == (T,)
    return stats, weight, d_logp, -wt * ent_coef


@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("N,T", [(5000, 90000), (300000, 200000), (4300000, 150000)])
def test_policy_of_many_sequences(N, T, reduction):
    """A search in three steps (over 4096 sequences) and in four (over 262144), and more than
    65536 workgroups' sequences; short and empty ones, many more than tokens at the last."""
    log(f"policy {N} sequences {T} tokens {reduction}")
    rng = np.random.default_rng(N)
    inner = np.sort(rng.integers(0, T + 1, N - 1))
    inner[N // 3:N // 3 + 700] = inner[N // 3]  # a long run of empty ones
    cu = np.concatenate([[0], np.sort(inner), [T]]).astype(np.int32)
    f = lambda s: (rng.normal(size=T) * s).astype(np.float32)  # noqa: E731
    logp = -np.abs(f(1.0))
    old, ref, adv, ent = logp + f(0.3), logp + f(0.3), f(1.5), np.abs(f(1.0))
    mask = rng.random(T) < 0.7
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    junk = np.where(mask, logp, np.float32(np.nan))
    kw = dict(ref_logp=up(ref), entropy=up(ent), mask=up(mask), cu_seqlens=up(cu), clip_low=0.25,
              clip_high=0.25, kl_coef=0.05, entropy_coef=0.01, reduction=reduction)
    stats, weight = api.policy_loss_fwd(up(junk), up(old), up(adv), **kw)
    dl, de = api.policy_loss_bwd(up(junk), up(old), up(adv), weight, d_loss=0.5, **kw)
    ws, ww, wl, we = policy(logp, old, adv, ref, ent, mask, cu, 0.25, 0.05, 0.01, reduction)
    size = np.abs(ws[1:]).max() + 1.0
    R.check(stats, ws, torch.from_numpy(np.abs(ws) * R.POLICY_REL + R.POLICY_ABS * size), "stats")
    R.check(weight, ww, torch.from_numpy(np.abs(ww) * R.U), "weight")
    wl, we = 0.5 * wl, 0.5 * we
    R.check(dl, wl, torch.from_numpy(np.abs(wl) * R.POLICY_REL + R.POLICY_ABS * 1e-3), "d_logp")
    R.check(de, we, torch.from_numpy(np.abs(we) * R.POLICY_REL), "d_entropy")
    again, w2 = api.policy_loss_fwd(up(junk), up(old), up(adv), **kw)
    same_bits(again, stats, "a second launch's stats")
    same_bits(w2, weight, "a second launch's weights")
