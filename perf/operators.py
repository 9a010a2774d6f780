"""Cases of the policy-head operators: layer norm, the 8-bit integer linear region, the token
log-probability and the clipped policy loss, each in a plain form of elementary torch
operations (``own`` false) and through the library's entry points (``own`` true).

A case names its operator and sizes; ``prepare`` draws its inputs on the GPU from a seed,
``run`` makes one pass, ``exact`` gives the pass's outputs from the definitions in binary64.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
I8_K_ALIGN = 128  # int8 operands hold rows padded with zeros to this many values

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decode step's hidden rows: 256 sequences, width 32 heads x 128
        {"name": "norm_fwd_decode", "op": "norm_fwd", "kind": "layer", "rows": 256, "width": 4096,
         "dtype": "bf16"},
        # the trainer's packed batch of 16384 tokens, width 4096
        {"name": "norm_bwd_trainer", "op": "norm_bwd", "kind": "layer", "rows": 16384,
         "width": 4096, "dtype": "bf16"},
        # binary32 rows of odd length and number, the root-mean-square form
        {"name": "norm_bwd_odd", "op": "norm_bwd", "kind": "rms", "rows": 4099, "width": 2049,
         "dtype": "f32"},
        # a projection of 16 decoding sequences: the weights' bytes count
        {"name": "i8_decode", "op": "i8", "m": 16, "n": 4096, "k": 4096, "dtype": "bf16"},
        # the vocabulary projection of 256 decoding sequences
        {"name": "i8_vocabulary", "op": "i8", "m": 256, "n": 65536, "k": 4096, "dtype": "bf16"},
        # the linear region's benchmark size, for the trainer's forward
        {"name": "i8_trainer", "op": "i8", "m": 16384, "n": 4096, "k": 4096, "dtype": "f32"},
        # log-probability of the sampled token in one decode step, a few rows of a long vocabulary
        {"name": "logprob_fwd_decode", "op": "logprob_fwd", "rows": 8, "vocab": 131072,
         "dtype": "f32", "entropy": False},
        # the trainer's log-probabilities and entropies
        {"name": "logprob_fwd_trainer", "op": "logprob_fwd", "rows": 8192, "vocab": 65536,
         "dtype": "bf16", "entropy": True},
        # their gradient
        {"name": "logprob_bwd_trainer", "op": "logprob_bwd", "rows": 8192, "vocab": 65536,
         "dtype": "bf16", "entropy": True},
        # gradient over an odd vocabulary in binary32
        {"name": "logprob_bwd_odd", "op": "logprob_bwd", "rows": 1021, "vocab": 50021,
         "dtype": "f32", "entropy": False},
        # loss and gradient of a small packed batch, mean over tokens
        {"name": "policy_trainer", "op": "policy", "tokens": 16384, "seqs": 4,
         "reduction": "token"},
        # 64 ragged sequences of 262144 tokens, mean over sequences
        {"name": "policy_ragged", "op": "policy", "tokens": 262144, "seqs": 64,
         "reduction": "sequence"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "i8", "logprob_fwd", "logprob_bwd", "policy"])
    dtype = rng.choice(["bf16", "f32"])
    while True:
        if op in ("norm_fwd", "norm_bwd"):
            c = {"op": op, "kind": rng.choice(["layer", "rms"]), "dtype": dtype,
                 "rows": _log_uniform(rng, 1, 16384), "width": _log_uniform(rng, 64, 16384)}
            fits = c["rows"] * c["width"] * _BYTES[dtype] <= 16384 * 4096 * 2
        elif op == "i8":
            c = {"op": op, "dtype": dtype, "m": _log_uniform(rng, 1, 16384),
                 "n": _log_uniform(rng, 64, 65536), "k": _log_uniform(rng, 64, 16384)}
            fits = (c["m"] * c["n"] * c["k"] <= 16384 * 4096 * 4096
                    and c["m"] * c["n"] <= 16384 * 4096 and c["n"] * c["k"] <= 65536 * 4096)
        elif op in ("logprob_fwd", "logprob_bwd"):
            c = {"op": op, "dtype": dtype, "rows": _log_uniform(rng, 1, 8192),
                 "vocab": _log_uniform(rng, 1000, 131072), "entropy": rng.random() < 0.5}
            fits = c["rows"] * c["vocab"] * _BYTES[dtype] <= 8192 * 65536 * 2
        else:
            c = {"op": op, "tokens": _log_uniform(rng, 64, 262144),
                 "seqs": _log_uniform(rng, 1, 256), "reduction": rng.choice(["token", "sequence"])}
            fits = True
        if fits:
            return c


# ------------------------------------------------------------------------------- inputs

EPS = 1e-5
SCALE = 0.8           # logits are multiplied by it (the inverse of a sampling temperature)
CLIP_LOW, CLIP_HIGH = 0.2, 0.28
DUAL_CLIP = 3.0
KL_COEF, ENTROPY_COEF = 0.01, 0.001


def _normal(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale


def _lengths(rng, tokens, seqs):
    """Ragged lengths that add up to `tokens`; some may be zero or one."""
    w = rng.lognormal(0.0, 1.0, seqs)
    cuts = np.floor(np.cumsum(w) / w.sum() * tokens).astype(np.int64)
    cuts[-1] = tokens
    return np.concatenate([[0], cuts])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm_fwd", "norm_bwd"):
        M, D, dt = case["rows"], case["width"], _DTYPE[case["dtype"]]
        x = _normal(gen, (M, D)) * (0.5 + 1.5 * torch.rand((M, 1), generator=gen, device=DEV))
        x = (x + _normal(gen, (M, 1), 0.5)).to(dt)
        s["x"] = x
        s["weight"] = (1.0 + _normal(gen, (D,), 0.1)).to(dt)
        s["bias"] = _normal(gen, (D,), 0.1).to(dt) if case["kind"] == "layer" else None
        if op == "norm_bwd":
            s["dy"] = _normal(gen, (M, D)).to(dt)
            xf = x.double()
            if case["kind"] == "layer":
                mean = xf.mean(1)
                s["mean"] = mean.float()
                s["rstd"] = (((xf - mean[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
            else:
                s["mean"] = None
                s["rstd"] = ((xf * xf).mean(1) + EPS).rsqrt().float()
    elif op == "i8":
        M, N, K = case["m"], case["n"], case["k"]
        s["x"] = _normal(gen, (M, K)).to(torch.bfloat16)
        # the weights are quantised and laid out once, rows padded with zeros
        w = _normal(gen, (N, K), 1.0 / math.sqrt(K))
        amax = w.abs().amax(1)
        wq = torch.zeros((N, -(-K // I8_K_ALIGN) * I8_K_ALIGN), dtype=torch.int8, device=DEV)
        wq[:, :K] = torch.round(w * (127.0 / amax)[:, None]).to(torch.int8)
        s["wq"], s["w_scale"] = wq, amax / 127.0
    elif op in ("logprob_fwd", "logprob_bwd"):
        M, V, dt = case["rows"], case["vocab"], _DTYPE[case["dtype"]]
        logits = _normal(gen, (M, V), 2.5).to(dt)
        ids = torch.randint(0, V, (M,), generator=gen, device=DEV)
        # a policy samples likely tokens: raise the chosen logit
        lift = _normal(gen, (M,), 3.0) + 8.0
        logits[torch.arange(M, device=DEV), ids] = lift.to(dt)
        ids[torch.arange(M, device=DEV) % 16 == 15] = -1  # prompt tokens, not scored
        s["logits"], s["ids"] = logits, ids
        if op == "logprob_bwd":
            f = _plain_logprob(logits, ids, case["entropy"])
            s["lse"], s["entropy"] = f["lse"], f.get("entropy")
            s["d_logp"] = _normal(gen, (M,))
            s["d_entropy"] = _normal(gen, (M,), 0.1) if case["entropy"] else None
    else:
        T, N = case["tokens"], case["seqs"]
        rng = np.random.default_rng(seed)
        cu = _lengths(rng, T, N)
        s["cu_seqlens"] = torch.from_numpy(cu.astype(np.int32)).to(DEV)
        seq = np.repeat(np.arange(N), np.diff(cu))
        prompt = (np.diff(cu) * rng.uniform(0.0, 0.4, N)).astype(np.int64)
        if N > 2:
            prompt[rng.integers(N)] = T  # a sequence without a scored token
        mask = np.arange(T) - cu[seq] >= prompt[seq]
        s["mask"] = torch.from_numpy(mask).to(DEV)
        s["logp"] = -_normal(gen, (T,)).abs()
        s["old_logp"] = s["logp"] + _normal(gen, (T,), 0.2)
        s["ref_logp"] = s["logp"] + _normal(gen, (T,), 0.3)
        s["entropy"] = _normal(gen, (T,)).abs()
        adv = _normal(gen, (N,))[torch.from_numpy(seq).to(DEV)]
        s["advantages"] = adv.contiguous()
    return s


# --------------------------------------------------------------------------- plain forms

def _plain_norm_fwd(s):
    x = s["x"].float()
    if s["case"]["kind"] == "layer":
        mean = x.mean(1)
        xc = x - mean[:, None]
    else:
        mean, xc = None, x
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
    y = xc * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = {"y": y.to(s["x"].dtype), "rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    return out


def _plain_norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    layer = s["mean"] is not None
    xh = (x - s["mean"][:, None]) * rstd if layer else x * rstd
    g = dy * s["weight"].float()
    t = g - xh * (g * xh).mean(1, keepdim=True)
    if layer:
        t = t - g.mean(1, keepdim=True)
    out = {"dx": (t * rstd).to(s["x"].dtype), "d_weight": (dy * xh).sum(0)}
    if layer:
        out["d_bias"] = dy.sum(0)
    return out


def _plain_i8(s):
    K, dt = s["case"]["k"], _DTYPE[s["case"]["dtype"]]
    # next to a rounding border binary32 would pick either side: the quotient is binary64
    x = s["x"].double()
    amax = x.abs().amax(1)
    q = torch.round(127.0 * x / torch.where(amax > 0, amax, 1.0)[:, None]).float()
    x_scale = (amax / 127.0).float()
    acc = torch.matmul(q, s["wq"][:, :K].float().t())  # whole numbers below 2^24: exact
    y = acc * x_scale[:, None] * s["w_scale"][None, :]
    return {"y": y.to(dt), "x_scale": x_scale}


def _plain_logprob(logits, ids, entropy):
    x = logits.float() * SCALE
    use = ids >= 0
    m = x.amax(1)
    x = x - m[:, None]
    e = torch.exp(x)
    total = e.sum(1)
    log_total = torch.log(total)
    chosen = x.gather(1, ids.clamp(min=0)[:, None])[:, 0]
    out = {"logp": torch.where(use, chosen - log_total, 0.0),
           "lse": torch.where(use, log_total + m, 0.0)}
    if entropy:
        out["entropy"] = torch.where(use, log_total - (e * x).sum(1) / total, 0.0)
    return out


def _plain_logprob_bwd(s):
    x = s["logits"].float() * SCALE
    use = s["ids"] >= 0
    logq = x - s["lse"][:, None]
    p = torch.exp(logq)
    g = torch.where(use, s["d_logp"], 0.0)
    d = -p * g[:, None]
    if s["d_entropy"] is not None:
        h = torch.where(use, s["d_entropy"], 0.0)
        d = d - h[:, None] * p * (logq + s["entropy"][:, None])
    d.scatter_add_(1, s["ids"].clamp(min=0)[:, None], g[:, None])
    d = torch.where(use[:, None], d * SCALE, 0.0)
    return {"d_logits": d.to(s["logits"].dtype)}


def _plain_policy(s):
    # binary64: the ratio is compared with the clip borders, and the sums are long
    logp, old, ref = s["logp"].double(), s["old_logp"].double(), s["ref_logp"].double()
    adv, ent, cu = s["advantages"].double(), s["entropy"].double(), s["cu_seqlens"].long()
    T = logp.numel()
    use = s["mask"]
    ratio = torch.exp(logp - old)
    lo, hi = 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH
    plain, clipped = ratio * adv, ratio.clamp(lo, hi) * adv
    gain = torch.minimum(plain, clipped)
    floor = DUAL_CLIP * adv
    held = (adv < 0) & (gain < floor)
    moves = (plain <= clipped) & ~held
    pg = -torch.where(held, floor, gain)
    gap = ref - logp
    kl = torch.exp(gap) - gap - 1.0
    cut = (~moves).double()
    zero = torch.zeros(1, dtype=torch.float64, device=DEV)

    def sums(v):
        c = torch.cat([zero, torch.cumsum(torch.where(use, v, 0.0), 0)])
        return c[cu[1:]] - c[cu[:-1]]

    count = sums(torch.ones_like(logp))
    if s["case"]["reduction"] == "sequence":
        live = (count > 0).double()
        weight = live / count.clamp(min=1.0) / live.sum().clamp(min=1.0)
    else:
        weight = torch.ones_like(count) / count.sum().clamp(min=1.0)
    terms = [(weight * sums(v)).sum() for v in (pg, kl, ent, cut)]
    loss = terms[0] + KL_COEF * terms[1] - ENTROPY_COEF * terms[2]
    seq = torch.searchsorted(cu[1:], torch.arange(T, device=DEV), right=True)
    wt = torch.where(use, weight[seq], 0.0)
    d = -torch.where(moves, plain, 0.0) + KL_COEF * (1.0 - torch.exp(gap))
    return {"stats": torch.stack([loss] + terms).float(),
            "d_logp": torch.where(use, wt * d, 0.0).float(),
            "d_entropy": (-ENTROPY_COEF * wt).float()}


# --------------------------------------------------------------------- the library's calls

_lib = None


def _api():
    global _lib
    if _lib is None:
        from bitwise_consistent_linear_amd import api
        _lib = api
    return _lib


def _own_norm_fwd(s):
    y, mean, rstd = _api().layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS,
                                          kind=s["case"]["kind"])
    return {"y": y, "rstd": rstd} if mean is None else {"y": y, "rstd": rstd, "mean": mean}


def _own_norm_bwd(s):
    dx, dw, db = _api().layer_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"],
                                       kind=s["case"]["kind"])
    out = {"dx": dx, "d_weight": dw}
    if s["mean"] is not None:
        out["d_bias"] = db
    return out


def _own_i8(s):
    api = _api()
    xq, x_scale = api.quantize_rows(s["x"])
    y = api.linear_i8_fwd(xq, x_scale, s["wq"], s["w_scale"],
                          out_dtype=_DTYPE[s["case"]["dtype"]])
    return {"y": y, "x_scale": x_scale}


def _own_logprob_fwd(s):
    logp, lse, entropy = _api().token_logprob_fwd(s["logits"], s["ids"], scale=SCALE,
                                                  entropy=s["case"]["entropy"])
    out = {"logp": logp, "lse": lse}
    if entropy is not None:
        out["entropy"] = entropy
    return out


def _own_logprob_bwd(s):
    return {"d_logits": _api().token_logprob_bwd(
        s["logits"], s["ids"], s["lse"], s["d_logp"], scale=SCALE, entropy=s["entropy"],
        d_entropy=s["d_entropy"])}


def _own_policy(s):
    api = _api()
    kw = dict(ref_logp=s["ref_logp"], entropy=s["entropy"], mask=s["mask"],
              cu_seqlens=s["cu_seqlens"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
              dual_clip=DUAL_CLIP, kl_coef=KL_COEF, entropy_coef=ENTROPY_COEF,
              reduction=s["case"]["reduction"])
    stats, weight = api.policy_loss_fwd(s["logp"], s["old_logp"], s["advantages"], **kw)
    d_logp, d_entropy = api.policy_loss_bwd(s["logp"], s["old_logp"], s["advantages"], weight,
                                            **kw)
    return {"stats": stats, "d_logp": d_logp, "d_entropy": d_entropy}


def run(state):
    op = state["case"]["op"]
    if op == "norm_fwd":
        return _own_norm_fwd(state) if own else _plain_norm_fwd(state)
    if op == "norm_bwd":
        return _own_norm_bwd(state) if own else _plain_norm_bwd(state)
    if op == "i8":
        return _own_i8(state) if own else _plain_i8(state)
    if op == "logprob_fwd":
        if own:
            return _own_logprob_fwd(state)
        return _plain_logprob(state["logits"], state["ids"], state["case"]["entropy"])
    if op == "logprob_bwd":
        return _own_logprob_bwd(state) if own else _plain_logprob_bwd(state)
    return _own_policy(state) if own else _plain_policy(state)


# ---------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        M, D, e = case["rows"], case["width"], _BYTES[case["dtype"]]
        stats = 8 * M if case["kind"] == "layer" else 4 * M
        if op == "norm_fwd":
            params = 2 * D * e if case["kind"] == "layer" else D * e
            return {"bytes": 2 * M * D * e + params + stats, "flops": 8 * M * D}
        grads = 8 * D if case["kind"] == "layer" else 4 * D
        return {"bytes": 3 * M * D * e + D * e + grads + stats, "flops": 16 * M * D}
    if op == "i8":
        M, N, K = case["m"], case["n"], case["k"]
        return {"bytes": 2 * M * K + N * K + 4 * (M + N) + M * N * _BYTES[case["dtype"]],
                "flops": 2 * M * N * K}
    if op in ("logprob_fwd", "logprob_bwd"):
        M, V, e = case["rows"], case["vocab"], _BYTES[case["dtype"]]
        scored = M - M // 16  # rows that are not scored need no reading
        if op == "logprob_fwd":
            return {"bytes": scored * V * e + M * (8 + (12 if case["entropy"] else 8)),
                    "flops": (7 if case["entropy"] else 5) * scored * V}
        return {"bytes": (scored + M) * V * e + M * (16 + (8 if case["entropy"] else 0)),
                "flops": (9 if case["entropy"] else 6) * scored * V}
    T = case["tokens"]
    return {"bytes": T * (5 * 4 + 1 + 2 * 4) + 4 * (case["seqs"] + 1) + 20, "flops": 40 * T}


# --------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The outputs of run() for these inputs from the definitions, in binary64."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm_fwd":
        x = s["x"].to(f64)
        D = case["width"]
        mean = x.sum(1) / D if case["kind"] == "layer" else torch.zeros(x.shape[0], dtype=f64,
                                                                        device=DEV)
        var = (x - mean[:, None]).square().sum(1) / D
        rstd = (var + EPS) ** -0.5
        y = (x - mean[:, None]) * (rstd[:, None] * s["weight"].to(f64))
        if case["kind"] == "layer":
            return {"y": y + s["bias"].to(f64), "rstd": rstd, "mean": mean}
        return {"y": y, "rstd": rstd}
    if op == "norm_bwd":
        x, dy, w, r = (s[k].to(f64) for k in ("x", "dy", "weight", "rstd"))
        D = case["width"]
        if case["kind"] == "layer":
            x = x - s["mean"].to(f64)[:, None]
        xh = x * r[:, None]
        gw = dy * w
        dot = torch.linalg.vecdot(gw, xh)[:, None] / D
        mid = gw.sum(1, keepdim=True) / D if case["kind"] == "layer" else 0.0
        out = {"dx": r[:, None] * (gw - mid - xh * dot),
               "d_weight": torch.linalg.vecdot(dy, xh, dim=0)}
        if case["kind"] == "layer":
            out["d_bias"] = dy.sum(0)
        return out
    if op == "i8":
        x = s["x"].to(f64)
        peak = x.abs().max(1).values
        q = torch.round(x / torch.where(peak == 0, torch.ones_like(peak), peak)[:, None] * 127.0)
        # where the quotient lies within rounding of a half, take the even neighbour exactly
        t = 127.0 * x
        low = torch.floor(t / torch.where(peak == 0, torch.ones_like(peak), peak)[:, None])
        rest = 2.0 * (t - low * peak[:, None]) - peak[:, None]
        near = rest.abs() <= 1e-9 * peak[:, None]
        even = torch.where(torch.remainder(low, 2.0) == 0, low, low + 1.0)
        side = torch.where(rest > 0, low + 1.0, torch.where(rest < 0, low, even))
        q = torch.where(near, side, q)
        y = torch.mm(q * (peak / 127.0)[:, None],
                     (s["wq"][:, :case["k"]].to(f64) * s["w_scale"].to(f64)[:, None]).t())
        return {"y": y, "x_scale": peak / 127.0}
    if op == "logprob_fwd":
        x = s["logits"].to(f64) * SCALE
        use = s["ids"] >= 0
        lse = torch.logsumexp(x, 1)
        logq = x - lse[:, None]
        logp = logq[torch.arange(case["rows"], device=DEV), s["ids"].clamp(min=0)]
        out = {"logp": logp * use, "lse": lse * use}
        if case["entropy"]:
            out["entropy"] = -(logq.exp() * logq).sum(1) * use
        return out
    if op == "logprob_bwd":
        use = (s["ids"] >= 0).to(f64)[:, None]
        x = s["logits"].to(f64) * SCALE
        x -= s["lse"].to(f64)[:, None]
        p = x.exp()
        d = p * -s["d_logp"].to(f64)[:, None]
        if case["entropy"]:
            x += s["entropy"].to(f64)[:, None]
            d -= x * p * s["d_entropy"].to(f64)[:, None]
        rows = torch.arange(case["rows"], device=DEV)
        d[rows, s["ids"].clamp(min=0)] += s["d_logp"].to(f64)
        return {"d_logits": d.mul_(SCALE).mul_(use)}
    return _exact_policy(case, s)


def _exact_policy(case, s):
    """On the host, a sequence at a time."""
    h = {k: s[k].cpu().numpy().astype(np.float64) for k in
         ("logp", "old_logp", "ref_logp", "advantages", "entropy")}
    use, cu = s["mask"].cpu().numpy(), s["cu_seqlens"].cpu().numpy()
    T = case["tokens"]
    r = np.exp(h["logp"] - h["old_logp"])
    A = h["advantages"]
    # per token: the clipped surrogate as a loss, bounded for negative advantages
    a = -A * r
    b = -A * np.clip(r, 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    worst = np.maximum(a, b)
    limit = -DUAL_CLIP * A
    capped = (A < 0) & (worst > limit)
    pg = np.where(capped, limit, worst)
    flat = capped | (a < b)
    u = h["ref_logp"] - h["logp"]
    kl = np.expm1(u) - u
    per = {"pg": pg, "kl": kl, "ent": h["entropy"], "cut": flat.astype(np.float64)}
    wt = np.zeros(T)
    spans = [np.arange(cu[n], cu[n + 1])[use[cu[n]:cu[n + 1]]] for n in range(len(cu) - 1)]
    spans = [t for t in spans if t.size]
    total = sum(t.size for t in spans)
    for t in spans:
        wt[t] = 1.0 / (t.size * len(spans)) if case["reduction"] == "sequence" else 1.0 / total
    m = {k: math.fsum(wt * v) for k, v in per.items()}
    loss = m["pg"] + KL_COEF * m["kl"] - ENTROPY_COEF * m["ent"]
    d = np.where(flat, 0.0, a) - KL_COEF * np.expm1(u)
    return {"stats": np.array([loss, m["pg"], m["kl"], m["ent"], m["cut"]]),
            "d_logp": wt * d, "d_entropy": -ENTROPY_COEF * wt}
