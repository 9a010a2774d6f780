"""Plain forms of the operators of libgdn_step.so, on the CPU: 8-bit values by their format's
definition, the draw in whole numbers, AdamW operation by operation in binary32 and in binary64."""

import math

import numpy as np
import torch

EMAX = {"e4m3": 8, "e5m2": 15}
PLACES = {"e4m3": 3, "e5m2": 2}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def exponents(top, fmt):
    """The least whole e >= -127 with top <= 1.75 2^(emax + e), by trying; 0 for top = 0."""
    out = []
    for a in top.reshape(-1).tolist():
        e = 0
        if a > 0:
            e = -127
            if a > 1.75 * 2.0 ** (EMAX[fmt] + e):
                e = max(-127, math.frexp(a)[1] - EMAX[fmt] - 3)
                while a > 1.75 * 2.0 ** (EMAX[fmt] + e):
                    e += 1
        out.append(e)
    return torch.tensor(out, dtype=torch.int64).view(top.shape)


def round_f8(y, fmt):
    """Finite binary64 values of at most the format's largest, rounded to it, ties to even."""
    low = -6 if fmt == "e4m3" else -14
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** low))
    last = torch.ldexp(torch.ones_like(y), e - 1 - PLACES[fmt])
    return torch.round(y / last) * last


def quantize(x, fmt):
    """Values [R, 128 B] that q holds (in units of the scale) and exponents [R, B] of the rows of
    x, in binary64; NaN where the value is NaN (or an infinity, in e4m3)."""
    x = x.double()
    R, K = x.shape
    B = -(-K // 128)
    xb = torch.zeros((R, B * 128), dtype=torch.float64)
    xb[:, :K] = x
    xb = xb.view(R, B, 128)
    finite = torch.isfinite(xb)
    e = exponents(torch.where(finite, xb.abs(), 0.0).amax(2), fmt)
    y = torch.where(finite, xb, 0.0) * torch.pow(2.0, -e.double())[:, :, None]
    q = round_f8(y, fmt)
    bad = torch.full_like(q, float("nan"))
    if fmt == "e5m2":
        bad = torch.where(torch.isinf(xb), xb, bad)
    return torch.where(finite, q, bad).view(R, B * 128), e


def scale_bytes(e):
    """Exponents [R, B] in the layout of the scales."""
    R, B = e.shape
    out = np.full((-(-B // 4), -(-R // 4) * 4, 4), 127, np.uint8)
    for b in range(B):
        out[b // 4, :R, b % 4] = e[:, b].numpy() + 127
    return out


def values(q, e):
    return (q.view(e.shape[0], -1, 128) * torch.pow(2.0, e.double())[:, :, None]).view(q.shape)


def draw(x, u, T, top_k=0, top_p=1.0, min_p=0.0):
    """(id, logp) of one row of logits, weights as whole numbers."""
    x = np.asarray(x, np.float64)
    V = x.size
    if np.isnan(x).any() or x.max() == np.inf or x.max() == -np.inf:
        return -1, 0.0
    if not (0.0 <= T < np.inf):
        return -1, 0.0
    if T == 0.0:
        return int(np.argmax(x)), 0.0
    shift = min(45, 62 - max(0, (V - 1).bit_length()))
    z = (x - x.max()) / T
    w = np.rint(np.exp(z) * 2.0 ** shift).astype(np.int64)
    order = np.lexsort((np.arange(V), -x))
    n = V
    if 0 < top_k < V:
        n = int(top_k)
    if top_p < 1.0:
        cum = np.cumsum(w[order[:n]])
        a, b = float(top_p).as_integer_ratio() if top_p > 0 else (0, 1)
        target = max(1, -(-a * int(cum[-1]) // b))
        n = int(np.searchsorted(cum, target, side="left")) + 1
    kept = np.zeros(V, bool)
    kept[order[:n]] = True
    if min_p > 0:
        a, b = min(float(min_p), 1.0).as_integer_ratio()
        kept &= w >= -(-a * (1 << shift) // b)
    w = np.where(kept, w, 0)
    cum = np.cumsum(w)
    total = int(cum[-1])
    u = 0.0 if not u > 0 else float(u)
    if u >= 1.0:
        r = total - 1
    else:
        a, b = u.as_integer_ratio()
        r = a * total // b
    i = int(np.searchsorted(cum, r, side="right"))
    return i, float(z[i] - (math.log(total) - shift * math.log(2.0)))


# ------------------------------------------------------------------------------- optimiser

BLOCK = 256
ROOT_BASE = 119 << 23


def f32(v):
    return float(np.float32(v))


def constants(step, lr, b1, b2, wd):
    return dict(b1=f32(b1), c1=f32(1.0 - b1), b2=f32(b2), c2=f32(1.0 - b2),
                root=f32(1.0 / math.sqrt(1.0 - b2 ** step)), decay=f32(1.0 - lr * wd),
                rate=f32(lr / (1.0 - b1 ** step)))


def adamw32(p, g, m, v, step, lr, b1, b2, eps, wd, factor=1.0):
    """Flat binary32 tensors; every operation rounded by itself. Returns p, m, v, sqrt(v)."""
    k = {n: torch.tensor(c, dtype=torch.float32) for n, c in constants(step, lr, b1, b2, wd).items()}
    g = g.float() * torch.tensor(factor, dtype=torch.float32)
    m = m * k["b1"] + g * k["c1"]
    v = v * k["b2"] + (g * g) * k["c2"]
    # numpy's root is the correctly rounded one; torch's on the CPU is off by a unit in 0.6 %
    r = torch.from_numpy(np.sqrt(v.numpy()))
    u = m / (r * k["root"] + torch.tensor(f32(eps)))
    return p * k["decay"] - u * k["rate"], m, v, r


def adamw64(p, g, m, v, step, lr, b1, b2, eps, wd, factor=1.0):
    p, g, m, v = (t.double() for t in (p, g, m, v))
    g = g * factor
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * wd * p - lr * mh / (vh.sqrt() + eps), m, v


def _blocks(x, top):
    n = x.numel()
    xb = torch.zeros(-(-n // BLOCK) * BLOCK)
    xb[:n] = x
    xb = xb.view(-1, BLOCK)
    peak = xb.abs().amax(1)
    live = peak >= 2.0 ** -100
    one = torch.tensor(1.0)
    up = torch.where(live, one / torch.where(live, peak, one) * torch.tensor(top), 0.0)
    return xb * up[:, None], torch.where(live, peak * torch.tensor(f32(1.0 / top)), 0.0)


def pack_m(m):
    y, scale = _blocks(m, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:m.numel()], scale


def pack_r(r):
    y, scale = _blocks(r, 248.0)
    bits = y.view(torch.int32).long()
    c = ((bits - ROOT_BASE + 0x3FFFF + ((bits >> 19) & 1)) >> 19).clamp(1, 255)
    return torch.where(y > 0, c, 0).to(torch.uint8).view(-1)[:r.numel()], scale


def _spread(scale, n):
    return scale.repeat_interleave(BLOCK)[:n]


def unpack_m(c, scale):
    return c.view(torch.float8_e4m3fn).float() * _spread(scale, c.numel())


def unpack_r(c, scale):
    c = c.long()
    r = torch.where(c > 0, ((c << 19) + ROOT_BASE).to(torch.int32).view(torch.float32), 0.0)
    return r * _spread(scale, c.numel())
