"""Cases of the operators that close an on-policy step: tokens drawn from logits, the linear
region in 8-bit floating point with its gradients, and the AdamW update behind a clipped gradient
norm, each in a plain form of elementary torch operations (``own`` false) and through the
library's entry points (``own`` true).

A case names its operator and sizes; ``prepare`` draws its inputs on the GPU from a seed,
``run`` makes one pass, ``exact`` gives the pass's outputs from the definitions in binary64.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BLOCK = 128         # values that share a scale in the 8-bit products
GROUP = 4           # blocks whose scales lie side by side
STATE_BLOCK = 256   # values that share a scale in AdamW's 8-bit states

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_F8_EMAX = {"e4m3": 8, "e5m2": 15}


def listed():
    return [
        # a projection of 16 decoding sequences, width 32 heads x 128: the weights' bytes count
        {"name": "f8_fwd_decode", "op": "f8_fwd", "m": 16, "n": 4096, "k": 4096, "dtype": "bf16"},
        # the linear region's benchmark size, the trainer's 16384 tokens forward
        {"name": "f8_fwd_trainer", "op": "f8_fwd", "m": 16384, "n": 4096, "k": 4096,
         "dtype": "bf16"},
        # gradients through the vocabulary projection of 4096 tokens
        {"name": "f8_bwd_vocabulary", "op": "f8_bwd", "m": 4096, "n": 65536, "k": 4096,
         "dtype": "bf16", "fmt": "e4m3"},
        # gradients of odd sizes, binary32 in and out, the wider format for dy
        {"name": "f8_bwd_odd", "op": "f8_bwd", "m": 1021, "n": 2049, "k": 1111, "dtype": "f32",
         "fmt": "e5m2"},
        # one decode step of 8 sequences over a long vocabulary, temperature only
        {"name": "sample_decode", "op": "sample", "rows": 8, "vocab": 131072, "dtype": "f32",
         "top_k": 0, "top_p": 1.0, "min_p": 0.0},
        # 256 decoding sequences with a nucleus of their own each
        {"name": "sample_top_p", "op": "sample", "rows": 256, "vocab": 65536, "dtype": "bf16",
         "top_k": 0, "top_p": 0.95, "min_p": 0.0},
        # every filter at once over an odd vocabulary
        {"name": "sample_all", "op": "sample", "rows": 100, "vocab": 50021, "dtype": "f32",
         "top_k": 50, "top_p": 0.9, "min_p": 0.05},
        # a large rollout batch, temperature only
        {"name": "sample_rollout", "op": "sample", "rows": 512, "vocab": 131072, "dtype": "bf16",
         "top_k": 0, "top_p": 1.0, "min_p": 0.0},
        # a small layer and its policy head: a dozen tensors, most of them short
        {"name": "adamw_small", "op": "adamw", "tensors": 12, "values": 600000, "dtype": "f32",
         "state": "f32"},
        # layers in bfloat16 with binary32 master weights, many tensors of odd sizes
        {"name": "adamw_layers", "op": "adamw", "tensors": 200, "values": 60000000,
         "dtype": "bf16", "state": "f32"},
        # the vocabulary projection (65536 x 4096) and its neighbours with 8-bit states
        {"name": "adamw_8bit", "op": "adamw", "tensors": 6, "values": 280000000, "dtype": "bf16",
         "state": "8bit"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["f8_fwd", "f8_bwd", "sample", "sample", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "f32"])
    while True:
        if op in ("f8_fwd", "f8_bwd"):
            c = {"op": op, "dtype": dtype, "m": _log_uniform(rng, 1, 16384),
                 "n": _log_uniform(rng, 64, 65536), "k": _log_uniform(rng, 64, 16384)}
            if op == "f8_bwd":
                c["fmt"] = rng.choice(["e4m3", "e5m2"])
            fits = (c["m"] * c["n"] * c["k"] <= 16384 * 4096 * 4096
                    and max(c["m"] * c["n"], c["n"] * c["k"], c["m"] * c["k"]) <= 16384 * 8192)
        elif op == "sample":
            c = {"op": op, "dtype": dtype, "rows": _log_uniform(rng, 1, 2048),
                 "vocab": _log_uniform(rng, 1000, 262144),
                 "top_k": rng.choice([0, 0, _log_uniform(rng, 1, 2000)]),
                 "top_p": rng.choice([1.0, rng.uniform(0.5, 0.999)]),
                 "min_p": rng.choice([0.0, rng.uniform(0.001, 0.2)])}
            fits = c["rows"] * c["vocab"] * _BYTES[dtype] <= 512 * 131072 * 2
        else:
            c = {"op": op, "dtype": dtype, "state": rng.choice(["f32", "8bit"]),
                 "tensors": _log_uniform(rng, 1, 400), "values": _log_uniform(rng, 1000, 1e8)}
            fits = True
        if fits:
            return c


# ------------------------------------------------------------------------------- inputs

TEMPERATURE = 0.8
LR, BETAS, EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.1
MAX_NORM = 1.0


def _normal(gen, shape, scale=1.0):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale


def _sizes(rng, tensors, values):
    """Ragged sizes of at least one value that add up to `values`."""
    w = rng.lognormal(0.0, 1.5, tensors)
    cuts = np.floor(np.cumsum(w) / w.sum() * (values - tensors)).astype(np.int64)
    cuts[-1] = values - tensors
    return (np.diff(np.concatenate([[0], cuts])) + 1).tolist()


def _hidden(gen, rows, width, dt):
    """Rows of different size with a few large channels, as a layer's outputs have them."""
    x = _normal(gen, (rows, width))
    x *= 0.5 + 1.5 * torch.rand((rows, 1), generator=gen, device=DEV)
    x[:, torch.randint(0, width, (max(1, width // 100),), generator=gen, device=DEV)] *= 20.0
    return x.to(dt)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "f8_fwd":
        s["x"] = _hidden(gen, case["m"], case["k"], _DTYPE[case["dtype"]])
        # the weights are quantised and laid out once
        w = _normal(gen, (case["n"], case["k"]), 1.0 / math.sqrt(case["k"]))
        s["wq"], s["w_scale"] = _plain_quantize(w, "e4m3")
    elif op == "f8_bwd":
        dt = _DTYPE[case["dtype"]]
        m, n, k = case["m"], case["n"], case["k"]
        s["dy"] = (_normal(gen, (m, n)) * torch.exp(_normal(gen, (m, 1), 2.0)) * 1e-4).to(dt)
        # what the forward pass and the weights' layout leave: both by columns
        s["xtq"], s["xt_scale"] = _plain_quantize(_hidden(gen, m, k, dt).float().t(), "e4m3")
        w = _normal(gen, (n, k), 1.0 / math.sqrt(k))
        s["wtq"], s["wt_scale"] = _plain_quantize(w.t(), "e4m3")
    elif op == "sample":
        M, V, dt = case["rows"], case["vocab"], _DTYPE[case["dtype"]]
        logits = _normal(gen, (M, V), 2.0)
        # a policy prefers a few tokens of each row
        like = torch.randint(0, V, (M, 1), generator=gen, device=DEV)
        like = (like + torch.arange(40, device=DEV) * (V // 40)) % V
        logits.scatter_(1, like, _normal(gen, (M, 40), 3.0) + 9.0)
        s["logits"] = logits.to(dt)
        s["u"] = torch.rand((M,), generator=gen, device=DEV)
        # requests bring parameters of their own; what no request uses is a plain number
        s["temperature"] = TEMPERATURE + 0.4 * torch.rand((M,), generator=gen, device=DEV)
        s["top_k"], s["top_p"], s["min_p"] = case["top_k"], case["top_p"], case["min_p"]
        if case["top_k"]:
            s["top_k"] = torch.randint(1, 2 * case["top_k"] + 1, (M,), generator=gen, device=DEV,
                                       dtype=torch.int32)
        if case["top_p"] < 1.0:
            low = 0.5 * torch.rand((M,), generator=gen, device=DEV)
            s["top_p"] = 1.0 - (1.0 - case["top_p"]) * (0.5 + low)
        if case["min_p"]:
            s["min_p"] = case["min_p"] * (0.5 + torch.rand((M,), generator=gen, device=DEV))
    else:
        dt, eight = _DTYPE[case["dtype"]], case["state"] == "8bit"
        rng = np.random.default_rng(case["tensors"])  # a model's shapes stay as they are
        sizes = _sizes(rng, min(case["tensors"], case["values"]), case["values"])
        # flat buffers; every tensor starts at a multiple of the states' block
        room = [-(-n // STATE_BLOCK) * STATE_BLOCK for n in sizes]
        at = np.concatenate([[0], np.cumsum(room)]).tolist()
        total = at[-1]
        weights = _normal(gen, (total,), 0.02)
        s["param"] = weights.to(dt)
        s["master"] = weights if case["dtype"] == "bf16" and not eight else None
        s["grad"] = (_normal(gen, (total,), 1e-3)
                     * torch.exp(_normal(gen, (total // STATE_BLOCK, 1), 1.0))
                     .expand(-1, STATE_BLOCK).reshape(-1)).to(dt)
        m = _normal(gen, (total,), 3e-4)
        v = torch.square(_normal(gen, (total,), 1e-3)) + 1e-9
        inside = torch.zeros((total,), dtype=torch.bool, device=DEV)
        for n, a in zip(sizes, at):
            inside[a:a + n] = True
        for t in (s["param"], s["master"], s["grad"], m, v):
            if t is not None:
                t *= inside
        del inside
        if eight:
            s["m"], s["m_scale"] = _plain_pack_m(m)
            s["v"], s["v_scale"] = _plain_pack_v(torch.sqrt(v))
        else:
            s["m"], s["v"] = m, v
        s["step"] = 10

        def cut(t, per=1):
            return None if t is None else [t[a // per:a // per + -(-n // per)]
                                           for n, a in zip(sizes, at)]

        s["lists"] = {name: cut(s[name]) for name in ("param", "master", "grad", "m", "v")}
        if eight:
            s["lists"]["m_scale"] = cut(s["m_scale"], STATE_BLOCK)
            s["lists"]["v_scale"] = cut(s["v_scale"], STATE_BLOCK)
    return s


# --------------------------------------------------------------------------- plain forms

def _power(e):
    """2^e in binary32 for whole e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _plain_exponents(x, fmt):
    """Blocks [R, B, 128] of the rows of x, zeros behind their end, and the blocks' exponents."""
    R, K = x.shape
    B = -(-K // BLOCK)
    xb = torch.zeros((R, B * BLOCK), dtype=torch.float32, device=x.device)
    xb[:, :K] = x
    xb = xb.view(R, B, BLOCK)
    top = xb.abs().amax(2)
    part, e = torch.frexp(top)  # top = part 2^e, part in [0.5, 1)
    e = e - 1 - _F8_EMAX[fmt] + (part > 0.875).to(torch.int32)
    return xb, torch.where(top > 0, e.clamp(min=-127), 0).to(torch.int32)


def _plain_quantize(x, fmt):
    """Values [R, 128 B] in 8 bits and scales [ceil(B / 4), R rounded up to 4, 4]."""
    xb, e = _plain_exponents(x, fmt)
    R, B = e.shape
    q = (xb * _power(-e)[:, :, None]).to(_F8[fmt]).view(R, B * BLOCK)
    G = -(-B // GROUP)
    scale = torch.full((G, -(-R // 4) * 4, GROUP), 127, dtype=torch.uint8, device=x.device)
    padded = torch.full((R, G * GROUP), 127, dtype=torch.uint8, device=x.device)
    padded[:, :B] = (e + 127).to(torch.uint8)
    scale[:, :R] = padded.view(R, G, GROUP).transpose(0, 1)
    return q, scale.view(torch.float8_e8m0fnu)


def _plain_values(q, scale):
    """The values that q [R, Kp] and its scales stand for, in binary32."""
    R, K = q.shape
    e = scale.view(torch.uint8)[:, :R].transpose(0, 1).reshape(R, -1)[:, :K // BLOCK].to(
        torch.int32)
    # two factors: 2^-127 is no normal number
    half = (e - 127) >> 1
    x = q.float().view(R, -1, BLOCK) * _power(half)[:, :, None]
    return (x * _power(e - 127 - half)[:, :, None]).view(R, K)


def _plain_f8_fwd(s):
    xq, x_scale = _plain_quantize(s["x"].float(), "e4m3")
    y = torch.matmul(_plain_values(xq, x_scale), _plain_values(s["wq"], s["w_scale"]).t())
    return {"y": y.to(_DTYPE[s["case"]["dtype"]])}


def _plain_f8_bwd(s):
    c = s["case"]
    dt, dy = _DTYPE[c["dtype"]], s["dy"].float()
    dq = _plain_values(*_plain_quantize(dy, c["fmt"]))
    dx = torch.matmul(dq, _plain_values(s["wtq"], s["wt_scale"]).t())
    dtq = _plain_values(*_plain_quantize(dy.t(), c["fmt"]))
    dw = torch.matmul(dtq, _plain_values(s["xtq"], s["xt_scale"]).t())
    return {"dx": dx.to(dt), "dw": dw}


def _column(v):
    return v.double()[:, None] if torch.is_tensor(v) else v


def _plain_sample(s):
    # binary64: one random number is compared with sums over the vocabulary
    z = s["logits"].double()
    M, V = z.shape
    z = (z - z.amax(1, keepdim=True)) / _column(s["temperature"])
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    es = torch.exp(zs)
    keep = torch.ones((M, V), dtype=torch.bool, device=DEV)
    if torch.is_tensor(s["top_k"]):
        keep &= torch.arange(V, device=DEV)[None] < s["top_k"].long()[:, None]
    if torch.is_tensor(s["top_p"]):
        w = torch.where(keep, es, 0.0)
        cum = torch.cumsum(w, 1)
        keep &= cum - w < _column(s["top_p"]) * cum[:, -1:]
    if torch.is_tensor(s["min_p"]):
        keep &= es >= _column(s["min_p"])
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    cum = torch.cumsum(torch.where(kept, torch.exp(z), 0.0), 1)
    ids = (cum <= _column(s["u"]) * cum[:, -1:]).sum(1)
    logp = z.gather(1, ids[:, None])[:, 0] - torch.log(cum[:, -1])
    return {"ids": ids, "logp": logp.float()}


# AdamW's 8-bit states: m in e4m3 with its block's largest magnitude at 448; the root r of v in
# an unsigned float of 4 exponent and 4 fraction bits (code c > 0 stands for the binary32 whose
# bits are (c << 19) + _R_BASE, from 2^-8 (1 + 1/16) to 2^7 (1 + 15/16) = 248), its block's
# largest at 248. A root above 0 has a code above 0.
_R_BASE = 119 << 23
_R_TOP = 248.0
_M_TOP = 448.0
_TINY = 2.0 ** -100  # blocks whose largest value is below hold zeros


def _block_scales(x, top):
    """Blocks of x, 1 over their scales and the scales; blocks of (almost) nothing have 0, 0."""
    xb = x.view(-1, STATE_BLOCK)
    peak = xb.abs().amax(1)
    live = peak >= _TINY
    inv = torch.where(live, top / torch.where(live, peak, 1.0), 0.0)
    return xb, inv[:, None], torch.where(live, peak / top, 0.0)


def _plain_pack_m(m):
    xb, inv, scale = _block_scales(m, _M_TOP)
    return (xb * inv).to(torch.float8_e4m3fn).view(-1), scale


def _plain_pack_v(r):
    xb, inv, scale = _block_scales(r, _R_TOP)
    y = xb * inv
    bits = y.view(torch.int32)
    code = ((bits - _R_BASE + 0x3FFFF + ((bits >> 19) & 1)) >> 19).clamp(1, 255)
    return torch.where(y > 0, code, 0).to(torch.uint8).view(-1), scale


def _plain_unpack_m(m, scale):
    return (m.float().view(-1, STATE_BLOCK) * scale[:, None]).view(-1)


def _plain_unpack_r(v, scale):
    c = v.to(torch.int32)
    r = torch.where(c > 0, ((c << 19) + _R_BASE).view(torch.float32), 0.0)
    return (r.view(-1, STATE_BLOCK) * scale[:, None]).view(-1)


def _plain_adamw(s):
    # the buffers hold zeros between the tensors, which stay zeros
    eight = s["case"]["state"] == "8bit"
    (b1, b2), t = BETAS, s["step"]
    s["step"] += 1
    norm = s["grad"].double().square().sum().sqrt()
    factor = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0).float()
    g = s["grad"].float() * factor
    m = _plain_unpack_m(s["m"], s["m_scale"]) if eight else s["m"]
    m = m * b1 + g * (1.0 - b1)
    if eight:
        r = _plain_unpack_r(s["v"], s["v_scale"])
        v = r * r
    else:
        v = s["v"]
    v = v * b2 + (g * g) * (1.0 - b2)
    r = torch.sqrt(v)
    u = m / (r * (1.0 / math.sqrt(1.0 - b2 ** t)) + EPS)
    w = s["param"].float() if s["master"] is None else s["master"]
    w = w * (1.0 - LR * DECAY) - u * (LR / (1.0 - b1 ** t))
    s["param"].copy_(w)
    out = {"norm": norm.float(), "param": s["param"]}
    if s["master"] is not None:
        s["master"].copy_(w)
        out["master"] = s["master"]
    if eight:
        for name, packed in (("m", _plain_pack_m(m)), ("v", _plain_pack_v(r))):
            s[name].copy_(packed[0])
            s[name + "_scale"].copy_(packed[1])
        r = _plain_unpack_r(s["v"], s["v_scale"])
        return {**out, "m": _plain_unpack_m(s["m"], s["m_scale"]), "v": r * r}
    s["m"].copy_(m)
    s["v"].copy_(v)
    return {**out, "m": s["m"], "v": s["v"]}


# --------------------------------------------------------------------- the library's calls

_lib = None


def _api():
    global _lib
    if _lib is None:
        from bitwise_consistent_linear_amd import api
        _lib = api
    return _lib


def _own_f8_fwd(s):
    api = _api()
    xq, x_scale = api.quantize_f8(s["x"])
    return {"y": api.linear_f8_fwd(xq, x_scale, s["wq"], s["w_scale"],
                                   out_dtype=_DTYPE[s["case"]["dtype"]])}


def _own_f8_bwd(s):
    dx, dw = _api().linear_f8_bwd(s["dy"], s["wtq"], s["wt_scale"], s["xtq"], s["xt_scale"],
                                  fmt=s["case"]["fmt"], dx_dtype=_DTYPE[s["case"]["dtype"]])
    return {"dx": dx, "dw": dw}


def _own_sample(s):
    ids, logp = _api().sample_tokens(s["logits"], s["u"], temperature=s["temperature"],
                                     top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return {"ids": ids, "logp": logp}


def _own_adamw(s):
    api = _api()
    q, t = s["lists"], s["step"]
    s["step"] += 1
    eight = s["case"]["state"] == "8bit"
    norm, factor = api.grad_norm(q["grad"], max_norm=MAX_NORM)
    api.adamw_step(q["param"], q["grad"], q["m"], q["v"], t, m_scale=q.get("m_scale"),
                   v_scale=q.get("v_scale"), master=q["master"], lr=LR, betas=BETAS, eps=EPS,
                   weight_decay=DECAY, grad_scale=factor)
    out = {"norm": norm.view(()), "param": s["param"]}
    if s["master"] is not None:
        out["master"] = s["master"]
    if eight:
        return {**out, "m": api.adamw_state_values(s["m"], s["m_scale"]),
                "v": api.adamw_state_values(s["v"], s["v_scale"])}
    return {**out, "m": s["m"], "v": s["v"]}


def run(state):
    op = state["case"]["op"]
    if op == "f8_fwd":
        return _own_f8_fwd(state) if own else _plain_f8_fwd(state)
    if op == "f8_bwd":
        return _own_f8_bwd(state) if own else _plain_f8_bwd(state)
    if op == "sample":
        return _own_sample(state) if own else _plain_sample(state)
    return _own_adamw(state) if own else _plain_adamw(state)


# ---------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    e = _BYTES[case["dtype"]]
    if op == "f8_fwd":
        M, N, K = case["m"], case["n"], case["k"]
        return {"bytes": M * K * e + N * K + N * K // BLOCK + M * N * e, "flops": 2 * M * N * K}
    if op == "f8_bwd":
        M, N, K = case["m"], case["n"], case["k"]
        held = (N + M) * K
        return {"bytes": M * N * e + held + held // BLOCK + M * K * e + N * K * 4,
                "flops": 4 * M * N * K}
    if op == "sample":
        M, V = case["rows"], case["vocab"]
        return {"bytes": M * V * e + M * 20, "flops": 8 * M * V}
    n = case["values"]
    if case["state"] == "8bit":  # codes read and written; their values, which a pass returns
        each = 3 * e + 4 + 16 / STATE_BLOCK + 8
    else:
        each = 3 * e + 16 if e == 4 else 2 * e + 24
    return {"bytes": int(each * n), "flops": 20 * n}


# --------------------------------------------------------------------------------- exact

def _exact_f8(x, fmt):
    """The values that rows of x keep in 8 bits, from the format's definition, in binary64."""
    x = x.to(torch.float64)
    R, K = x.shape
    places, emax, low = (3, 8, -6) if fmt == "e4m3" else (2, 15, -14)
    xb = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(R, -1, BLOCK)
    top = xb.abs().amax(2, keepdim=True)
    unit = torch.exp2(torch.ceil(torch.log2(top / (1.75 * 2.0 ** emax))).clamp(min=-127.0))
    # beside a power of two the logarithm may round either way
    unit = torch.where(top > unit * 1.75 * 2.0 ** emax, unit * 2.0, unit)
    unit = torch.where((unit > 2.0 ** -127) & (top <= unit * 0.875 * 2.0 ** emax), unit * 0.5, unit)
    unit = torch.where(top > 0, unit, torch.ones_like(unit))
    y = xb / unit
    scale = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** low))))
    scale = torch.where(scale > y.abs().clamp(min=2.0 ** low), scale * 0.5, scale)
    scale = torch.where(2.0 * scale <= y.abs(), scale * 2.0, scale)
    last = scale * 2.0 ** -places
    return (torch.round(y / last) * last * unit).view(R, -1)


def _exact_held(q, scale):
    """Held values in binary64."""
    R, K = q.shape
    e = scale.view(torch.uint8)[:, :R].permute(1, 0, 2).reshape(R, -1)[:, :K // BLOCK]
    return q.to(torch.float32).to(torch.float64) * torch.exp2(
        e.to(torch.float64) - 127.0).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    """The outputs of run() for these inputs from the definitions, in binary64."""
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "f8_fwd":
        return {"y": _exact_f8(s["x"], "e4m3") @ _exact_held(s["wq"], s["w_scale"]).t()}
    if op == "f8_bwd":
        dx = _exact_f8(s["dy"], case["fmt"]) @ _exact_held(s["wtq"], s["wt_scale"]).t()
        return {"dx": dx, "dw": _exact_f8(s["dy"].t(), case["fmt"])
                @ _exact_held(s["xtq"], s["xt_scale"]).t()}
    if op == "sample":
        return _exact_sample(s)
    (b1, b2), t = BETAS, s["step"]
    g = s["grad"].to(f64)
    norm = torch.linalg.vector_norm(g)
    g = g * min(1.0, MAX_NORM / (float(norm) + 1e-6))
    eight = case["state"] == "8bit"
    if eight:
        # in binary32, as the states are held: beside a border the neighbours differ by a step
        m, r = _plain_unpack_m(s["m"], s["m_scale"]).to(f64), _plain_unpack_r(s["v"], s["v_scale"])
        v = r.to(f64) ** 2
    else:
        m, v = s["m"].to(f64), s["v"].to(f64)
    m = torch.lerp(m, g, 1.0 - b1)
    v = torch.lerp(v, g ** 2, 1.0 - b2)
    step = (m / (1.0 - b1 ** t)) / ((v / (1.0 - b2 ** t)) ** 0.5 + EPS)
    w = (s["param"] if s["master"] is None else s["master"]).to(f64)
    w = w - LR * (DECAY * w + step)
    out = {"norm": norm, "param": w}
    if s["master"] is not None:
        out["master"] = w
    if eight:
        # which neighbour a state rounds to hangs on its last bits: no value of its own
        return {**out, "m": None, "v": None}
    return {**out, "m": m, "v": v}


def _exact_sample(s):
    """On the host, a row at a time."""
    M, V = s["logits"].shape
    if M * V > 1 << 26:
        return None

    def host(v):
        v = v.double().cpu().numpy() if torch.is_tensor(v) else np.asarray(float(v))
        return np.broadcast_to(v, (M,))

    T, p, least, u = (host(s[k]) for k in ("temperature", "top_p", "min_p", "u"))
    k = host(s["top_k"]).astype(np.int64)
    rows = s["logits"].float().cpu().numpy()
    ids, logp = np.zeros(M, np.int64), np.zeros(M)
    for i in range(M):
        x = rows[i].astype(np.float64)
        z = (x - x.max()) / T[i]
        w = np.exp(z)
        floor = least[i]
        if k[i] or p[i] < 1.0:
            order = np.lexsort((np.arange(V), -x))
            n = k[i] if 0 < k[i] < V else V
            cum = np.cumsum(w[order[:n]])
            if p[i] < 1.0:
                n = int(np.searchsorted(cum, p[i] * cum[-1], side="left")) + 1
            kept = np.zeros(V, bool)
            kept[order[:n]] = True
            w = np.where(kept, w, 0.0)
        w = np.where(w >= floor, w, 0.0)
        cum = np.cumsum(w)
        ids[i] = np.searchsorted(cum, u[i] * cum[-1], side="right")
        logp[i] = z[ids[i]] - math.log(math.fsum(w))
    return {"ids": ids, "logp": logp}
