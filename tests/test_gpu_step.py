"""The operators around the policy head on the GPU against their plain forms (tests/step_ref.py):
8-bit quantisation and product with its gradients, sampling, AdamW and the gradient norm; rows that
do not depend on the batch around them, graphs, streams, outputs between patterns and the binding's
refusals."""

import math

import numpy as np
import pytest
import torch

import step_ref as R
from bitwise_consistent_linear_amd import api
from gpu_util import DEV

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rand(g, *shape, scale=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def same(a, b, label=""):
    """The same bits (8-bit types too)."""
    a, b = a.detach().cpu(), b.detach().cpu()
    assert a.dtype == b.dtype and a.shape == b.shape, label
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    equal = torch.equal(a.contiguous().view(view), b.contiguous().view(view))
    assert equal, f"the bits differ: {label}"


# --------------------------------------------------------------------------- quantisation

def held(q, scale):
    """Values and exponents that a quantised matrix holds, by its layout."""
    q, s = q.cpu(), scale.cpu().view(torch.uint8)
    rows, k = q.shape
    e = s.transpose(0, 1)[:rows].reshape(rows, -1)[:, :k // 128].long() - 127
    return q.float().double(), e


def check_quantized(x, q, scale, fmt):
    """Codes as values, NaN alike, and every byte of the scales, the padding included."""
    want, e = R.quantize(x, fmt)
    got, _ = held(q, scale)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))
    assert np.array_equal(scale.cpu().view(torch.uint8).numpy(), R.scale_bytes(e))


@pytest.mark.parametrize("rows,k", [(1, 1), (1, 7), (2, 8), (1, 127), (3, 128), (5, 129), (4, 512),
                                    (7, 513), (130, 640), (129, 1111), (257, 300)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize(rows, k, dtype, fmt):
    g = gen(rows * 10000 + k)
    x = (rand(g, rows, k) * torch.exp(4 * rand(g, rows, 1))).to(DTYPES[dtype])
    x[:, ::5] *= 2.0 ** -14  # values beside the format's lowest
    x[rows // 2, :k // 2] = 0.0
    d = x.to(DEV)
    q, s, qt, st = api.quantize_f8(d, fmt=fmt, layout="both")
    assert q.dtype == R.F8[fmt] and q.shape == (rows, -(-k // 128) * 128)
    assert qt.shape == (k, -(-rows // 128) * 128) and s.dtype == torch.float8_e8m0fnu
    check_quantized(x, q, s, fmt)
    check_quantized(x.t(), qt, st, fmt)
    for a, b in zip(api.quantize_f8(d, fmt=fmt), (q, s)):
        same(a, b, "rows alone")
    for a, b in zip(api.quantize_f8(d, fmt=fmt, layout="columns"), (qt, st)):
        same(a, b, "columns alone")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_values_that_matter(fmt):
    """Largest values at a border of the scale, beside it, subnormal, huge, nothing but zeros, and
    values that are not finite."""
    top = 1.75 * 2.0 ** R.EMAX[fmt]
    up, down = (float(np.nextafter(np.float32(top), np.float32(s))) for s in (np.inf, 0))
    peaks = [top, up, down, top * 2.0 ** -3, up * 2.0 ** 20, 2.0 ** -149, 2.0 ** -127, 2.0 ** -119,
             1.75 * 2.0 ** -119, 3.4e38, 1.75 * 2.0 ** 127, 1.0, 0.0]
    x = torch.zeros(len(peaks) + 3, 128)
    g = gen(9)
    for i, p in enumerate(peaks):
        x[i] = (torch.rand(128, generator=g) * 2 - 1) * torch.tensor(p)
        x[i, 3 * i % 128] = p
    x[-3, :4] = torch.tensor([float("nan"), 1.0, -3.0, 0.5])
    x[-2, :4] = torch.tensor([float("inf"), 1.0, -float("inf"), 0.5])
    x[-1] = float("nan")
    for layout, y in (("rows", x), ("both", x.t().contiguous())):
        out = api.quantize_f8(y.to(DEV), fmt=fmt, layout=layout)
        check_quantized(x, *out[-2:], fmt)


def test_quantize_strides():
    g = gen(11)
    wide = rand(g, 70, 400, dtype=BF16).to(DEV)
    for x in (wide[:, 3:303], wide[::2], wide[5:6], torch.as_strided(wide, (9, 200), (0, 1), 7)):
        for a, b in zip(api.quantize_f8(x, layout="both"),
                        api.quantize_f8(x.contiguous(), layout="both")):
            same(a, b)


def test_quantize_no_rows():
    q, s, qt, st = api.quantize_f8(torch.zeros(0, 200, device=DEV), layout="both")
    assert q.shape == (0, 256) and s.shape == (1, 0, 4) and qt.shape == (200, 0)
    assert st.shape == (0, 200, 4)


# -------------------------------------------------------------------------------- product

def operands(g, m, n, k, fmt="e4m3", whole=False):
    """X and W in 8 bits; whole: whole numbers to 3 (every sum of their products is exact)."""
    if whole:
        x, w = (torch.randint(-3, 4, s, generator=g).float() for s in ((m, k), (n, k)))
    else:
        x = rand(g, m, k) * torch.exp(2 * rand(g, m, 1))
        w = rand(g, n, k, scale=k ** -0.5)
    return (*api.quantize_f8(x.to(DEV), fmt=fmt), *api.quantize_f8(w.to(DEV)))


# Sizes of every kernel: few rows (16 columns a wave; 32 and 64 rows), tiles from 64 x 64 to 256 x
# 256; k of one block, of part and of several words of scales.
SIZES = [(1, 1, 1), (1, 64, 128), (16, 100, 130), (33, 70, 512), (40, 4100, 640), (70, 2500, 256),
         (64, 4200, 1100), (300, 1500, 700), (700, 1300, 520), (1000, 2100, 384), (515, 4500, 1536),
         (2050, 2050, 300), (4100, 4200, 260)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_product_of_whole_numbers(m, n, k, dtype):
    """Sums of at most 9 k whole numbers: exact in binary32, rounded once to bf16."""
    xq, xs, wq, ws = operands(gen(m + n + k), m, n, k, whole=True)
    y = api.linear_f8_fwd(xq, xs, wq, ws, out_dtype=DTYPES[dtype])
    x, w = (R.values(*held(q, s)).float().to(DEV) for q, s in ((xq, xs), (wq, ws)))
    same(y, (x @ w.t()).to(DTYPES[dtype]))


def bounds(xq, xs, wq, ws, dtype):
    """The exact product and how far the kernel's may be off: binary32 adds K products (2^-24 of
    sum |x w| each); bf16 cuts each product off 13 bits below the largest of its eight (8 2^-13 of
    that), adds likewise and rounds."""
    x, w = (R.values(*held(q, s)) for q, s in ((xq, xs), (wq, ws)))
    y, size = x @ w.t(), x.abs() @ w.abs().t()
    off = x.shape[1] * 2.0 ** -24 * size
    if dtype is BF16:
        p = x.abs().view(x.shape[0], 1, -1, 8) * w.abs().view(1, w.shape[0], -1, 8)
        off = off + 2.0 ** -10 * p.amax(3).sum(2)
        off = off + 2.0 ** -8 * (y.abs() + off)
    return y, off + 2.0 ** -149


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 33, 130), (33, 70, 640), (65, 300, 1100),
                                   (130, 260, 513)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_product(m, n, k, dtype, fmt):
    ops = operands(gen(m * n + k), m, n, k, fmt)
    y = api.linear_f8_fwd(*ops, out_dtype=DTYPES[dtype]).cpu().double()
    want, off = bounds(*ops, DTYPES[dtype])
    assert bool(((y - want).abs() <= off).all()), float(((y - want).abs() / off).max())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_product_rows_do_not_depend_on_the_batch(dtype, fmt):
    """A row of X, or of W, in products of other sizes (that take every kernel) gives the same
    bits: of operands 128 K k wide, in k that end inside a word of scales too."""
    for k in (4096, 1408):
        xq, xs, wq, ws = operands(gen(21), 2100, 4200, k, fmt)
        run = lambda a, b: api.linear_f8_fwd(  # noqa: E731
            xq[a].contiguous(), cut(xs, a), wq[b].contiguous(), cut(ws, b), out_dtype=DTYPES[dtype])
        whole = run(slice(0, 2100), slice(0, 4200))
        for a, b in [(slice(0, 1), slice(0, 4200)), (slice(3, 40), slice(0, 4200)),
                     (slice(7, 70), slice(100, 1000)), (slice(9, 500), slice(0, 2000)),
                     (slice(0, 1000), slice(17, 2000)), (slice(1000, 2100), slice(4100, 4200)),
                     (slice(2099, 2100), slice(4199, 4200)), (slice(0, 200), slice(0, 4200))]:
            same(run(a, b), whole[a, b], (k, a, b))


def cut(scale, rows):
    """The scales of some rows."""
    part = scale.view(torch.uint8)[:, rows]
    out = torch.full((part.shape[0], -(-part.shape[1] // 4) * 4, 4), 127, dtype=torch.uint8,
                     device=scale.device)
    out[:, :part.shape[1]] = part
    return out.view(torch.float8_e8m0fnu)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m", [5, 70, 600])
def test_product_of_values_next_to_nothing(m, fmt):
    """Blocks whose largest value is near 2^-116. A product to binary32 takes its values in bf16,
    whose least number is 2^-133: 2^-134 is a tie and becomes 0, powers of two above are held.
    Sums of powers of two 21 bits apart at most are exact."""
    g = gen(33)
    k, n = 384, 520
    x = torch.exp2(torch.randint(-131, -115, (m, k), generator=g).float())
    x[torch.rand(m, k, generator=g) < 0.2] = 0.0
    x[1, :] = 2.0 ** -134
    w = torch.exp2(torch.randint(100, 103, (n, k), generator=g).float())
    xq, xs = api.quantize_f8(x.to(DEV), fmt=fmt)
    wq, ws = api.quantize_f8(w.to(DEV))
    held_x, held_w = (R.values(*held(q, s)) for q, s in ((xq, xs), (wq, ws)))
    in_bf16 = held_x.clone()
    in_bf16[1] = 0.0
    same(api.linear_f8_fwd(xq, xs, wq, ws), (in_bf16 @ held_w.t()).float())
    y = api.linear_f8_fwd(xq, xs, wq, ws, out_dtype=BF16).cpu().double()
    want, off = bounds(xq, xs, wq, ws, BF16)
    assert bool(((y - want).abs() <= off).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_product_of_far_scales(dtype):
    """Scales at both ends, products that stay in binary32's range: whole numbers, so exact."""
    g = gen(31)
    x = torch.randint(-3, 4, (40, 256), generator=g).float()
    w = torch.randint(-3, 4, (50, 256), generator=g).float()
    for ex, ew in ((100, -100), (-110, 100), (60, 60), (-60, -40)):
        xq, xs = api.quantize_f8((x * 2.0 ** ex).to(DEV))
        wq, ws = api.quantize_f8((w * 2.0 ** ew).to(DEV))
        y = api.linear_f8_fwd(xq, xs, wq, ws, out_dtype=DTYPES[dtype])
        want = ((x @ w.t()).double() * 2.0 ** (ex + ew)).float().to(DTYPES[dtype])
        same(y.cpu(), want, (ex, ew))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m", [3, 200])
def test_product_of_nan(dtype, fmt, m):
    """What is multiplied out of a NaN or an infinity is not finite, and nothing else."""
    g = gen(33)
    x, w = rand(g, m, 300), rand(g, 5000, 300)
    x[1, 7] = float("nan")
    x[2, 200] = float("inf")
    w[4, 100] = float("nan")
    xq, xs = api.quantize_f8(x.to(DEV), fmt=fmt)
    wq, ws = api.quantize_f8(w.to(DEV))
    y = api.linear_f8_fwd(xq, xs, wq, ws, out_dtype=DTYPES[dtype]).cpu()
    bad = torch.zeros(y.shape, dtype=torch.bool)
    bad[1] = bad[2] = True
    bad[:, 4] = True
    assert torch.equal(~torch.isfinite(y), bad)


def test_product_over_no_k_and_of_nothing():
    e = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    f = lambda t: t.view(torch.float8_e4m3fn)  # noqa: E731
    z = lambda t: t.view(torch.float8_e8m0fnu)  # noqa: E731
    y = torch.full((3, 5), 7.0, device=DEV)
    out = api.linear_f8_fwd(f(e(3, 0)), z(e(0, 4, 4)), f(e(5, 0)), z(e(0, 8, 4)), y=y)
    assert out is y and float(y.abs().max()) == 0.0
    assert api.linear_f8_fwd(f(e(0, 128)), z(e(1, 0, 4)), f(e(5, 128)), z(e(1, 8, 4))).shape == (0, 5)


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 3, 130), (100, 300, 70), (300, 129, 700),
                                   (1000, 520, 260)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_backward(m, n, k, dtype, fmt):
    g = gen(m + 7 * n + k)
    x, w = rand(g, m, k), rand(g, n, k, scale=k ** -0.5)
    dy = (rand(g, m, n) * torch.exp(2 * rand(g, m, 1)) * 1e-4).to(DTYPES[dtype])
    wtq, wts = api.quantize_f8(w.to(DEV), layout="columns")
    xtq, xts = api.quantize_f8(x.to(DEV), layout="columns")
    dx, dw = api.linear_f8_bwd(dy.to(DEV), wtq, wts, xtq, xts, fmt=fmt)
    assert dx.dtype == DTYPES[dtype] and dw.dtype == F32
    dq, dqs, dtq, dts = api.quantize_f8(dy.to(DEV), fmt=fmt, layout="both")
    for got, ops, dt in ((dx, (dq, dqs, wtq, wts), DTYPES[dtype]), (dw, (dtq, dts, xtq, xts), F32)):
        if got.numel() * ops[0].shape[1] > 5e7 and dt is BF16:
            dt_got, ops = got[:64, :64], (ops[0][:64], cut(ops[1], slice(0, 64)), ops[2][:64],
                                          cut(ops[3], slice(0, 64)))
        else:
            dt_got = got
        want, off = bounds(*ops, dt)
        assert bool(((dt_got.cpu().double() - want).abs() <= off).all())
    # either alone, in other types, from strided rows
    same(api.linear_f8_bwd(dy.to(DEV), wtq, wts, fmt=fmt)[0], dx)
    none, dw16 = api.linear_f8_bwd(dy.to(DEV), xtq=xtq, xt_scale=xts, fmt=fmt, dw_dtype=BF16)
    assert none is None and dw16.dtype == BF16
    assert float((dw16.float() - dw).abs().max()) <= 0.02 * float(dw.abs().max())
    wide = torch.zeros(m, n + 5, dtype=dy.dtype, device=DEV)
    wide[:, 2:2 + n] = dy.to(DEV)
    for a, b in zip(api.linear_f8_bwd(wide[:, 2:2 + n], wtq, wts, xtq, xts, fmt=fmt), (dx, dw)):
        same(a, b)


@pytest.mark.parametrize("m,n,k", [(1024, 1024, 1024), (1021, 2049, 1111), (2048, 2048, 2048),
                                   (300, 700, 5000), (2000, 130, 900), (17, 2100, 4100)])
@pytest.mark.parametrize("dtypes", [(F32, F32), (BF16, BF16), (BF16, F32)], ids=str)
def test_backward_together_and_alone(m, n, k, dtypes):
    """Both gradients of one call, in one launch or two, are those of two calls."""
    g = gen(m + n + k)
    dy = rand(g, m, n).to(DEV)
    w = api.quantize_f8(rand(g, n, k, scale=k ** -0.5).to(DEV), layout="columns")
    x = api.quantize_f8(rand(g, m, k).to(DEV), layout="columns")
    dx, dw = api.linear_f8_bwd(dy, *w, *x, fmt="e5m2", dx_dtype=dtypes[0], dw_dtype=dtypes[1])
    same(dx, api.linear_f8_bwd(dy, *w, fmt="e5m2", dx_dtype=dtypes[0])[0])
    same(dw, api.linear_f8_bwd(dy, None, None, *x, fmt="e5m2", dw_dtype=dtypes[1])[1])


def test_backward_against_differences():
    """sum(dy Y) along steps of X and W that 8 bits hold, with dy that they hold: linear, so a
    difference is the gradient times the step, up to binary32's sums."""
    g = gen(41)
    m, n, k = 9, 11, 200
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).float().to(DEV)  # noqa: E731
    x, w, dy, vx, vw = whole(m, k), whole(n, k), whole(m, n), whole(m, k), whole(n, k)

    def loss(x, w):
        return float((dy * api.linear_f8_fwd(*api.quantize_f8(x), *api.quantize_f8(w))).sum())

    dx, dw = api.linear_f8_bwd(dy, *api.quantize_f8(w, layout="columns"),
                               *api.quantize_f8(x, layout="columns"))
    # whole numbers below 2^24 all through: equal
    assert loss(x + vx, w) - loss(x, w) == float((dx * vx).sum())
    assert loss(x, w + vw) - loss(x, w) == float((dw * vw).sum())


def test_backward_without_rows():
    g = gen(43)
    wtq, wts = api.quantize_f8(rand(g, 20, 30).to(DEV), layout="columns")
    xtq, xts = api.quantize_f8(torch.zeros(0, 30, device=DEV), layout="columns")
    dw = torch.full((20, 30), 3.0, device=DEV)
    dx, got = api.linear_f8_bwd(torch.zeros(0, 20, device=DEV), wtq, wts, xtq, xts, dw=dw)
    assert dx.shape == (0, 30) and got is dw and float(dw.abs().max()) == 0.0


# ------------------------------------------------------------------------------- sampling

def check_draw(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, label=""):
    """Ids equal; logp within binary32's rounding of differences of up to 64 and the library's
    logarithm (2^-23 of its size, 1e-6 in all)."""
    M = logits.shape[0]
    on = lambda v: v.to(DEV) if torch.is_tensor(v) else v  # noqa: E731
    of = lambda v, i: v[i].item() if torch.is_tensor(v) else v  # noqa: E731
    ids, logp = api.sample_tokens(logits if logits.is_cuda else logits.to(DEV), u.to(DEV),
                                  temperature=on(temperature), top_k=on(top_k), top_p=on(top_p),
                                  min_p=on(min_p))
    z = logits.cpu().float().numpy()
    for i in range(M):
        k = of(top_k, i)
        p = of(top_p, i)
        want, lp = R.draw(z[i], u[i].item(), of(temperature, i), k if k > 0 else 0,
                          1.0 if math.isnan(p) else p, of(min_p, i))
        assert int(ids[i]) == want, (label, i, int(ids[i]), want)
        assert abs(float(logp[i]) - lp) <= 1e-6 + 2.0 ** -23 * abs(lp), (label, i)
    return ids, logp


FILTERS = [dict(), dict(temperature=0.5), dict(temperature=3.0), dict(temperature=0.0),
           dict(top_k=1), dict(top_k=7), dict(top_k=900), dict(top_p=0.9), dict(top_p=1e-6),
           dict(top_p=0.0), dict(min_p=0.05), dict(min_p=1.0), dict(min_p=7.0),
           dict(top_k=40, top_p=0.8), dict(top_p=0.99, min_p=0.002),
           dict(temperature=0.7, top_k=60, top_p=0.9, min_p=0.01)]


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 64, 511, 513, 1000, 5003, 20000])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sample(vocab, dtype):
    g = gen(vocab)
    x = (rand(g, 6, vocab, scale=2.5)).to(DTYPES[dtype])
    x[1:3, :40] += 6.0
    u = torch.rand(6, generator=g)
    for f in FILTERS:
        check_draw(x, u, **f, label=f)


@pytest.mark.parametrize("rows,vocab", [(3, 131072), (300, 4000), (2, 262147)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sample_large(rows, vocab, dtype):
    g = gen(rows + vocab)
    x = rand(g, rows, vocab, scale=2.0).to(DTYPES[dtype])
    u = torch.rand(rows, generator=g)
    for f in (dict(), dict(top_k=50), dict(top_k=20000), dict(top_p=0.95),
              dict(top_k=3000, top_p=0.9, min_p=0.001), dict(temperature=8.0, top_p=0.7)):
        check_draw(x, u, **f, label=f)


@pytest.mark.parametrize("value", [0.0, -3.5, 1e30, -3.3895313892515355e38])
def test_sample_of_equal_logits(value):
    """One value all through, the type's lowest among them: ids go by their order alone."""
    for vocab in (100, 5000, 70000):
        x = torch.full((5, vocab), value, dtype=BF16)
        u = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.99999994])
        for f in (dict(), dict(top_k=30), dict(top_k=6000), dict(top_p=0.5), dict(top_p=0.001)):
            check_draw(x, u, **f, label=(vocab, f))


def test_sample_of_masked_logits():
    g = gen(51)
    inf, nan = float("inf"), float("nan")
    x = rand(g, 12, 3001, scale=2.0)
    x[0, :] = -inf                      # nothing left
    x[1, :] = -inf
    x[1, 2999] = -50.0                  # one token
    x[2, 5] = nan
    x[3, 5] = inf
    x[4, 10:] = -inf
    x[5, :] = torch.finfo(F32).min
    x[6, :] = torch.finfo(F32).min
    x[6, 17] = 0.0
    x[7, ::2] = -inf
    x[8] = -nan
    x[9, 0] = -nan
    x[10, :] = 0.0
    x[10, ::2] = -0.0                   # equal to 0: ids decide
    x[11, :] = torch.finfo(F32).max
    u = torch.rand(12, generator=g)
    for f in FILTERS:
        ids, logp = check_draw(x, u, **f, label=f)
        assert ids[[0, 2, 3, 8, 9]].tolist() == [-1] * 5 and not logp[[0, 2, 3, 8, 9]].any()


def test_sample_random_numbers():
    """The ends of [0, 1), what lies outside, binary64, and a comb of numbers that draws every
    token as often as its probability says, to one."""
    g = gen(53)
    x = rand(g, 1, 700, scale=2.0)
    for u in (0.0, 2.0 ** -149, 0.99999994, 1.0, 1.5, -0.5, float("inf"), float("nan")):
        check_draw(x, torch.tensor([u]), label=u)
    check_draw(x, torch.tensor([1.0 - 2.0 ** -53], dtype=torch.float64))
    check_draw(x, torch.tensor([0.1], dtype=torch.float64))
    n = 3000
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    few = x[:, :20]
    ids, _ = api.sample_tokens(few.to(DEV).expand(n, 20), u.to(DEV), temperature=0.7)
    p = torch.softmax(few[0].double() / 0.7, 0)
    counts = torch.bincount(ids.cpu(), minlength=20)
    assert float((counts - n * p).abs().max()) <= 1.0


def test_sample_parameters_of_each_row():
    g = gen(55)
    nan, inf = float("nan"), float("inf")
    n = 12
    x = rand(g, n, 2000, scale=2.0, dtype=BF16)
    u = torch.rand(n, generator=g)
    t = torch.tensor([1.0, 0.5, 0.0, nan, inf, -1.0, 1e-30, 2.0, 1.0, 1.0, 0.9, 1e30])
    k = torch.tensor([0, 5, 5, 5, 5, 5, 5, -3, 2000, 2 ** 31 - 1, 100, 3], dtype=torch.int32)
    p = torch.tensor([1.0, 0.9, 0.5, 0.5, 0.5, 0.5, 0.5, nan, -1.0, 0.3, 2.0, 0.9])
    least = torch.tensor([0.0, 0.1, 0.1, 0.1, 0.1, 0.1, 0.1, nan, -2.0, 0.01, 5.0, inf])
    ids, logp = check_draw(x, u, t, k, p, least)
    assert ids[3:6].tolist() == [-1] * 3 and not logp[3:6].any()
    # a row alone, with its parameters as numbers, and in int32
    for i in (0, 1, 2, 10):
        one = api.sample_tokens(x[i:i + 1].to(DEV), u[i:i + 1].to(DEV), temperature=t[i].item(),
                                top_k=k[i].item(), top_p=p[i].item(), min_p=least[i].item(),
                                id_dtype=torch.int32)
        assert one[0].dtype == torch.int32 and int(one[0]) == int(ids[i])
        same(one[1], logp[i:i + 1])


@pytest.mark.parametrize("rows,vocab", [(1, 32768), (2, 50021), (9, 40007), (70, 33001), (128, 33000)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sample_few_long_rows(rows, vocab, dtype):
    """Rows that several workgroups share: every kind of row among them, with every filter."""
    g = gen(rows * vocab)
    x = rand(g, rows, vocab, scale=2.0)
    inf = float("inf")
    kinds = [lambda r: r.mul_(0.001), lambda r: r.fill_(3.0), lambda r: r[1:].fill_(-inf),
             lambda r: r[:vocab - 2].fill_(-inf), lambda r: r.fill_(-inf), lambda r: r[5:6].fill_(inf),
             lambda r: r[vocab - 1:].fill_(float("nan")), lambda r: r.mul_(1e4),
             lambda r: r.fill_(torch.finfo(F32 if dtype == "f32" else BF16).min),
             lambda r: r[::2].fill_(7.5)]
    for i in range(rows):
        if i % 12 < len(kinds) and rows > 1:
            kinds[(i + rows) % 12 % len(kinds)](x[i])
    x = x.to(DTYPES[dtype])
    u = torch.rand(rows, generator=g)
    some = FILTERS if rows < 10 else [dict(top_k=50, top_p=0.95), dict(top_p=0.9)]
    for f in some + [dict(top_k=vocab // 2, top_p=0.5), dict(top_p=1 - 2.0 ** -24),
                     dict(temperature=0.01, top_k=300), dict(temperature=1e-9, top_p=0.9)]:
        check_draw(x, u, **f, label=f)


def test_sample_parameters_of_few_long_rows():
    g = gen(66)
    n, vocab = 12, 34567
    x = rand(g, n, vocab, scale=2.0, dtype=BF16)
    u = torch.rand(n, generator=g)
    t = torch.tensor([1.0, 0.5, 0.0, float("nan"), 1e30, -1.0, 1e-30, 2.0, 1.0, 1.0, 0.9, 0.8])
    k = torch.tensor([0, 5, 5, 5, 5, 5, 5, -3, 20000, 2 ** 31 - 1, 0, 0], dtype=torch.int32)
    p = torch.tensor([1.0, 0.9, 0.5, 0.5, 0.5, 0.5, 0.5, float("nan"), -1.0, 0.3, 0.999, 1.0])
    least = torch.tensor([0.0, 0.1, 0.1, 0.1, 0.1, 0.1, 0.1, float("nan"), -2.0, 0.01, 0.0, 0.2])
    check_draw(x, u, t, k, p, least)
    check_draw(x, u, t, 0, p, least)


def test_sample_rows_do_not_depend_on_the_batch():
    """Batches of other sizes, and so of other schedules."""
    g = gen(57)
    for dtype, vocab in ((F32, 150000), (BF16, 33333)):
        x = rand(g, 500, vocab, scale=2.0, dtype=dtype).to(DEV)
        u = torch.rand(500, generator=g).to(DEV)
        for f in (dict(), dict(top_p=0.9), dict(top_k=50, min_p=0.01)):
            ids, logp = api.sample_tokens(x, u, **f)
            for a, b in ((0, 1), (3, 11), (100, 180), (499, 500), (0, 300)):
                i, lp = api.sample_tokens(x[a:b], u[a:b], **f)
                same(i, ids[a:b], (f, a, b))
                same(lp, logp[a:b], (f, a, b))


def test_sample_strides():
    g = gen(59)
    wide = rand(g, 40, 3000, scale=2.0, dtype=BF16).to(DEV)
    u = torch.rand(40, generator=g).to(DEV)
    for x in (wide[:, 1:2002], wide[::2, 7:], torch.as_strided(wide, (9, 200), (0, 1), 7)):
        for f in (dict(), dict(top_k=20, top_p=0.9)):
            a = api.sample_tokens(x, u[:x.shape[0]], **f)
            b = api.sample_tokens(x.contiguous(), u[:x.shape[0]], **f)
            for s, t in zip(a, b):
                same(s, t)


def test_sample_far_rows():
    """Rows whose first element is more than 2^31 elements from the tensor's."""
    x = torch.zeros((5, 2 ** 29 + 64), dtype=BF16, device=DEV)
    g = gen(61)
    x[:, :1000] = rand(g, 5, 1000, scale=2.0, dtype=BF16).to(DEV)
    check_draw(x[:, :1000], torch.rand(5, generator=g), top_p=0.9)


def test_sample_no_rows():
    ids, logp = api.sample_tokens(torch.zeros(0, 9, device=DEV), torch.zeros(0, device=DEV))
    assert ids.shape == (0,) and logp.shape == (0,)


def test_sample_agrees_with_token_logprob():
    """Without filters the log-probability is token_logprob_fwd's (each within 1e-5 of the exact)."""
    g = gen(63)
    x = rand(g, 50, 9000, scale=3.0).to(DEV)
    u = torch.rand(50, generator=g).to(DEV)
    ids, logp = api.sample_tokens(x, u, temperature=0.8)
    other, _, _ = api.token_logprob_fwd(x, ids, scale=1 / 0.8)
    assert float((logp - other).abs().max()) <= 2e-5


# ------------------------------------------------------------------------------ optimiser

NUMELS = [1, 3, 4, 255, 256, 257, 0, 2047, 2048, 2049, 70001]


def make(seed, numels, pt, gt, eight, master, odd=False):
    """Lists of CPU tensors; odd: views that start one value into a buffer."""
    g = gen(seed)

    def each(dtype, scale=1.0, f=None):
        out = []
        for n in numels:
            t = torch.randn(n + 1, generator=g) * scale
            t = (f(t) if f else t).to(dtype)
            out.append(t[1:] if odd else t[:n].clone())
        return out

    s = {"p": each(pt), "g": each(gt, 0.1), "m": each(F32, 0.01),
         "v": each(F32, 0.01, lambda t: t * t)}
    if numels and numels[-1] > 600:
        s["m"][-1][:300] = 0.0
        s["v"][-1][:300] = 0.0
        s["g"][-1][:256] = 0.0
    s["master"] = [t.float() + 1e-4 * torch.randn(t.shape, generator=g) for t in s["p"]] if master else None
    if eight:
        packed = [R.pack_m(t) for t in s["m"]], [R.pack_r(t.sqrt()) for t in s["v"]]
        s["mc"], s["ms"] = ([a[i] for a in packed[0]] for i in (0, 1))
        s["vc"], s["vs"] = ([a[i] for a in packed[1]] for i in (0, 1))
    return s


HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def on_gpu(tensors, odd):
    if tensors is None:
        return None
    out = []
    for t in tensors:
        room = torch.zeros(t.numel() + 1, dtype=t.dtype, device=DEV)
        v = room[1:] if odd else room[:-1]
        v.copy_(t)
        out.append(v)
    return out


def step_both(s, eight, step, factor, odd):
    """One update on the GPU and in the plain form; the GPU's tensors and the plain ones."""
    d = {k: on_gpu(s[k], odd) for k in ("p", "g", "master")}
    kw = dict(HYPER, master=d["master"])
    if factor is not None:
        kw["grad_scale"] = torch.tensor([factor], device=DEV)
    if eight:
        d["m"] = [t.view(torch.float8_e4m3fn) for t in on_gpu(s["mc"], odd)]
        d["v"] = on_gpu(s["vc"], odd)
        d["ms"], d["vs"] = on_gpu(s["ms"], odd), on_gpu(s["vs"], odd)
        kw.update(m_scale=d["ms"], v_scale=d["vs"])
    else:
        d["m"], d["v"] = on_gpu(s["m"], odd), on_gpu(s["v"], odd)
    api.adamw_step(d["p"], d["g"], d["m"], d["v"], step, **kw)
    want = {k: [] for k in ("p", "m", "v", "ms", "vs", "master")}
    for i, p in enumerate(s["p"]):
        m = R.unpack_m(s["mc"][i], s["ms"][i]) if eight else s["m"][i]
        v = R.unpack_r(s["vc"][i], s["vs"][i]) ** 2 if eight else s["v"][i]
        w = s["master"][i] if s["master"] else p.float()
        w, m, v, r = R.adamw32(w, s["g"][i], m, v, step, HYPER["lr"], *HYPER["betas"],
                               HYPER["eps"], HYPER["weight_decay"], factor or 1.0)
        want["p"].append(w.to(p.dtype))
        want["master"].append(w)
        if eight:
            (m, ms), (v, vs) = R.pack_m(m), R.pack_r(r)
            want["ms"].append(ms)
            want["vs"].append(vs)
            m = m.view(torch.float8_e4m3fn)
        want["m"].append(m)
        want["v"].append(v)
    return d, want


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32), (F32, BF16)], ids=str)
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("step,factor,master", [(1, None, False), (1000, 0.37, True)])
def test_adamw(types, eight, odd, step, factor, master):
    """Every bit: parameters, states, scales, master weights."""
    master = master and types[0] is BF16
    s = make(step + odd, NUMELS, *types, eight, master, odd)
    d, want = step_both(s, eight, step, factor, odd)
    for name in ("p", "m", "v") + (("ms", "vs") if eight else ()) + (("master",) if master else ()):
        for i, n in enumerate(NUMELS):
            same(d[name][i], want[name][i], (name, n))
    if eight:
        for c, sc in ((d["m"], d["ms"]), (d["v"], d["vs"])):
            got = api.adamw_state_values(c[-1], sc[-1])
            code, scale = c[-1].cpu(), sc[-1].cpu()
            same(got, R.unpack_m(code, scale) if code.dtype != torch.uint8
                 else R.unpack_r(code, scale) ** 2)


def test_adamw_many_tensors():
    """More than one launch holds, empty ones between; the binary64 update within the roundings of
    one step of binary32 (12 of 2^-24 of values to 5)."""
    numels = [(37 * i) % 700 * (i % 3 > 0) for i in range(173)]
    s = make(5, numels, F32, F32, False, False)
    d, want = step_both(s, False, 3, None, False)
    for i in range(len(numels)):
        for name in ("p", "m", "v"):
            same(d[name][i], want[name][i], (name, i))
        p, _, _ = R.adamw64(s["p"][i], s["g"][i], s["m"][i], s["v"][i], 3, HYPER["lr"],
                            *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
        if numels[i]:
            assert float((d["p"][i].cpu().double() - p).abs().max()) <= 12 * 2.0 ** -24 * 5


def test_adamw_large_tensor():
    """A tensor past the launch's workgroups, whose places pass 2^31 bytes."""
    n = 600_000_007
    p = torch.ones(n, device=DEV)
    g, m, v = torch.full((n,), 0.5, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    api.adamw_step([p], [g], [m], [v], 1, **HYPER)
    for t in (p, m, v):
        assert float(t[0]) == float(t[-1]) and bool((t == t[0]).all())
    assert float(p[0]) != 1.0


def test_adamw_skips_a_factor_that_is_not_finite():
    for eight in (False, True):
        s = make(7, [300, 1000], BF16, BF16, eight, True)
        for bad in (float("nan"), float("inf"), -float("inf")):
            d, _ = step_both(s, eight, 2, bad, False)
            names = ["p", "master"] + (["ms", "vs"] if eight else ["m", "v"])
            for name in names:
                for got, was in zip(d[name], s[name]):
                    same(got, was, name)
            if eight:
                for got, was in zip(d["v"], s["vc"]):
                    same(got, was)


def test_adamw_step_and_rate_on_the_device():
    """int64 step and float32 rate in tensors: the same bits as numbers, and in a captured call
    that is replayed while they change."""
    s = make(9, [1000, 5], F32, F32, False, False)
    step, lr = torch.tensor([1], device=DEV), torch.tensor([1e-2], device=DEV)
    mine = {k: on_gpu(s[k], False) for k in "pgmv"}
    other = {k: on_gpu(s[k], False) for k in "pgmv"}
    call = lambda d, t, r: api.adamw_step(*[d[k] for k in "pgmv"], t, **dict(HYPER, lr=r))  # noqa: E731
    call({k: on_gpu(s[k], False) for k in "pgmv"}, step, lr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(mine, step, lr)
    for t in (1, 2, 3, 50, 100000):
        rate = 1e-2 / t
        step.fill_(t)
        lr.fill_(rate)
        graph.replay()
        call(other, t, float(torch.tensor(rate)))
        torch.cuda.synchronize()
        for k in "pmv":
            for a, b in zip(mine[k], other[k]):
                same(a, b, (t, k))


def test_adamw_marks_what_it_writes():
    p = torch.nn.Parameter(torch.ones(300, device=DEV))
    before = p._version
    api.adamw_step([p], [torch.ones(300, device=DEV)], [torch.zeros(300, device=DEV)],
                   [torch.zeros(300, device=DEV)], 1)
    assert p._version > before


def test_adamw_from_nothing():
    """8-bit states of zeros, steps in a row: blocks of zero gradients stay as they are but for the
    decay; the others move by the rate at first, as AdamW's first steps do (up to the rounding of
    the states from the second step on)."""
    n = 1024
    p = torch.zeros(n, device=DEV)
    g = torch.full((n,), 0.25, device=DEV)
    g[256:512] = 0.0
    m, v = torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn), torch.zeros(
        n, dtype=torch.uint8, device=DEV)
    ms, vs = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    for t in range(1, 6):
        api.adamw_step([p], [g], [m], [v], t, m_scale=[ms], v_scale=[vs], lr=1e-2, weight_decay=0.0)
    assert not p[256:512].any() and float(ms[1]) == float(vs[1]) == 0.0
    moved = p[g > 0]
    assert float((moved + 5e-2).abs().max()) <= 5e-2 * 2.0 ** -4


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("numels", [[], [0], [1], [5, 0, 300, 8191, 8192, 8193], [1000003],
                                    [17 * i % 400 for i in range(500)], [40_000_000, 3]], ids=len)
def test_grad_norm(dtype, numels):
    """Against binary64: rounded once."""
    g = gen(len(numels))
    lists = [rand(g, n, dtype=DTYPES[dtype]).to(DEV) for n in numels]
    norm, factor = api.grad_norm(lists, max_norm=2.0)
    want = math.sqrt(sum(float(t.double().square().sum()) for t in lists))
    assert abs(float(norm) - want) <= want * 2.0 ** -23
    assert abs(float(factor) - min(1.0, 2.0 / (want + 1e-6))) <= 2.0 ** -23
    assert float(api.grad_norm(lists)[1]) == 1.0
    again = api.grad_norm(lists, max_norm=2.0)
    same(again[0], norm)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_grad_norm_that_is_not_finite(bad):
    t = torch.ones(20000, device=DEV)
    t[12345] = bad
    norm, factor = api.grad_norm([torch.ones(5, device=DEV), t], max_norm=1.0)
    assert not math.isfinite(float(norm)) and math.isnan(float(factor))


def test_grad_norm_of_large_values():
    """Squares past binary32's range."""
    norm, factor = api.grad_norm([torch.full((4,), 1e30, device=DEV)], max_norm=1.0)
    assert float(norm) == pytest.approx(2e30, rel=1e-6) and float(factor) == pytest.approx(5e-31, rel=1e-6)


# ------------------------------------------------------- together, graphs, streams, refusals

def policy_step(s):
    """From hidden rows to updated weights: norm, 8-bit product, draw, log-probability, loss,
    gradients, clipped AdamW. In place on s['w'], s['m'] and so on."""
    y, mean, rstd = api.layer_norm_fwd(s["h"], s["gamma"], kind="rms")
    xq, xs, xtq, xts = api.quantize_f8(y, layout="both")
    wq, ws, wtq, wts = api.quantize_f8(s["w"], layout="both")
    logits = api.linear_f8_fwd(xq, xs, wq, ws, out_dtype=BF16)
    ids, _ = api.sample_tokens(logits, s["u"], temperature=0.8, top_p=0.9)
    logp, lse, _ = api.token_logprob_fwd(logits, ids, scale=1.25)
    stats, weight = api.policy_loss_fwd(logp, s["old"], s["adv"])
    d_logp, _ = api.policy_loss_bwd(logp, s["old"], s["adv"], weight)
    d_logits = api.token_logprob_bwd(logits, ids, lse, d_logp, scale=1.25)
    d_y, d_w = api.linear_f8_bwd(d_logits, wtq, wts, xtq, xts, fmt="e5m2", dx_dtype=F32)
    d_h, d_gamma, _ = api.layer_norm_bwd(d_y.to(BF16), s["h"], s["gamma"], mean, rstd, kind="rms")
    grads = [d_w, d_gamma]
    norm, factor = api.grad_norm(grads, max_norm=0.5)
    api.adamw_step([s["w"], s["gamma"]], grads, s["m"], s["v"], s["step"], m_scale=s["ms"],
                   v_scale=s["vs"], grad_scale=factor, lr=1e-2)
    return [logits, ids, logp, stats, d_logits, d_y, d_w, d_h, d_gamma, norm, factor]


def policy_state(seed):
    g = gen(seed)
    T, D, V = 200, 320, 1500
    sizes = [V * D, D]
    s = {"h": rand(g, T, D, dtype=BF16), "gamma": 1 + 0.1 * rand(g, D), "w": rand(g, V, D, scale=0.1),
         "u": torch.rand(T, generator=g), "old": -rand(g, T).abs() - 5, "adv": rand(g, T),
         "step": torch.tensor([4])}
    s = {k: v.to(DEV) for k, v in s.items()}
    s["m"] = [torch.zeros(n, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for n in sizes]
    s["v"] = [torch.zeros(n, dtype=torch.uint8, device=DEV) for n in sizes]
    s["ms"], s["vs"] = ([torch.zeros(-(-n // 256), device=DEV) for n in sizes] for _ in range(2))
    return s


def flat(s):
    return [t for v in s.values() for t in (v if isinstance(v, list) else [v])]


def test_step_together_and_in_a_graph():
    """One step as a user's program makes it, again, and captured: the same bits each time, with
    eager work between the replays."""
    eager = policy_state(71)
    want = policy_step(eager)
    torch.cuda.synchronize()
    for t in want:
        assert t.dtype == torch.int64 or bool(torch.isfinite(t).all())
    assert float(want[6].abs().max()) > 0 and float(want[9]) > 0
    s = policy_state(71)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = policy_step(s)
    for seed in (71, 72, 73, 71):
        for a, b in zip(flat(s), flat(policy_state(seed))):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        mine = policy_state(seed)
        for a, b in zip(out, policy_step(mine)):
            same(a, b, seed)
        for a, b in zip(flat(s), flat(mine)):
            same(a, b, seed)
    assert not torch.equal(eager["w"], policy_state(71)["w"])


def test_projection_gradients_are_near_the_linear_regions():
    """d_w and d_y against products of the unrounded operands: an 8-bit value is within 2^-4 (e4m3)
    or 2^-3 (e5m2) of it, so a product within 0.2 of sum |x w|."""
    s = policy_state(75)
    y = torch.randn(200, 320, device=DEV)
    dy = torch.randn(200, 1500, device=DEV)
    xtq, xts = api.quantize_f8(y, layout="columns")
    wtq, wts = api.quantize_f8(s["w"], layout="columns")
    dx, dw = api.linear_f8_bwd(dy, wtq, wts, xtq, xts, fmt="e5m2")
    for got, a, b in ((dx, dy, s["w"]), (dw, dy.t(), y)):
        want, size = a.cpu().double() @ b.cpu().double(), a.cpu().abs().double() @ b.cpu().abs().double()
        assert bool(((got.cpu().double() - want).abs() <= 0.2 * size).all())


def test_side_stream():
    s = policy_state(77)
    other = policy_state(77)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    xq, xs = api.quantize_f8(s["h"], stream=side)
    wq, ws, wtq, wts = api.quantize_f8(s["w"], layout="both", stream=side)
    logits = api.linear_f8_fwd(xq, xs, wq, ws, stream=side)
    ids, logp = api.sample_tokens(logits, s["u"], top_k=9, stream=side)
    dx, _ = api.linear_f8_bwd(logits, wtq, wts, stream=side)
    norm, factor = api.grad_norm([dx], max_norm=1.0, stream=side)
    api.adamw_step([s["w"]], [s["w"].clone()], s["m"][:1], s["v"][:1], 1, m_scale=s["ms"][:1],
                   v_scale=s["vs"][:1], grad_scale=factor, stream=side)
    val = api.adamw_state_values(s["v"][0], s["vs"][0], stream=side)
    side.synchronize()
    got = [xq, xs, wq, wts, logits, ids, logp, dx, norm, s["w"], val]
    xq, xs = api.quantize_f8(other["h"])
    wq, ws, wtq, wts = api.quantize_f8(other["w"], layout="both")
    logits = api.linear_f8_fwd(xq, xs, wq, ws)
    ids, logp = api.sample_tokens(logits, other["u"], top_k=9)
    dx, _ = api.linear_f8_bwd(logits, wtq, wts)
    norm, factor = api.grad_norm([dx], max_norm=1.0)
    api.adamw_step([other["w"]], [other["w"].clone()], other["m"][:1], other["v"][:1], 1,
                   m_scale=other["ms"][:1], v_scale=other["vs"][:1], grad_scale=factor)
    val = api.adamw_state_values(other["v"][0], other["vs"][0])
    for a, b in zip(got, [xq, xs, wq, wts, logits, ids, logp, dx, norm, other["w"], val]):
        same(a, b)


def framed(dtype, *shape):
    """A tensor inside a larger buffer of a pattern, and a check that the pattern stands."""
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    room = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    t = room[256:256 + n].view(dtype).view(shape)
    return t, lambda: bool((room[:256] == 0xA5).all() and (room[256 + n:] == 0xA5).all())


@pytest.mark.parametrize("m,n,k", [(3, 37, 200), (130, 5001, 333), (513, 1030, 129)])
def test_outputs_between_patterns(m, n, k):
    """Nothing is written outside an output, and no value of it is left."""
    g = gen(m)
    x, w = rand(g, m, k, dtype=BF16).to(DEV), rand(g, n, k).to(DEV)
    pad = lambda c: -(-c // 128) * 128  # noqa: E731
    shapes = {"q": (torch.float8_e4m3fn, m, pad(k)), "qt": (torch.float8_e4m3fn, k, pad(m)),
              "scale": (torch.float8_e8m0fnu, -(-k // 512), -(-m // 4) * 4, 4),
              "scale_t": (torch.float8_e8m0fnu, -(-m // 512), -(-k // 4) * 4, 4)}
    out = {name: framed(*s) for name, s in shapes.items()}
    api.quantize_f8(x, layout="both", **{name: t for name, (t, _) in out.items()})
    for name, (t, intact) in out.items():
        assert intact(), name
    for a, b in zip(api.quantize_f8(x, layout="both"), (out["q"], out["scale"], out["qt"],
                                                        out["scale_t"])):
        same(a, b[0])
    wq, ws, wtq, wts = api.quantize_f8(w, layout="both")
    for dtype in (F32, BF16):
        y, intact = framed(dtype, m, n)
        api.linear_f8_fwd(out["q"][0], out["scale"][0], wq, ws, y=y)
        assert intact()
        same(y, api.linear_f8_fwd(out["q"][0], out["scale"][0], wq, ws, out_dtype=dtype))
        dx, intact_x = framed(dtype, m, k)
        dw, intact_w = framed(dtype, n, k)
        api.linear_f8_bwd(y, wtq, wts, out["qt"][0], out["scale_t"][0], dx=dx, dw=dw)
        assert intact_x() and intact_w()
        ids, intact_i = framed(torch.int64, m)
        logp, intact_l = framed(F32, m)
        api.sample_tokens(y, torch.rand(m, device=DEV), top_p=0.9, ids=ids, logp=logp)
        assert intact_i() and intact_l() and bool((ids >= 0).all()) and bool((ids < n).all())
    for size in (n, 1, 255, 257):
        tensors = [framed(F32, size), framed(torch.float8_e4m3fn, size), framed(torch.uint8, size),
                   framed(F32, -(-size // 256)), framed(F32, -(-size // 256))]
        p, cm, cv, ms, vs = (t for t, _ in tensors)
        for t in (p, ms, vs):
            t.zero_()
        cm.view(torch.uint8).zero_()
        cv.zero_()
        api.adamw_step([p], [torch.ones(size, device=DEV)], [cm], [cv], 1, m_scale=[ms], v_scale=[vs])
        val, intact_v = framed(F32, size)
        api.adamw_state_values(cv, vs, out=val)
        assert intact_v() and all(intact() for _, intact in tensors)


def test_workspaces_may_hold_anything():
    g = gen(81)
    dy, w, x = rand(g, 70, 200).to(DEV), rand(g, 200, 300).to(DEV), rand(g, 70, 300).to(DEV)
    ops = (*api.quantize_f8(w, layout="columns"), *api.quantize_f8(x, layout="columns"))
    want = api.linear_f8_bwd(dy, *ops)
    shape = api.GdnLinearF8Shape(70, 200, 300, 200, 0, 0, 0, 0)
    for fill in (0, 0x7F, 0xFF):
        ws = torch.full((api.linear_f8_bwd_workspace_bytes(shape),), fill, dtype=torch.uint8, device=DEV)
        for a, b in zip(api.linear_f8_bwd(dy, *ops, workspace=ws), want):
            same(a, b)
        room = torch.full((1 << 16,), fill, dtype=torch.uint8, device=DEV)
        same(api.grad_norm([dy, w], workspace=room)[0], api.grad_norm([dy, w])[0])
        size = api.sample_tokens_workspace_bytes(api.GdnSampleShape(2, 150000, 150000, 0, 4, 8, 0, 1.0, 1.0, 0.0))
        logits, u = torch.zeros(2, 150000, device=DEV), torch.rand(2, generator=g).to(DEV)
        logits[:, ::3] = 1.0
        room = torch.full((max(size, 1),), fill, dtype=torch.uint8, device=DEV)
        for f in (dict(), dict(top_p=0.5), dict(top_k=9), dict(top_k=60000)):
            a = api.sample_tokens(logits, u, workspace=room if size else None, **f)
            for s, t in zip(a, api.sample_tokens(logits, u, **f)):
                same(s, t)


def test_binding_refuses():
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    q, s = api.quantize_f8(f(10, 200))
    w, ws = api.quantize_f8(f(20, 300))
    with pytest.raises(ValueError, match="rows of 256"):
        api.linear_f8_fwd(q, s, w, ws)
    with pytest.raises(ValueError, match="x_scale"):
        api.linear_f8_fwd(q, s[:, :4].contiguous(), q, s)
    with pytest.raises(TypeError, match="wq has dtype"):
        api.linear_f8_fwd(q, s, *api.quantize_f8(f(20, 200), fmt="e5m2"))
    with pytest.raises(ValueError, match="y must be"):
        api.linear_f8_fwd(q, s, q, s, y=f(10, 11))
    with pytest.raises(ValueError, match="wtq or xtq"):
        api.linear_f8_bwd(f(10, 20))
    with pytest.raises(ValueError, match="without its 8-bit operand"):
        api.linear_f8_bwd(f(10, 20), *api.quantize_f8(f(20, 30), layout="columns"), dw=f(20, 30))
    with pytest.raises(ValueError, match="xtq must be"):
        api.linear_f8_bwd(f(10, 20), xtq=q, xt_scale=s)
    with pytest.raises(ValueError, match="layout 'rows' has no qt"):
        api.quantize_f8(f(10, 20), qt=q)
    with pytest.raises(api.GdnError, match="k must be"):
        api.quantize_f8(f(1, 2 ** 20 + 1))
    with pytest.raises(ValueError, match="u must be"):
        api.sample_tokens(f(3, 9), f(4))
    with pytest.raises(TypeError, match="top_k has dtype"):
        api.sample_tokens(f(3, 9), f(3), top_k=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="top_k must be >= 0"):
        api.sample_tokens(f(3, 9), f(3), top_k=-1)
    with pytest.raises(api.GdnError, match="temperature"):
        api.sample_tokens(f(3, 9), f(3), temperature=-1.0)
    with pytest.raises(ValueError, match="contiguous inside a row"):
        api.sample_tokens(f(9, 3).t(), f(3))
    with pytest.raises(TypeError, match=r"grads\[1\] has dtype"):
        api.grad_norm([f(3), f(3).bfloat16()])
    with pytest.raises(ValueError, match=r"grads\[0\] must be contiguous"):
        api.grad_norm([f(9, 3).t()])
    one = [f(300)]
    with pytest.raises(ValueError, match=r"grads\[0\] must have 300 values"):
        api.adamw_step(one, [f(299)], [f(300)], [f(300)], 1)
    with pytest.raises(ValueError, match="together"):
        api.adamw_step(one, [f(300)], [f(300)], [f(300)], 1, m_scale=[f(2)])
    with pytest.raises(TypeError, match=r"m\[0\] has dtype"):
        api.adamw_step(one, [f(300)], [f(300)], [f(300)], 1, m_scale=[f(2)], v_scale=[f(2)])
    with pytest.raises(ValueError, match="master needs bfloat16"):
        api.adamw_step(one, [f(300)], [f(300)], [f(300)], 1, master=[f(300)])
    with pytest.raises(api.GdnError, match="step"):
        api.adamw_step(one, [f(300)], [f(300)], [f(300)], 0)
    with pytest.raises(ValueError, match="params has a tensor twice"):
        api.adamw_step(one * 2, [f(300), f(300)], [f(300), f(300)], [f(300), f(300)], 1)
    with pytest.raises(api.GdnError, match="two buffers of a tensor are the same"):
        m = f(300)
        api.adamw_step(one, [f(300)], [m], [m], 1)
    with pytest.raises(ValueError, match="scale must be"):
        api.adamw_state_values(torch.zeros(300, dtype=torch.uint8, device=DEV), f(1))
