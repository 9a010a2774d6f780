"""The policy-head operators on the GPU against their plain 64-bit forms (policy_ref), at the
sizes, masks, strides and types where they can go wrong; the 8-bit product bit for bit; rows
that do not depend on the batch around them; graphs, streams and the binding's refusals."""

import numpy as np
import pytest
import torch

import policy_ref as R
from bitwise_consistent_linear_amd import api
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}


def rand(gen, *shape, scale=1.0, dtype=F32):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def same_bits(a, b, label):
    assert a.dtype == b.dtype and a.shape == b.shape, label
    kind = {4: torch.int32, 2: torch.int16, 1: torch.int8}[a.element_size()]
    assert torch.equal(a.contiguous().view(kind), b.contiguous().view(kind)), label


# ------------------------------------------------------------------------------------ norm

NORM_SIZES = [(1, 1), (3, 7), (5, 8), (300, 64), (17, 127), (9, 129), (700, 500), (33, 513),
              (5, 2048), (130, 2049), (257, 4096), (19, 4100), (7, 8192), (11, 8193), (5, 16384),
              (1100, 96)]


def norm_inputs(M, D, xt, wt, seed):
    g = gen(seed)
    x = rand(g, M, D, scale=1.5) + rand(g, M, 1, scale=0.7)
    return (x.to(xt), (1 + rand(g, D, scale=0.2)).to(wt), rand(g, D, scale=0.3, dtype=wt),
            rand(g, M, D, dtype=xt))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"),
                                   ("f32", "bf16")])
@pytest.mark.parametrize("M,D", NORM_SIZES)
def test_norm(M, D, xt, wt, kind):
    log(f"norm {kind} M={M} D={D} x={xt} w={wt}")
    x, w, b, dy = norm_inputs(M, D, DTYPES[xt], DTYPES[wt], M * 7 + D)
    b = b if kind == "layer" else None
    bias = None if b is None else b.to(DEV)
    y, mean, rstd = api.layer_norm_fwd(x.to(DEV), w.to(DEV), bias, eps=1e-5, kind=kind)
    (wy, ey), (wm, em), (wr, er) = R.norm_fwd_bounds(x, w, b, 1e-5, kind, x.dtype)
    R.check(y, wy, ey, "y")
    R.check(rstd, wr, er, "rstd")
    if kind == "layer":
        R.check(mean, wm, em, "mean")
    else:
        assert mean is None
    dx, dw, db = api.layer_norm_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd, kind=kind)
    hm = None if mean is None else mean.cpu()
    (wx, ex), (ww, ew), (wb, eb) = R.norm_bwd_bounds(dy, x, w, hm, rstd.cpu(), kind, x.dtype)
    R.check(dx, wx, ex, "dx")
    R.check(dw, ww, ew, "d_weight")
    if kind == "layer":
        R.check(db, wb, eb, "d_bias")
    else:
        assert db is None


@pytest.mark.parametrize("M,D", [(5000, 72), (6000, 1030)])
def test_norm_many_rows(M, D):
    """Rows enough for several walks of a workgroup, forward and backward."""
    x, w, b, dy = norm_inputs(M, D, BF16, BF16, 5)
    y, mean, rstd = api.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV))
    (wy, ey), _, _ = R.norm_fwd_bounds(x, w, b, 1e-5, "layer", BF16)
    R.check(y, wy, ey, "y")
    dx, dw, db = api.layer_norm_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd)
    (wx, ex), (ww, ew), (wb, eb) = R.norm_bwd_bounds(dy, x, w, mean.cpu(), rstd.cpu(), "layer",
                                                     BF16)
    R.check(dx, wx, ex, "dx")
    R.check(dw, ww, ew, "d_weight")
    R.check(db, wb, eb, "d_bias")


def test_norm_strides_in_place_and_no_rows():
    x, w, b, dy = (t.to(DEV) for t in norm_inputs(37, 200, F32, F32, 11))
    wide = torch.full((37, 331), float("nan"), device=DEV)
    wide[:, 100:300] = x
    wdy = torch.full((37, 203), float("nan"), device=DEV)
    wdy[:, 3:] = dy
    y0, m0, r0 = api.layer_norm_fwd(x, w, b)
    y1, m1, r1 = api.layer_norm_fwd(wide[:, 100:300], w, b)
    for p, q in ((y0, y1), (m0, m1), (r0, r1)):
        same_bits(p, q, "strided forward")
    for p, q in zip(api.layer_norm_bwd(dy, x, w, m0, r0),
                    api.layer_norm_bwd(wdy[:, 3:], wide[:, 100:300], w, m0, r0)):
        same_bits(p, q, "strided backward")
    one = x[:1].expand(37, 200)  # a stride of 0
    same_bits(api.layer_norm_fwd(one, w, b)[0], y0[:1].expand(37, 200), "repeated row")
    dx0, dw0, _ = api.layer_norm_bwd(dy, x, w, m0, r0)
    xin, din = x.clone(), dy.clone()
    api.layer_norm_fwd(xin, w, b, y=xin)
    same_bits(xin, y0, "y in x's place")
    api.layer_norm_bwd(din, x, w, m0, r0, dx=din)
    same_bits(din, dx0, "dx in dy's place")
    no = torch.empty((0, 200), device=DEV)
    assert api.layer_norm_fwd(no, w, b)[0].shape == (0, 200)
    _, dw, db = api.layer_norm_bwd(no, no, w, m0[:0], r0[:0])
    assert float(dw.abs().sum()) == 0.0 and float(db.abs().sum()) == 0.0
    dx, dw, db = api.layer_norm_bwd(dy, x, w, m0, r0, bias=False)
    assert db is None
    same_bits(dw, dw0, "without d_bias")


def test_norm_rms_with_bias():
    x, w, b, dy = norm_inputs(21, 300, BF16, F32, 12)
    y, _, rstd = api.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), kind="rms")
    (wy, ey), _, _ = R.norm_fwd_bounds(x, w, b, 1e-5, "rms", BF16)
    R.check(y, wy, ey, "y")
    _, _, db = api.layer_norm_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), None, rstd, kind="rms",
                                  bias=True)
    _, _, (wb, eb) = R.norm_bwd_bounds(dy, x, w, None, rstd.cpu(), "rms", BF16)
    R.check(db, wb, eb, "d_bias")


def test_norm_large_offset_constant_and_nonfinite_rows():
    """A mean a thousand times the spread costs the variance nothing; a constant row has
    variance 0 and eps alone; a NaN stays in its row."""
    g = gen(13)
    x = rand(g, 4, 1500) + 1000.0
    x[1] = 3.0
    w, b = torch.ones(1500), torch.zeros(1500)
    y, mean, rstd = api.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), eps=1e-5)
    (wy, ey), (wm, em), (wr, er) = R.norm_fwd_bounds(x, w, b, 1e-5, "layer", F32)
    R.check(y, wy, ey, "y")
    R.check(mean, wm, em, "mean")
    R.check(rstd, wr, er, "rstd")
    x[2, 700] = float("nan")
    z, _, _ = api.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), eps=1e-5)
    assert bool(z[2].isnan().all())
    for i in (0, 1, 3):
        same_bits(z[i], y[i], "rows beside a NaN")


@pytest.mark.parametrize("M,D", [(600, 4096), (600, 2049), (900, 100)])
def test_norm_rows_do_not_depend_on_the_batch(M, D):
    x, w, b, dy = (t.to(DEV) for t in norm_inputs(M, D, BF16, BF16, 14))
    y, mean, rstd = api.layer_norm_fwd(x, w, b)
    dx, _, _ = api.layer_norm_bwd(dy, x, w, mean, rstd)
    for lo, hi in ((0, 1), (M - 3, M), (57, 400)):
        y1, m1, r1 = api.layer_norm_fwd(x[lo:hi], w, b)
        d1, _, _ = api.layer_norm_bwd(dy[lo:hi], x[lo:hi], w, m1, r1)
        for p, q in ((y1, y), (m1, mean), (r1, rstd), (d1, dx)):
            same_bits(p, q[lo:hi], f"rows {lo}:{hi}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 513, 1038, 8195])
def test_rows_of_every_ending(D, dt):
    """A row's last values, 1 to 8 of a run of eight, through every kernel that reads rows: next
    to NaN on both sides, which must stay outside."""
    dt, M = DTYPES[dt], 5
    x, w, b, dy = norm_inputs(M, D, dt, dt, 80 + D)

    def guarded(t):
        wide = torch.full((t.shape[0] * t.shape[1] + 32,), float("nan"), dtype=dt, device=DEV)
        inner = wide[16:-16].view(t.shape)
        inner.copy_(t)
        return inner

    xd, dyd = guarded(x), guarded(dy)
    y, mean, rstd = api.layer_norm_fwd(xd, guarded(w[None])[0], guarded(b[None])[0])
    (wy, ey), _, _ = R.norm_fwd_bounds(x, w, b, 1e-5, "layer", dt)
    R.check(y, wy, ey, "y")
    dx, dw, db = api.layer_norm_bwd(dyd, xd, w.to(DEV), mean, rstd)
    (wx, ex), (ww, ew), (wb, eb) = R.norm_bwd_bounds(dy, x, w, mean.cpu(), rstd.cpu(), "layer", dt)
    R.check(dx, wx, ex, "dx")
    R.check(dw, ww, ew, "d_weight")
    R.check(db, wb, eb, "d_bias")
    q, s = api.quantize_rows(xd)
    wq, ws = R.quantize(x, -(-D // 128) * 128)
    assert torch.equal(q.cpu().to(torch.int64), wq)
    same_bits(s.cpu(), ws, "scale")
    ids = torch.tensor([0, D - 1, D // 2, -1, D - 1])
    logp, lse, ent = api.token_logprob_fwd(xd, ids.to(DEV), scale=0.8, entropy=True)
    for got, (want, bound), name in zip((logp, lse, ent), R.logprob_bounds(x, ids, 0.8),
                                        ("logp", "lse", "entropy")):
        R.check(got, want, bound, name)
    dlp = torch.ones(M)
    d = api.token_logprob_bwd(xd, ids.to(DEV), lse, dlp.to(DEV), scale=0.8, entropy=ent,
                              d_entropy=dlp.to(DEV))
    want, bound = R.logprob_bwd_bounds(x, ids, lse.cpu(), dlp, 0.8, ent.cpu(), dlp, dt)
    R.check(d, want, bound, "d_logits")
    # in place
    api.layer_norm_bwd(dyd, xd, w.to(DEV), mean, rstd, dx=dyd)
    same_bits(dyd, dx, "dx in dy's place")
    z = xd.clone()
    api.token_logprob_bwd(z, ids.to(DEV), lse, dlp.to(DEV), scale=0.8, entropy=ent,
                          d_entropy=dlp.to(DEV), d_logits=z)
    same_bits(z, d, "d_logits in the logits' place")
    api.layer_norm_fwd(xd, w.to(DEV), b.to(DEV), y=xd)
    same_bits(xd, y, "y in x's place")


# --------------------------------------------------------------------------- 8-bit product

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 5), (70, 127), (33, 129), (5, 500), (9, 2047),
                                 (130, 4096), (3, 8200), (2, 33000), (2, 65536)])
def test_quantize(M, K, dt):
    log(f"quantize M={M} K={K} {dt}")
    x = rand(gen(M + K), M, K, scale=3.0, dtype=DTYPES[dt])
    x[0, 0] = 0.0
    q, s = api.quantize_rows(x.to(DEV))
    wq, ws = R.quantize(x, -(-K // 128) * 128)
    assert torch.equal(q.cpu().to(torch.int64), wq)
    same_bits(s.cpu(), ws, "scale")


def test_quantize_ties_tiny_and_nonfinite_rows():
    """Every tie k + 1/2 of a row whose maximum is 127 and 63.5 (2^n / 254 steps), both signs;
    rows of zeros, of subnormal and of the largest values; NaN and infinities."""
    ties = (torch.arange(-127, 127) + 0.5)
    x = torch.zeros(9, 300)
    x[0, :254] = ties
    x[0, 299] = 127.0
    x[1] = x[0] / 2
    x[3, :254] = ties * 2.0 ** -133
    x[3, 299] = 127 * 2.0 ** -133
    x[4] = x[0] * 2.0 ** 120
    x[5, :7] = torch.tensor([1.0, -2.0, float("inf"), -float("inf"), 3.4e38, 0.0, -1.0])
    x[6, 5], x[6, 7] = float("nan"), 4.0
    x[7, 0] = 2.0 ** -133  # bfloat16's smallest
    x[8, 2], x[8, 3] = 2.0 ** -133, -3 * 2.0 ** -133
    for dt in (F32, BF16):
        xd = x.to(dt)
        finite = [0, 1, 2, 3, 4, 7, 8]
        q, s = (t.cpu() for t in api.quantize_rows(xd.to(DEV)))
        wq, ws = R.quantize(xd[finite], 384)
        assert torch.equal(q[finite].to(torch.int64), wq)
        same_bits(s[finite], ws, "scale")
        assert float(s[5]) == float("inf") and bool(s[6].isnan())
        assert q[5, :7].tolist() == ([0, 0, 127, -127, 0, 0, 0] if dt == F32 else
                                     q[5, :7].tolist()) and int(q[6].abs().sum()) == 0
        assert int(q[5, 2]) == 127 and int(q[5, 3]) == -127 and int(q[5, 0]) == 0


def test_quantize_strided_rows():
    x = rand(gen(3), 40, 301, dtype=BF16).to(DEV)
    a, b = api.quantize_rows(x[:, 7:280]), api.quantize_rows(x[:, 7:280].contiguous())
    for p, q in zip(a, b):
        same_bits(p, q, "strided rows")


I8_SIZES = [(1, 1, 128), (1, 300, 256), (3, 17, 128), (16, 64, 4096), (17, 130, 384),
            (33, 257, 1024), (64, 48, 8192), (65, 1000, 640), (100, 129, 128), (129, 255, 2048),
            (200, 1030, 512), (256, 512, 1152), (257, 300, 256), (513, 640, 384),
            (1000, 96, 256), (1300, 1100, 896), (8, 5000, 128), (2, 64, 65536),
            # tiles of 64 x 64, 64 x 128, 128 x 128 and 256 x 256, whole and ragged, with K of
            # an even and an odd number of 128-byte lines, one line among them
            (300, 4000, 128), (320, 4032, 512), (600, 4100, 384), (1024, 2048, 256),
            (1100, 4100, 384), (2048, 2048, 128), (3500, 3700, 384), (3841, 3585, 128),
            (200, 65537, 256),
            # K split over workgroups: few rows, tiles, parts of unequal length, odd columns
            (85, 69, 15744), (21, 568, 10752), (208, 2162, 13696), (400, 511, 16512),
            (130, 1001, 65536), (1, 1, 65536), (700, 700, 9344)]


@pytest.mark.parametrize("M,N,K", I8_SIZES)
def test_linear_i8(M, N, K):
    """All values of 8 bits, -128 among them: integer sums are exact, so are the outputs."""
    log(f"linear_i8 M={M} N={N} K={K}")
    g = gen(M + 3 * N + K)
    xq = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(M, generator=g) + 0.01, torch.rand(N, generator=g) + 0.01
    for dt in (F32, BF16):
        y = api.linear_i8_fwd(xq.to(DEV), xs.to(DEV), wq.to(DEV), ws.to(DEV), out_dtype=dt)
        same_bits(y.cpu(), R.linear_i8(xq, xs, wq, ws, dt), f"y {dt}")


def test_linear_i8_workspace():
    g = gen(23)
    xq = torch.randint(-128, 128, (20, 20480), generator=g, dtype=torch.int8).to(DEV)
    wq = torch.randint(-128, 128, (33, 20480), generator=g, dtype=torch.int8).to(DEV)
    s = torch.rand(33, generator=g).to(DEV)
    need = api.linear_i8_fwd_workspace_bytes(20, 33, 20480)
    assert need > 0
    room = torch.full((need + 64,), 85, dtype=torch.uint8, device=DEV)
    y = api.linear_i8_fwd(xq, s[:20], wq, s, workspace=room[:need])
    same_bits(y.cpu(), R.linear_i8(xq.cpu(), s[:20].cpu(), wq.cpu(), s.cpu(), F32), "y")
    assert bool((room[need:] == 85).all())
    with pytest.raises(api.GdnError, match="workspace"):
        api.linear_i8_fwd(xq, s[:20], wq, s, workspace=room[:need - 16])


def test_linear_i8_largest_sums():
    """65536 products of (-128)^2 reach 2^30; of 127 * -128, -2^30 and some."""
    for a, b in ((-128, -128), (127, -128)):
        xq = torch.full((20, 65536), a, dtype=torch.int8)
        wq = torch.full((40, 65536), b, dtype=torch.int8)
        one = torch.ones(40)
        y = api.linear_i8_fwd(xq.to(DEV), one[:20].to(DEV), wq.to(DEV), one.to(DEV))
        assert bool((y == float(np.float32(a * b * 65536))).all())


def test_linear_i8_rows_do_not_depend_on_the_batch():
    g = gen(21)
    xq, xs = api.quantize_rows(rand(g, 700, 1000, dtype=BF16).to(DEV))
    wq, ws = api.quantize_rows(rand(g, 900, 1000, dtype=BF16).to(DEV))
    y = api.linear_i8_fwd(xq, xs, wq, ws, out_dtype=BF16)
    for lo, hi in ((0, 1), (5, 21), (100, 150), (3, 400), (699, 700)):
        z = api.linear_i8_fwd(xq[lo:hi], xs[lo:hi], wq, ws, out_dtype=BF16)
        same_bits(z, y[lo:hi], f"rows {lo}:{hi}")


def test_quantized_product_is_near_the_exact_one():
    """Through both calls: each operand is off by half of its step, so a product of rows by
    half a step of one times the other's absolute sum (and the product of both halves)."""
    g = gen(22)
    x, w = rand(g, 50, 900, dtype=BF16), rand(g, 70, 900, scale=0.03, dtype=BF16)
    xq, xs = api.quantize_rows(x.to(DEV))
    wq, ws = api.quantize_rows(w.to(DEV))
    y = api.linear_i8_fwd(xq, xs, wq, ws)
    xd, wd = x.double(), w.double()
    hx, hw = xs.cpu().double()[:, None] / 2, ws.cpu().double()[None, :] / 2
    bound = (hx * wd.abs().sum(1)[None, :] + hw * xd.abs().sum(1)[:, None] + 900 * hx * hw)
    R.check(y, xd @ wd.t(), bound * 1.001, "y")


# ------------------------------------------------------------------------- log-probability

LP_SIZES = [(1, 1), (2, 2), (3, 7), (5, 8), (7, 9), (40, 1000), (9, 4096), (6, 4097), (5, 50021),
            (3, 65536), (17, 16385), (2, 131072)]


def lp_inputs(M, V, dt, seed, int32=False):
    g = gen(seed)
    z = rand(g, M, V, scale=2.5)
    ids = torch.randint(0, V, (M,), generator=g)
    z[torch.arange(M), ids] += 6.0
    if M > 2:
        ids[1], ids[2] = -1, V
    return z.to(dt), ids.to(torch.int32) if int32 else ids, rand(g, M), rand(g, M, scale=0.3)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.8, 1.7])
@pytest.mark.parametrize("M,V", LP_SIZES)
def test_logprob(M, V, scale, dt):
    log(f"logprob M={M} V={V} scale={scale} {dt}")
    z, ids, dlp, de = lp_inputs(M, V, DTYPES[dt], M + V, int32=scale == 1.0)
    zd, idd = z.to(DEV), ids.to(DEV)
    logp, lse, ent = api.token_logprob_fwd(zd, idd, scale=scale, entropy=True)
    for got, (want, bound), name in zip((logp, lse, ent), R.logprob_bounds(z, ids, scale),
                                        ("logp", "lse", "entropy")):
        R.check(got, want, bound, name)
    l1, s1, none = api.token_logprob_fwd(zd, idd, scale=scale)
    assert none is None
    same_bits(l1, logp, "logp without the entropy")
    same_bits(s1, lse, "lse without the entropy")
    d = api.token_logprob_bwd(zd, idd, lse, dlp.to(DEV), scale=scale, entropy=ent,
                              d_entropy=de.to(DEV))
    want, bound = R.logprob_bwd_bounds(z, ids, lse.cpu(), dlp, scale, ent.cpu(), de, z.dtype)
    R.check(d, want, bound, "d_logits with entropy")
    d = api.token_logprob_bwd(zd, idd, lse, dlp.to(DEV), scale=scale)
    want, bound = R.logprob_bwd_bounds(z, ids, lse.cpu(), dlp, scale, None, None, z.dtype)
    R.check(d, want, bound, "d_logits")
    api.token_logprob_bwd(zd, idd, lse, dlp.to(DEV), scale=scale, d_logits=zd)
    same_bits(zd, d, "in the logits' place")


def test_logprob_masks():
    """Masks of -inf and of the type's lowest value; a row of nothing else; one admissible
    token; the chosen token masked; NaN and +inf rows stay theirs."""
    inf, V = float("inf"), 3000
    for dt in (F32, BF16):
        low = torch.finfo(dt).min
        z, _, _, _ = lp_inputs(10, V, F32, 31)
        z = z.to(dt)
        ids = torch.tensor([5, 6, 7, 8, 9, 10, 11, 12, 13, 14])
        z[0, 100:] = -inf
        z[1, 100:] = low
        z[2, :] = -inf
        z[3, :] = low
        z[4, :] = -inf
        z[4, 9] = 2.0
        z[5, 10] = -inf
        z[6, 50] = float("nan")
        z[7, 50] = inf
        z[8, 1500:] = -inf
        z[8, :1400] = -inf
        z[9, :] = low
        z[9, 14] = torch.finfo(dt).max
        for scale in (0.8, 1.5):
            logp, lse, ent = (t.cpu().double() for t in api.token_logprob_fwd(
                z.to(DEV), ids.to(DEV), scale=scale, entropy=True))
            ok = [0, 1, 2, 4, 5, 8]
            for got, (want, bound), name in zip((logp, lse, ent),
                                                R.logprob_bounds(z[ok], ids[ok], scale),
                                                ("logp", "lse", "entropy")):
                R.check(got[ok], want, bound, f"{name} {dt} {scale}")
            # a row of the lowest value alone is uniform
            u = np.log(V)
            assert abs(float(logp[3]) + u) < 1e-5 and abs(float(ent[3]) - u) < 1e-5
            assert float(logp[4]) == 0.0 and float(ent[4]) == 0.0
            assert float(logp[9]) == 0.0 and float(ent[9]) == 0.0
            assert all(bool(v[i].isnan()) for v in (logp, lse) for i in (6, 7))
            dlp, de = torch.ones(10), torch.ones(10)
            d = api.token_logprob_bwd(z.to(DEV), ids.to(DEV), lse.float().to(DEV), dlp.to(DEV),
                                      scale=scale, entropy=ent.float().to(DEV),
                                      d_entropy=de.to(DEV))
            want, bound = R.logprob_bwd_bounds(z[ok], ids[ok], lse[ok].float(), dlp[ok], scale,
                                               ent[ok].float(), de[ok], dt)
            R.check(d[ok], want, bound, f"d_logits {dt} {scale}")
            assert float(d[2].abs().sum()) == 0.0  # nothing admissible


def test_logprob_strides_and_rows_alone():
    z, ids, dlp, de = lp_inputs(50, 20001, BF16, 32)
    wide = torch.full((50, 20100), 7.0, dtype=BF16)
    wide[:, :20001] = z
    zd, idd, wd = z.to(DEV), ids.to(DEV), wide.to(DEV)
    full = api.token_logprob_fwd(zd, idd, scale=0.9, entropy=True)
    for p, q in zip(full, api.token_logprob_fwd(wd[:, :20001], idd, scale=0.9, entropy=True)):
        same_bits(p, q, "strided rows")
    kw = dict(scale=0.9, entropy=full[2], d_entropy=de.to(DEV))
    d = api.token_logprob_bwd(zd, idd, full[1], dlp.to(DEV), **kw)
    same_bits(api.token_logprob_bwd(wd[:, :20001], idd, full[1], dlp.to(DEV), **kw), d, "strided")
    with pytest.raises(ValueError, match="contiguous"):
        api.token_logprob_bwd(zd, idd, full[1], dlp.to(DEV), d_logits=wd[:, :20001])
    for lo, hi in ((0, 1), (7, 11), (3, 49)):
        part = api.token_logprob_fwd(zd[lo:hi], idd[lo:hi], scale=0.9, entropy=True)
        for p, q in zip(part, full):
            same_bits(p, q[lo:hi], f"rows {lo}:{hi}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [98304, 98305, 131072, 196609, 262147])
def test_logprob_few_long_rows(V, dt):
    """Few rows of a long vocabulary are split over workgroups: against the 64-bit form, with
    whole parts masked, and the same bits as in a batch whose rows are not split."""
    inf = float("inf")
    z, ids, _, _ = lp_inputs(70, V, DTYPES[dt], V)
    z[3, :65536] = -inf
    z[4, 65536:] = -inf
    z[5, :] = -inf
    z[6, 1:] = torch.finfo(z.dtype).min
    z[7, V - 1] = inf
    z[8, 0] = float("nan")
    ids[3], ids[4], ids[9] = V - 1, 0, V - 1
    zd, idd = z.to(DEV), ids.to(DEV)
    full = api.token_logprob_fwd(zd, idd, scale=0.8, entropy=True)
    part = api.token_logprob_fwd(zd[:64], idd[:64], scale=0.8, entropy=True)
    for p, q in zip(part, full):
        same_bits(p.nan_to_num(7.0), q[:64].nan_to_num(7.0), "64 rows of 70")
    one = api.token_logprob_fwd(zd[9:10], idd[9:10], scale=0.8)
    same_bits(one[0], full[0][9:10], "a row alone, without the entropy")
    own = torch.empty(api.token_logprob_fwd_workspace_bytes(api.GdnLogprobShape(
        1, V, V, int(dt == "bf16"), 8, 0.8)), dtype=torch.uint8, device=DEV)
    assert own.numel() == (0 if V == 98304 else 1024 * 6 * (-(-V // 65536)))
    same_bits(api.token_logprob_fwd(zd[9:10], idd[9:10], scale=0.8, workspace=own)[1], one[1],
              "the caller's workspace")
    ok = [0, 1, 2, 3, 4, 5, 9, 63]
    for got, (want, bound), name in zip(part, R.logprob_bounds(z[ok], ids[ok], 0.8),
                                        ("logp", "lse", "entropy")):
        R.check(got[ok], want, bound, name)
    for v in part[:2]:
        assert bool(v[7].isnan()) and bool(v[8].isnan())


def test_logprob_gradient_against_differences():
    """The kernel's gradient against central differences of the 64-bit log-probability: off by
    the gradient's own bound and by the difference's step (h^2 / 6 times a third derivative of
    order 1, relative to the sums of |d|)."""
    z, ids, dlp, de = lp_inputs(8, 301, F32, 33)
    logp, lse, ent = api.token_logprob_fwd(z.to(DEV), ids.to(DEV), scale=0.8, entropy=True)
    d = api.token_logprob_bwd(z.to(DEV), ids.to(DEV), lse, dlp.to(DEV), scale=0.8, entropy=ent,
                              d_entropy=de.to(DEV)).cpu().double()
    v = torch.randn(8, 301, generator=gen(34), dtype=torch.float64)
    h = 1e-4

    def f(z):
        a, _, c = R.logprob(z, ids, 0.8)
        return float((a * dlp + c * de).sum())

    want = (f(z.double() + h * v) - f(z.double() - h * v)) / (2 * h)
    size = float(dlp.abs().sum() + de.abs().sum())
    assert abs(want - float((d * v).sum())) < 1e-5 * size


# ----------------------------------------------------------------------------- policy loss

def cut(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


POLICY_CASES = [("many", [37] * 513 + [0, 2, 70000] + [5] * 700), ("one", [1]), ("none scored", [5, 3]), ("tiny", [0, 1, 0, 0, 2, 1]),
                ("block edges", [256, 256, 255, 1, 257, 0, 513]), ("many short", [1] * 700),
                ("many empty", [0] * 300 + [40] + [0] * 300 + [1, 0]), ("long", [5000, 1, 9000]),
                ("mixed", [0, 3, 1000, 17, 2, 2, 2, 2500, 0]),
                # sequences inside 256 tokens, over their borders, and 62 to 65 of them at once
                ("ragged", [int(v) for v in np.random.default_rng(1).geometric(0.03, 200) - 1]),
                ("short and long", [int(v) for v in np.random.default_rng(2).choice(
                    [0, 1, 7, 60, 200, 255, 256, 257, 600], 90)]),
                ("63 in a chunk", [4] * 62 + [8] + [4] * 63 + [4] * 64 + [1] * 256 + [2] * 65),
                ("chunk of empty ones", [250] + [0] * 200 + [3] + [0] * 70 + [9])]


def policy_inputs(name, lengths, seed):
    rng = np.random.default_rng(seed)
    cu = cut(lengths)
    T = int(cu[-1])
    f = lambda s: (rng.normal(size=T) * s).astype(np.float32)  # noqa: E731
    logp = -np.abs(f(1.0))
    old, ref = logp + f(0.3), logp + f(0.3)
    mask = np.zeros(T, bool) if name == "none scored" else rng.random(T) < 0.7
    if name == "one":
        mask[:] = True
    return cu, logp, old, f(1.5), ref, np.abs(f(1.0)), mask


@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("terms", ["all", "plain"])
@pytest.mark.parametrize("name,lengths", POLICY_CASES, ids=[c[0] for c in POLICY_CASES])
def test_policy(name, lengths, terms, reduction):
    log(f"policy {name} {terms} {reduction}")
    cu, logp, old, adv, ref, ent, mask = policy_inputs(name, lengths, len(lengths))
    dual = 3.0
    if terms == "plain":
        ref = ent = dual = None
    up = lambda v: None if v is None else torch.from_numpy(v).to(DEV)  # noqa: E731
    junk = logp.copy()  # what is not scored may hold anything
    junk[~mask] = np.nan
    kw = dict(ref_logp=up(ref), entropy=up(ent), mask=up(mask), cu_seqlens=up(cu), clip_low=0.2,
              clip_high=0.28, dual_clip=dual, kl_coef=0.05, entropy_coef=0.01,
              reduction=reduction)
    stats, weight = api.policy_loss_fwd(up(junk), up(old), up(adv), **kw)
    dl, de = api.policy_loss_bwd(up(junk), up(old), up(adv), weight, d_loss=0.5, **kw)
    ws, ww, wl, we = R.policy(logp, old, adv, ref, ent, mask, cu, 0.2, 0.28, dual or 0.0, 0.05,
                              0.01, reduction)
    size = np.abs(ws[1:]).max(initial=0.0) + 1.0  # the loss's terms cancel
    R.check(stats, ws, torch.from_numpy(np.abs(ws) * R.POLICY_REL + R.POLICY_ABS * size), "stats")
    R.check(weight, ww, torch.from_numpy(np.abs(ww) * R.U), "weight")
    R.check(dl, 0.5 * wl, torch.from_numpy(np.abs(wl) * R.POLICY_REL + R.POLICY_ABS * 1e-3), "d_logp")
    if ent is None:
        assert de is None
    else:
        R.check(de, 0.5 * we, torch.from_numpy(np.abs(we) * R.POLICY_REL), "d_entropy")


def test_policy_without_mask_and_offsets():
    _, logp, old, adv, _, _, _ = policy_inputs("x", [3001], 8)
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    stats, weight = api.policy_loss_fwd(up(logp), up(old), up(adv))
    dl, de = api.policy_loss_bwd(up(logp), up(old), up(adv), weight)
    assert de is None
    ws, ww, wl, _ = R.policy(logp, old, adv, None, None, None, [0, 3001], 0.2, 0.2, 0.0, 0.0,
                             0.0, "token")
    R.check(stats, ws, torch.from_numpy(np.abs(ws) * R.POLICY_REL + R.POLICY_ABS), "stats")
    R.check(dl, wl, torch.from_numpy(np.abs(wl) * R.POLICY_REL + R.POLICY_ABS * 1e-3), "d_logp")
    no = torch.empty(0, device=DEV)
    stats, weight = api.policy_loss_fwd(no, no, no)
    assert stats.tolist() == [0.0] * 5 and weight.tolist() == [0.0]
    none = torch.zeros(1, dtype=torch.int32, device=DEV)
    stats, weight = api.policy_loss_fwd(no, no, no, cu_seqlens=none)
    assert stats.tolist() == [0.0] * 5 and weight.tolist() == []
    # no sequences and some tokens: none is any sequence's
    stats, weight = api.policy_loss_fwd(up(logp), up(old), up(adv), cu_seqlens=none)
    dl, _ = api.policy_loss_bwd(up(logp), up(old), up(adv), weight, cu_seqlens=none)
    assert stats.tolist() == [0.0] * 5 and float(dl.abs().sum()) == 0.0


def test_policy_long_batch():
    """More tokens than one chunk for each of the most spans: a wave walks over several chunks
    and carries a sequence from one to the next."""
    lengths = [700001, 3, 0, 255, 600000, 1]
    cu, logp, old, adv, ref, ent, mask = policy_inputs("x", lengths, 9)
    mask &= np.random.default_rng(10).random(len(mask)) < 0.02
    mask[-1] = True
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    for reduction in ("token", "sequence"):
        kw = dict(ref_logp=up(ref), entropy=up(ent), mask=up(mask), cu_seqlens=up(cu),
                  kl_coef=0.05, entropy_coef=0.01, reduction=reduction)
        stats, weight = api.policy_loss_fwd(up(logp), up(old), up(adv), **kw)
        dl, de = api.policy_loss_bwd(up(logp), up(old), up(adv), weight, **kw)
        ws, ww, wl, we = R.policy(logp, old, adv, ref, ent, mask, cu, 0.2, 0.2, 0.0, 0.05, 0.01,
                                  reduction)
        size = np.abs(ws[1:]).max() + 1.0
        R.check(stats, ws, torch.from_numpy(np.abs(ws) * R.POLICY_REL + R.POLICY_ABS * size),
                "stats")
        R.check(weight, ww, torch.from_numpy(np.abs(ww) * R.U), "weight")
        R.check(dl, wl, torch.from_numpy(np.abs(wl) * R.POLICY_REL + R.POLICY_ABS * 1e-3), "d_logp")
        R.check(de, we, torch.from_numpy(np.abs(we) * R.POLICY_REL), "d_entropy")


def test_policy_at_the_clip_borders():
    """Ratios a rounding away from the borders on either side: binary64 tells them apart as
    the definition does."""
    rows = []
    for border in (0.8, 1.28, 3.0):
        x = np.float32(np.log(border))
        for k in range(-6, 7):
            v = x
            for _ in range(abs(k)):
                v = np.nextafter(v, np.float32(np.inf if k > 0 else -np.inf))
            rows.append(v)
    logp = np.array(rows * 2, np.float32)
    adv = np.concatenate([np.ones(len(rows)), -np.ones(len(rows))]).astype(np.float32)
    old = np.zeros_like(logp)
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    kw = dict(clip_low=0.2, clip_high=0.28, dual_clip=3.0)
    stats, weight = api.policy_loss_fwd(up(logp), up(old), up(adv), **kw)
    dl, _ = api.policy_loss_bwd(up(logp), up(old), up(adv), weight, **kw)
    _, _, wl, _ = R.policy(logp, old, adv, None, None, None, [0, len(logp)], 0.2, 0.28, 3.0, 0.0,
                           0.0, "token")
    assert np.array_equal(dl.cpu().numpy() == 0.0, wl == 0.0)
    R.check(dl, wl, torch.from_numpy(np.abs(wl) * R.POLICY_REL), "d_logp")


def test_policy_next_to_the_reference():
    """A policy a few steps of binary32 from its reference: the KL term and its slope keep
    their relative accuracy, which exp(u) - u - 1 and 1 - exp(u) lose. Without an advantage
    nothing else is in the gradient. u in binary64 is exact, the KL's series too, so what is
    left are the outputs' roundings."""
    logp = np.full(64, -1e-4, np.float32)
    ref = logp.copy()
    for i in range(1, 64):
        ref[i] = np.nextafter(ref[i - 1], np.float32(0.0))
    ref[-9:] = logp[-9:] + np.float32([2**-7, -2**-7, 2**-6, -2**-6, 0.0157, -0.0157, 0.1, -1, 2])
    zero = np.zeros_like(logp)
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    u = ref.astype(np.float64) - logp.astype(np.float64)
    near = np.abs(u) < 0.1
    kl = np.where(near, u**2 / 2 + u**3 / 6 + u**4 / 24 + u**5 / 120 + u**6 / 720 + u**7 / 5040
                  + u**8 / 40320 + u**9 / 362880, np.expm1(u) - u)
    for part in (slice(0, 55), slice(55, 64)):
        kw = dict(ref_logp=up(ref[part].copy()), kl_coef=1.0)
        args = [up(v[part].copy()) for v in (logp, logp, zero)]
        stats, weight = api.policy_loss_fwd(*args, **kw)
        dl, _ = api.policy_loss_bwd(*args, weight, **kw)
        n = len(logp[part])
        want = -np.expm1(u[part]) / n
        R.check(dl, want, torch.from_numpy(np.abs(want) * R.POLICY_REL), "d_logp")
        mean = float(kl[part].mean())
        R.check(stats[2:3], torch.tensor([mean]), torch.tensor([mean * R.POLICY_REL]), "kl")


def test_policy_nan_stays():
    """A NaN among a scored token's inputs reaches the loss and that token's gradient alone."""
    _, logp, old, adv, _, _, _ = policy_inputs("x", [300], 71)
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    clean, weight = api.policy_loss_fwd(up(logp), up(old), up(adv))
    want, _ = api.policy_loss_bwd(up(logp), up(old), up(adv), weight)
    for k in range(3):
        args = [v.copy() for v in (logp, old, adv)]
        args[k][77] = np.nan
        args = [up(v) for v in args]
        stats, weight = api.policy_loss_fwd(*args)
        dl, _ = api.policy_loss_bwd(*args, weight)
        assert bool(stats[0].isnan()) and bool(stats[1].isnan()) and bool(dl[77].isnan())
        dl[77] = want[77]
        same_bits(dl, want, "the other tokens")


def test_policy_bad_offsets_stay_inside():
    """Offsets that fall, go below zero or past the end give wrong numbers, nothing else: the
    kernels clamp every start to [0, T] and every slot is below the number of slots."""
    T = 1000
    up = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    z = np.zeros(T, np.float32)
    for cu in ([0, 900, 100, 2**31 - 1], [-5, -7, 400, 1000], [1000, 0, 1000, 0]):
        c = up(np.array(cu, np.int64).astype(np.int32))
        stats, weight = api.policy_loss_fwd(up(z), up(z), up(z), cu_seqlens=c)
        dl, _ = api.policy_loss_bwd(up(z), up(z), up(z), weight, cu_seqlens=c)
        torch.cuda.synchronize()
        assert dl.shape == (T,) and weight.shape == (3,)


# ------------------------------------------------------------- buffers at odd elements

def odd(t):
    """The same values in a dense buffer that starts one element past an aligned place."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
    flat.copy_(t.reshape(-1))
    return flat.view(t.shape)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_buffers_at_odd_elements(dt):
    dt = DTYPES[dt]
    x, w, b, dy = (t.to(DEV) for t in norm_inputs(70, 1032, dt, dt, 61))
    y, mean, rstd = api.layer_norm_fwd(x, w, b)
    y1, _, _ = api.layer_norm_fwd(odd(x), odd(w), odd(b), y=odd(x))
    same_bits(y1, y, "norm")
    dx, dw, db = api.layer_norm_bwd(dy, x, w, mean, rstd)
    out = dict(dx=odd(x), d_weight=odd(dw), d_bias=odd(db))
    for p, q in zip(api.layer_norm_bwd(odd(dy), odd(x), odd(w), odd(mean), odd(rstd), **out),
                    (dx, dw, db)):
        same_bits(p, q, "norm backward")
    xq, xs = api.quantize_rows(x)
    xq1, xs1 = api.quantize_rows(odd(x), scale=odd(xs))
    same_bits(xq1, xq, "quantised")
    same_bits(xs1, xs, "scale")
    for rows, cols in ((5, 70), (70, 3000), (3000, 3000)):
        q = torch.randint(-127, 128, (max(rows, cols), 128), dtype=torch.int8).to(DEV)
        s = torch.rand(max(rows, cols)).to(DEV)
        want = api.linear_i8_fwd(q[:rows], s[:rows], q[:cols], s[:cols], out_dtype=dt)
        got = api.linear_i8_fwd(q[:rows], odd(s[:rows]), q[:cols], odd(s[:cols]), y=odd(want))
        same_bits(got, want, f"product {rows} x {cols}")
    z, ids, dlp, de = (t.to(DEV) for t in lp_inputs(9, 5000, dt, 62))
    logp, lse, ent = api.token_logprob_fwd(z, ids, entropy=True)
    for p, q in zip(api.token_logprob_fwd(odd(z), odd(ids), entropy=True, logp=odd(lse),
                                          lse=odd(lse)), (logp, lse, ent)):
        same_bits(p, q, "logp")
    kw = dict(entropy=ent, d_entropy=de)
    same_bits(api.token_logprob_bwd(odd(z), odd(ids), odd(lse), odd(dlp), d_logits=odd(z), **kw),
              api.token_logprob_bwd(z, ids, lse, dlp, **kw), "d_logits")


def test_product_of_tiny_scales():
    """Results among binary32's and bfloat16's subnormals are rounded, not flushed."""
    g = gen(63)
    xq = torch.randint(-127, 128, (300, 128), generator=g, dtype=torch.int8)
    wq = torch.randint(-127, 128, (500, 128), generator=g, dtype=torch.int8)
    xs, ws = torch.rand(300, generator=g) * 1e-20, torch.rand(500, generator=g) * 1e-23
    for m in (3, 300):
        for dt in (F32, BF16):
            y = api.linear_i8_fwd(xq[:m].to(DEV), xs[:m].to(DEV), wq.to(DEV), ws.to(DEV),
                                  out_dtype=dt)
            same_bits(y.cpu(), R.linear_i8(xq[:m], xs[:m], wq, ws, dt), f"y {m} {dt}")


# ------------------------------------------------------- element offsets past 2^31, bytes past 2^32

def test_long_norm_and_quantize():
    M, D = 540000, 4096
    x = torch.full((M, D), 0.5, dtype=BF16, device=DEV)
    tail = rand(gen(51), 70, D, dtype=BF16).to(DEV)
    x[-70:] = tail
    w = torch.ones(D, dtype=BF16, device=DEV)
    y, mean, rstd = api.layer_norm_fwd(x, w, w)
    y1, m1, r1 = api.layer_norm_fwd(tail, w, w)
    for p, q in ((y[-70:], y1), (mean[-70:], m1), (rstd[-70:], r1)):
        same_bits(p, q, "norm's last rows")
    dx, dw, db = api.layer_norm_bwd(x, x, w, mean, rstd)
    d1, dw1, _ = api.layer_norm_bwd(tail, tail, w, m1, r1)
    same_bits(dx[-70:], d1, "dx's last rows")
    # the constant rows' normalised values are 0: d_weight is the last rows' alone; the bound
    # is the sums' own, twice (two orders of addition)
    xh = (tail.double() - m1.double()[:, None]) * r1.double()[:, None]
    bound = 2 * (R.ROWS_DEPTH + 4) * R.U * (tail.double() * xh).abs().sum(0).cpu()
    R.check(dw, dw1.cpu().double(), bound, "d_weight")
    q, s = api.quantize_rows(x)
    q1, s1 = api.quantize_rows(tail)
    same_bits(q[-70:], q1, "q's last rows")
    same_bits(s[-70:], s1, "scale's last rows")


def test_long_product():
    g = gen(52)
    M, N = 33000, 66000
    xq = torch.randint(-127, 128, (M, 128), generator=g, dtype=torch.int8).to(DEV)
    wq = torch.randint(-127, 128, (N, 128), generator=g, dtype=torch.int8).to(DEV)
    xs, ws = torch.rand(M, generator=g).to(DEV), torch.rand(N, generator=g).to(DEV)
    y = api.linear_i8_fwd(xq, xs, wq, ws, out_dtype=BF16)
    z = api.linear_i8_fwd(xq[-90:], xs[-90:], wq, ws, out_dtype=BF16)
    same_bits(y[-90:], z, "last rows")
    want = R.linear_i8(xq[-90:].cpu(), xs[-90:].cpu(), wq[-200:].cpu(), ws[-200:].cpu(), BF16)
    same_bits(z[:, -200:].contiguous().cpu(), want, "last rows and columns")


def test_long_logits():
    M, V = 33000, 65537
    z = torch.zeros((M, V), dtype=BF16, device=DEV)
    tail, ids, dlp, de = (t.to(DEV) for t in lp_inputs(60, V, BF16, 53))
    z[-60:] = tail
    every = torch.full((M,), -1, dtype=torch.int64, device=DEV)
    every[-60:] = ids
    dl = torch.zeros(M, device=DEV)
    dl[-60:] = dlp
    logp, lse, _ = api.token_logprob_fwd(z, every)
    logp1, lse1, _ = api.token_logprob_fwd(tail, ids)
    same_bits(logp[-60:], logp1, "logp's last rows")
    same_bits(lse[-60:], lse1, "lse's last rows")
    assert float(logp[:-60].abs().sum()) == 0.0
    d1 = api.token_logprob_bwd(tail, ids, lse1, dlp)
    d = api.token_logprob_bwd(z, every, lse, dl, d_logits=z)
    same_bits(d[-60:], d1, "d_logits' last rows")


def test_more_rows_than_one_launch_holds():
    """2^26 rows and some of a small vocabulary: more threads than one launch can have."""
    M, V = 2**26 + 70, 5
    z = torch.zeros((M, V), dtype=BF16, device=DEV)
    tail, ids, dlp, de = (t.to(DEV) for t in lp_inputs(70, V, BF16, 54))
    z[-70:] = tail
    every = torch.zeros(M, dtype=torch.int32, device=DEV)
    every[-70:] = ids
    dl = torch.ones(M, device=DEV)
    dl[-70:] = dlp
    logp, lse, ent = api.token_logprob_fwd(z, every, entropy=True)
    logp1, lse1, ent1 = api.token_logprob_fwd(tail, ids.to(torch.int32), entropy=True)
    for p, q in ((logp, logp1), (lse, lse1), (ent, ent1)):
        same_bits(p[-70:], q, "last rows")
        assert bool((p[:-70] == p[0]).all())
    dh = torch.zeros(M, device=DEV)
    dh[-70:] = de
    d1 = api.token_logprob_bwd(tail, ids, lse1, dlp, entropy=ent1, d_entropy=de)
    d = api.token_logprob_bwd(z, every, lse, dl, entropy=ent, d_entropy=dh)
    same_bits(d[-70:], d1, "last rows' gradient")
    assert bool((d[:-70] == d[0]).all())


# ------------------------------------------------------------ graphs, streams and refusals

def head_step(s):
    """The operators in the order a training step uses them, on fixed buffers."""
    y, mean, rstd = api.layer_norm_fwd(s["x"], s["w"], s["b"])
    xq, xs = api.quantize_rows(y)
    logits = api.linear_i8_fwd(xq, xs, s["wq"], s["ws"], out_dtype=BF16)
    logp, lse, ent = api.token_logprob_fwd(logits, s["ids"], scale=0.8, entropy=True)
    kw = dict(entropy=ent, mask=s["mask"], cu_seqlens=s["cu"], entropy_coef=0.01)
    stats, weight = api.policy_loss_fwd(logp, s["old"], s["adv"], **kw)
    dl, de = api.policy_loss_bwd(logp, s["old"], s["adv"], weight, **kw)
    d = api.token_logprob_bwd(logits, s["ids"], lse, dl, scale=0.8, entropy=ent, d_entropy=de)
    dx, dw, db = api.layer_norm_bwd(s["dy"], s["x"], s["w"], mean, rstd)
    return [y, logits, logp, lse, ent, stats, weight, dl, de, d, dx, dw, db]


def head_state(seed):
    g = gen(seed)
    T, D, V = 300, 512, 1500
    wq, ws = api.quantize_rows(rand(g, V, D, scale=0.05).to(DEV))
    s = {"x": rand(g, T, D, dtype=BF16), "w": rand(g, D, dtype=BF16), "b": rand(g, D, dtype=BF16),
         "dy": rand(g, T, D, dtype=BF16), "ids": torch.randint(0, V, (T,), generator=g),
         "old": -rand(g, T).abs() - 6, "adv": rand(g, T),
         "mask": torch.rand(T, generator=g) < 0.8,
         "cu": torch.tensor([0, 100, 100, 300], dtype=torch.int32)}
    return {**{k: v.to(DEV) for k, v in s.items()}, "wq": wq, "ws": ws}


def test_captured_step_replays():
    s = head_state(41)
    eager = [t.clone() for t in head_step(s)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = head_step(s)
    for seed in (41, 42, 43, 41):
        new = head_state(seed)
        for k in s:
            s[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = head_step(s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same_bits(a, b, f"replay, seed {seed}")
    for k, v in head_state(41).items():
        s[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, eager):
        same_bits(a, b, "replay and the first eager step")


def test_side_stream():
    s = head_state(44)
    want = head_step(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y, mean, rstd = api.layer_norm_fwd(s["x"], s["w"], s["b"], stream=side)
    xq, xs = api.quantize_rows(y, stream=side)
    logits = api.linear_i8_fwd(xq, xs, s["wq"], s["ws"], out_dtype=BF16, stream=side)
    logp, lse, ent = api.token_logprob_fwd(logits, s["ids"], scale=0.8, entropy=True, stream=side)
    side.synchronize()
    for a, b in zip((y, logits, logp, lse, ent), want):
        same_bits(a, b, "side stream")


def test_binding_refusals_leave_outputs():
    x = torch.ones((4, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    y = torch.full((4, 63), 5.0, device=DEV)
    with pytest.raises(ValueError, match="y must be"):
        api.layer_norm_fwd(x, w, w, y=y)
    assert bool((y == 5.0).all())
    with pytest.raises(ValueError, match="weight must be"):
        api.layer_norm_fwd(x, w[:63])
    with pytest.raises(TypeError, match="bias"):
        api.layer_norm_fwd(x, w, w.to(BF16))
    with pytest.raises(ValueError, match="contiguous inside"):
        api.layer_norm_fwd(x.t(), torch.ones(4, device=DEV))
    with pytest.raises(ValueError, match="differ"):
        api.layer_norm_bwd(x[:3], x, w, w[:4], w[:4])
    with pytest.raises(ValueError, match="no mean"):
        api.layer_norm_bwd(x, x, w, w[:4], w[:4], kind="rms")
    with pytest.raises(api.GdnError, match="workspace"):
        api.layer_norm_bwd(x, x, w, w[:4], w[:4],
                           workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(api.GdnError, match="eps"):
        api.layer_norm_fwd(x, w, w, eps=-1.0)
    with pytest.raises(TypeError, match="dtype"):
        api.quantize_rows(x.half())
    q = torch.zeros((4, 192), dtype=torch.int8, device=DEV)
    with pytest.raises(api.GdnError, match="k_pad"):
        api.linear_i8_fwd(q, w[:4], q, w[:4])
    with pytest.raises(ValueError, match="but wq is"):
        api.linear_i8_fwd(q, w[:4], q[:, :128].contiguous(), w[:4])
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError, match="ids must be"):
        api.token_logprob_fwd(x, ids[:3])
    with pytest.raises(TypeError, match="ids"):
        api.token_logprob_fwd(x, ids.to(torch.int16))
    with pytest.raises(api.GdnError, match="scale"):
        api.token_logprob_fwd(x, ids, scale=0.0)
    with pytest.raises(ValueError, match="entropy"):
        api.token_logprob_bwd(x, ids, w[:4], w[:4], d_entropy=w[:4])
    with pytest.raises(ValueError, match="mask must be"):
        api.policy_loss_fwd(w, w, w, mask=torch.ones(63, dtype=torch.bool, device=DEV))
    with pytest.raises(api.GdnError, match="dual_clip"):
        api.policy_loss_fwd(w, w, w, dual_clip=0.5)
