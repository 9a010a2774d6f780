"""The norm's backward where a row's mean times its rstd is past binary32's range: places past
the row's end, which hold zeros, must not reach the row's sums."""

import pytest
import torch

import policy_ref as R
from bitwise_consistent_linear_amd import api
from gpu_util import DEV
from test_gpu_policy import DTYPES, gen, rand, same_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("eps,value", [(1e-5, 1.5e36), (1e-12, 4e32), (1e-5, -1.5e36)])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 100, 129, 500, 513, 2049, 5341, 8193, 9000, 16377])
def test_constant_rows_of_large_values(D, eps, value, dt):
    """A constant row has normalised values 0: dx = rstd (g - mean(g)), d_weight 0 from it."""
    dt = DTYPES[dt]
    g = gen(D)
    x = rand(g, 6, D).to(dt)
    x[1] = x[4] = value
    dy, w = rand(g, 6, D).to(dt), (1 + rand(g, D, scale=0.2)).to(dt)
    # mean and rstd of the constant rows as the definition gives them
    xd = x.double()
    mean = xd.mean(1)
    mean[1] = mean[4] = x[1, 0].double()
    rstd = ((xd - mean[:, None]).square().mean(1) + eps).rsqrt().float()
    mean = mean.float()
    up = [t.to(DEV) for t in (dy, x, w, mean, rstd)]
    dx, dw, db = api.layer_norm_bwd(*up)
    (wx, ex), (ww, ew), (wb, eb) = R.norm_bwd_bounds(dy, x, w, mean, rstd, "layer", dt)
    R.check(dx, wx, ex, "dx")
    R.check(dw, ww, ew, "d_weight")
    R.check(db, wb, eb, "d_bias")


@pytest.mark.parametrize("eps", [1e-5, 1e-12])
def test_forward_and_backward_of_a_constant_row(eps):
    """Through both calls: 64 equal values sum exactly, so the mean is the value itself."""
    x = torch.full((3, 64), 1.5e36)
    x[1] = rand(gen(1), 64)
    w, b, dy = torch.ones(64), torch.full((64,), 0.25), rand(gen(2), 3, 64)
    y, mean, rstd = api.layer_norm_fwd(x.to(DEV), w.to(DEV), b.to(DEV), eps=eps)
    assert bool((y[0] == 0.25).all()) and float(mean[0]) == float(x[0, 0])
    dx, dw, db = api.layer_norm_bwd(dy.to(DEV), x.to(DEV), w.to(DEV), mean, rstd)
    (wx, ex), (ww, ew), (wb, eb) = R.norm_bwd_bounds(dy, x, w, mean.cpu(), rstd.cpu(), "layer",
                                                     x.dtype)
    R.check(dx, wx, ex, "dx")
    R.check(dw, ww, ew, "d_weight")
    R.check(db, wb, eb, "d_bias")
    same_bits(dx[1:2], api.layer_norm_bwd(dy[1:2].to(DEV), x[1:2].to(DEV), w.to(DEV), mean[1:2],
                                          rstd[1:2])[0], "the row beside, alone")
