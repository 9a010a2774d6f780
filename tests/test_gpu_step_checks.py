"""The operators around the policy head where a first set of tests did not look: rows past 2^31
elements in every kernel that draws or quantises, all that a skipped update leaves alone, products
that cancel, and calls made again that give the same bits."""

import pytest
import torch

from bitwise_consistent_linear_amd import api
from gpu_util import DEV
from test_gpu_step import BF16, F32, check_draw, gen, make, on_gpu, rand, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far():
    """Five rows 2^29 + 64 elements apart: the last one's offset is past 2^31."""
    x = torch.zeros((5, 2 ** 29 + 64), dtype=BF16, device=DEV)
    x[:, :20011] = rand(gen(83), 5, 20011, dtype=BF16).to(DEV)
    yield x
    del x
    torch.cuda.empty_cache()


# the columns and filters that lead to each kernel: one workgroup a row without cuts; rows in
# slices; cuts with the row in LDS; candidates of a top-k; a top-p whose run LDS holds, then one
# that it does not (normal logits: 0.9 of the weight is three fifths of the tokens); what is left
# of a long top-k
FAR = [(1000, dict()), (1000, dict(temperature=0.0)), (20011, dict()), (20011, dict(min_p=0.1)),
       (20011, dict(temperature=0.0)), (1000, dict(top_k=30, top_p=0.9)), (20011, dict(top_k=50)),
       (20011, dict(top_k=50, temperature=0.0)), (20011, dict(top_p=0.9, temperature=0.2)),
       (20011, dict(top_p=0.9)), (20011, dict(top_k=1500)), (20011, dict(top_k=9000, top_p=0.8))]


@pytest.mark.parametrize("vocab,filters", FAR, ids=str)
def test_sample_far_rows(far, vocab, filters):
    u = torch.rand(5, generator=gen(vocab))
    check_draw(far[:, :vocab], u, **filters)


def test_quantize_far_rows(far):
    x = far[:, :1001]
    for layout in ("rows", "columns", "both"):
        for a, b in zip(api.quantize_f8(x, layout=layout),
                        api.quantize_f8(x.contiguous(), layout=layout)):
            same(a, b, layout)
    w = api.quantize_f8(rand(gen(85), 1001, 200).to(DEV), layout="columns")
    h = api.quantize_f8(rand(gen(86), 5, 200).to(DEV), layout="columns")
    for a, b in zip(api.linear_f8_bwd(x, *w, *h), api.linear_f8_bwd(x.contiguous(), *w, *h)):
        same(a, b)


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_adamw_leaves_everything_without_a_factor(eight, bad):
    """Every buffer of a step that a factor skips, the codes of both moments among them."""
    s = make(7, [300, 1000, 5], BF16, BF16, eight, True)
    d = {name: on_gpu(s[name], False) for name in ("p", "g", "master")}
    if eight:
        d["m"] = [t.view(torch.float8_e4m3fn) for t in on_gpu(s["mc"], False)]
        d["v"], d["ms"], d["vs"] = (on_gpu(s[name], False) for name in ("vc", "ms", "vs"))
    else:
        d["m"], d["v"] = on_gpu(s["m"], False), on_gpu(s["v"], False)
    before = {name: [t.clone() for t in ts] for name, ts in d.items()}
    api.adamw_step(d["p"], d["g"], d["m"], d["v"], 2, m_scale=d.get("ms"), v_scale=d.get("vs"),
                   master=d["master"], grad_scale=torch.tensor([bad], device=DEV))
    for name, ts in d.items():
        for a, b in zip(ts, before[name]):
            same(a, b, name)


@pytest.mark.parametrize("m,n,k", [(5, 100, 512), (40, 300, 1024), (300, 1000, 512), (700, 2500, 640)])
def test_products_that_cancel(m, n, k):
    """Of every eight k two products are 2^16 and -2^16, the others whole numbers to 3. To binary32
    every partial sum is a whole number below 2^24 (k / 8 pairs of 2^16, of which at most 16 k are
    added at a time: under 2^18 and 3 k): exact. To bf16 every product is cut off 13 bits below 2^16
    at most, so each eight is off by 8 2^-13 2^16, k additions round by 2^-24 of at most (k / 4)
    2^16 + 3 k each, and Y by 2^-8 of itself."""
    g = gen(m + k)
    x = torch.randint(-3, 4, (m, k), generator=g).float()
    w = torch.randint(0, 2, (n, k), generator=g).float() * 2 - 1
    x[:, ::8], x[:, 5::8] = 256.0, -256.0
    w[:, ::8] = w[:, 5::8] = 256.0
    ops = (*api.quantize_f8(x.to(DEV)), *api.quantize_f8(w.to(DEV)))
    want = x.double() @ w.double().t()
    same(api.linear_f8_fwd(*ops), want.float())
    off = k / 8 * 8 * 2.0 ** 3 + k * 2.0 ** -24 * (k / 4 * 2.0 ** 16 + 3 * k)
    got = api.linear_f8_fwd(*ops, out_dtype=BF16).cpu().double()
    assert bool(((got - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)).all())


@pytest.mark.parametrize("m,n,k", [(16, 4096, 4096), (1021, 2049, 1111), (1024, 1024, 1024),
                                   (4096, 4096, 1024)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=str)
def test_products_again(m, n, k, dtype):
    """Both gradients in one launch, with grids that fit both products and only one, or in two."""
    g = gen(m + n)
    dy = rand(g, m, n).to(DEV)
    wq, ws, wtq, wts = api.quantize_f8(rand(g, n, k, scale=k ** -0.5).to(DEV), layout="both")
    xq, xs, xtq, xts = api.quantize_f8(rand(g, m, k).to(DEV), layout="both")
    first = None
    for _ in range(8):
        out = [api.linear_f8_fwd(xq, xs, wq, ws, out_dtype=dtype),
               *api.linear_f8_bwd(dy, wtq, wts, xtq, xts, fmt="e5m2", dx_dtype=dtype, dw_dtype=dtype)]
        first = first or out
        for a, b in zip(out, first):
            same(a, b)


@pytest.mark.parametrize("rows,vocab", [(8, 131072), (200, 30011)])
def test_draws_again(rows, vocab):
    """Sums of whole numbers by atomics, lists filled in any order."""
    g = gen(rows)
    x = rand(g, rows, vocab, scale=2.0, dtype=BF16).to(DEV)
    u = torch.rand(rows, generator=g).to(DEV)
    for f in (dict(), dict(top_p=0.95), dict(top_k=50, min_p=0.01), dict(top_k=3000, top_p=0.9)):
        first = api.sample_tokens(x, u, **f)
        for _ in range(5):
            for a, b in zip(api.sample_tokens(x, u, **f), first):
                same(a, b, f)
