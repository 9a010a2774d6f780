"""The operators around the policy head on the host: exports, refusals before anything is launched
(fake pointers are never read), the kernels' instructions, and the plain forms' gradients against
differences."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import step_ref as R
from bitwise_consistent_linear_amd import api, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_step.h")
FAKE = 0x100000  # never dereferenced: every call below is refused on the host
F32, BF16 = api.GDN_DTYPE_F32, api.GDN_DTYPE_BF16
NULL, SHAPE, UNSUP, OK = api.GDN_E_NULL, api.GDN_E_SHAPE, api.GDN_E_UNSUPPORTED, api.GDN_OK
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return api.step_lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 12, names
    out = subprocess.run(["nm", "-D", "--defined-only", api.STEP_LIB_PATH],
                         capture_output=True, text=True, check=True).stdout
    assert set(re.findall(r"\s[TW]\s+(gdn_\w+)$", out, flags=re.M)) == names
    for name, value in (("GDN_STEP_ABI_VERSION", api.step_abi_version()),
                        ("GDN_F8_BLOCK", api.F8_BLOCK), ("GDN_ADAMW_BLOCK", api.ADAMW_BLOCK)):
        assert int(re.search(rf"#define {name} (\d+)", open(HEADER).read()).group(1)) == value


def qf(L, x=2 * FAKE, rows=4, k=64, stride=64, dt=F32, fmt=0, q=FAKE, s=FAKE, qt=FAKE, st=FAKE):
    return L.gdn_quantize_f8(x, rows, k, stride, dt, fmt, q, s, qt, st, None)


def lf(L, m=4, n=4, k=128, fmt=0, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, dt=F32, y=FAKE):
    return L.gdn_linear_f8_fwd(m, n, k, fmt, xq, xs, wq, ws, dt, y, None)


def lb_shape(**kw):
    d = dict(m=4, n=4, k=4, dy_stride=4, dy_dtype=F32, dy_format=0, dx_dtype=F32, dw_dtype=F32)
    d.update(kw)
    return ctypes.byref(api.GdnLinearF8Shape(*d.values()))


def lb(L, sh=None, dy=FAKE, wtq=FAKE, wts=FAKE, xtq=FAKE, xts=FAKE, dx=FAKE, dw=FAKE, ws=FAKE,
       b=1 << 30):
    return L.gdn_linear_f8_bwd(lb_shape() if sh is None else sh, dy, wtq, wts, xtq, xts, dx, dw,
                               ws, b, None)


def sa_shape(**kw):
    d = dict(rows=4, vocab=64, logits_stride=64, logits_dtype=F32, u_bytes=4, id_bytes=8, top_k=0,
             temperature=1.0, top_p=1.0, min_p=0.0)
    d.update(kw)
    return ctypes.byref(api.GdnSampleShape(*d.values()))


def sa(L, sh=None, logits=FAKE, u=FAKE, t=None, k=None, p=None, least=None, ids=FAKE, logp=FAKE,
       ws=FAKE, b=1 << 30):
    return L.gdn_sample_tokens(sa_shape() if sh is None else sh, logits, u, t, k, p, least, ids,
                               logp, ws, b, None)


def grads(*sizes, at=FAKE):
    return (api.GdnGradTensor * max(1, len(sizes)))(*[(n, at) for n in sizes])


def gn(L, t=None, count=2, dt=F32, most=1.0, norm=FAKE, factor=FAKE, ws=FAKE, b=1 << 30):
    return L.gdn_grad_norm(grads(8, 8) if t is None else t, count, dt, most, norm, factor, ws, b,
                           None)


def tensors(**kw):
    d = dict(numel=300, param=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE,
             master=None)
    d.update(kw)
    return (api.GdnAdamwTensor * 1)(tuple(d.values()))


def aw(L, t=None, count=1, sh=True, factor=None, step_at=None, lr_at=None, **kw):
    d = dict(param_dtype=F32, grad_dtype=F32, state=1, reserved=0, lr=1e-3, beta1=0.9, beta2=0.999,
             eps=1e-8, weight_decay=0.01, step=1)
    d.update(kw)
    shape = ctypes.byref(api.GdnAdamwShape(*d.values())) if sh else ctypes.POINTER(
        api.GdnAdamwShape)()
    return L.gdn_adamw_step(shape, tensors() if t is None else t, count, factor, step_at, lr_at,
                            None)


def av(L, c=FAKE, s=FAKE, n=300, moment=0, out=FAKE):
    return L.gdn_adamw_state_values(c, s, n, moment, out, None)


NO_F8 = ctypes.POINTER(api.GdnLinearF8Shape)()
NO_SA = ctypes.POINTER(api.GdnSampleShape)()
NO_GT = ctypes.POINTER(api.GdnGradTensor)()
NO_AT = ctypes.POINTER(api.GdnAdamwTensor)()
SIZE = ctypes.byref(ctypes.c_size_t())
REFUSALS = [
    ("quantize negative rows", lambda L: qf(L, rows=-1), SHAPE),
    ("quantize rows 2^31", lambda L: qf(L, rows=2**31), SHAPE),
    ("quantize k 0", lambda L: qf(L, k=0), UNSUP),
    ("quantize k over 2^20", lambda L: qf(L, k=2**20 + 1), UNSUP),
    ("quantize rows over 2^20 by columns", lambda L: qf(L, rows=2**20 + 1), SHAPE),
    ("quantize negative stride", lambda L: qf(L, stride=-1), SHAPE),
    ("quantize stride over 2^31", lambda L: qf(L, stride=2**31 + 1), SHAPE),
    ("quantize dtype", lambda L: qf(L, dt=2), UNSUP),
    ("quantize format", lambda L: qf(L, fmt=2), UNSUP),
    ("quantize null x", lambda L: qf(L, x=None), NULL),
    ("quantize values without scales", lambda L: qf(L, s=None), NULL),
    ("quantize scales without values", lambda L: qf(L, qt=None), NULL),
    ("quantize no output", lambda L: qf(L, q=None, s=None, qt=None, st=None), NULL),
    ("quantize misaligned x", lambda L: qf(L, x=FAKE + 2), SHAPE),
    ("quantize misaligned q", lambda L: qf(L, q=FAKE + 8), SHAPE),
    ("quantize misaligned scales", lambda L: qf(L, st=FAKE + 4), SHAPE),
    ("product negative m", lambda L: lf(L, m=-1), SHAPE),
    ("product n 2^31", lambda L: lf(L, n=2**31), SHAPE),
    ("product k 64", lambda L: lf(L, k=64), UNSUP),
    ("product k over 2^20", lambda L: lf(L, k=2**20 + 128), UNSUP),
    ("product negative k", lambda L: lf(L, k=-128), UNSUP),
    ("product format", lambda L: lf(L, fmt=-1), UNSUP),
    ("product dtype", lambda L: lf(L, dt=5), UNSUP),
    ("product null x", lambda L: lf(L, xq=None), NULL),
    ("product null scales", lambda L: lf(L, ws=None), NULL),
    ("product null y", lambda L: lf(L, y=None), NULL),
    ("product null y over no k", lambda L: lf(L, k=0, y=None), NULL),
    ("product misaligned w", lambda L: lf(L, wq=FAKE + 8), SHAPE),
    ("product misaligned scales", lambda L: lf(L, xs=FAKE + 4), SHAPE),
    ("product misaligned y", lambda L: lf(L, y=FAKE + 2), SHAPE),
    ("product too many tiles", lambda L: lf(L, m=2**20, n=2**20), SHAPE),
    ("backward null shape", lambda L: lb(L, NO_F8), NULL),
    ("backward negative m", lambda L: lb(L, lb_shape(m=-1)), SHAPE),
    ("backward m over 2^20", lambda L: lb(L, lb_shape(m=2**20 + 1)), SHAPE),
    ("backward n 0", lambda L: lb(L, lb_shape(n=0)), SHAPE),
    ("backward k over 2^20", lambda L: lb(L, lb_shape(k=2**20 + 1)), SHAPE),
    ("backward stride", lambda L: lb(L, lb_shape(dy_stride=-4)), SHAPE),
    ("backward dtype", lambda L: lb(L, lb_shape(dw_dtype=3)), UNSUP),
    ("backward format", lambda L: lb(L, lb_shape(dy_format=3)), UNSUP),
    ("backward no gradient", lambda L: lb(L, dx=None, dw=None), NULL),
    ("backward dx without w", lambda L: lb(L, wtq=None), NULL),
    ("backward dw without scales of x", lambda L: lb(L, xts=None), NULL),
    ("backward null dy", lambda L: lb(L, dy=None), NULL),
    ("backward null workspace", lambda L: lb(L, ws=None), NULL),
    ("backward misaligned workspace", lambda L: lb(L, ws=FAKE + 16), SHAPE),
    ("backward short workspace", lambda L: lb(L, b=512), SHAPE),
    ("backward misaligned dy", lambda L: lb(L, dy=FAKE + 2), SHAPE),
    ("backward misaligned operand", lambda L: lb(L, xtq=FAKE + 8), SHAPE),
    ("backward workspace null", lambda L: L.gdn_linear_f8_bwd_workspace(lb_shape(), None), NULL),
    ("sample null shape", lambda L: sa(L, NO_SA), NULL),
    ("sample negative rows", lambda L: sa(L, sa_shape(rows=-1)), SHAPE),
    ("sample vocab 0", lambda L: sa(L, sa_shape(vocab=0)), SHAPE),
    ("sample vocab 2^31", lambda L: sa(L, sa_shape(vocab=2**31)), SHAPE),
    ("sample stride", lambda L: sa(L, sa_shape(logits_stride=-1)), SHAPE),
    ("sample dtype", lambda L: sa(L, sa_shape(logits_dtype=2)), UNSUP),
    ("sample u bytes", lambda L: sa(L, sa_shape(u_bytes=2)), UNSUP),
    ("sample id bytes", lambda L: sa(L, sa_shape(id_bytes=2)), UNSUP),
    ("sample negative temperature", lambda L: sa(L, sa_shape(temperature=-1.0)), SHAPE),
    ("sample temperature nan", lambda L: sa(L, sa_shape(temperature=NAN)), SHAPE),
    ("sample temperature infinite", lambda L: sa(L, sa_shape(temperature=INF)), SHAPE),
    ("sample temperature tiny", lambda L: sa(L, sa_shape(temperature=2.0**-41)), SHAPE),
    ("sample negative top_k", lambda L: sa(L, sa_shape(top_k=-1)), SHAPE),
    ("sample negative top_p", lambda L: sa(L, sa_shape(top_p=-0.1)), SHAPE),
    ("sample top_p nan", lambda L: sa(L, sa_shape(top_p=NAN)), SHAPE),
    ("sample min_p infinite", lambda L: sa(L, sa_shape(min_p=INF)), SHAPE),
    ("sample null logits", lambda L: sa(L, logits=None), NULL),
    ("sample null u", lambda L: sa(L, u=None), NULL),
    ("sample null ids", lambda L: sa(L, ids=None), NULL),
    ("sample null logp", lambda L: sa(L, logp=None), NULL),
    ("sample misaligned u", lambda L: sa(L, sa_shape(u_bytes=8), u=FAKE + 4), SHAPE),
    ("sample misaligned ids", lambda L: sa(L, ids=FAKE + 4), SHAPE),
    ("sample misaligned top_k", lambda L: sa(L, k=FAKE + 2), SHAPE),
    ("sample workspace null", lambda L: L.gdn_sample_tokens_workspace(sa_shape(), None), NULL),
    ("norm negative count", lambda L: gn(L, count=-1), SHAPE),
    ("norm count over 2^20", lambda L: gn(L, count=2**20 + 1), SHAPE),
    ("norm null list", lambda L: gn(L, NO_GT), NULL),
    ("norm negative numel", lambda L: gn(L, grads(8, -1)), SHAPE),
    ("norm numel 2^40", lambda L: gn(L, grads(8, 2**40)), SHAPE),
    ("norm dtype", lambda L: gn(L, dt=2), UNSUP),
    ("norm negative most", lambda L: gn(L, most=-1.0), SHAPE),
    ("norm most nan", lambda L: gn(L, most=NAN), SHAPE),
    ("norm null norm", lambda L: gn(L, norm=None), NULL),
    ("norm null gradient", lambda L: gn(L, grads(8, 8, at=None)), NULL),
    ("norm misaligned gradient", lambda L: gn(L, grads(8, 8, at=FAKE + 2)), SHAPE),
    ("norm misaligned factor", lambda L: gn(L, factor=FAKE + 2), SHAPE),
    ("norm null workspace", lambda L: gn(L, ws=None), NULL),
    ("norm misaligned workspace", lambda L: gn(L, ws=FAKE + 8), SHAPE),
    ("norm short workspace", lambda L: gn(L, b=8), SHAPE),
    ("norm workspace null", lambda L: L.gdn_grad_norm_workspace(grads(8), 1, None), NULL),
    ("adamw null shape", lambda L: aw(L, sh=False), NULL),
    ("adamw null list", lambda L: aw(L, NO_AT), NULL),
    ("adamw negative count", lambda L: aw(L, count=-1), SHAPE),
    ("adamw numel", lambda L: aw(L, tensors(numel=-1)), SHAPE),
    ("adamw param dtype", lambda L: aw(L, param_dtype=2), UNSUP),
    ("adamw grad dtype", lambda L: aw(L, grad_dtype=-1), UNSUP),
    ("adamw state", lambda L: aw(L, state=2), UNSUP),
    ("adamw beta1 1", lambda L: aw(L, beta1=1.0), SHAPE),
    ("adamw beta2 negative", lambda L: aw(L, beta2=-0.1), SHAPE),
    ("adamw beta2 nan", lambda L: aw(L, beta2=NAN), SHAPE),
    ("adamw eps negative", lambda L: aw(L, eps=-1e-8), SHAPE),
    ("adamw lr infinite", lambda L: aw(L, lr=INF), SHAPE),
    ("adamw decay nan", lambda L: aw(L, weight_decay=NAN), SHAPE),
    ("adamw step 0", lambda L: aw(L, step=0), SHAPE),
    ("adamw null param", lambda L: aw(L, tensors(param=None)), NULL),
    ("adamw null grad", lambda L: aw(L, tensors(grad=None)), NULL),
    ("adamw null m", lambda L: aw(L, tensors(m=None)), NULL),
    ("adamw null scale", lambda L: aw(L, tensors(v_scale=None)), NULL),
    ("adamw master of binary32", lambda L: aw(L, tensors(master=FAKE)), UNSUP),
    ("adamw misaligned param", lambda L: aw(L, tensors(param=FAKE + 2)), SHAPE),
    ("adamw misaligned bf16 grad", lambda L: aw(L, tensors(grad=FAKE + 1), grad_dtype=BF16), SHAPE),
    ("adamw misaligned m", lambda L: aw(L, tensors(m=FAKE + 1), state=0), SHAPE),
    ("adamw misaligned scale", lambda L: aw(L, tensors(m_scale=FAKE + 2)), SHAPE),
    ("adamw misaligned factor", lambda L: aw(L, factor=FAKE + 2), SHAPE),
    ("adamw misaligned step", lambda L: aw(L, step_at=FAKE + 4), SHAPE),
    ("values numel", lambda L: av(L, n=-1), SHAPE),
    ("values moment", lambda L: av(L, moment=2), UNSUP),
    ("values null codes", lambda L: av(L, c=None), NULL),
    ("values null scale", lambda L: av(L, s=None), NULL),
    ("values misaligned out", lambda L: av(L, out=FAKE + 2), SHAPE),
]


@pytest.mark.parametrize("name,call,status", REFUSALS, ids=[r[0] for r in REFUSALS])
def test_refused_before_launch(L, name, call, status):
    assert call(L) == status
    assert re.match(r"gdn_(quantize_f8|linear_f8|sample_tokens|grad_norm|adamw)",
                    L.gdn_step_last_error().decode())


def test_a_tensor_needs_buffers_of_its_own(L):
    names = ("param", "grad", "m", "v", "m_scale", "v_scale", "master")
    apart = {n: FAKE + 4096 * i for i, n in enumerate(names)}
    for a in names:
        for b in names:
            if a < b:
                assert aw(L, tensors(**dict(apart, **{a: apart[b]})), param_dtype=BF16) == SHAPE
                assert L.gdn_step_last_error().endswith(b"two buffers of a tensor are the same")


def test_empty_sizes_launch_nothing(L):
    assert qf(L, rows=0, x=None) == OK
    assert lf(L, m=0) == OK and lf(L, n=0, y=None) == OK
    assert lb(L, lb_shape(m=0), dy=None, dw=None, ws=None) == OK
    assert sa(L, sa_shape(rows=0), logits=None) == OK
    assert aw(L, NO_AT, count=0) == OK
    assert aw(L, tensors(numel=0, param=None, grad=None)) == OK
    assert av(L, n=0, c=None) == OK
    assert L.gdn_step_last_error() == b""


def test_workspaces_grow_with_the_sizes():
    f = api.linear_f8_bwd_workspace_bytes
    small = f(api.GdnLinearF8Shape(100, 200, 300, 200, F32, 0, F32, F32))
    big = f(api.GdnLinearF8Shape(1000, 2000, 300, 2000, F32, 0, F32, F32))
    # both forms of dy and their scales
    assert small >= 100 * 256 + 200 * 128 and big >= 1000 * 2048 + 2000 * 1024
    assert small % 256 == big % 256 == 0
    n = ctypes.c_size_t()
    sizes = []
    for numel in (1, 10**6, 10**9):
        assert api.step_lib().gdn_grad_norm_workspace(grads(numel), 1, ctypes.byref(n)) == OK
        sizes.append(n.value)
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] > sizes[0]


def test_binding_refuses_host_tensors_and_wrong_arguments():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        api.quantize_f8(x)
    with pytest.raises(ValueError, match="layout"):
        api.quantize_f8(x, layout="tiles")
    with pytest.raises(ValueError, match="fmt"):
        api.quantize_f8(x, fmt="e3m4")
    with pytest.raises(ValueError, match="GPU"):
        api.linear_f8_fwd(x.to(torch.float8_e4m3fn), x, x, x)
    with pytest.raises(TypeError, match="out_dtype"):
        api.linear_f8_fwd(x, x, x, x, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="torch tensor"):
        api.linear_f8_bwd(x.numpy())
    with pytest.raises(ValueError, match="GPU"):
        api.sample_tokens(x, torch.zeros(4))
    with pytest.raises(TypeError, match="id_dtype"):
        api.sample_tokens(x, torch.zeros(4), id_dtype=torch.int16)
    with pytest.raises(TypeError, match="list or tuple"):
        api.grad_norm(x)
    with pytest.raises(ValueError, match="grads.0. must be on a GPU"):
        api.grad_norm([x])
    with pytest.raises(ValueError, match="params.0. must be on a GPU"):
        api.adamw_step([x], [x], [x], [x], 1)
    with pytest.raises(ValueError, match="as many"):
        api.adamw_step([x], [], [x], [x], 1)
    with pytest.raises(ValueError, match="GPU"):
        api.adamw_state_values(x, x)


def test_library_and_binding_missing_are_errors(monkeypatch, tmp_path):
    import sys

    import bitwise_consistent_linear_amd as package
    with monkeypatch.context() as mp:
        mp.setattr(api, "_step_lib", None)
        mp.setattr(api, "STEP_LIB_PATH", str(tmp_path / "absent.so"))
        with pytest.raises(RuntimeError, match="missing"):
            api.step_lib()
    monkeypatch.setattr(api, "_step_calls", None)
    monkeypatch.delattr(package, "_step_binding", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._step_binding", None)
    with pytest.raises(RuntimeError, match="_step_binding"):
        api.quantize_f8(torch.zeros(4, 8))


def test_binding_refuses_wrong_calls():
    calls = api._step()
    with pytest.raises(TypeError, match="number of arguments"):
        calls.quantize_f8(torch.zeros(4, 8))
    with pytest.raises(TypeError, match="setup takes"):
        calls.setup(1, 2)


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("isa") / "step.s")
    sources = [s for s in build.STEP_SOURCES if s.endswith(".hip")]
    return open(build.device_asm(path, sources)).read()


def test_instructions(asm):
    """No packed fp32 arithmetic, no floating-point atomics, denormals kept; the matrix code is the
    scaled 8-bit instruction and the bf16 one."""
    assert not re.search(r"^\s+v_pk_(add|mul|fma)_f32", asm, flags=re.M)
    assert not re.search(r"^\s+(global|buffer|flat|ds)_(atomic_)?(pk_)?add\w*_f(16|32|64)", asm,
                         flags=re.M)
    modes = re.findall(r"\.amdhsa_float_denorm_mode_32 (\d)", asm)
    assert modes and all(m == "3" for m in modes)
    mfma = set(re.findall(r"^\s+(v_mfma_\w+)", asm, flags=re.M))
    assert mfma == {"v_mfma_scale_f32_32x32x64_f8f6f4", "v_mfma_f32_32x32x16_bf16"}, mfma


# ------------------------------------------------- the plain forms against differences

def test_product_gradient_against_differences():
    """Y = X W^T is linear in the values that X and W stand for: for a dy that 8 bits hold, the
    gradients are exact, and a difference of sum(dy Y) over a step of one value is them times the
    step, up to binary64's rounding of sums of 300 products of order 1."""
    g = torch.Generator().manual_seed(3)
    m, n, k = 5, 7, 300
    x, w, dy = (torch.randn(*s, generator=g) for s in ((m, k), (n, k), (m, n)))
    xv = R.values(*R.quantize(x, "e4m3"))[:, :k]
    wv = R.values(*R.quantize(w, "e4m3"))[:, :k]
    dyv = R.values(*R.quantize(dy, "e4m3"))[:, :n]
    assert torch.equal(R.values(*R.quantize(dyv.t(), "e4m3"))[:, :m].t(), dyv)
    dx, dw = dyv @ wv, dyv.t() @ xv
    f = lambda a, b: float((dyv * (a @ b.t())).sum())  # noqa: E731
    vx, vw = torch.randn(m, k, generator=g).double(), torch.randn(n, k, generator=g).double()
    assert abs(f(xv + vx, wv) - f(xv, wv) - float((dx * vx).sum())) < 1e-9
    assert abs(f(xv, wv + vw) - f(xv, wv) - float((dw * vw).sum())) < 1e-9


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_rounding_to_8_bits(fmt):
    """The reference's rounding is torch's, for every bf16 value in the format's range."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    x = x[torch.isfinite(x) & (x.abs() <= 1.75 * 2.0 ** R.EMAX[fmt])]
    assert torch.equal(R.round_f8(x, fmt), x.float().to(R.F8[fmt]).double())


def test_draw_by_counting():
    """Evenly spaced random numbers draw every token as often as its probability says, to one."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=20) * 2
    p = np.exp(x / 0.7) / np.exp(x / 0.7).sum()
    n = 4000
    ids = [R.draw(x, (i + 0.5) / n, 0.7)[0] for i in range(n)]
    assert np.abs(np.bincount(ids, minlength=20) - n * p).max() <= 1.0


def test_adamw_forms_agree():
    """Binary32 against binary64: a value of order 1 moves by at most lr / (1 - beta1) in a step;
    a dozen roundings of 2^-24 each."""
    g = torch.Generator().manual_seed(5)
    p, gr, m = (torch.randn(1000, generator=g) for _ in range(3))
    v = torch.rand(1000, generator=g)
    args = (7, 1e-2, 0.9, 0.95, 1e-8, 0.1)
    a = R.adamw32(p, gr, m, v, *args)
    b = R.adamw64(p, gr, m, v, *args)
    for x, y in zip(a, b):
        assert float((x.double() - y).abs().max()) <= 12 * 2.0 ** -24 * float(y.abs().max())


def test_8bit_states_keep_their_values():
    g = torch.Generator().manual_seed(6)
    m = torch.randn(1000, generator=g)
    got = R.unpack_m(*R.pack_m(m))
    # half a step of e4m3, or of its smallest values, 2^-9 448ths of the block's largest
    peak = m.abs().max()
    assert bool(((got - m).abs() <= m.abs() * 2.0 ** -4 * 1.001 + peak / 448 * 2.0 ** -10 * 1.001).all())
    r = torch.rand(1000, generator=g) ** 4
    got = R.unpack_r(*R.pack_r(r))
    lowest = r.max() / 248 * 2.0 ** -8 * (17 / 16)
    close = (got - r).abs() <= r * 2.0 ** -5 * 1.001
    assert bool((close | (r <= lowest * 1.05)).all()) and bool((got > 0).all())
