"""The policy-head operators on the host: exports, refusals before anything is launched (fake
pointers are never read), the kernels' instructions, and the plain 64-bit forms' gradients
against differences."""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import policy_ref as R
from bitwise_consistent_linear_amd import api, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_policy.h")
FAKE = 0x100000  # never dereferenced: every call below is refused on the host
F32, BF16 = api.GDN_DTYPE_F32, api.GDN_DTYPE_BF16
NULL, SHAPE, UNSUP = api.GDN_E_NULL, api.GDN_E_SHAPE, api.GDN_E_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    return api.policy_lib()


def test_exports_every_declared_function(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text))
    assert len(names) == 14, names
    out = subprocess.run(["nm", "-D", "--defined-only", api.POLICY_LIB_PATH],
                         capture_output=True, text=True, check=True).stdout
    assert set(re.findall(r"\s[TW]\s+(gdn_\w+)$", out, flags=re.M)) == names
    m = re.search(r"#define GDN_POLICY_ABI_VERSION (\d+)", open(HEADER).read())
    assert api.policy_abi_version() == int(m.group(1))
    m = re.search(r"#define GDN_I8_K_ALIGN (\d+)", open(HEADER).read())
    assert api.I8_K_ALIGN == int(m.group(1))


def norm_shape(rows=4, width=64, kind=0, x=F32, w=F32):
    return ctypes.byref(api.GdnNormShape(rows, width, kind, x, w))


def nf(L, sh=None, x=2 * FAKE, stride=64, w=FAKE, b=FAKE, eps=1e-5, y=FAKE, mean=FAKE, rstd=FAKE):
    return L.gdn_layer_norm_fwd(norm_shape() if sh is None else sh, x, stride, w, b, eps, y,
                                mean, rstd, None)


def nb(L, sh=None, dy=FAKE, ds=64, x=2 * FAKE, xs=64, w=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE,
       dw=FAKE, db=FAKE, ws=FAKE, n=1 << 30):
    return L.gdn_layer_norm_bwd(norm_shape() if sh is None else sh, dy, ds, x, xs, w, mean,
                                rstd, dx, dw, db, ws, n, None)


def qr(L, x=FAKE, rows=4, k=64, stride=64, dt=F32, q=FAKE, scale=FAKE):
    return L.gdn_quantize_rows(x, rows, k, stride, dt, q, scale, None)


def li(L, m=4, n=4, k=128, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, dt=F32, y=FAKE, room=None, b=0):
    return L.gdn_linear_i8_fwd(m, n, k, xq, xs, wq, ws, dt, y, room, b, None)


def lp_shape(rows=4, vocab=64, stride=64, dt=F32, idb=8, scale=1.0):
    return ctypes.byref(api.GdnLogprobShape(rows, vocab, stride, dt, idb, scale))


def lf(L, sh=None, logits=FAKE, ids=FAKE, logp=FAKE, lse=FAKE, ent=FAKE, ws=None, n=0):
    return L.gdn_token_logprob_fwd(lp_shape() if sh is None else sh, logits, ids, logp, lse,
                                   ent, ws, n, None)


def lb(L, sh=None, logits=FAKE, ids=FAKE, lse=FAKE, dlp=FAKE, ent=FAKE, de=FAKE, out=2 * FAKE):
    return L.gdn_token_logprob_bwd(lp_shape() if sh is None else sh, logits, ids, lse, dlp, ent,
                                   de, out, None)


def po_shape(**kw):
    d = dict(tokens=8, seqs=2, reduction=0, reserved=0, clip_low=0.2, clip_high=0.2,
             dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0)
    d.update(kw)
    return ctypes.byref(api.GdnPolicyShape(*d.values()))


def pf(L, sh=None, logp=FAKE, old=FAKE, adv=FAKE, ref=None, ent=None, mask=None, cu=FAKE,
       stats=FAKE, w=FAKE, ws=FAKE, n=1 << 30):
    return L.gdn_policy_loss_fwd(po_shape() if sh is None else sh, logp, old, adv, ref, ent,
                                 mask, cu, stats, w, ws, n, None)


def pb(L, sh=None, logp=FAKE, old=FAKE, adv=FAKE, ref=None, mask=None, cu=FAKE, w=FAKE, dl=1.0,
       dlp=FAKE, de=None):
    return L.gdn_policy_loss_bwd(po_shape() if sh is None else sh, logp, old, adv, ref, mask,
                                 cu, w, dl, dlp, de, None)


NAN, INF = float("nan"), float("inf")
NO_NORM = ctypes.POINTER(api.GdnNormShape)()
NO_LP = ctypes.POINTER(api.GdnLogprobShape)()
NO_PO = ctypes.POINTER(api.GdnPolicyShape)()
LONG = lp_shape(rows=1, vocab=1 << 20, stride=1 << 20)  # split over workgroups
REFUSALS = [
    ("norm null shape", lambda L: nf(L, NO_NORM), NULL),
    ("norm negative rows", lambda L: nf(L, norm_shape(rows=-1)), SHAPE),
    ("norm rows 2^31", lambda L: nf(L, norm_shape(rows=2**31)), SHAPE),
    ("norm width 0", lambda L: nf(L, norm_shape(width=0)), UNSUP),
    ("norm width 16385", lambda L: nf(L, norm_shape(width=16385)), UNSUP),
    ("norm kind", lambda L: nf(L, norm_shape(kind=2)), UNSUP),
    ("norm x dtype", lambda L: nf(L, norm_shape(x=2)), UNSUP),
    ("norm w dtype", lambda L: nf(L, norm_shape(w=-1)), UNSUP),
    ("norm negative stride", lambda L: nf(L, stride=-64), SHAPE),
    ("norm stride over 2^31", lambda L: nf(L, stride=2**31 + 1), SHAPE),
    ("norm eps negative", lambda L: nf(L, eps=-1e-5), SHAPE),
    ("norm eps nan", lambda L: nf(L, eps=NAN), SHAPE),
    ("norm eps infinite", lambda L: nf(L, eps=INF), SHAPE),
    ("norm null x", lambda L: nf(L, x=None), NULL),
    ("norm null weight", lambda L: nf(L, w=None), NULL),
    ("norm null mean", lambda L: nf(L, mean=None), NULL),
    ("norm null rstd", lambda L: nf(L, rstd=None), NULL),
    ("norm misaligned y", lambda L: nf(L, y=FAKE + 2), SHAPE),
    ("norm misaligned bf16 x", lambda L: nf(L, norm_shape(x=BF16), x=FAKE + 1), SHAPE),
    ("norm misaligned bias", lambda L: nf(L, b=FAKE + 2), SHAPE),
    ("norm in place with a stride", lambda L: nf(L, x=FAKE, stride=80), SHAPE),
    ("norm bwd in place with a stride", lambda L: nb(L, ds=80), SHAPE),
    ("norm bwd dx is x", lambda L: nb(L, dx=2 * FAKE), SHAPE),
    ("norm bwd null dy", lambda L: nb(L, dy=None), NULL),
    ("norm bwd null d_weight", lambda L: nb(L, dw=None), NULL),
    ("norm bwd null mean", lambda L: nb(L, mean=None), NULL),
    ("norm bwd null workspace", lambda L: nb(L, ws=None), NULL),
    ("norm bwd misaligned workspace", lambda L: nb(L, ws=FAKE + 16), SHAPE),
    ("norm bwd short workspace", lambda L: nb(L, n=64), SHAPE),
    ("norm bwd negative stride", lambda L: nb(L, ds=-1), SHAPE),
    ("norm bwd misaligned d_bias", lambda L: nb(L, db=FAKE + 1), SHAPE),
    ("norm bwd workspace null", lambda L: L.gdn_layer_norm_bwd_workspace(norm_shape(), None), NULL),
    ("quantize negative rows", lambda L: qr(L, rows=-1), SHAPE),
    ("quantize k 0", lambda L: qr(L, k=0), UNSUP),
    ("quantize k 65537", lambda L: qr(L, k=65537), UNSUP),
    ("quantize dtype", lambda L: qr(L, dt=7), UNSUP),
    ("quantize null q", lambda L: qr(L, q=None), NULL),
    ("quantize misaligned q", lambda L: qr(L, q=FAKE + 8), SHAPE),
    ("quantize stride", lambda L: qr(L, stride=-1), SHAPE),
    ("linear negative m", lambda L: li(L, m=-1), SHAPE),
    ("linear n 2^31", lambda L: li(L, n=2**31), SHAPE),
    ("linear k not padded", lambda L: li(L, k=192), UNSUP),
    ("linear k 0", lambda L: li(L, k=0), UNSUP),
    ("linear k over 65536", lambda L: li(L, k=65536 + 128), UNSUP),
    ("linear dtype", lambda L: li(L, dt=3), UNSUP),
    ("linear null w_scale", lambda L: li(L, ws=None), NULL),
    ("linear misaligned wq", lambda L: li(L, wq=FAKE + 4), SHAPE),
    ("linear misaligned y", lambda L: li(L, y=FAKE + 2), SHAPE),
    ("linear too many tiles", lambda L: li(L, m=2**31 - 1, n=2**31 - 1), SHAPE),
    ("linear rows past one launch", lambda L: li(L, m=2**30, n=1), SHAPE),
    ("linear columns past one launch", lambda L: li(L, m=1, n=2**31 - 1), SHAPE),
    ("linear no workspace", lambda L: li(L, k=65536), NULL),
    ("linear short workspace", lambda L: li(L, k=65536, room=FAKE, b=16), SHAPE),
    ("linear misaligned workspace", lambda L: li(L, k=65536, room=FAKE + 4, b=1 << 30), SHAPE),
    ("linear workspace null", lambda L: L.gdn_linear_i8_fwd_workspace(4, 4, 128, None), NULL),
    ("linear workspace k", lambda L: L.gdn_linear_i8_fwd_workspace(
        4, 4, 130, ctypes.byref(ctypes.c_size_t(0))), UNSUP),
    ("logprob null shape", lambda L: lf(L, NO_LP), NULL),
    ("logprob vocab 0", lambda L: lf(L, lp_shape(vocab=0)), SHAPE),
    ("logprob rows", lambda L: lf(L, lp_shape(rows=-1)), SHAPE),
    ("logprob dtype", lambda L: lf(L, lp_shape(dt=2)), UNSUP),
    ("logprob id bytes", lambda L: lf(L, lp_shape(idb=2)), UNSUP),
    ("logprob scale 0", lambda L: lf(L, lp_shape(scale=0.0)), SHAPE),
    ("logprob scale nan", lambda L: lf(L, lp_shape(scale=NAN)), SHAPE),
    ("logprob scale infinite", lambda L: lf(L, lp_shape(scale=INF)), SHAPE),
    ("logprob stride", lambda L: lf(L, lp_shape(stride=-1)), SHAPE),
    ("logprob null ids", lambda L: lf(L, ids=None), NULL),
    ("logprob null lse", lambda L: lf(L, lse=None), NULL),
    ("logprob misaligned ids", lambda L: lf(L, ids=FAKE + 4), SHAPE),
    ("logprob misaligned logits", lambda L: lf(L, logits=FAKE + 2), SHAPE),
    ("logprob no workspace", lambda L: lf(L, LONG), NULL),
    ("logprob short workspace", lambda L: lf(L, LONG, ws=FAKE, n=8), SHAPE),
    ("logprob misaligned workspace", lambda L: lf(L, LONG, ws=FAKE + 2, n=1 << 30), SHAPE),
    ("logprob workspace null", lambda L: L.gdn_token_logprob_fwd_workspace(lp_shape(), None), NULL),
    ("logprob bwd entropy alone", lambda L: lb(L, de=None), NULL),
    ("logprob bwd d_entropy alone", lambda L: lb(L, ent=None), NULL),
    ("logprob bwd null d_logits", lambda L: lb(L, out=None), NULL),
    ("logprob bwd in place with a stride", lambda L: lb(L, lp_shape(stride=80), out=FAKE), SHAPE),
    ("logprob bwd too large", lambda L: lb(L, lp_shape(rows=2**31 - 1, vocab=2**31 - 1)), SHAPE),
    ("policy null shape", lambda L: pf(L, NO_PO), NULL),
    ("policy tokens", lambda L: pf(L, po_shape(tokens=-1)), SHAPE),
    ("policy negative sequences", lambda L: pf(L, po_shape(seqs=-1)), SHAPE),
    ("policy no sequence, no cu_seqlens", lambda L: pf(L, po_shape(seqs=0), cu=None), NULL),
    ("policy reduction", lambda L: pf(L, po_shape(reduction=2)), UNSUP),
    ("policy clip_low over 1", lambda L: pf(L, po_shape(clip_low=1.5)), SHAPE),
    ("policy clip_high negative", lambda L: pf(L, po_shape(clip_high=-0.1)), SHAPE),
    ("policy clip_high nan", lambda L: pf(L, po_shape(clip_high=NAN)), SHAPE),
    ("policy dual_clip under 1", lambda L: pf(L, po_shape(dual_clip=0.5)), SHAPE),
    ("policy kl_coef nan", lambda L: pf(L, po_shape(kl_coef=NAN)), SHAPE),
    ("policy null logp", lambda L: pf(L, logp=None), NULL),
    ("policy null cu_seqlens", lambda L: pf(L, cu=None), NULL),
    ("policy null stats", lambda L: pf(L, stats=None), NULL),
    ("policy short workspace", lambda L: pf(L, n=8), SHAPE),
    ("policy misaligned workspace", lambda L: pf(L, ws=FAKE + 8), SHAPE),
    ("policy misaligned ref", lambda L: pf(L, ref=FAKE + 2), SHAPE),
    ("policy workspace null", lambda L: L.gdn_policy_loss_workspace(po_shape(), None), NULL),
    ("policy bwd null weight", lambda L: pb(L, w=None), NULL),
    ("policy bwd null d_logp", lambda L: pb(L, dlp=None), NULL),
    ("policy bwd d_loss nan", lambda L: pb(L, dl=NAN), SHAPE),
    ("policy bwd misaligned d_entropy", lambda L: pb(L, de=FAKE + 1), SHAPE),
]


@pytest.mark.parametrize("name,call,status", REFUSALS, ids=[r[0] for r in REFUSALS])
def test_refused_before_launch(L, name, call, status):
    assert call(L) == status
    assert re.match(r"gdn_(layer_norm|quantize_rows|linear_i8|token_logprob|policy_loss)",
                    L.gdn_policy_last_error().decode())


def test_empty_sizes_launch_nothing(L):
    """Fake pointers are never touched."""
    assert nf(L, norm_shape(rows=0), x=None) == api.GDN_OK
    assert qr(L, rows=0, x=None) == api.GDN_OK
    assert li(L, m=0) == api.GDN_OK and li(L, n=0, y=None) == api.GDN_OK
    assert lf(L, lp_shape(rows=0), logits=None) == api.GDN_OK
    assert lb(L, lp_shape(rows=0)) == api.GDN_OK
    assert pb(L, po_shape(tokens=0), logp=None, dlp=None) == api.GDN_OK
    assert L.gdn_policy_last_error() == b""


def test_workspaces_grow_with_the_sizes():
    small = api.layer_norm_bwd_workspace_bytes(api.GdnNormShape(1, 100, 0, F32, F32))
    big = api.layer_norm_bwd_workspace_bytes(api.GdnNormShape(4096, 100, 0, F32, F32))
    assert small >= 2 * 100 * 4 and big > small and small % 256 == big % 256 == 0
    a = api.policy_loss_workspace_bytes(api.GdnPolicyShape(100, 3, 0, 0, 0.2, 0.2, 0, 0, 0))
    d = api.linear_i8_fwd_workspace_bytes
    assert d(16, 4096, 4096) == d(16384, 4096, 65536) == d(0, 4, 65536) == d(4, 4, 128) == 0
    assert d(85, 69, 15744) % (85 * 69 * 4) == 0 < d(85, 69, 15744)
    c = lambda rows, vocab: api.token_logprob_fwd_workspace_bytes(  # noqa: E731
        api.GdnLogprobShape(rows, vocab, vocab, F32, 8, 1.0))
    assert c(1, 1000) == c(100000, 1 << 20) == 0 < c(1, 1 << 20) < c(2, 1 << 20) < c(2, 1 << 21)
    b = api.policy_loss_workspace_bytes(api.GdnPolicyShape(10**6, 300, 0, 0, 0.2, 0.2, 0, 0, 0))
    assert b > a > 0 and a % 256 == b % 256 == 0


def test_binding_refuses_host_tensors_and_wrong_arguments():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        api.layer_norm_fwd(x, w)
    with pytest.raises(ValueError, match="kind"):
        api.layer_norm_fwd(x, w, kind="batch")
    with pytest.raises(TypeError, match="torch tensor"):
        api.quantize_rows(x.numpy())
    with pytest.raises(ValueError, match="GPU"):
        api.linear_i8_fwd(torch.zeros(4, 128, dtype=torch.int8), w, w, w)
    with pytest.raises(ValueError, match="GPU"):
        api.token_logprob_fwd(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="reduction"):
        api.policy_loss_fwd(w, w, w, reduction="mean")


def test_library_missing_is_an_error(monkeypatch, tmp_path):
    monkeypatch.setattr(api, "_policy_lib", None)
    monkeypatch.setattr(api, "POLICY_LIB_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(RuntimeError, match="missing"):
        api.policy_lib()


def test_binding_missing_is_an_error(monkeypatch):
    import sys

    import bitwise_consistent_linear_amd as package
    monkeypatch.setattr(api, "_policy_calls", None)
    monkeypatch.delattr(package, "_policy_binding", raising=False)
    monkeypatch.setitem(sys.modules, package.__name__ + "._policy_binding", None)
    with pytest.raises(RuntimeError, match="_policy_binding"):
        api.quantize_rows(torch.zeros(4, 8))


def test_binding_refuses_wrong_calls():
    """The module's own checks: the number of arguments, and values that are no numbers."""
    calls = api._policy()
    with pytest.raises(TypeError, match="number of arguments"):
        calls.quantize_rows(torch.zeros(4, 8))
    with pytest.raises(TypeError, match="setup takes"):
        calls.setup(1, 2)
    for bad in (torch.zeros(4, 8), None, 3, torch.zeros(4, 8, dtype=torch.bfloat16).to_sparse()):
        with pytest.raises((TypeError, ValueError)):
            api.layer_norm_fwd(bad, torch.ones(8))


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    path = str(tmp_path_factory.mktemp("isa") / "policy.s")
    sources = [s for s in build.POLICY_SOURCES if s.endswith(".hip")]
    return open(build.device_asm(path, sources)).read()


def test_instructions(asm):
    """No packed fp32 arithmetic, no floating-point atomics, denormals kept, and the only
    matrix code is the int8 product's."""
    assert not re.search(r"^\s+v_pk_(add|mul|fma)_f32", asm, flags=re.M)
    assert not re.search(r"^\s+(global|buffer|flat|ds)_(atomic_)?(pk_)?add\w*_f(16|32|64)", asm,
                         flags=re.M)
    modes = re.findall(r"\.amdhsa_float_denorm_mode_32 (\d)", asm)
    assert modes and all(m == "3" for m in modes)
    mfma = set(re.findall(r"^\s+(v_mfma_\w+)", asm, flags=re.M))
    assert mfma <= {"v_mfma_i32_16x16x64_i8", "v_mfma_i32_32x32x32_i8"} and mfma


# ------------------------------------------------- the plain forms against differences

def slope(f, x, v, h):
    return float((f(x + h * v) - f(x - h * v)) / (2 * h))


# A central difference with step h of values of order 1 in binary64 is off by h^2 / 6 of the
# third derivative (order 1 to 100 here) and 2^-52 / h: under 1e-7 for h = 1e-5.
H, DIFF = 1e-5, 1e-7


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_gradient_against_differences(kind):
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = r(5, 33), r(33), r(33), r(5, 33)
    f = lambda x, w, b: (R.norm_fwd(x, w, b, 1e-5, kind)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = R.norm_fwd(x, w, b, 1e-5, kind)
    dx, dw, db = R.norm_bwd(dy, x, w, mean, rstd, kind)
    vx, vw = r(5, 33), r(33)
    size = float(dy.abs().sum())
    assert abs(slope(lambda t: f(t, w, b), x, vx, H) - float((dx * vx).sum())) < DIFF * size
    assert abs(slope(lambda t: f(x, t, b), w, vw, H) - float((dw * vw).sum())) < DIFF * size
    assert abs(slope(lambda t: f(x, w, t), b, vw, H) - float((db * vw).sum())) < DIFF * size


def test_logprob_gradient_against_differences():
    g = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    z, dlp, de, v = 2 * r(6, 41), r(6), r(6), r(6, 41)
    ids = torch.tensor([0, 40, 7, -1, 3, 41])

    def f(z):
        logp, _, ent = R.logprob(z, ids, 0.75)
        return (logp * dlp + ent * de).sum()

    _, lse, ent = R.logprob(z, ids, 0.75)
    d = R.logprob_bwd(z, ids, lse, dlp, 0.75, ent, de)
    assert abs(slope(f, z, v, H) - float((d * v).sum())) < DIFF * float(dlp.abs().sum() + de.abs().sum()) * 10
    assert float(d[3].abs().sum()) == 0.0 and float(d[5].abs().sum()) == 0.0


@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_gradient_against_differences(reduction):
    rng = np.random.default_rng(5)
    T, cu = 40, [0, 7, 7, 8, 40]
    logp, ref, ent, adv = (rng.normal(size=T) for _ in range(4))
    # ratios away from the borders 0.8, 1.28 and 3, where the loss has a kink
    old = logp - np.log(rng.choice([0.5, 0.9, 1.1, 1.5, 4.0], size=T))
    mask = rng.random(T) < 0.8
    args = (ref, ent, mask, cu, 0.2, 0.28, 3.0, 0.1, 0.05, reduction)
    _, _, dl, de = R.policy(logp, old, adv, *args)
    v = rng.normal(size=T)
    loss = lambda lp, en: R.policy(lp, old, adv, ref, en, *args[2:])[0][0]  # noqa: E731
    got = (loss(logp + H * v, ent) - loss(logp - H * v, ent)) / (2 * H)
    assert abs(got - float((dl * v).sum())) < DIFF * 10
    got = (loss(logp, ent + H * v) - loss(logp, ent - H * v)) / (2 * H)
    assert abs(got - float((de * v).sum())) < DIFF * 10
