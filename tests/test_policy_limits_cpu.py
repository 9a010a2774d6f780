"""The sizes that the policy head's header admits and refuses, against the library's answers.
Fake pointers: every call is refused on the host."""

import re

import pytest

from bitwise_consistent_linear_amd import api
from test_policy_cpu import BF16, F32, HEADER, SHAPE, lb, li, lp_shape, nb, nf, qr


@pytest.fixture(scope="module")
def L():
    return api.policy_lib()


def header(name):
    """The comment in front of a declaration, its lines joined."""
    text = open(HEADER).read()
    comment = text[:text.index(f"gdn_status_t {name}(")].rsplit("/*", 1)[1]
    return re.sub(r"\s*\n \*\s*", " ", comment)


@pytest.mark.parametrize("dt,run", [(F32, 2048), (BF16, 4096)])
def test_gradient_of_the_logits(L, dt, run):
    """2^30 rows of one value more than a run are 2^31 runs."""
    assert lb(L, lp_shape(rows=2**30, vocab=run + 1, stride=run + 1, dt=dt)) == SHAPE
    assert f"{run}" in L.gdn_policy_last_error().decode()
    assert "2^31" in L.gdn_policy_last_error().decode()
    assert "rows * ceil(vocab / 2048) (4096 for BF16) passes 2^31 - 1" in header("gdn_token_logprob_bwd")


def test_product(L):
    """Tiles of 64 x 64 values hold 256 threads: 2^20 rows and columns are far past a launch's
    2^32 - 1 even in tiles of 256 x 256, which hold 512."""
    for m, n in ((2**20, 2**20), (2**30, 1), (1, 2**31 - 1)):
        assert li(L, m=m, n=n) == SHAPE, (m, n)
        assert -(-m // 64) * 64 * (-(-n // 64) * 64) >= 2**35
    assert "under 2^35, m and n rounded up to multiples of 64" in header("gdn_linear_i8_fwd")


def test_strides(L):
    over = 2**31 + 1
    assert nf(L, stride=over) == nb(L, ds=over) == nb(L, xs=over) == qr(L, stride=over) == SHAPE
    assert lb(L, lp_shape(stride=over)) == SHAPE
    text = re.sub(r"\s*\n \*\s*", " ", open(HEADER).read())
    assert "An input's stride may be any value in [0, 2^31]" in text
