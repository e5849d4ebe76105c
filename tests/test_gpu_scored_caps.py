"""Caps of scored attention at the ends of what is accepted, against the plain 64-bit form."""
import pytest
import torch

from range_helpers import Scored
from tree_helpers import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_272_gb300 import ops as o
    return o


def check(ops, w, what=""):
    out, d = w.run(ops)
    assert_within(out, *w.reference(), what)
    assert int(d["err"]) == 0


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [1e-38, 1e-30, 1e-12, 3e-8, 1e-3, 30.0, 4096.0])
def test_scores_of_zero(ops, cap, D, f8):
    """Queries that are zero, and key tiles that are, beside others: their scores are zero, whatever
    the cap, and their weights those of the definition."""
    for bias in (False, True):
        w = Scored([(200, 9), (70, 33)], 8, 2, D, "causal", cap=cap, bias=bias, seed=23, f8=f8)
        w.q[:] = 0
        check(ops, w, "queries")
        w = Scored([(200, 9), (70, 33)], 8, 2, D, "causal", cap=cap, bias=bias, seed=24, f8=f8)
        for t in range(64):
            w.k[int(w.bt[0, t // 16]), :, t % 16] = 0
        check(ops, w, "keys")


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [128.0, 1000.0, 4096.0])
def test_large_caps_within_the_bound_of_all(ops, cap, D, f8):
    """Scores to about 35, far below the cap: off by 2^-23.6 of the cap at most (at 4096 3.2e-4), and by
    the products' rounding (128 of magnitude 16 at 2^-24 each, 1.2e-4): a weight moves by less than
    2^-11 of itself, the result by twice that, within the 2^-10 of every other case."""
    w = Scored([(300, 9), (700, 1)], 8, 2, D, "causal", cap=cap, seed=25, f8=f8)
    w.q *= 4
    check(ops, w)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("part", [0.1, 0.16, 0.32, 0.44])
@pytest.mark.parametrize("cap", [64.0, 65.0, 4096.0])
def test_tiles_of_both_forms(ops, cap, part, f8):
    """Equal scores in two tiles, one of which holds a far score of the other sign: the two forms of
    the tanh agree, so that V of 1 and of -1 cancel.  Each is within 2^-21 of the cap (at 4096 0.002;
    their difference of 0.0013, as their sources add up: 2^-23.6 and 1.2 2^-22, moves the result by half
    of that, below the bound's 2^-10)."""
    w = Scored([(128, 1)], 2, 1, 64, "causal", cap=cap, seed=26, f8=f8)
    w.q[:] = 1
    b = torch.as_tensor(w.bt[0]).long()
    x = part * cap          # the score of all keys but one, whose score is -16 x
    v = torch.where(torch.arange(128) < 64, 1.0, -1.0).view(8, 16)
    if f8:
        code = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)
        w.ks[:], w.vs[:] = x / 8, 1.0
        k = torch.ones(8, 1, 16, 64)
        k[5, 0, 3] = -16
        w.k[b], w.v.view(w.NB, 1, 64, 16)[b] = code(k), code(v.view(8, 1, 1, 16).expand(8, 1, 64, 16))
    else:
        k = torch.full((8, 1, 16, 64), x / 8)
        k[5, 0, 3] = -2 * x
        w.k[b] = k.to(torch.bfloat16)
        w.v[b] = v.view(8, 1, 16, 1).expand(8, 1, 16, 64).to(torch.bfloat16)
    check(ops, w, (cap, part))
