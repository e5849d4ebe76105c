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
