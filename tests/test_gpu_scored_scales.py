"""One scale per E4M3 cache (floats) in scored attention, as the other calls take it."""
import pytest
import torch

from range_helpers import Scored
from tree_helpers import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (50.0, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_one_scale_per_cache(D, cap, bias):
    from paged_kv_cache_272_gb300 import ops
    w = Scored([(600, 1), (130, 40), (33, 33)], 8, 2, D, "window", 100, cap, bias, seed=27, f8=True)
    w.ks[:], w.vs[:] = 0.02, 0.03
    d = w.cuda(q=w.q, qs=w.qs, kb=w.key_begin, ke=w.key_end, sl=w.slopes)
    heads, _ = w.run(ops, d)
    d["ks"], d["vs"] = 0.02, 0.03
    out, _ = w.run(ops, d)
    assert_within(out, *w.reference())
    # scale k_scale is rounded once with one scale, twice with one a head: 2^-24 of a score more
    _, bound = w.reference()
    assert_within(out, heads.cpu().double(), 2 * bound)
    assert int(d["err"]) == 0
    for bad in (0.0, -1.0, float("nan")):
        for n in ("ks", "vs"):
            e = dict(d)
            e[n] = bad
            with pytest.raises(ops.PagedKVError):
                w.run(ops, e)
