"""How the kernels of a shared-prefix decode wait for one another, read from a captured call: two of
them read the plan without waiting for the launch before them, so the launch behind the plan starts
once the plan is complete and the others start behind that one."""
import ctypes

import pytest
import torch

from range_helpers import Scored, Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


class EdgeData(ctypes.Structure):
    _fields_ = [("from_port", ctypes.c_ubyte), ("to_port", ctypes.c_ubyte),
                ("type", ctypes.c_ubyte), ("reserved", ctypes.c_ubyte * 5)]


FULL, PROGRAMMATIC = 0, 1


def edges(call):
    """The kinds of the edges of a captured chain of kernels, in its order."""
    cu = ctypes.CDLL("libcuda.so.1")
    ok = lambda r: r == 0 or pytest.fail(f"driver error {r}")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g, n = ctypes.c_void_p(), ctypes.c_size_t()
    ok(cu.cuStreamBeginCapture_v2(ctypes.c_void_p(st.cuda_stream), 2))
    try:
        call(st.cuda_stream)
    finally:
        ok(cu.cuStreamEndCapture(ctypes.c_void_p(st.cuda_stream), ctypes.byref(g)))
    get = cu.cuGraphGetEdges_v2
    ok(get(g, None, None, None, ctypes.byref(n)))
    src, dst = (ctypes.c_void_p * n.value)(), (ctypes.c_void_p * n.value)()
    kind = (EdgeData * n.value)()
    ok(get(g, src, dst, kind, ctypes.byref(n)))
    ok(cu.cuGraphDestroy(g))
    after = {s: (d, k.type) for s, d, k in zip(src, dst, kind)}
    assert len(after) == n.value  # a chain
    at = (set(after) - {d for d, _ in after.values()}).pop()
    out = []
    while at in after:
        at, k = after[at]
        out.append(k)
    return out


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_shared(D, f8):
    from paged_kv_cache_272_gb300 import ops
    w = Shared([(3, 64, 5)], 8, 2, D, f8=f8)
    d = w.cuda(q=w.q, starts=w.starts, prefix=w.prefix)
    ws = ops.alloc_shared_workspace(w.S, 1, w.Hq, w.Hkv, w.D)
    out, _ = w.run(ops, d, ws)
    # plan, prefixes, own keys, join
    assert edges(lambda st: w.run(ops, d, ws, out, st)) == [FULL, PROGRAMMATIC, PROGRAMMATIC]


def test_scored():
    from paged_kv_cache_272_gb300 import ops
    w = Scored([(64, 5)], 8, 2, 64)
    d = w.cuda(q=w.q, qs=w.qs, kb=None, ke=None, sl=None)
    ws = ops.alloc_scored_workspace(w.S, w.T, w.Hq, w.Hkv, w.D)
    out, _ = w.run(ops, d, ws)
    # each waits for the one before: plan, attention, join
    assert edges(lambda st: w.run(ops, d, ws, out, st)) == [PROGRAMMATIC, PROGRAMMATIC]
