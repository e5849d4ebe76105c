"""Shared-prefix decode, scored attention and verification at the ends of their sizes: more query heads a
KV head than a row tile has rows, as many sequences as a call takes, vocabularies of one, no tokens."""
import numpy as np
import pytest
import torch

import verify_helpers as VH
from range_helpers import Scored, Shared
from tree_helpers import assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_272_gb300 import ops as o
    prev = o.set_shared_variant(o.PKV_SHARED_ALWAYS)
    yield o
    o.set_shared_variant(prev)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("G,Hkv,D", [(127, 2, 64), (129, 1, 128), (200, 1, 64), (256, 2, 128)])
def test_more_heads_than_rows(ops, G, Hkv, D, f8):
    """A token's rows lie in two row tiles or more, and a row tile begins within a token's."""
    w = Shared([(3, 200, [5, 0, 70]), (2, 96, 33)], G * Hkv, Hkv, D, seed=1, f8=f8)
    out, d = w.run(ops)
    assert_within(out, *w.reference())
    assert int(d["err"]) == 0
    for mask, cap, bias in (("causal", 0.0, False), ("window", 30.0, True), ("odd", 0.0, True)):
        w = Scored([(90, 7), (200, 1), (3, 3)], G * Hkv, Hkv, D, mask, 40, cap, bias, seed=2, f8=f8,
                   pad_rows=1)
        out, d = w.run(ops)
        n = int(w.qs[-1])
        assert_within(out[:n], *w.reference(), mask)
        assert (out[n:] == 9).all() and int(d["err"]) == 0


class Short:
    """65535 sequences of up to 40 tokens over a few blocks, which many of them name."""

    def __init__(self, f8, seed):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.w = Shared([(64, 0, 47)], 2, 1, 64, seed=seed, f8=f8)
        self.S = 65535
        w = self.w
        w.bt = w.bt[rng.integers(0, 64, self.S)]
        w.ctx = rng.integers(0, 41, self.S).astype(np.int32)
        w.S = self.S
        w.q = torch.randn(self.S, 2, 64, generator=g).to(torch.bfloat16)
        self.some = rng.choice(self.S, 300, replace=False)

    def check(self, out):
        w = self.w
        ref, bound = zip(*(w.row64(w.q[s], *w.kv64(s), w.scale) for s in self.some))
        assert torch.isfinite(out).all()
        assert_within(out[torch.from_numpy(self.some).cuda()], torch.stack(ref), torch.stack(bound))


@pytest.mark.parametrize("f8", [False, True])
def test_most_sequences(ops, f8):
    x = Short(f8, 3)
    w = x.w
    # groups of every size, without anything in common but that is named so: no whole block
    cuts = np.sort(np.random.default_rng(4).choice(np.arange(1, x.S), 4000, replace=False))
    w.starts = np.concatenate([[0], cuts, [x.S]]).astype(np.int32)
    w.prefix = np.zeros(len(w.starts) - 1, np.int32)
    out, d = w.run(ops)
    x.check(out)
    assert int(d["err"]) == 0
    # one token each, as scored attention (a sequence without tokens in its context has no row)
    L = (w.ctx > 0).astype(np.int32)
    qs = np.concatenate([[0], np.cumsum(L)]).astype(np.int32)
    rows = torch.from_numpy(np.flatnonzero(L))
    d = w.cuda(q=w.q[rows], qs=qs)
    T = len(rows)
    o = torch.full((T, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = ops.alloc_scored_workspace(x.S, T, 2, 1, 64)
    f = ops.paged_attention_scored_fp8 if f8 else ops.paged_attention_scored
    f(o, d["q"], d["k"], d["v"], d["bt"], d["ctx"], d["qs"], w.scale,
      *((d["ks"], d["vs"]) if f8 else ()), ws, err_flag=d["err"])
    full = torch.zeros(x.S, 2, 64, dtype=torch.bfloat16, device="cuda")
    full[rows.cuda()] = o
    x.check(full)
    assert int(d["err"]) == 0


@pytest.mark.parametrize("f8", [False, True])
def test_one_group_of_all_sequences(ops, f8):
    """One prefix of 32 tokens for all: 1024 row tiles."""
    x = Short(f8, 5)
    w = x.w
    first = w.bt[0, :2].copy()
    w.bt = np.concatenate([np.tile(first, (x.S, 1)), w.bt[:, 2:]], 1)
    w.ctx = np.maximum(w.ctx, 32)
    w.starts, w.prefix = np.array([0, x.S], np.int32), np.array([32], np.int32)
    out, d = w.run(ops)
    x.check(out)
    assert int(d["err"]) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafts", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 9])
def test_small_vocabularies(ops, V, drafts, dtype):
    for kind in ("chain", "star"):
        w = VH.Drafts([3, 1, 0, 5] * 20, V, kind, drafts, dtype, seed=V)
        out, t = VH.run_verify(ops, w)
        VH.assert_same(out, VH.plain_verify(w), (V, kind))
        assert int(t["err"]) == 0


@pytest.mark.parametrize("drafts", [False, True])
def test_no_tokens(ops, drafts):
    w = VH.Drafts([0, 0, 0], 10, "chain", drafts)
    w.A = 4
    out, t = VH.run_verify(ops, w)
    assert out[0].tolist() == [[-1] * 4] * 3 and out[1].tolist() == [0] * 3
    assert out[2].tolist() == [-1] * 3 and int(t["err"]) == 0
