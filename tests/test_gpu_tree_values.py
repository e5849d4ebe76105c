"""Tree attention where values or scores are unusual."""
import copy

import numpy as np
import pytest
import torch

import tree_helpers as TH
from tree_helpers import BS, Tree, assert_within, run_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_272_gb300 import ops as o
    return o


def set_v(w, s, t, head, d, value):
    """V of cached token t of sequence s (value: a number, or an E4M3 code)."""
    b, o = int(w.bt[s, t // BS]), t % BS
    if w.f8:
        w.v.view(w.NB, w.Hkv, w.D, BS)[b, head, d, o] = value
    else:
        w.v[b, head, o, d] = value


def check_odd_values(ops, w, odd):
    """odd: (sequence, tree token, head, column, value).  A row that sees the token gets the
    value in that column (their sum, where it sees several), and no other element changes:
    each weight is above zero and finite, and times a value that is not finite that value."""
    clean = copy.copy(w)
    clean.v = w.v.clone()
    special = {}
    for s, j, h, d, val in odd:
        t = int(w.ctx[s] - w.L[s]) + j
        set_v(clean, s, t, h, d, 0)
        set_v(w, s, t, h, d, 0x7F if w.f8 else val)
        for i in range(int(w.L[s])):
            r = int(w.qs[s]) + i
            if w.visible[r][j]:
                special.setdefault((r, h, d), []).append(val)
    out, dev = run_tree(ops, w)
    assert int(dev["err"]) == 0
    ref, bound = clean.attention64()
    G = w.Hq // w.Hkv
    want = torch.zeros_like(ref)  # 0: finite
    for (r, h, d), vals in special.items():
        want[r, h * G:(h + 1) * G, d] = sum(vals)
    got = out[:int(w.qs[-1])].cpu().double()
    fine = want == 0
    assert torch.isfinite(got[fine]).all()
    assert ((got - ref).abs() <= bound)[fine].all()
    assert torch.equal(torch.isnan(got[~fine]), torch.isnan(want[~fine]))
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf])
    return int((~fine).sum())


def odd_values(w, tokens, values, seed=0):
    rng = np.random.default_rng(seed)
    out = []
    for s in range(w.S):
        for j in tokens:
            if j < w.L[s]:
                out.append((s, j, int(rng.integers(w.Hkv)), int(rng.integers(w.D)),
                            values[int(rng.integers(len(values)))]))
    return out


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([(400, 20)], 4, 2, 64),     # few parts
    ([(9000, 100)], 8, 2, 128),  # many
])
def test_values_not_finite_under_vanishing_weights(ops, lens, Hq, Hkv, D, f8):
    """One cached token outscores the tree by more than fp32's range of weights.  A row that
    sees a value that is not finite there gets it all the same, as its weight is above zero,
    whether the two lie in one CTA's run or in parts that are joined."""
    w = Tree(lens, Hq, Hkv, D, seed=52, f8=f8)
    w.q[:, :, 0] = 1024.0
    t = 5  # K in column 0: this token's largest, the others' none
    b, o = int(w.bt[0, t // BS]), t % BS
    if f8:
        w.k[:, :, :, 0] = 0
        w.k[b, :, o, 0] = 0x7E  # 448, in value at least 448 / 64
    else:
        w.k[:, :, :, 0] = 0
        w.k[b, :, o, 0] = 8.0
    # scores: 1024 x 7 x D^-1/2 >= 633 in front of what the normals give (below 50); the outlier
    # leaves q's small elements 2^-7 in E4M3 terms, which cannot bring them near
    assert w.scale * 1024 * 7 > 600
    odd = odd_values(w, (0, 7, 19, 40, 63, 64, 99), [NAN] if f8 else [INF, -INF, NAN], seed=1)
    assert check_odd_values(ops, w, odd) > 0
