"""Tree attention where values or scores are unusual: V elements that are not finite under a
finite score, in short contexts (one CTA) and long ones (parts that are joined), scores far
apart, queries with an outlier channel, caches past 2^31 bytes."""
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


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


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
    ([(150, 40), (30, 30), (200, 70)], 8, 4, 64),  # a tree inside one or two tiles
    ([(700, 300)] * 12, 16, 16, 64),               # several tree tiles of one CTA's run
    ([(700, 300)] * 6, 16, 16, 128),
    ([(6000, 300)], 4, 2, 128),                    # parts of one to a few tiles, joined
    ([(6000, 300), (4100, 20)], 4, 2, 64),
])
def test_values_not_finite_under_finite_scores(ops, lens, Hq, Hkv, D, f8):
    w = Tree(lens, Hq, Hkv, D, seed=50 + len(lens), f8=f8)
    odd = odd_values(w, (0, 3, 63, 64, 130, 199, 255, 256, 299), [NAN] if f8 else [INF, -INF, NAN])
    n = check_odd_values(ops, w, odd)
    assert 0 < n < w.q.numel() // 10


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


def split_error(w):
    """How far E4M3 scores may be off by the two-term form of q: it is exact for elements down
    to 2^-9 of the row's largest, and within 2^-17 of the largest below."""
    q = w.q.double().abs()
    top = q.amax(-1, keepdim=True)
    err = torch.where(q < top * 2.0 ** -9, top * 2.0 ** -17, torch.zeros_like(q))
    worst = torch.zeros(w.q.shape[0], w.Hq, dtype=torch.float64)
    G = w.Hq // w.Hkv
    for s in range(w.S):
        k, _ = w.kv64(s)
        rows = slice(int(w.qs[s]), int(w.qs[s + 1]))
        e = err[rows].view(-1, w.Hkv, G, w.D)
        worst[rows] = torch.einsum("nhgd,chd->nhgc", e, k.abs()).amax(-1).reshape(-1, w.Hq)
    return worst * w.scale


def check_scores(ops, w):
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    n = int(w.qs[-1])
    if w.f8:
        # a score off by e moves a weight by e of itself and the sum as much; |out| <= max |V|
        vmax = max(float(w.kv64(s)[1].abs().max()) for s in range(w.S))
        bound = bound + (2 * split_error(w)[:n, :, None] * vmax)
    assert_within(out[:n], ref, bound)
    assert int(d["err"]) == 0


@pytest.mark.parametrize("lens", [[(700, 30)], [(5000, 30)], [(2000, 5)] * 40])
@pytest.mark.parametrize("D", [64, 128])
def test_e4m3_scores_far_apart(ops, lens, D):
    """The running maximum jumps by tens to hundreds, early and late in a run."""
    w = Tree(lens, 8, 2, D, seed=60, f8=True)
    # scores up to ~150, their fp32 rounding below 2^-24 x 2^13: inside the bound's 2^-10
    w.q = (w.q.float() * 40).to(torch.bfloat16)
    check_scores(ops, w)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lens", [[(333, 40), (64, 64)], [(5000, 9)]])
def test_queries_with_an_outlier_channel(ops, lens, f8):
    w = Tree(lens, 8, 2, 128, seed=61, f8=f8)
    w.q[:, :, 17] *= 60
    w.q[::3, :, 90] *= 2.0 ** -12
    check_scores(ops, w)


def test_e4m3_cache_offsets_past_32_bits(ops):
    """Blocks at the far end of E4M3 caches of more than 2^31 bytes: written, read, moved."""
    Hkv, D = 8, 128
    w = Tree([(200, 20), (90, 7)], 8, Hkv, D, seed=15, f8=True, poison=False)
    NB = 2**31 // (Hkv * BS * D) + 40
    if torch.cuda.mem_get_info()[0] < 4 * NB * Hkv * BS * D:
        pytest.skip("not enough free memory")
    d = w.cuda()
    far = torch.arange(w.NB, device="cuda") + NB - w.NB
    for n in ("k", "v"):
        big = torch.empty(NB, Hkv, BS, D, dtype=torch.uint8, device="cuda")
        big[far] = d[n]
        d[n] = big
    d["bt"] = torch.where(d["bt"] >= 0, d["bt"] + NB - w.NB, d["bt"])
    out, _ = run_tree(ops, w, d=d)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    assert int(d["err"]) == 0
    slots = d["slots"] + (NB - w.NB) * BS
    v = d["v"].view(NB, Hkv, D, BS)
    take = lambda i: (d["k"][slots[i] // BS, :, slots[i] % BS].clone(),
                      v[slots[i] // BS, :, :, slots[i] % BS].clone())
    want = take(19)
    ops.paged_tree_commit_fp8(d["k"], d["v"], slots, d["qs"], i32([[19, 3], [0, 6]]), i32([2, 2]))
    assert all(torch.equal(a, b) for a, b in zip(take(0), want))
    rows = torch.randn(27, 16, D, device="cuda").to(torch.bfloat16)
    ops.paged_qk_norm_rope_write_fp8(rows[:, :8].clone(), rows[:, :8], rows[:, 8:], rows[:, 8:],
                                     None, None, slots, d["k"], d["v"], 1.0, 1.0)
    codes = rows[:, 8:].to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(d["k"][slots // BS, :, slots % BS], codes)
    assert torch.equal(v[slots // BS, :, :, slots % BS], codes)


def test_e4m3_long_tail_of_small_weights(ops):
    """One token that outweighs each of half a million others by 2^25.3: their share of the
    result, 1.2 percent, is not lost.  Every CTA's run is one whole sequence (all share the
    same few blocks), so that one reference serves all of its keys."""
    n, D, x = 1 << 19, 64, 25.3
    S = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")
    k, v = z(2, 1, BS, D, t=torch.uint8), z(2, 1, BS, D, t=torch.uint8)
    one = int(torch.tensor(1.0).to(torch.float8_e4m3fn).view(torch.uint8))
    k[0, 0, 0, 0] = one  # the token that outweighs: score q . K = 1, the others' 0; V 0, theirs 1
    v.view(2, 1, D, BS)[:] = one
    v.view(2, 1, D, BS)[0, 0, :, 0] = 0
    bt = z(S, n // BS).fill_(1)
    bt[:, 0] = 0
    q = z(S, 1, D, t=torch.bfloat16)
    q[..., 0] = 1
    out, err = torch.empty_like(q), z(1)
    ws = ops.alloc_tree_workspace(1, 1, D, 1)
    masks = torch.ones(S, 1, dtype=torch.int64, device="cuda")
    ops.paged_attention_tree_fp8(out, q, k, v, bt, z(S).fill_(n),
                                 torch.arange(S + 1, dtype=torch.int32, device="cuda"), masks,
                                 x * np.log(2.0), 1.0, 1.0, 1, ws, err_flag=err)
    w = (n - 1) * 2.0 ** -x
    want = w / (1 + w)
    # bf16's half step; a weight of 2^-25.3 lifted by 2^7 is within 2^-25 in f16 (2^-32 of the
    # largest); the product's sum grows by 4 x 8192 terms of equal size, each truncated to 2^-23
    # of what has been summed (2^-24 on average); l, above 2^7, takes 8192 terms within 2^-17
    tol = want * (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -11) + n * 2.0 ** -32
    assert tol < want / 20
    assert int(err) == 0
    assert float((out.double() - want).abs().max()) <= tol
