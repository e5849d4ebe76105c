"""The drafted-tree operators on the GPU against their plain 64-bit forms (tree_helpers): each
element within a bound that counts the roundings of the kernel's types."""
import numpy as np
import pytest
import torch

import oracle
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


# ---- masks ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("sizes,words", [([1], 1), ([8, 1, 0, 64, 33], 1), ([65, 128, 2], 2),
                                         ([200, 7, 131], 5), ([1024, 3], 16)])
def test_masks(ops, sizes, words, kind):
    w = Tree([(n + 5 * s, n) for s, n in enumerate(sizes)], 1, 1, 64, seed=sum(sizes), words=words,
             kind=kind, pad_rows=3, poison=False)
    d = w.cuda()
    for base in (None, i32(np.arange(w.S) * 1000 - 7)):
        masks = torch.full((w.T, words), 77, dtype=torch.int64, device="cuda")
        pos = torch.full((w.T,), 55, dtype=torch.int32, device="cuda")
        ops.paged_tree_masks(masks, pos, d["parents"], d["qs"], d["ctx"], base, err_flag=d["err"])
        n = int(w.qs[-1])
        assert torch.equal(masks[:n].cpu(), w.masks[:n])
        want = []
        for s in range(w.S):
            b = int(base[s]) if base is not None else int(w.ctx[s] - w.L[s])
            want += [b + int(w.visible[r].sum()) - 1 for r in range(w.qs[s], w.qs[s + 1])]
        assert pos[:n].tolist() == want
        assert (masks[n:] == 77).all() and (pos[n:] == 55).all()
        assert int(d["err"]) == 0
    ops.paged_tree_masks(masks, None, d["parents"], d["qs"], d["ctx"])


def test_masks_bad_input(ops):
    """A parent that does not come first is flagged and taken as the context; a tree beyond
    the mask words, or beyond its context, is flagged and left unwritten."""
    par = i32([-1, 0, 2, 5, -2, 1])
    masks = torch.zeros(6, 1, dtype=torch.int64, device="cuda")
    err = i32([0])
    ops.paged_tree_masks(masks, None, par, i32([0, 6]), i32([20]), err_flag=err)
    assert masks.flatten().tolist() == [1, 3, 4, 8, 16, 35] and int(err) == ops.DEV_BAD_TREE
    big = torch.full((70, 1), 5, dtype=torch.int64, device="cuda")
    for qs, ctx in (([0, 66, 70], [99, 99]), ([0, 4, 70], [3, 99])):
        err.zero_()
        big.fill_(5)
        ops.paged_tree_masks(big, None, i32([-1] * 70), i32(qs), i32(ctx), err_flag=err)
        assert int(err) == ops.DEV_BAD_CONTEXT
        left = torch.tensor([qs[0] <= r < qs[1] if ctx[0] == 3 or qs[1] > 64 else False
                             for r in range(70)])
        assert (big.cpu()[left] == 5).all()


# ---- norm, rotation, write -----------------------------------------------------------
def rope_case(T, Hq, Hkv, D, seed, far=40000, axes=1):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16)
    NB = -(-T // BS) + 2
    slots = torch.randperm(NB * BS, generator=g)[:T].to(torch.int64)
    pos = torch.randint(0, far, (axes, T), generator=g).to(torch.int32)
    qw = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16)
    kw = (1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16)
    return g, qkv, NB, slots, pos, qw, kw


def split(qkv, Hq, Hkv, D):
    T = qkv.shape[0]
    q = qkv[:, :Hq * D].view(T, Hq, D) if qkv.is_contiguous() and Hq * D == qkv.shape[1] else \
        qkv[:, :Hq * D].unflatten(1, (Hq, D))
    return (q, qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),
            qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D)))


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,axes,order,inter,norm,scale", [
    (1, 8, 8, 128, 128, 1, None, False, True, 1.0),
    (3, 7, 1, 64, 64, 1, None, True, True, 1.0),
    (33, 12, 4, 128, 64, 3, "blocked", False, True, 1.0),
    (33, 4, 2, 64, 48, 2, "cyclic", True, False, 1.25),
    (17, 6, 3, 128, 16, 4, "cyclic", False, False, 1.0),
    (16, 4, 4, 64, 0, 1, None, False, True, 1.0),
    (2600, 5, 5, 64, 32, 1, None, False, True, 1.0),
    (2603, 8, 2, 128, 128, 3, "cyclic", True, True, 0.75),
])
def test_qk_norm_rope_write(ops, f8, T, Hq, Hkv, D, rot, axes, order, inter, norm, scale):
    g, qkv, NB, slots, pos, qw, kw = rope_case(T, Hq, Hkv, D, T + D + axes, axes=axes)
    slots[2::5] = -1  # padding tokens: q only
    half = rot // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    ax = [0] * half if order is None else [i * axes // half if order == "blocked" else i % axes
                                           for i in range(half)]
    dq = qkv.cuda()
    q, k, v = split(dq, Hq, Hkv, D)
    qo = torch.full((T, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    err = i32([0])
    kw_ = dict(q_weight=qw.cuda() if norm else None, k_weight=kw.cuda() if norm else None,
               eps=1e-5, pair_axes=ax if axes > 1 else None, interleaved=inter, rope_scale=scale,
               err_flag=err)
    p = pos.cuda() if axes > 1 else pos[0].cuda()
    fr = freq.cuda() if rot else None
    if f8:
        ks, vs = (torch.rand(Hkv, generator=g) + 0.5) / 40, (torch.rand(Hkv, generator=g) + 0.5) / 40
        kc = torch.full((NB, Hkv, BS, D), 3, dtype=torch.uint8, device="cuda")
        vc = kc.clone()
        ops.paged_qk_norm_rope_write_fp8(qo, q, k, v, p, fr, slots.cuda(), kc, vc, ks.cuda(),
                                         vs.cuda(), **kw_)
    else:
        kc = torch.full((NB, Hkv, BS, D), 3.0, dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
        ops.paged_qk_norm_rope_write(qo, q, k, v, p, fr, slots.cuda(), kc, vc, **kw_)
    assert int(err) == 0 and torch.equal(dq.cpu(), qkv)
    hq, hk, hv = split(qkv, Hq, Hkv, D)
    y, b = TH.rope64(hq, qw if norm else None, 1e-5, pos, ax, freq, rot, inter, scale)
    assert_within(qo, y, b + TH.BF16_HALF * y.abs() + 2.0 ** -134, "q")
    y, b = TH.rope64(hk, kw if norm else None, 1e-5, pos, ax, freq, rot, inter, scale)
    on = slots >= 0
    blk, off = slots[on] // BS, slots[on] % BS
    got = kc.cpu()
    rest = torch.ones(NB, BS, dtype=torch.bool)
    rest[blk, off] = False
    if not f8:
        assert_within(got[blk, :, off], y[on], (b + TH.BF16_HALF * y.abs() + 2.0 ** -134)[on], "k")
        assert torch.equal(vc.cpu()[blk, :, off], hv[on])
        assert (got.transpose(1, 2)[rest] == 3).all() and (vc.cpu().transpose(1, 2)[rest] == 3).all()
        return
    z = y / ks.double().view(1, -1, 1)
    bz = b / ks.double().view(1, -1, 1) + z.abs() * 2.0 ** -23
    assert_within(got[blk, :, off].view(torch.float8_e4m3fn).double(), z[on].clamp(-448, 448),
                  (bz + TH.E4M3_HALF * z.abs().clamp(max=448) + 2.0 ** -10)[on], "k codes")
    # v codes are those of the plain quantising write
    k2, v2 = torch.full_like(kc, 3), torch.full_like(vc, 3)
    ops.paged_kv_write_fp8_per_head(k.contiguous(), v.contiguous(), slots.cuda(), k2, v2, ks.cuda(),
                                    vs.cuda())
    assert torch.equal(vc, v2)
    assert (got.transpose(1, 2)[rest] == 3).all()
    if not rot and not norm:
        assert torch.equal(kc, k2)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,D", [(1215, 64), (1217, 64), (3647, 128), (3651, 128), (400, 128)])
@pytest.mark.parametrize("inter", [False, True])
def test_qk_norm_rope_write_around_the_launch_shapes(ops, f8, T, D, inter):
    """One and two tokens per CTA, and a token's heads over several CTAs."""
    test_qk_norm_rope_write(ops, f8, T, 12, 2, D, 32, 1, None, inter, True, 1.0)


@pytest.mark.parametrize("f8", [False, True])
def test_write_without_norm_or_rotation_is_the_plain_write(ops, f8):
    g, qkv, NB, slots, _, _, _ = rope_case(50, 4, 2, 128, 5)
    dq = qkv.cuda()
    q, k, v = split(dq, 4, 2, 128)
    qo = torch.empty(50, 4, 128, dtype=torch.bfloat16, device="cuda")
    dt = torch.uint8 if f8 else torch.bfloat16
    c = [torch.zeros(NB, 2, BS, 128, dtype=dt, device="cuda") for _ in range(4)]
    if f8:
        ops.paged_qk_norm_rope_write_fp8(qo, q, k, v, None, None, slots.cuda(), c[0], c[1], 0.02,
                                         0.03)
        ops.paged_kv_write_fp8(k.contiguous(), v.contiguous(), slots.cuda(), c[2], c[3], 0.02, 0.03)
    else:
        ops.paged_qk_norm_rope_write(qo, q, k, v, None, None, slots.cuda(), c[0], c[1])
        ops.paged_kv_write(k.contiguous(), v.contiguous(), slots.cuda(), c[2], c[3])
    assert torch.equal(qo, q) and torch.equal(c[0], c[2]) and torch.equal(c[1], c[3])


@pytest.mark.parametrize("scales", [(0.02, 0.015), (1.0, 3.0e-3), (0.5, 448.0), (1e-30, 1e30),
                                    (3e38, 1e-38), (1.1e-18, 9e17), (0.0078125, 1 / 3)])
def test_e4m3_codes_of_every_bf16(ops, scales):
    """Every bf16 pattern as k and as v: the codes of the plain quantising write (a NaN's sign
    aside), for scales inside and far outside the range of the shared reciprocal."""
    D, Hkv = 128, 4
    T = 65536 // (D * Hkv)
    k = torch.arange(65536, dtype=torch.int32).sub(32768).to(torch.int16).view(T, Hkv, D)
    k = k.view(torch.bfloat16).cuda()
    v = k.flip(0).contiguous()
    slots = torch.arange(T, device="cuda")
    q = torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    c = [torch.zeros(T // BS, Hkv, BS, D, dtype=torch.uint8, device="cuda") for _ in range(4)]
    ops.paged_qk_norm_rope_write_fp8(q.clone(), q, k, v, None, None, slots, c[0], c[1], *scales)
    ops.paged_kv_write_fp8(k, v, slots, c[2], c[3], *scales)
    for a, b in ((c[0], c[2]), (c[1], c[3])):
        nan = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
        assert bool(((a == b) | nan).all()), int((a != b).sum())


def test_rope_in_place_far_positions_and_shared_axes(ops):
    """q rotated where it stands in the packed projection, positions up to the largest int32
    (and negative ones), one row of positions for all axes."""
    T, Hq, Hkv, D = 9, 4, 2, 128
    _, qkv, NB, slots, _, _, _ = rope_case(T, Hq, Hkv, D, 11)
    pos = torch.tensor([0, 1, -1, 131072, 1000003, 2**31 - 1, -2**31, 99999999, 7],
                       dtype=torch.int32)
    freq = 500000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    dq = qkv.cuda()
    q, k, v = split(dq, Hq, Hkv, D)
    kc = torch.zeros(NB, Hkv, BS, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ops.paged_qk_norm_rope_write(q, q, k, v, pos.cuda().expand(3, T), freq.cuda(), slots.cuda(), kc,
                                 vc, pair_axes=bytes(i % 3 for i in range(64)))
    hq, hk, hv = split(qkv, Hq, Hkv, D)
    y, b = TH.rope64(hq, None, 0, pos.expand(3, T), [0] * 64, freq, D, False)
    # the 64-bit form's own angle is off by 2^-53 x 2^31 rad at most: below 2^-20
    assert_within(q, y, b * 32 + TH.BF16_HALF * y.abs(), "q")
    assert torch.equal(dq.cpu()[:, Hq * D:], qkv[:, Hq * D:])


def test_rope_flags(ops):
    T, Hq, Hkv, D = 6, 2, 2, 64
    _, qkv, NB, slots, pos, _, _ = rope_case(T, Hq, Hkv, D, 13)
    slots[1] = NB * BS
    dq = qkv.cuda()
    q, k, v = split(dq, Hq, Hkv, D)
    qo = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(NB, Hkv, BS, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    err = i32([0])
    ops.paged_qk_norm_rope_write(qo, q, k, v, None, None, slots.cuda(), kc, vc, err_flag=err)
    assert int(err) == ops.DEV_BAD_SLOT and torch.equal(qo, q)
    assert int((kc != 0).any(-1).any(1).sum()) == T - 1
    c8 = torch.zeros(NB, Hkv, BS, D, dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(c8)
    sc = torch.tensor([0.02, 0.0], device="cuda")
    slots[1] = -1
    err.zero_()
    ops.paged_qk_norm_rope_write_fp8(qo, q, k, v, None, None, slots.cuda(), c8, v8, sc, sc,
                                     err_flag=err)
    assert int(err) == ops.DEV_BAD_SCALE and (c8[:, 1] == 0).all() and (c8[:, 0] != 0).any()
    with pytest.raises(ValueError):
        ops.paged_qk_norm_rope_write(qo, q.transpose(0, 1), k, v, None, None, slots.cuda(), kc, vc)
    with pytest.raises(ValueError):
        ops.paged_qk_norm_rope_write(qo, q, k, v, pos.cuda().expand(2, T),
                                     torch.ones(32, dtype=torch.float64, device="cuda"),
                                     slots.cuda(), kc, vc)


# ---- attention -----------------------------------------------------------------------
CASES = [
    # (context with the drafts, drafts) per sequence, Hq, Hkv, D
    ([(1, 1)], 1, 1, 64),
    ([(1, 1), (2, 2), (17, 1), (16, 16), (0, 0)], 4, 2, 128),
    ([(300, 8)], 32, 8, 128),
    ([(65, 1), (64, 64), (129, 65), (63, 3), (500, 33)], 8, 2, 64),
    ([(2100, 5), (40, 40), (777, 20)], 12, 2, 128),     # groups of 6
    ([(1500, 130), (131, 131), (200, 1)], 7, 1, 128),   # groups of 7, three mask words
    ([(90, 90), (1024, 50)], 16, 16, 64),               # no shared heads
    ([(400, 24)] * 9, 24, 2, 64),                       # groups of 12
    ([(3000, 17), (33, 17)], 64, 8, 128),
    ([(5000, 2)], 8, 8, 128),
]


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("kind", ["random", "chain", "star"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(ops, case, kind, f8):
    lens, Hq, Hkv, D = CASES[case]
    w = Tree(lens, Hq, Hkv, D, seed=case, kind=kind, f8=f8, pad_rows=2)
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    n = int(w.qs[-1])
    assert_within(out[:n], ref, bound, (lens, kind))
    assert (out[n:] == 9).all() and int(d["err"]) == 0
    again, _ = run_tree(ops, w, d=d)
    assert torch.equal(again[:n], out[:n])  # the same bits every time


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,D,maxq", [
    # more sequences than threads of a CTA, most of them shorter than a tile
    ([(1 + (7 * s) % 90, 1 + (7 * s) % 90 % 3) for s in range(701)], 2, 1, 64, None),
    # row tiles that only some sequences have
    ([(260, 70), (300, 3), (129, 129), (40, 1), (64, 64), (900, 33)], 16, 2, 128, None),
    # more row tiles than one launch takes, for one of two sequences
    ([(1030, 1024), (80, 5)], 12, 1, 64, None),
    # many KV heads; a bound on the tree sizes that none reaches
    ([(100, 5), (33, 9)], 40, 40, 64, 64),
])
def test_attention_many_sequences_heads_and_row_tiles(ops, lens, Hq, Hkv, D, maxq, f8):
    w = Tree(lens, Hq, Hkv, D, seed=len(lens), f8=f8)
    if maxq:
        w.maxq = maxq
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    assert int(d["err"]) == 0


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    # one row tile more than a launch takes: the second launch has a single one
    ([(80, 5), (930, 920)], 9, 1, 64),
    # row tiles of very different lengths, none of them shared
    ([(4000, 8), (20, 17), (600, 40), (33, 33), (2500, 1)], 8, 1, 128),
    # empty sequences between the others
    ([(0, 0), (700, 8), (64, 0), (5, 5), (0, 0), (129, 3)], 8, 8, 64),
    # as many sequences as a warp, a CTA and a CTA with one more have threads
    ([(40 + s % 60, 1 + s % 2) for s in range(256)], 2, 1, 64),
    ([(40 + s % 60, 1 + s % 2) for s in range(385)], 2, 1, 64),
])
def test_attention_cut_into_runs(ops, lens, Hq, Hkv, D, f8):
    w = Tree(lens, Hq, Hkv, D, seed=Hq, f8=f8)
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    assert int(d["err"]) == 0
    again, _ = run_tree(ops, w, d=d)
    assert torch.equal(again, out)


@pytest.mark.parametrize("f8", [False, True])
def test_attention_arbitrary_masks(ops, f8):
    """Masks that are no tree: random bits, rows that see nothing of the tree, a whole tree
    with no context and empty rows (zeros), bits past the tree's end, more words than
    needed."""
    lens = [(100, 70), (20, 20), (333, 64), (5, 5)]
    w = Tree(lens, 8, 2, 128, seed=4, words=3, f8=f8)
    rng = np.random.default_rng(5)
    for r in range(len(w.visible)):
        w.visible[r] = rng.random(w.visible[r].shape[0]) < 0.3
    for r in (3, 70 + 2, 70 + 19, 90 + 7, 154):
        w.visible[r][:] = False
    w.masks = TH.pack(w.visible, 3)
    for r, s in ((0, 0), (75, 1), (154, 3)):  # garbage past the end
        n = int(w.L[s])
        for b in range(n, 192):
            w.masks[r, b // 64] |= torch.tensor(1).to(torch.int64) << (b % 64)
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    assert (out[72] == 0).all() and (out[154] == 0).all() and int(d["err"]) == 0


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("bad", ["nan", "inf"])
def test_masked_rows_take_no_part(ops, bad, f8):
    """A drafted token whose K and V rows are NaN or infinite spoils the rows that see it and
    no other."""
    if f8 and bad == "inf":
        pytest.skip("E4M3 has no infinities")
    lens = [(150, 40), (30, 30), (200, 70)]
    w = Tree(lens, 8, 4, 64, seed=8, f8=f8)
    val = float(bad)
    for s, j in ((0, 11), (1, 0), (2, 66), (2, 3)):
        t = int(w.ctx[s] - w.L[s]) + j
        b, o = w.bt[s, t // BS], t % BS
        if f8:
            w.k[b, :, o], w.v.view(w.NB, 4, 64, BS)[b, :, :, o] = 0x7F, 0x7F
        else:
            w.k[b, :, o], w.v[b, :, o] = val, val
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    good = torch.isfinite(ref).all(-1)
    assert good.any() and not good.all()
    o = out.cpu().double()
    assert ((o - ref).abs() <= bound)[good].all()
    assert not torch.isfinite(o[~good]).all(-1).any()


def test_infinite_value_with_finite_score(ops):
    """An infinite V element seen with a positive weight gives that infinity; rows that do
    not see it are untouched."""
    w = Tree([(90, 30)], 4, 2, 128, seed=9)
    j = 7
    t = 60 + j
    w.v[w.bt[0, t // BS], :, t % BS, 5] = float("inf")
    out, _ = run_tree(ops, w)
    ref, bound = w.attention64()
    o = out.cpu().double()
    assert torch.equal(torch.isinf(o), torch.isinf(ref))
    fine = torch.isfinite(ref)
    b = torch.where(torch.isfinite(bound), bound, torch.zeros_like(bound))
    assert ((o - ref).abs() <= b)[fine].all()


def test_extreme_scores(ops):
    """Scores far apart (the running maximum jumps by hundreds) and all equal."""
    w = Tree([(700, 30)], 8, 2, 128, seed=10)
    w.q = (w.q.float() * 40).to(torch.bfloat16)
    out, _ = run_tree(ops, w)
    # a score's own fp32 rounding now moves weights: 128 products of magnitude up to ~500,
    # 2^-24 x 2^13 absolute at most, inside 2^-10 relative
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    w.q.zero_()
    out, _ = run_tree(ops, w)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)


def test_chain_is_prefill_and_single_token_is_decode(ops):
    w = Tree([(500, 100), (77, 77), (130, 1)], 8, 2, 128, seed=11, kind="chain")
    out, d = run_tree(ops, w)
    pre = torch.empty_like(out)
    ops.paged_attention_prefill(pre, d["q"], d["k"], d["v"], d["bt"], d["ctx"], d["qs"], w.scale,
                                w.maxq)
    ref, bound = w.attention64()
    assert_within(pre, ref, bound)
    assert ((out - pre).abs().cpu().double() <= 2 * bound).all()
    w = Tree([(n, 1) for n in (1, 16, 17, 900, 4000)], 16, 4, 64, seed=12)
    out, d = run_tree(ops, w)
    dec = torch.empty_like(out)
    ws = ops.alloc_workspace(5, 16, 64, 4000)
    ops.paged_attention_decode(dec, d["q"], d["k"], d["v"], d["bt"], d["ctx"], w.scale, 4000, ws)
    ref, bound = w.attention64()
    assert ((out - dec).abs().cpu().double() <= 2 * bound).all()


def test_attention_flags(ops):
    """Bad lengths leave the sequence's rows unwritten, bad blocks are flagged; the other
    sequences are served."""
    w = Tree([(50, 10), (60, 20), (70, 5)], 4, 2, 128, seed=14)
    ref, bound = w.attention64()

    def go(**ch):
        d = w.cuda()
        d.update(ch)
        out, d = run_tree(ops, w, d=d)
        return out, int(d["err"])
    # 65 tokens fit the table's five columns but reach its unused entry (-1)
    for ctx, want in (([50, 19, 70], ops.DEV_BAD_CONTEXT), ([50, 65, 70], ops.DEV_BAD_BLOCK),
                      ([50, -1, 70], ops.DEV_BAD_CONTEXT), ([50, 81, 70], ops.DEV_BAD_CONTEXT),
                      ([50, 2**31 - 1, 70], ops.DEV_BAD_CONTEXT)):
        out, err = go(ctx=i32(ctx))
        assert err == want, ctx
        if want == ops.DEV_BAD_CONTEXT:
            assert (out[10:30] == 9).all()
        assert_within(out[:10], ref[:10], bound[:10])
        assert_within(out[30:], ref[30:], bound[30:])
    out, err = go(qs=i32([0, 10, 30, 36]))  # past the last row
    assert err == ops.DEV_BAD_CONTEXT and (out[30:] == 9).all()
    bt = w.bt.copy()
    bt[1, 2] = w.NB
    out, err = go(bt=torch.as_tensor(bt, device="cuda"))
    assert err == ops.DEV_BAD_BLOCK
    assert_within(out[:10], ref[:10], bound[:10])
    assert_within(out[30:], ref[30:], bound[30:])


@pytest.mark.parametrize("bad", [-1, -2**31, 2**31 - 1])
@pytest.mark.parametrize("f8", [False, True])
def test_attention_bad_block_ids(ops, f8, bad):
    w = Tree([(50, 10), (60, 20), (70, 5)], 4, 2, 128, seed=16, f8=f8)
    ref, bound = w.attention64()
    w.bt[1, 1] = bad
    out, d = run_tree(ops, w)
    assert int(d["err"]) == ops.DEV_BAD_BLOCK
    assert_within(out[:10], ref[:10], bound[:10])
    assert_within(out[30:], ref[30:], bound[30:])


@pytest.mark.parametrize("q_size,k_scale", [(1e-20, 1e-30), (1e-38, 1e-8), (1.0, 1e-44)])
def test_e4m3_scores_that_vanish(ops, q_size, k_scale):
    """Scores below fp32's range weigh every visible token alike, and masked ones not at all."""
    w = Tree([(70, 40), (30, 30), (700, 9)], 8, 2, 128, seed=17, f8=True)
    w.q = (w.q.float() * q_size).to(torch.bfloat16)
    w.ks.fill_(k_scale)
    out, d = run_tree(ops, w)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    assert int(d["err"]) == 0


@pytest.mark.parametrize("f8", [False, True])
def test_two_calls_at_once(ops, f8):
    """Calls on two streams, each with its own workspace and inputs, interleaved."""
    ws = [Tree([(900, 30), (1500, 20)], 8, 2, 128, seed=18, f8=f8),
          Tree([(64, 64), (2000, 3), (17, 2)], 8, 4, 64, seed=19, f8=f8)]
    ds = [w.cuda() for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    outs = [torch.empty(w.T, w.Hq, w.D, dtype=torch.bfloat16, device="cuda") for w in ws]
    scratch = [ops.alloc_tree_workspace(w.Hq, w.Hkv, w.D, w.maxq) for w in ws]
    torch.cuda.synchronize()
    for _ in range(10):
        for w, d, st, o, sc in zip(ws, ds, streams, outs, scratch):
            run_tree(ops, w, d=d, ws=sc, out=o, stream=st)
    torch.cuda.synchronize()
    for w, d, o in zip(ws, ds, outs):
        ref, bound = w.attention64()
        assert_within(o, ref, bound)
        assert int(d["err"]) == 0


def test_cache_offsets_past_32_bits(ops):
    """Blocks at the far end of a cache of more than 2^31 elements."""
    w = Tree([(200, 20), (90, 7)], 8, 8, 128, seed=15, poison=False)
    NB = 2**31 // (8 * BS * 128) + 40
    if torch.cuda.mem_get_info()[0] < 3 * NB * 8 * BS * 128 * 2:
        pytest.skip("not enough free memory")
    d = w.cuda()
    far = torch.arange(w.NB, device="cuda") + NB - w.NB
    for n in ("k", "v"):
        big = torch.empty(NB, 8, BS, 128, dtype=torch.bfloat16, device="cuda")
        big[far] = d[n]
        d[n] = big
    d["bt"] = torch.where(d["bt"] >= 0, d["bt"] + NB - w.NB, d["bt"])
    out, _ = run_tree(ops, w, d=d)
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
    slots = d["slots"] + (NB - w.NB) * BS
    acc, al = i32([[19, 3], [0, 6]]), i32([2, 2])
    want = d["k"][slots[19] // BS, :, slots[19] % BS].clone()
    ops.paged_tree_commit(d["k"], d["v"], slots, d["qs"], acc, al)
    assert torch.equal(d["k"][slots[0] // BS, :, slots[0] % BS], want)
    rows = torch.randn(27, 16, 128, device="cuda").to(torch.bfloat16)
    ops.paged_qk_norm_rope_write(rows[:, :8].clone(), rows[:, :8], rows[:, 8:], rows[:, 8:], None,
                                 None, slots, d["k"], d["v"])
    assert torch.equal(d["v"][slots // BS, :, slots % BS], rows[:, 8:])


# ---- commit --------------------------------------------------------------------------
def commit64(k, v, f8, slots, qs, acc, lens, dst=None):
    """Host reference on [NB][Hkv][16][D] arrays (E4M3 V as [NB][Hkv][D][16])."""
    for s, n in enumerate(lens):
        src = [int(slots[qs[s] + acc[s][r]]) for r in range(n)]
        to = [int(dst[s][r]) if dst is not None else int(slots[qs[s] + r]) for r in range(n)]
        rows = [(k[a // BS, :, a % BS].clone(),
                 (v[a // BS, :, :, a % BS] if f8 else v[a // BS, :, a % BS]).clone()) for a in src]
        for (rk, rv), a, b in zip(rows, src, to):
            if a < 0 or b < 0:
                continue
            k[b // BS, :, b % BS] = rk
            if f8:
                v[b // BS, :, :, b % BS] = rv
            else:
                v[b // BS, :, b % BS] = rv


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("Hkv,D,lens,A,order", [
    (1, 64, [(20, 5)], 5, "sorted"), (3, 128, [(70, 40), (9, 9), (33, 1), (64, 30)], 9, "random"),
    (8, 128, [(300, 200), (50, 3)], 150, "random"), (2, 64, [(1100, 1024)], 1024, "reverse"),
])
def test_commit(ops, f8, Hkv, D, lens, A, order):
    w = Tree(lens, Hkv, Hkv, D, seed=A, f8=f8, poison=False, words=16)
    rng = np.random.default_rng(A)
    acc = np.full((w.S, A), -1, np.int32)
    al = np.zeros(w.S, np.int32)
    for s in range(w.S):
        n = min(A, int(w.L[s]))
        p = rng.permutation(int(w.L[s]))[:n]
        acc[s, :n] = {"sorted": np.sort(p), "random": p, "reverse": np.sort(p)[::-1]}[order]
        al[s] = n if s != 1 else n // 2
    for dst_on in (False, True):
        d = w.cuda()
        dst = None
        if dst_on:  # other slots: the spare blocks
            free = np.setdiff1d(np.arange(w.NB * BS), [b * BS + o for b in w.bt[w.bt >= 0]
                                                       for o in range(BS)])
            if free.size < al.sum():
                continue
            dst = np.full((w.S, A), -1, np.int64)
            at = 0
            for s in range(w.S):
                dst[s, :al[s]] = free[at:at + al[s]]
                at += int(al[s])
            dst[0, 0] = -1  # skipped
        k, v = w.k.clone(), w.v.clone().view(w.NB, Hkv, D, BS) if f8 else w.v.clone()
        commit64(k, v, f8, w.slots, w.qs, acc, al, dst)
        f = ops.paged_tree_commit_fp8 if f8 else ops.paged_tree_commit
        f(d["k"], d["v"], d["slots"], d["qs"], i32(acc), i32(al),
          dst_slots=None if dst is None else torch.as_tensor(dst, device="cuda"),
          err_flag=d["err"])
        assert int(d["err"]) == 0
        bits = lambda t: t.cpu().contiguous().view(torch.uint8 if f8 else torch.int16)
        assert torch.equal(bits(d["k"]), bits(k))
        assert torch.equal(bits(d["v"]), bits(v.view(w.v.shape)))


def test_commit_flags(ops):
    w = Tree([(40, 8), (30, 4)], 2, 2, 64, seed=3, poison=False)
    for acc, al, slot, want in (([[9, 1], [0, 1]], [2, 0], None, "DEV_BAD_ROW"),
                                ([[-1, 1], [0, 1]], [1, 0], None, "DEV_BAD_ROW"),
                                ([[2, 1], [0, 1]], [3, 0], None, "DEV_BAD_CONTEXT"),
                                ([[2, 1], [0, 1]], [-1, 0], None, "DEV_BAD_CONTEXT"),
                                ([[2, 1], [0, 1]], [1, 0], 2, "DEV_BAD_SLOT")):
        d = w.cuda()
        if slot is not None:
            d["slots"][slot] = w.NB * BS
        before = d["k"].clone()
        ops.paged_tree_commit(d["k"], d["v"], d["slots"], d["qs"], i32(acc), i32(al),
                              err_flag=d["err"])
        assert int(d["err"]) == getattr(ops, want)
        rest = torch.ones(w.NB * BS, dtype=torch.bool, device="cuda")
        rest[d["slots"][1]] = False  # the second row of the first case is moved
        same = (d["k"] == before).all(-1).all(1).flatten()
        assert same[rest].all()


# ---- together ------------------------------------------------------------------------
@pytest.mark.parametrize("f8", [False, True])
def test_whole_step_over_the_block_pool(ops, f8):
    """Three verification steps of a batch on the native block pool: each sequence is forked
    for its drafts, the drafts' K/V go to the fork's slots, the tree is scored, the accepted
    path moves to slots appended to the sequence, the fork is freed.  K and V kept by hand in
    64-bit order are what the cache holds at the end, and every tree's output is that of the
    definition over them."""
    from paged_kv_cache_272_gb300.block_pool import BlockPool
    rng = np.random.default_rng(21)
    g = torch.Generator().manual_seed(21)
    S, Hq, Hkv, D, NB = 4, 8, 2, 64, 80
    pool = BlockPool(NB)
    dt = torch.uint8 if f8 else torch.bfloat16
    kc = torch.zeros(NB, Hkv, BS, D, dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)
    ks = vs = torch.full((Hkv,), 1 / 64, device="cuda")
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    qw = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda()
    err = i32([0])

    def project(n):
        return torch.randn(n, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).cuda()

    def write(qkv, pos, slots):
        q, k, v = split(qkv, Hq, Hkv, D)
        qo = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        a = (qo, q, k, v, pos, freq, slots, kc, vc)
        kw = dict(q_weight=qw, k_weight=qw, err_flag=err)
        if f8:
            ops.paged_qk_norm_rope_write_fp8(*a, ks, vs, **kw)
        else:
            ops.paged_qk_norm_rope_write(*a, **kw)
        return qo

    def copy(pairs):
        if len(pairs):
            f = ops.paged_block_copy_fp8 if f8 else ops.paged_block_copy
            f(kc, vc, i32(pairs))

    def row(slot):
        b, o = slot // BS, slot % BS
        return kc[b, :, o].cpu(), (vc.view(NB, Hkv, D, BS)[b, :, :, o] if f8 else vc[b, :, o]).cpu()

    held = [[] for _ in range(S)]  # (k row, v row) bytes per token
    for s in range(S):
        pool.add_seq(s)
        n = int(rng.integers(1, 60))
        slots, _ = pool.append_tokens(s, n)
        write(project(n), torch.arange(n, dtype=torch.int32, device="cuda"),
              torch.as_tensor(slots, device="cuda"))
        held[s] = [row(int(x)) for x in slots]
    for step in range(3):
        sizes = [int(rng.integers(1, 12)) for _ in range(S)]
        qs = np.concatenate([[0], np.cumsum(sizes)])
        parents = np.concatenate([TH.random_parents(rng, n) for n in sizes])
        slots, pairs = [], []
        for s in range(S):
            pool.fork(s, 100 + s)
            sl, pr = pool.append_tokens(100 + s, sizes[s])
            slots += list(sl)
            pairs += [p for p in pr.tolist()]
        copy(pairs)
        bt, ctx = pool.export([100 + s for s in range(S)], 8)
        masks = torch.empty(qs[-1], 1, dtype=torch.int64, device="cuda")
        pos = torch.empty(qs[-1], dtype=torch.int32, device="cuda")
        ops.paged_tree_masks(masks, pos, i32(parents), i32(qs), i32(ctx), err_flag=err)
        dslots = torch.as_tensor(np.array(slots, np.int64), device="cuda")
        q = write(project(int(qs[-1])), pos, dslots)
        out = torch.empty_like(q)
        ws = ops.alloc_tree_workspace(Hq, Hkv, D, max(sizes))
        a = (out, q, kc, vc, torch.as_tensor(bt, device="cuda"), i32(ctx), i32(qs), masks, D ** -0.5)
        if f8:
            ops.paged_attention_tree_fp8(*a, ks, vs, max(sizes), ws, err_flag=err)
        else:
            ops.paged_attention_tree(*a, max(sizes), ws, err_flag=err)
        # the definition, over the rows kept by hand
        val = lambda r: (r.view(torch.float8_e4m3fn).double() / 64 if f8 else r.double())
        path = []
        for s in range(S):
            drafts = [row(int(slots[i])) for i in range(qs[s], qs[s + 1])]
            see = TH.ancestors(parents[qs[s]:qs[s + 1]].tolist())
            for i in range(sizes[s]):
                rows = held[s] + [drafts[j] for j in np.flatnonzero(see[i])]
                k = torch.stack([val(r[0]) for r in rows])
                v = torch.stack([val(r[1]) for r in rows])
                qq = q[qs[s] + i].cpu().double().view(Hkv, Hq // Hkv, D)
                p = torch.softmax(torch.einsum("hgd,chd->hgc", qq, k) * D ** -0.5, -1)
                ref = torch.einsum("hgc,chd->hgd", p, v).reshape(Hq, D)
                mag = torch.einsum("hgc,chd->hgd", p, v.abs()).reshape(Hq, D)
                assert_within(out[qs[s] + i], ref, TH.BF16_HALF * ref.abs() + 2.0 ** -7.5 * mag)
            leaf = int(rng.integers(sizes[s]))
            path.append([int(j) for j in np.flatnonzero(see[leaf])])
            held[s] += [drafts[j] for j in path[s]]
        A = max(len(p) for p in path)
        acc, dst = np.zeros((S, A), np.int32), np.full((S, A), -1, np.int64)
        pairs = []
        for s in range(S):
            acc[s, :len(path[s])] = path[s]
            sl, pr = pool.append_tokens(s, len(path[s]))
            dst[s, :len(path[s])] = sl
            pairs += pr.tolist()
        copy(pairs)
        f = ops.paged_tree_commit_fp8 if f8 else ops.paged_tree_commit
        f(kc, vc, dslots, i32(qs), i32(acc), i32([len(p) for p in path]),
          dst_slots=torch.as_tensor(dst, device="cuda"), err_flag=err)
        for s in range(S):
            pool.free_seq(100 + s)
            table = pool.block_table(s)
            for t, (rk, rv) in enumerate(held[s]):
                gk, gv = row(table[t // BS] * BS + t % BS)
                assert torch.equal(gk.view(torch.uint8), rk.view(torch.uint8)), (step, s, t)
                assert torch.equal(gv.view(torch.uint8), rv.view(torch.uint8)), (step, s, t)
    assert int(err) == 0


@pytest.mark.parametrize("f8", [False, True])
def test_captured_step_replays_on_new_inputs(ops, f8):
    """masks -> attention -> commit captured once and replayed on new lengths, tables, masks
    and queries; the eager calls on another stream give the same bits."""
    lens = [[(300, 20), (40, 9), (900, 30)], [(33, 1), (700, 30), (520, 2)]]
    ws_ = [Tree(l, 8, 2, 128, seed=30 + i, f8=f8, poison=False, spare_blocks=60)
           for i, l in enumerate(lens)]
    NB, T, MB = max(w.NB for w in ws_), max(w.T for w in ws_), max(w.MB for w in ws_)
    W, maxq = 1, 30
    dt = torch.uint8 if f8 else torch.bfloat16
    z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")
    b = dict(k=z(NB, 2, BS, 128, t=dt), v=z(NB, 2, BS, 128, t=dt), q=z(T, 8, 128, t=torch.bfloat16),
             out=z(T, 8, 128, t=torch.bfloat16), masks=z(T, W, t=torch.int64), par=z(T), qs=z(4),
             ctx=z(3), bt=z(3, MB), slots=z(T, t=torch.int64), acc=z(3, 2), al=z(3), err=z(1),
             ks=z(2, t=torch.float32), vs=z(2, t=torch.float32))
    scratch = ops.alloc_tree_workspace(8, 2, 128, maxq)

    def fill(w):
        d = w.cuda()
        n = w.T
        b["k"][:w.NB], b["v"][:w.NB] = d["k"], d["v"]
        b["q"][:n], b["par"][:n], b["slots"][:n] = d["q"], d["parents"], d["slots"]
        b["qs"].copy_(d["qs"]), b["ctx"].copy_(d["ctx"]), b["bt"].fill_(-1)
        b["bt"][:, :w.MB] = d["bt"]
        b["ks"].copy_(d["ks"]), b["vs"].copy_(d["vs"])
        b["acc"].copy_(torch.tensor([[min(2, int(x) - 1), 0] for x in w.L], device="cuda"))
        b["al"].copy_(torch.tensor([min(2, int(x)) for x in w.L], device="cuda"))

    def step():
        ops.paged_tree_masks(b["masks"], None, b["par"], b["qs"], b["ctx"], err_flag=b["err"])
        a = (b["out"], b["q"], b["k"], b["v"], b["bt"], b["ctx"], b["qs"], b["masks"], 128 ** -0.5)
        if f8:
            ops.paged_attention_tree_fp8(*a, b["ks"], b["vs"], maxq, scratch, err_flag=b["err"])
            ops.paged_tree_commit_fp8(b["k"], b["v"], b["slots"], b["qs"], b["acc"], b["al"],
                                      err_flag=b["err"])
        else:
            ops.paged_attention_tree(*a, maxq, scratch, err_flag=b["err"])
            ops.paged_tree_commit(b["k"], b["v"], b["slots"], b["qs"], b["acc"], b["al"],
                                  err_flag=b["err"])
    fill(ws_[0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 0, 1):
        w = ws_[i]
        fill(w)
        graph.replay()
        torch.cuda.synchronize()
        got = {n: b[n].clone() for n in ("out", "k", "v", "masks")}
        ref, bound = w.attention64()
        assert_within(got["out"][:w.T], ref, bound)
        side = torch.cuda.Stream()
        fill(w)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        for n in ("masks", "k", "v"):
            assert torch.equal(got[n], b[n]), n
        assert torch.equal(got["out"][:w.T], b["out"][:w.T])
    assert int(b["err"]) == 0


def test_misplaced_arguments(ops):
    """A workspace too small, tensors of other types, a stream object of this device."""
    w = Tree([(40, 4)], 4, 2, 64, seed=40)
    d = w.cuda()
    with pytest.raises(ops.PagedKVError):
        run_tree(ops, w, d=d, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        run_tree(ops, w, d=dict(d, masks=d["masks"].to(torch.int32)))
    with pytest.raises(ValueError):
        run_tree(ops, w, d=dict(d, masks=d["masks"][:3]))
    with pytest.raises(TypeError):
        run_tree(ops, w, d=dict(d, q=d["q"].float()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = run_tree(ops, w, d=d, stream=side)
    side.synchronize()
    ref, bound = w.attention64()
    assert_within(out, ref, bound)
