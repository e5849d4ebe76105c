"""Refusals of the drafted-tree entry points, on the host and before anything is queued, and
the plain forms their GPU tests compare with."""
import ctypes

import numpy as np
import pytest
import torch

import tree_helpers as TH

fake = 1 << 20  # never dereferenced: every call fails validation, or has nothing to do
F = ctypes.c_float


def lib():
    from paged_kv_cache_272_gb300.ops import lib as l
    return l


def test_masks_refusals():
    f = lib().paged_tree_masks
    a = lambda **k: [k.get("m", fake), k.get("pos", fake), k.get("par", fake), k.get("qs", fake),
                     k.get("ctx", fake), None, k.get("S", 2), k.get("T", 9), k.get("W", 1), None,
                     None]
    assert f(*a(W=0)) == -2 and f(*a(W=17)) == -2 and f(*a(S=-1)) == -2 and f(*a(T=-1)) == -2
    for n in ("m", "par", "qs", "ctx"):
        assert f(*a(**{n: None})) == -1
    assert f(*a(S=0, m=None)) == 0 and f(*a(T=0, m=None)) == 0


def rope_args(fp8=False, **k):
    D, Hq, Hkv = k.get("D", 128), k.get("Hq", 8), k.get("Hkv", 2)
    ax = (ctypes.c_uint8 * 64)(*k.get("axes_of", []))
    a = [k.get("qo", fake), k.get("qos", Hq * D), k.get("q", fake), k.get("qst", Hq * D),
         k.get("k", fake), k.get("kst", Hkv * D), k.get("v", fake), k.get("vst", Hkv * D),
         k.get("qw", None), None, F(k.get("eps", 1e-6)), k.get("pos", fake), 0,
         k.get("axes", 1), ax if "axes_of" in k else None, k.get("freq", fake),
         k.get("rot", D), 0, F(1.0), k.get("slots", fake), k.get("T", 4), k.get("kc", fake),
         fake, 8, Hq, Hkv, D, k.get("bs", 16)]
    if fp8:
        a += [F(k.get("ks", 1.0)), F(k.get("vs", 1.0)), k.get("kss", None), k.get("vss", None)]
    return a + [None, None]


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_refusals(fp8):
    f = lib().paged_qk_norm_rope_write_fp8 if fp8 else lib().paged_qk_norm_rope_write
    c = lambda **k: f(*rope_args(fp8, **k))
    assert c(bs=8) == -3
    for k in (dict(D=96), dict(Hq=6, Hkv=4), dict(rot=24), dict(rot=144), dict(rot=-16),
              dict(axes=0), dict(axes=5, axes_of=[0]), dict(T=-1), dict(eps=-1.0),
              dict(eps=float("nan")), dict(qst=8 * 128 - 8), dict(kst=2 * 128 - 8),
              dict(vst=0), dict(qos=0)):
        assert c(**k) == -2, k
    for n in ("qo", "q", "k", "v", "pos", "freq", "slots", "kc"):
        assert c(**{n: None}) == -1, n
    assert c(axes=2) == -1                              # several axes, no map
    assert c(axes=2, axes_of=[0] * 63 + [2]) == -14     # an axis that is not there
    for k in (dict(q=fake + 2), dict(qo=fake + 8), dict(kc=fake + 4), dict(qw=fake + 8),
              dict(qst=8 * 128 + 4), dict(kst=2 * 128 + 1)):
        assert c(**k) == -4, k
    assert c(T=0, q=None) == 0
    if fp8:
        assert c(ks=0.0) == -2 and c(vs=float("nan")) == -2
        assert c(kss=fake) == -1 and c(vss=fake) == -1


def tree_args(fp8=False, **k):
    a = [k.get("out", fake), k.get("q", fake), fake, k.get("vc", fake), k.get("bt", fake),
         k.get("ctx", fake), k.get("qs", fake), k.get("masks", fake), k.get("W", 1),
         k.get("S", 2), k.get("T", 9), k.get("MB", 4), k.get("Hq", 8), k.get("Hkv", 2),
         k.get("D", 128), k.get("bs", 16), k.get("NB", 64), F(k.get("scale", 0.1))]
    if fp8:
        a += [F(k.get("ks", 1.0)), F(1.0), k.get("kss", None), k.get("vss", None)]
    return a + [k.get("maxq", 8), k.get("ws", fake), k.get("wsb", 1 << 40), None, None]


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_refusals(fp8):
    f = lib().paged_attention_tree_fp8 if fp8 else lib().paged_attention_tree
    c = lambda **k: f(*tree_args(fp8, **k))
    assert c(bs=32) == -3
    for k in (dict(D=80), dict(Hq=6, Hkv=4), dict(W=0), dict(W=17), dict(maxq=65), dict(maxq=-1),
              dict(scale=0.0), dict(scale=float("nan")), dict(S=-1), dict(S=65536), dict(T=-1),
              dict(MB=0), dict(NB=0), dict(NB=1 << 27, Hkv=1)):
        assert c(**k) == -2, k
    for n in ("out", "q", "vc", "bt", "ctx", "qs", "masks", "ws"):
        assert c(**{n: None}) == -1, n
    assert c(q=fake + 8) == -4 and c(ws=fake + 128) == -4
    need = lib().paged_attention_tree_workspace_size(8, 2, 128, 8)
    assert need > 0 and c(wsb=need - 1) == -5
    for k in (dict(S=0), dict(T=0), dict(maxq=0)):
        assert c(out=None, **k) == 0
    if fp8:
        assert c(ks=0.0) == -2 and c(kss=fake) == -1 and c(vss=fake) == -1
    assert lib().paged_attention_tree_workspace_size(7, 2, 128, 8) == 0
    assert lib().paged_attention_tree_workspace_size(8, 2, 128, -1) == 0


def test_workspace_of_sizes_out_of_range():
    """No size for what the call itself refuses."""
    f = lib().paged_attention_tree_workspace_size
    for k in ((8, 2, 96, 8), (8, 2, 128, 1025), (0, 1, 64, 8), (8, 0, 64, 8)):
        assert f(*k) == 0, k


@pytest.mark.parametrize("fp8", [False, True])
def test_commit_refusals(fp8):
    f = lib().paged_tree_commit_fp8 if fp8 else lib().paged_tree_commit
    a = lambda **k: [k.get("kc", fake), fake, k.get("sl", fake), k.get("qs", fake),
                     k.get("acc", fake), k.get("al", fake), None, k.get("S", 2), k.get("T", 9),
                     k.get("A", 4), k.get("NB", 8), k.get("H", 2), k.get("D", 128),
                     k.get("bs", 16), None, None]
    assert f(*a(bs=8)) == -3
    for k in (dict(D=80), dict(A=-1), dict(A=1025), dict(S=-1), dict(T=-1), dict(NB=0),
              dict(H=0)):
        assert f(*a(**k)) == -2, k
    for n in ("kc", "sl", "qs", "acc", "al"):
        assert f(*a(**{n: None})) == -1, n
    assert f(*a(kc=fake + 8)) == -4
    for k in (dict(S=0), dict(T=0), dict(A=0)):
        assert f(*a(kc=None, **k)) == 0


def test_binding_refuses_cpu_tensors():
    from paged_kv_cache_272_gb300 import ops
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(TypeError):
        ops.paged_tree_masks(torch.zeros(4, 1, dtype=torch.int64), None, i(4), i(2), i(1))
    kv = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ops.paged_tree_commit(kv, kv, torch.zeros(4, dtype=torch.int64), i(2), i(1, 2), i(1))


def test_plain_forms_agree():
    """The two plain forms of the masks, and attention of a chain against causal softmax."""
    w = TH.Tree([(37, 9), (64, 64), (5, 5)], 4, 2, 64, seed=3, kind="chain")
    for r in range(9):
        assert list(np.flatnonzero(w.visible[r])) == list(range(r + 1))
    assert w.masks[9 + 63, 0] == -1 and w.masks[9 + 5, 0] == 0b111111
    out, bound = w.attention64()
    k, v = w.kv64(1)
    i = 20
    x = torch.einsum("gd,cd->gc", w.q[9 + i, :2].double(), k[:i + 1, 0]) * w.scale
    assert torch.allclose(out[9 + i, :2], torch.softmax(x, -1) @ v[:i + 1, 0])
    assert (bound >= 0).all()
