"""Timed cases of the tree-verification operators: a serving step that checks a tree of
drafted tokens against the paged cache.

Four operators, in the order a step runs them:

  masks    parents of the drafted tokens -> ancestor bit masks and positions
  rope     head-wise RMS norm of q and k, rotary positions on one or several axes, and the
           write of k and v into the paged cache (bf16, or E4M3 with a scale per KV head)
  tree     attention of every drafted token over its sequence's cached prefix and its own
           ancestors in the tree (bf16 or E4M3 cache)
  commit   the K/V rows of the accepted path moved to the sequence's next slots

``own`` false computes them with elementary torch operations in 32 bits, ``own`` true calls
the library.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 16
DEV = "cuda"


# -------------------------------------------------------------------------------------
# Cases
# -------------------------------------------------------------------------------------
def listed():
    return [
        # One user, a short answer so far, a small tree: the latency of a single call.
        dict(name="tree-one-short", op="tree", S=1, ctx=700, L=8, ragged=False, Hq=32, Hkv=8,
             D=128, kv="bf16"),
        # A chat batch in mid-answer: ragged contexts and ragged trees.
        dict(name="tree-chat-batch", op="tree", S=32, ctx=4096, L=16, ragged=True, Hq=64,
             Hkv=8, D=128, kv="bf16"),
        # Long documents with a wide tree: the most cache bytes and the most products.
        dict(name="tree-long", op="tree", S=8, ctx=65536, L=48, ragged=False, Hq=64, Hkv=8,
             D=128, kv="bf16"),
        # No shared heads, head_dim 64, odd lengths, a tree of more than one mask word.
        dict(name="tree-mha-d64", op="tree", S=5, ctx=2501, L=77, ragged=True, Hq=32, Hkv=32,
             D=64, kv="bf16"),
        # A large batch over a quantised cache.
        dict(name="tree-e4m3-batch", op="tree", S=64, ctx=8192, L=13, ragged=True, Hq=64,
             Hkv=8, D=128, kv="e4m3"),
        # One drafted chain of a single user, plain one-axis positions.
        dict(name="rope-one-chain", op="rope", T=4, Hq=32, Hkv=8, D=128, rot=128, axes=1,
             order="blocked", inter=False, norm=True, kv="bf16", far=4096),
        # The trees of a batch over a quantised cache, three axes (time, height, width).
        dict(name="rope-e4m3-axes", op="rope", T=1021, Hq=64, Hkv=8, D=128, rot=128, axes=3,
             order="cyclic", inter=False, norm=True, kv="e4m3", far=32768),
        # A prompt chunk far into a long document; half of head_dim rotates, pairs adjacent.
        dict(name="rope-prompt-d64", op="rope", T=16384, Hq=32, Hkv=8, D=64, rot=32, axes=1,
             order="blocked", inter=True, norm=False, kv="bf16", far=1000000),
        # One small tree.
        dict(name="masks-one", op="masks", S=1, L=8, ragged=False),
        # A large batch of wide, ragged trees.
        dict(name="masks-batch", op="masks", S=256, L=200, ragged=True),
        # A batch that accepts a few tokens each, in place.
        dict(name="commit-batch", op="commit", S=64, L=32, accept=6, Hkv=8, D=128, kv="bf16"),
        # The same over a quantised cache with more heads and longer paths.
        dict(name="commit-e4m3", op="commit", S=200, L=64, accept=17, Hkv=16, D=64, kv="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "rope", "masks", "commit"])
    kv = rng.choice(["bf16", "e4m3"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "tree":
        S, ctx, L = _log(rng, 1, 64), _log(rng, 20, 65536), _log(rng, 1, 130)
        G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12])
        G = min(G, max(1, 96 // Hkv))
        # no more work than the largest listed case: cached tokens, and products
        S = max(1, min(S, 500000 // ctx, 100000000 // (ctx * L)))
        while S * ctx * Hkv * D * L * G > 8 * 65536 * 48 * 64 * 128 or \
                S * ctx * Hkv > 8 * 65536 * 8:
            if S > 1:
                S = S // 2
            else:
                ctx = ctx // 2
        return dict(op=op, S=S, ctx=max(ctx, L + 1), L=L, ragged=rng.random() < 0.6, Hq=Hkv * G,
                    Hkv=Hkv, D=D, kv=kv)
    if op == "rope":
        G = rng.choice([1, 2, 3, 4, 7, 8])
        T = _log(rng, 1, max(2, 16384 * 48 * 64 // ((G + 2) * Hkv * D)))
        return dict(op=op, T=T, Hq=Hkv * G, Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, 32]), axes=rng.choice([1, 1, 3, 4]),
                    order=rng.choice(["blocked", "cyclic"]), inter=rng.random() < 0.4,
                    norm=rng.random() < 0.6, kv=kv, far=_log(rng, 100, 1000000))
    if op == "masks":
        return dict(op=op, S=_log(rng, 1, 256), L=_log(rng, 1, 200), ragged=rng.random() < 0.6)
    L = _log(rng, 2, 130)
    return dict(op=op, S=_log(rng, 1, 200), L=L, accept=rng.randint(1, min(L, 17)), Hkv=Hkv, D=D,
                kv=kv)


def _lens(case):
    """Context lengths (drafted tokens included) and tree sizes of a case's sequences."""
    S, L = case["S"], case["L"]
    ctx = case.get("ctx", 4 * L + 100)
    r = random.Random("%d-%d-%d" % (S, ctx, L))
    if not case.get("ragged"):
        return [ctx] * S, [L] * S
    ls = [r.randint(max(1, L // 3), L) for _ in range(S)]
    ls[0] = L
    cs = [max(n, r.randint(ctx // 4, ctx)) for n in ls]
    cs[0] = max(ctx, L)
    return cs, ls


# -------------------------------------------------------------------------------------
# Inputs
# -------------------------------------------------------------------------------------
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _starts(ls):
    s = [0]
    for n in ls:
        s.append(s[-1] + n)
    return s


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _codes(g, *shape):
    """E4M3 codes of normal values over a scale of 1/32."""
    x = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
    return (x * 32).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _tables(g, cs):
    """Block tables (a random permutation of the pool) and the number of blocks."""
    nb = [-(-c // BLOCK) for c in cs]
    total, mb = sum(nb), max(nb)
    perm = torch.randperm(total + 7, generator=g, device=DEV)
    first = _ints(_starts(nb)[:-1], torch.int64)[:, None]
    col = torch.arange(mb, device=DEV)[None, :]
    inside = col < _ints(nb, torch.int64)[:, None]
    bt = torch.where(inside, perm[(first + col).clamp(max=total - 1)], torch.full_like(col, -1))
    return bt.to(torch.int32).contiguous(), total + 7


def _parents(g, ls):
    """A random tree per sequence: token i hangs under one of the tokens before it, or
    under the cached context (-1)."""
    T = sum(ls)
    i = torch.cat([torch.arange(n, device=DEV) for n in ls])
    u = torch.rand(T, generator=g, device=DEV)
    return (torch.floor(u * (i + 1)).to(torch.int64).clamp(max=i) - 1).to(torch.int32)


def _closure(parents, qs, L, dtype):
    """[S][L][L] 0/1: token j is token i itself or one of its ancestors.  With A the
    parent relation, sum of A^k = (I - A)^-1, a unit lower triangular solve (whole
    numbers throughout)."""
    S = qs.numel() - 1
    i = torch.arange(L, device=DEV)
    start = qs[:-1].to(torch.int64)[:, None]
    n = (qs[1:] - qs[:-1]).to(torch.int64)[:, None]
    par = parents.to(torch.int64)[(start + i).clamp(max=parents.numel() - 1)]
    par = torch.where(i[None, :] < n, par, torch.full_like(par, -1))
    A = (par[:, :, None] == i[None, None, :]).to(dtype)
    eye = torch.eye(L, device=DEV, dtype=dtype).expand(S, L, L)
    R = torch.linalg.solve_triangular(eye - A, eye, upper=False, unitriangular=True)
    return torch.where(R > 0.5, torch.ones_like(R), torch.zeros_like(R))


def _pack(R, qs, words):
    """Rows of 0/1 -> int64 words per drafted token, bit j of word w = token 64 w + j."""
    S, L, _ = R.shape
    bits = torch.zeros(S, L, words * 64, dtype=torch.int64, device=DEV)
    bits[:, :, :L] = R.to(torch.int64)
    bits = bits.view(S, L, words, 64) << torch.arange(64, device=DEV)
    n = (qs[1:] - qs[:-1]).to(torch.int64)[:, None]
    rows = torch.arange(L, device=DEV)[None, :] < n
    return bits.sum(-1)[rows].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    s["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    op = case["op"]
    if op == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        qkv = _randn(g, T, (Hq + 2 * Hkv) * D)  # the fused projection's rows
        s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["qw"] = (1 + 0.1 * _randn(g, D).float()).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1 + 0.1 * _randn(g, D).float()).to(torch.bfloat16) if case["norm"] else None
        half = case["rot"] // 2
        s["freq"] = 500000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        base = torch.randint(0, case["far"], (case["axes"], 1), generator=g, device=DEV)
        step = torch.randint(0, 64, (case["axes"], T), generator=g, device=DEV)
        pos = base + torch.arange(T, device=DEV) + (step if case["axes"] > 1 else 0)
        s["pos"] = pos.to(torch.int32).contiguous()
        pair = torch.arange(half)
        ax = pair * case["axes"] // half if case["order"] == "blocked" else pair % case["axes"]
        s["pair_axes"] = bytes(ax.tolist())
        s["axis_of"] = ax.to(DEV)
        nblocks = -(-T // BLOCK) + 3
        # consecutive slots of shuffled blocks, as a prompt's chunk has them
        blocks = torch.randperm(nblocks, generator=g, device=DEV)
        t = torch.arange(T, device=DEV)
        s["slots"] = blocks[t // BLOCK] * BLOCK + t % BLOCK
        _caches(s, g, nblocks)
        return s
    cs, ls = _lens(case)
    qs = _starts(ls)
    s["qs"], s["ctx_lens"] = _ints(qs), _ints(cs)
    s["maxq"] = max(ls)
    s["words"] = -(-max(ls) // 64)
    s["parents"] = _parents(g, ls)
    if op == "masks":
        T = qs[-1]
        s["masks"] = torch.zeros(T, s["words"], dtype=torch.int64, device=DEV)
        s["pos"] = torch.zeros(T, dtype=torch.int32, device=DEV)
        return s
    s["bt"], nblocks = _tables(g, cs)
    _caches(s, g, nblocks)
    if op == "tree":
        T, Hq, D = qs[-1], case["Hq"], case["D"]
        R = _closure(s["parents"], s["qs"], s["maxq"], torch.float32)
        s["masks"] = _pack(R, s["qs"], s["words"])
        s["q"] = _randn(g, T, Hq, D)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = D ** -0.5
        return s
    # commit: the tree's slots and a path of increasing tree indices per sequence
    S, A, L = case["S"], case["accept"], case["L"]
    s["acc_lens"] = torch.randint(1, A + 1, (S,), generator=g, device=DEV).to(torch.int32)
    pick = torch.rand(S, L, generator=g, device=DEV).argsort(1)[:, :A].sort(1).values
    s["acc"] = pick.to(torch.int32).contiguous()
    start = _ints(cs, torch.int64)[:, None] - _ints(ls, torch.int64)[:, None]
    p = start + torch.arange(L, device=DEV)
    s["slots"] = (s["bt"].to(torch.int64).gather(1, p // BLOCK) * BLOCK + p % BLOCK).flatten()
    return s


def _caches(s, g, nblocks):
    Hkv, D = s["Hkv"], s["D"]
    if s["kv"] == "bf16":
        s["kc"], s["vc"] = _randn(g, nblocks, Hkv, BLOCK, D), _randn(g, nblocks, Hkv, BLOCK, D)
        return
    s["kc"] = _codes(g, nblocks, Hkv, BLOCK, D)
    s["vc"] = _codes(g, nblocks, Hkv, D, BLOCK).view(nblocks, Hkv, BLOCK, D)  # [D][16] blocks
    s["ks"] = (torch.rand(Hkv, generator=g, device=DEV) + 0.5) / 32
    s["vs"] = (torch.rand(Hkv, generator=g, device=DEV) + 0.5) / 32


# -------------------------------------------------------------------------------------
# One pass
# -------------------------------------------------------------------------------------
def run(s):
    if own:
        return _RUN_OWN[s["op"]](s)
    return _RUN_PLAIN[s["op"]](s)


def _state(s, *first):
    """Outputs with the caches (E4M3 codes as the values they stand for, over the scale)."""
    if s["kv"] == "bf16":
        return (*first, s["kc"], s["vc"])
    return (*first, s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn))


def _own_masks(s):
    from paged_kv_cache_272_gb300 import ops
    ops.paged_tree_masks(s["masks"], s["pos"], s["parents"], s["qs"], s["ctx_lens"],
                         err_flag=s["err"])
    return s["masks"], s["pos"]


def _own_rope(s):
    from paged_kv_cache_272_gb300 import ops
    if s["kv"] == "bf16":
        ops.paged_qk_norm_rope_write(
            s["q_out"], s["q"], s["k"], s["v"], s["pos"], s["freq"], s["slots"], s["kc"], s["vc"],
            q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, pair_axes=s["pair_axes"],
            interleaved=s["inter"], err_flag=s["err"])
    else:
        ops.paged_qk_norm_rope_write_fp8(
            s["q_out"], s["q"], s["k"], s["v"], s["pos"], s["freq"], s["slots"], s["kc"], s["vc"],
            s["ks"], s["vs"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
            pair_axes=s["pair_axes"], interleaved=s["inter"], err_flag=s["err"])
    return _state(s, s["q_out"])


def _own_tree(s):
    from paged_kv_cache_272_gb300 import ops
    if "ws" not in s:  # the program's scratch, allocated once
        s["ws"] = ops.alloc_tree_workspace(s["Hq"], s["Hkv"], s["D"], s["maxq"])
    if s["kv"] == "bf16":
        ops.paged_attention_tree(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["ctx_lens"],
                                 s["qs"], s["masks"], s["scale"], s["maxq"], s["ws"],
                                 err_flag=s["err"])
    else:
        ops.paged_attention_tree_fp8(s["out"], s["q"], s["kc"], s["vc"], s["bt"], s["ctx_lens"],
                                     s["qs"], s["masks"], s["scale"], s["ks"], s["vs"],
                                     s["maxq"], s["ws"], err_flag=s["err"])
    return s["out"]


def _own_commit(s):
    from paged_kv_cache_272_gb300 import ops
    f = ops.paged_tree_commit if s["kv"] == "bf16" else ops.paged_tree_commit_fp8
    f(s["kc"], s["vc"], s["slots"], s["qs"], s["acc"], s["acc_lens"], err_flag=s["err"])
    return _state(s)


_RUN_OWN = {"masks": _own_masks, "rope": _own_rope, "tree": _own_tree, "commit": _own_commit}


# ---- plain forms ---------------------------------------------------------------------
def _plain_masks(s):
    qs = s["qs"]
    R = _closure(s["parents"], qs, s["maxq"], torch.float32)
    n = (qs[1:] - qs[:-1]).to(torch.int64)[:, None]
    rows = torch.arange(s["maxq"], device=DEV)[None, :] < n
    depth = R.sum(-1).to(torch.int64) - 1
    pos = (s["ctx_lens"].to(torch.int64)[:, None] - n + depth)[rows]
    return _pack(R, qs, s["words"]), pos.to(torch.int32)


def _norm(x, w, eps):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()


def _rotate(x, cos, sin, rot, inter):
    """x [T][H][D] float; cos, sin [T][rot / 2]."""
    cos, sin = cos[:, None, :], sin[:, None, :]
    a = x[..., 0:rot:2] if inter else x[..., :rot // 2]
    b = x[..., 1:rot:2] if inter else x[..., rot // 2:rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((ra, rb), -1).flatten(-2) if inter else torch.cat((ra, rb), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_rope(s):
    pos = s["pos"].to(torch.float64)[s["axis_of"]].t()  # [T][rot / 2]
    angle = pos * s["freq"]  # 64 bits: far positions
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _rotate(_norm(s["q"], s["qw"], 1e-6), cos, sin, s["rot"], s["inter"])
    k = _rotate(_norm(s["k"], s["kw"], 1e-6), cos, sin, s["rot"], s["inter"])
    s["q_out"].copy_(q)
    blk, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    if s["kv"] == "bf16":
        s["kc"][blk, :, off] = k.to(torch.bfloat16)
        s["vc"][blk, :, off] = s["v"]
        return _state(s, s["q_out"])
    kq = (k / s["ks"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    vq = (s["v"].float() / s["vs"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    s["kc"][blk, :, off] = kq
    vc = s["vc"].view(-1, s["Hkv"], s["D"], BLOCK)
    vc[blk, :, :, off] = vq.view(torch.uint8)
    return _state(s, s["q_out"])


def _plain_tree(s):
    S, MB = s["bt"].shape
    Hq, Hkv, D, L = s["Hq"], s["Hkv"], s["D"], s["maxq"]
    G, N = Hq // Hkv, MB * BLOCK
    qs, ctx = s["qs"].to(torch.int64), s["ctx_lens"].to(torch.int64)
    n = qs[1:] - qs[:-1]
    i, t = torch.arange(L, device=DEV), torch.arange(N, device=DEV)
    live = i[None, :] < n[:, None]
    row = (qs[:-1, None] + i).clamp(max=int(s["q"].shape[0]) - 1)
    q = s["q"][row].float().view(S, L, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, L * G, D)
    bt = s["bt"].to(torch.int64).clamp(min=0)
    if s["kv"] == "bf16":
        k = s["kc"][bt].permute(0, 2, 1, 3, 4).reshape(S, Hkv, N, D).float()
        v = s["vc"][bt].permute(0, 2, 1, 3, 4).reshape(S, Hkv, N, D).float()
    else:
        k = s["kc"].view(torch.float8_e4m3fn)[bt].float() * s["ks"][:, None, None]
        k = k.permute(0, 2, 1, 3, 4).reshape(S, Hkv, N, D)
        v = s["vc"].view(-1, Hkv, D, BLOCK).view(torch.float8_e4m3fn)[bt].float()
        v = (v * s["vs"][:, None, None]).permute(0, 2, 1, 4, 3).reshape(S, Hkv, N, D)
    j = t[None, :] - (ctx - n)[:, None]  # index in the tree; negative: the cached prefix
    jc = j.clamp(0, L - 1)
    words = s["masks"][row].gather(2, (jc // 64)[:, None, :].expand(S, L, N))
    bit = (words >> (jc % 64)[:, None, :]) & 1
    seen = (j < 0)[:, None, :] | ((bit == 1) & (j < n[:, None])[:, None, :])
    seen = (seen & live[:, :, None])[:, None, :, None, :]  # [S][1][L][1][N]
    x = (q @ k.transpose(2, 3) * s["scale"]).view(S, Hkv, L, G, N)
    x = torch.where(seen, x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
    o = p.view(S, Hkv, L * G, N) @ v
    l = p.sum(-1).view(S, Hkv, L * G, 1)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).view(S, Hkv, L, G, D)
    return o.permute(0, 2, 1, 3, 4).reshape(S, L, Hq, D)[live].to(torch.bfloat16)


def _plain_commit(s):
    S, A = s["acc"].shape
    used = torch.arange(A, device=DEV)[None, :] < s["acc_lens"][:, None]
    first = s["qs"][:-1].to(torch.int64)[:, None]
    src = s["slots"][first + s["acc"].to(torch.int64)][used]
    dst = s["slots"][first + torch.arange(A, device=DEV)][used]
    sb, so, db, do = src // BLOCK, src % BLOCK, dst // BLOCK, dst % BLOCK
    s["kc"][db, :, do] = s["kc"][sb, :, so]
    v = s["vc"] if s["kv"] == "bf16" else s["vc"].view(-1, s["Hkv"], s["D"], BLOCK).transpose(2, 3)
    v[db, :, do] = v[sb, :, so]
    return _state(s)


_RUN_PLAIN = {"masks": _plain_masks, "rope": _plain_rope, "tree": _plain_tree,
              "commit": _plain_commit}


# -------------------------------------------------------------------------------------
# Work and the definition in 64 bits
# -------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rope":
        T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
        e = 2 if case["kv"] == "bf16" else 1
        rows = T * D * (Hq + 2 * Hkv) * 2 + T * D * (Hq * 2 + 2 * Hkv * e)
        return {"bytes": rows + T * (8 + 4 * case["axes"]) + case["rot"] * 4,
                "flops": T * (Hq + Hkv) * (case["rot"] * 3 + (4 * D if case["norm"] else 0))}
    cs, ls = _lens(case)
    T = sum(ls)
    if op == "masks":
        return {"bytes": T * (4 + 4 + 8 * -(-max(ls) // 64)) + 8 * len(ls), "flops": T}
    e = 2 if case["kv"] == "bf16" else 1
    if op == "commit":
        moved = case["S"] * (case["accept"] + 1) / 2  # accepted lengths are even over 1..accept
        return {"bytes": moved * case["Hkv"] * case["D"] * 2 * e * 2, "flops": 0}
    kv = sum(cs) * case["Hkv"] * case["D"] * 2 * e
    io = 2 * T * case["Hq"] * case["D"] * 2 + T * 8 * -(-max(ls) // 64)
    # every drafted token meets its whole prefix and at least itself
    keys = sum(n * (c - n + 1) for c, n in zip(cs, ls))
    return {"bytes": kv + io, "flops": 4 * case["Hq"] * case["D"] * keys}


def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _exact_masks(s):
    return None  # whole numbers: compared as they are


def _exact_rope(s):
    D, rot = s["D"], s["rot"]
    ax = s["axis_of"].tolist()
    ang = torch.stack([s["pos"][ax[i]].double() * s["freq"][i] for i in range(rot // 2)], 1)
    turn = torch.polar(torch.ones_like(ang), ang)[:, None, :]  # unit complex numbers

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + 1e-6) * w.double()
        if s["inter"]:
            z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * turn
            x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
        else:
            h = rot // 2
            z = torch.complex(x[..., :h].contiguous(), x[..., h:rot].contiguous()) * turn
            x[..., :h], x[..., h:rot] = z.real, z.imag
        return x

    q, k, v = one(s["q"].clone(), s["qw"]), one(s["k"].clone(), s["kw"]), s["v"].double()
    blk, off = torch.div(s["slots"], BLOCK, rounding_mode="floor"), s["slots"].remainder(BLOCK)
    if s["kv"] == "bf16":
        kc, vc = s["kc"].double(), s["vc"].double()
        kc[blk, :, off], vc[blk, :, off] = k, v
        return q, kc, vc
    kc = s["kc"].view(torch.float8_e4m3fn).double()
    vc = s["vc"].view(torch.float8_e4m3fn).double().view(-1, s["Hkv"], D, BLOCK)
    # the values before their rounding to 8 bits, in units of the scale
    kc[blk, :, off] = (k / s["ks"].double()[:, None]).clamp(-448, 448)
    vc[blk, :, :, off] = (v / s["vs"].double()[:, None]).clamp(-448, 448)
    return q, kc, vc.view(-1, s["Hkv"], BLOCK, D)


def _exact_tree(s):
    cs, ls = _lens(s)
    Hkv, D = s["Hkv"], s["D"]
    G = s["Hq"] // Hkv
    out, at = [], 0
    for b, (c, n) in enumerate(zip(cs, ls)):
        blocks = s["bt"][b, :-(-c // BLOCK)].long()
        if s["kv"] == "bf16":
            k, v = s["kc"][blocks].double(), s["vc"][blocks].double()
        else:
            k = s["kc"][blocks].view(torch.float8_e4m3fn).double()
            k = k * s["ks"].double().view(1, -1, 1, 1)
            v = s["vc"][blocks].view(-1, Hkv, D, BLOCK).view(torch.float8_e4m3fn).double()
            v = (v * s["vs"].double().view(1, -1, 1, 1)).transpose(2, 3)
        k = k.transpose(0, 1).reshape(Hkv, -1, D)[:, :c]
        v = v.transpose(0, 1).reshape(Hkv, -1, D)[:, :c]
        # visible: the prefix, and the ancestors found by walking up from each token
        par = s["parents"][at:at + n].tolist()
        see = torch.zeros(n, c, dtype=torch.bool)
        see[:, :c - n] = True
        for i in range(n):
            a = i
            while a >= 0:
                see[i, c - n + a] = True
                a = par[a]
        see = see.to(DEV)
        q = s["q"][at:at + n].double().view(n, Hkv, G, D)
        for h in range(Hkv):
            x = torch.einsum("ngd,cd->ngc", q[:, h], k[h]) * s["scale"]
            x = x.masked_fill(~see[:, None, :], float("-inf"))
            out.append((b, h, torch.softmax(x, -1) @ v[h]))
        at += n
    rows = []
    for b in range(len(cs)):
        rows.append(torch.stack([o for bb, _, o in out if bb == b], 1))
    return torch.cat(rows, 0).reshape(at, s["Hq"], D)


def _exact_commit(s):
    qs, acc, lens = s["qs"].tolist(), s["acc"].tolist(), s["acc_lens"].tolist()
    f8 = s["kv"] != "bf16"
    kc = (s["kc"].view(torch.float8_e4m3fn) if f8 else s["kc"]).double()
    vc = (s["vc"].view(torch.float8_e4m3fn) if f8 else s["vc"]).double()
    vt = vc.view(-1, s["Hkv"], s["D"], BLOCK).transpose(2, 3) if f8 else vc
    slots = s["slots"].tolist()
    src = [slots[qs[b] + acc[b][i]] for b in range(len(lens)) for i in range(lens[b])]
    dst = [slots[qs[b] + i] for b in range(len(lens)) for i in range(lens[b])]
    a, b = torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV)
    for c in (kc, vt):
        rows = c[a // BLOCK, :, a % BLOCK].clone()
        c[b // BLOCK, :, b % BLOCK] = rows
    return kc, vc


_EXACT = {"masks": _exact_masks, "rope": _exact_rope, "tree": _exact_tree,
          "commit": _exact_commit}
