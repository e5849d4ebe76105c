"""Plain 64-bit forms of the drafted-tree operators (CPU tensors, loops), and the inputs of
their tests."""
from __future__ import annotations

import numpy as np
import torch

BS = 16
BF16_HALF = 2.0 ** -8   # half a step of bf16, relative
F16_HALF = 2.0 ** -11
E4M3_HALF = 2.0 ** -4


def ancestors(parents):
    """bool [L][L]: token j is token i or one of its ancestors."""
    L = len(parents)
    m = np.zeros((L, L), bool)
    for i in range(L):
        a = i
        while a >= 0:
            m[i, a] = True
            a = parents[a]
    return m


def pack(rows, words):
    """bool [T][<= 64 words] -> int64 [T][words]."""
    out = np.zeros((len(rows), words), np.uint64)
    for i, r in enumerate(rows):
        for j in np.flatnonzero(r):
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(out.view(np.int64).copy())


def random_parents(rng, L, kind="random"):
    if kind == "chain":
        return [i - 1 for i in range(L)]
    if kind == "star":
        return [-1] * L
    return [int(rng.integers(-1, i)) if i else -1 for i in range(L)]


class Tree:
    """One drafted-tree step: lens[s] = (context with the drafts, drafts)."""

    def __init__(self, lens, Hq, Hkv, D, seed=0, words=None, kind="random", pad_rows=0,
                 f8=False, poison=True, spare_blocks=3):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.f8 = lens, Hq, Hkv, D, f8
        self.S = len(lens)
        self.ctx = np.array([c for c, _ in lens], np.int32)
        self.L = np.array([n for _, n in lens], np.int32)
        self.qs = np.concatenate([[0], np.cumsum(self.L)]).astype(np.int32)
        self.T = int(self.qs[-1]) + pad_rows
        self.maxq = max(1, int(self.L.max()))
        self.words = words or -(-self.maxq // 64)
        nb = -(-self.ctx.astype(np.int64) // BS)
        self.NB = int(nb.sum()) + spare_blocks
        perm = rng.permutation(self.NB)
        self.MB = max(1, int(nb.max()))
        self.bt = np.full((self.S, self.MB), -1, np.int32)
        at = 0
        for s in range(self.S):
            self.bt[s, :nb[s]] = perm[at:at + nb[s]]
            at += nb[s]
        self.parents = np.full(self.T, 7, np.int32)  # padding rows hold anything
        rows = []
        for s in range(self.S):
            p = random_parents(rng, int(self.L[s]), kind)
            self.parents[self.qs[s]:self.qs[s + 1]] = p
            rows += list(ancestors(p))
        self.visible = rows  # per drafted token, over its tree
        self.masks = torch.cat([pack(rows, self.words),
                                torch.full((pad_rows, self.words), -1, dtype=torch.int64)])
        self.slots = np.zeros(self.T, np.int64)
        for s in range(self.S):
            p = np.arange(self.ctx[s] - self.L[s], self.ctx[s])
            self.slots[self.qs[s]:self.qs[s + 1]] = (
                self.bt[s, p // BS].astype(np.int64) * BS + p % BS)
        self.q = torch.randn(self.T, Hq, D, generator=g).to(torch.bfloat16)
        self.scale = D ** -0.5
        shape = (self.NB, Hkv, BS, D)
        self.ks = (torch.rand(Hkv, generator=g) + 0.5) / 32
        self.vs = (torch.rand(Hkv, generator=g) + 0.5) / 32
        if f8:
            # a quarter of the range: the drawn codes span subnormals to 448
            code = lambda *sh: (torch.randn(*sh, generator=g) * 32).to(
                torch.float8_e4m3fn).view(torch.uint8)
            self.k, self.v = code(*shape), code(self.NB, Hkv, D, BS).view(shape)
        else:
            self.k = torch.randn(*shape, generator=g).to(torch.bfloat16)
            self.v = torch.randn(*shape, generator=g).to(torch.bfloat16)
        if poison:  # every token slot that no sequence holds is NaN
            used = np.zeros((self.NB, BS), bool)
            for s in range(self.S):
                p = np.arange(self.ctx[s])
                used[self.bt[s, p // BS], p % BS] = True
            u = torch.from_numpy(~used)
            if f8:
                self.k[u[:, None, :, None].expand(shape)] = 0x7F
                v = self.v.view(self.NB, Hkv, D, BS)
                v[u[:, None, None, :].expand(v.shape)] = 0x7F
            else:
                self.k[u[:, None, :, None].expand(shape)] = float("nan")
                self.v[u[:, None, :, None].expand(shape)] = float("nan")

    def kv64(self, s):
        """K and V of sequence s in 64 bits, [ctx][Hkv][D]."""
        c = int(self.ctx[s])
        b = torch.from_numpy(self.bt[s, :-(-c // BS)].astype(np.int64))
        if self.f8:
            k = self.k[b].view(torch.float8_e4m3fn).double() * self.ks.double().view(1, -1, 1, 1)
            v = self.v[b].view(-1, self.Hkv, self.D, BS).view(torch.float8_e4m3fn).double()
            v = (v * self.vs.double().view(1, -1, 1, 1)).transpose(2, 3)
        else:
            k, v = self.k[b].double(), self.v[b].double()
        f = lambda x: x.transpose(1, 2).reshape(-1, self.Hkv, self.D)[:c]
        return f(k), f(v)

    def attention64(self, visible=None):
        """(out [rows][Hq][D], bound): the definition in 64 bits, and per element how far a
        result in the kernel's types may be from it.  The result is a mean of V rows by
        weights: each weight is rounded once on its way into the product (half a step h of
        bf16 or f16), the sum once to bf16 at the end; scores, sums and the merge are in 32
        bits, which moves a weight by less than 2^-10 of itself at these sizes (128 products
        of magnitude about 1 summed, 2^-24 each, exponent up to ~30 rounded at 2^-24: below
        2^-12).  f16 weights below 2^-14 of the row's largest lose up to 2^-25 each."""
        visible = self.visible if visible is None else visible
        G = self.Hq // self.Hkv
        rows = int(self.qs[-1])
        out = torch.zeros(rows, self.Hq, self.D, dtype=torch.float64)
        bound = torch.zeros_like(out)
        h = F16_HALF if self.f8 else BF16_HALF
        for s in range(self.S):
            c, n = int(self.ctx[s]), int(self.L[s])
            k, v = self.kv64(s)
            for i in range(n):
                r = int(self.qs[s]) + i
                see = np.concatenate([np.ones(c - n, bool), np.asarray(visible[r])[:n]])
                idx = torch.from_numpy(np.flatnonzero(see))
                if idx.numel() == 0:
                    continue
                q = self.q[r].double().view(self.Hkv, G, self.D)
                kk, vv = k[idx], v[idx]
                p = torch.softmax(torch.einsum("hgd,chd->hgc", q, kk) * self.scale, -1)
                out[r] = torch.einsum("hgc,chd->hgd", p, vv).reshape(self.Hq, self.D)
                mag = torch.einsum("hgc,chd->hgd", p, vv.abs()).reshape(self.Hq, self.D)
                bound[r] = BF16_HALF * out[r].abs() + (h + 2.0 ** -10) * mag + 2.0 ** -40
                if self.f8:
                    bound[r] += idx.numel() * 2.0 ** -25 * float(vv.abs().max())
        return out, bound

    def cuda(self):
        d = "cuda"
        t = lambda a: torch.as_tensor(a, device=d)
        return dict(q=self.q.to(d), k=self.k.to(d).clone(), v=self.v.to(d).clone(), bt=t(self.bt),
                    ctx=t(self.ctx), qs=t(self.qs), masks=self.masks.to(d), slots=t(self.slots),
                    parents=t(self.parents), ks=self.ks.to(d), vs=self.vs.to(d),
                    err=torch.zeros(1, dtype=torch.int32, device=d))


def run_tree(ops, w, d=None, ws=None, out=None, stream=None):
    """paged_attention_tree(_fp8) of w through the public call; returns (out, device dict)."""
    d = d or w.cuda()
    if out is None:
        out = torch.full((w.T, w.Hq, w.D), 9.0, dtype=torch.bfloat16, device="cuda")
    if ws is None:
        ws = ops.alloc_tree_workspace(w.Hq, w.Hkv, w.D, w.maxq)
        ws.fill_(0xFF)  # stale contents must not matter
    if w.f8:
        ops.paged_attention_tree_fp8(out, d["q"], d["k"], d["v"], d["bt"], d["ctx"], d["qs"],
                                     d["masks"], w.scale, d["ks"], d["vs"], w.maxq, ws,
                                     err_flag=d["err"], stream=stream)
    else:
        ops.paged_attention_tree(out, d["q"], d["k"], d["v"], d["bt"], d["ctx"], d["qs"],
                                 d["masks"], w.scale, w.maxq, ws, err_flag=d["err"],
                                 stream=stream)
    return out, d


def assert_within(got, ref, bound, what=""):
    g = got.detach().cpu().double()
    bad = ~((g - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(((g - ref).abs() / bound).max()),
                           torch.nonzero(bad)[0].tolist())


def rope64(x, w, eps, pos, axes, freq, rot, inter, scale=1.0):
    """(y, bound) of head rows x [T][H][D] in 64 bits: norm, then rotation.  bound: the fp32
    arithmetic before the final rounding -- the norm's sum of D squares and its root (D 2^-24
    at most, relative), three products and two sums, sines to 2^-22: below 2^-16 (|a| + |b|)
    for the pair's values."""
    T, H, D = x.shape
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    out, bound = y.clone(), y.abs() * 2.0 ** -16
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        t = (pos[axes[i]].double() * freq[i].double())[:, None]
        c, s = torch.cos(t) * scale, torch.sin(t) * scale
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        bound[..., a] = bound[..., b] = (y[..., a].abs() + y[..., b].abs()) * scale * 2.0 ** -16
    return out, bound
