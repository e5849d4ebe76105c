"""Shared prefixes of 24 MB and more: a group's row tiles run side by side, in lanes of their own, and a
pair of row tile and head is cut over runs that lie apart."""
import numpy as np
import pytest
import torch

from range_helpers import Shared
from tree_helpers import BS, assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


@pytest.fixture(scope="module")
def ops():
    from paged_kv_cache_272_gb300 import ops as o
    return o


class Long(Shared):
    """As Shared, each prefix in the cache once: (sequences, prefix, own tokens) per group."""

    def __init__(self, groups, Hq, Hkv, D, seed=0, f8=False):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.g, self.f8, self.Hq, self.Hkv, self.D = g, f8, Hq, Hkv, D
        rows, ctx, starts, used, copies = [], [], [0], 0, []
        for n, p, own in groups:
            m, rest = p // BS, p % BS
            prefix, used = list(range(used, used + m)), used + m
            for i in range(n):
                c = p + own[i % len(own)]
                nb = -(-c // BS) - m
                if i and rest:
                    copies.append((first, used, rest))
                elif rest:
                    first = used
                rows.append(prefix + list(range(used, used + nb)))
                used += nb
                ctx.append(c)
            starts.append(len(ctx))
        self.S, self.NB, self.MB = len(ctx), used + 3, max(len(r) for r in rows)
        perm = rng.permutation(self.NB)
        self.ctx, self.starts = np.array(ctx, np.int32), np.array(starts, np.int32)
        self.prefix = np.array([p for _, p, _ in groups], np.int32)
        self.bt = np.full((self.S, self.MB), -1, np.int32)
        for s, r in enumerate(rows):
            self.bt[s, :len(r)] = perm[r]
        shape = (self.NB, Hkv, BS, D)
        self.ks = (torch.rand(Hkv, generator=g) + 0.5) / 32
        self.vs = (torch.rand(Hkv, generator=g) + 0.5) / 32
        x = lambda: torch.randn(*shape, generator=g)
        code = lambda t: (t * 32).to(torch.float8_e4m3fn).view(torch.uint8)
        self.k, self.v = (code(x()), code(x())) if f8 else (x().bfloat16(), x().bfloat16())
        for a, b, rest in copies:
            a, b = perm[a], perm[b]
            self.k[b, :, :rest] = self.k[a, :, :rest]
            if f8:
                v = self.v.view(self.NB, Hkv, D, BS)
                v[b, :, :, :rest] = v[a, :, :, :rest]
            else:
                self.v[b, :, :rest] = self.v[a, :, :rest]
        held = np.zeros((self.NB, BS), bool)
        for s in range(self.S):
            p = np.arange(int(self.ctx[s]))
            held[self.bt[s, p // BS], p % BS] = True
        self.poison(torch.from_numpy(~held))
        self.q = torch.randn(self.S, Hq, D, generator=g).to(torch.bfloat16)
        self.scale = D ** -0.5


def lanes(w):
    """How the plan cuts these prefixes: (row tiles, runs) of each group's lanes and which of the run
    lengths tried is the first that fits; None where they do not run in lanes."""
    ctas = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    start, tile_bytes = (12, 128 * w.D) if w.f8 else (5, 256 * w.D)
    G = w.Hq // w.Hkv
    rows, lane, keys = [], [], 0
    for a, b, p in zip(w.starts, w.starts[1:], w.prefix):
        if b - a > 1 and p >= BS:
            tiles = -(-(int(p) // BS * BS) // 64)
            rows.append(-(-int(b - a) * G // 128))
            lane.append(w.Hkv * (tiles + start))
            keys += tiles * w.Hkv
    if keys <= (24 << 20) // tile_bytes:
        return None
    even = sum(r * x for r, x in zip(rows, lane)) // ctas + 1
    for i in range(32):
        cuts = [-(-x // (even + even * i // 128)) for x in lane]
        if sum(r * c for r, c in zip(rows, cuts)) <= ctas:
            return list(zip(rows, cuts)), i
    return None


OWN = [1, 0, 37, 300, 16]
# E4M3, (sequences, prefix) of each group, Hq, Hkv, D
CASES = [
    # two and three row tiles a group
    (False, [(9, 3500), (17, 2909)], 128, 8, 128),
    (True, [(9, 7001), (17, 6000)], 128, 8, 128),
    # one to three row tiles, a group of one beside them
    (False, [(5, 2000), (10, 3100), (1, 777), (18, 2700)], 128, 8, 128),
    (True, [(5, 4000), (10, 6200), (1, 777), (18, 5500)], 128, 8, 128),
    # groups' runs fit only where they are longer than the even share
    (False, [(6, 5322), (20, 1483), (17, 869), (4, 6182)], 128, 16, 64),
    (False, [(2, 3128), (9, 6152), (24, 1584), (15, 2871)], 64, 8, 128),
    (True, [(26, 5596), (12, 1046), (2, 5095)], 128, 16, 128),
    (True, [(7, 841), (9, 6553), (21, 1419)], 128, 16, 128),
    # short pairs, several heads of which make one run, beside long ones; 9 heads a KV head
    (False, [(60, 7000), (30, 100)], 72, 8, 128),
    (True, [(60, 14000), (30, 100)], 72, 8, 128),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_lanes(ops, case):
    f8, groups, Hq, Hkv, D = CASES[case]
    w = Long([(n, p, OWN) for n, p in groups], Hq, Hkv, D, seed=case, f8=f8)
    plan = lanes(w)
    assert plan and max(r for r, _ in plan[0]) > 1
    if 4 <= case < 8:
        assert plan[1] > 0
    if case >= 8:
        assert min(c for _, c in plan[0]) < Hkv
    ref, bound = w.reference()
    d = w.cuda(q=w.q, starts=w.starts, prefix=w.prefix)
    for variant in (ops.PKV_SHARED_ALWAYS, ops.PKV_SHARED_AUTO):
        was = ops.set_shared_variant(variant)
        try:
            out, _ = w.run(ops, d)
            assert_within(out, ref, bound, variant)
            again, _ = w.run(ops, d)
        finally:
            ops.set_shared_variant(was)
        assert torch.equal(again, out)  # the same bits every time
    assert int(d["err"]) == 0
