"""The sums that verification draws from, to the last places that a 24-bit uniform can tell."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import verify_helpers as VH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def close_draws(n, seed):
    """n sequences whose only draft is refused and leaves two tokens, A and B = p - d: (p, d, A, w,
    token), w the uniform next to A / (A + B), within 2^-27 of it and not within 2^-41 (the sums
    are within 2^-43 of each value)."""
    rng = np.random.default_rng(seed)
    found = []
    while len(found) < n:
        d = np.float32(rng.random() * 0.05 + 0.001)
        B = Fraction(int(2 * rng.integers(2 ** 20, 2 ** 21) + 1), 2 ** 22)
        p = np.float32(float(B) + float(d) + int(rng.integers(-2, 3)) * 2.0 ** -24)
        a = np.float32(rng.random() * 0.3 + 0.1)
        A, B = Fraction(float(a)), Fraction(float(p)) - Fraction(float(d))
        w = np.float32(float(A / (A + B)))
        w = np.nextafter(w, np.float32(rng.integers(0, 2)))
        for x in (w, np.nextafter(w, np.float32(0)), np.nextafter(w, np.float32(1))):
            gap = A - Fraction(float(x)) * (A + B)
            if Fraction(1, 2 ** 41) < abs(gap) < Fraction(1, 2 ** 27):
                found.append((p, d, a, x, 0 if gap > 0 else 1))
                break
    return found


@pytest.mark.parametrize("n", [3, 150, 700])  # eight, four CTAs a sequence, one
def test_draws_next_to_a_border(n):
    from paged_kv_cache_272_gb300 import ops
    cases = close_draws(n, n)
    w = VH.Drafts([2] * n, 4, "chain")
    w.p, w.d = torch.zeros(2 * n, 4), torch.zeros(2 * n, 4)
    w.tokens[1::2] = 2           # the draft had a probability, the target none: refused
    w.u[:] = 0.5
    want = np.zeros(n, np.int32)
    for s, (p, d, a, x, token) in enumerate(cases):
        w.p[2 * s] = torch.tensor([a, p, 0, 0])
        w.d[2 * s] = torch.tensor([0, d, 0.5, 0])
        w.w[s] = float(x)
        want[s] = token
    out, t = VH.run_verify(ops, w)
    assert (out[1] == 1).all() and int(t["err"]) == 0
    got = out[2].cpu().numpy()
    assert np.array_equal(got, want), (int((got != want).sum()), n)
