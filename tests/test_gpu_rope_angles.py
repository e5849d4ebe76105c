"""How exact the rotary write's angles are: frequencies and far positions whose product lies
close to whole turns, where the sine's own bits show the angle's error."""
from decimal import Decimal, getcontext

import pytest
import torch

pytestmark = pytest.mark.gpu
getcontext().prec = 80


def pi():
    """Machin's formula."""
    def atan_inv(n):
        total, power, k, sign = Decimal(0), Decimal(1) / n, 1, 1
        while power > Decimal(10) ** -78:
            total += sign * power / k
            power, k, sign = power / (n * n), k + 2, -sign
        return total
    return 4 * (4 * atan_inv(5) - atan_inv(239))


@pytest.mark.parametrize("size", [1e-3, 0.7, 6.0, 60.0, 4000.0, 1e6])
def test_angles_of_far_positions(size):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_272_gb300 import ops
    two_pi, D = 2 * pi(), 128
    pos = torch.tensor([2**31 - 1, -2**31, 2**30 + 12345, 1000003, -131071, 77], dtype=torch.int32)
    T, pairs = pos.numel(), D // 2
    # each token and pair: a frequency near `size` that takes the position a few 1e-7 of a turn
    # off a whole number of turns, or as near as a double can
    for t, p in enumerate(pos.tolist()):
        turns = [int(size * abs(p) / 6.283) + i for i in range(pairs)]
        freq = torch.tensor([float(two_pi * (n + Decimal(i - 32) * Decimal("2e-8")) / p)
                             for i, n in enumerate(turns)], dtype=torch.float64)
        q = torch.zeros(1, 1, D, dtype=torch.bfloat16, device="cuda")
        q[..., :pairs] = 1  # (1, 0) -> (cos, sin)
        out = torch.empty_like(q)
        kc = torch.zeros(1, 1, 16, D, dtype=torch.bfloat16, device="cuda")
        ops.paged_qk_norm_rope_write(out, q, q, q, pos[t:t + 1].cuda(), freq.cuda(),
                                     torch.tensor([-1], device="cuda"), kc, kc.clone())
        sin = out[0, 0, pairs:].cpu().double()
        for i, w in enumerate(freq.tolist()):
            x = Decimal(w) * p / two_pi
            x -= x.to_integral_value()  # turns, within half of one
            if abs(x) > Decimal("0.01"):
                continue  # doubles are too far apart here
            angle = float(x * two_pi)
            # radians: the product's 2^-33 + w 2^-41 of a turn, the 2^-32 cut off below the top 32
            # bits, the 24 bits kept (2^-24 of the angle, as of the sine); bf16's half step
            err = 6.2832 * (2.0 ** -33 + abs(w) * 2.0 ** -41 + 2.0 ** -32)
            assert abs(float(sin[i]) - angle) <= \
                err + (2.0 ** -8 + 2.0 ** -22) * abs(angle) + abs(angle) ** 3 / 6, (p, w)
