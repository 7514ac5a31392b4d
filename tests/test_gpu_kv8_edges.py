"""The 8-bit K/V cache at the ends of its ranges. Bounds as in test_gpu_kv8."""
import numpy as np
import pytest

from .test_gpu_kv8 import Pair

pytestmark = pytest.mark.gpu

# (rows of the call, queries, heads on one K/V head): few and many query rows, items in one part and in several
CALLS = [(1, 1, 1), (1, 10, 2), (1, 40, 2), (160, 10, 2), (160, 40, 2), (100, 80, 2)]


# ---- V scales

SPREADS = [(1e23, 0, 1e23, 0, 0), (1e30, 1e-20, 1, 0, 1e30), (0, 1, 1e25, 1e-17, 1e-5), (1e-20, 1e30, 0, 0, 1e20)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,nq,H", CALLS)
@pytest.mark.parametrize("spread", range(len(SPREADS)))
def test_v_scales_far_apart(D, B, nq, H, spread):
    """Scores of like size in blocks whose V scales lie up to 2^160 apart, in both orders: each
    key counts in the sum of the weights by its score, whatever its V."""
    rng = np.random.default_rng(spread)
    f = np.repeat(SPREADS[spread], 64)[:, None]
    p = Pair(1, 1, D, 320, 2)
    K, Vv = (rng.standard_normal((1, 2, 320, D)) for _ in range(2))
    p.write(K, Vv * np.stack([f, f[::-1]]))
    slots, lens = rng.integers(0, 2, B), rng.integers(280, 321, B)
    Q = 0.5 * rng.standard_normal((B, nq, H, D))
    p.check_attend(Q, lens, slots=slots)
    Q[:, ::3] *= 1e-6                                # equal scores
    p.check_attend(Q, lens, slots=slots, causal=True, window=200)
