"""The cache operators at the ends of their number ranges, against the float64 restatement.

Tolerances, from the roundings that an operator makes (half a step each):
  o     bf16 output: 2^-8 |o|.
  p     a weight that enters the P V product: 2^-11 of itself against an 8-bit cache (fp16), 2^-16 against
        a bf16 cache (two bf16 terms); its exponential and the scalings 2^-20; and the scores' own error
        twice over (numerator and denominator): all times sum_j p_j |v_j|. Sums in fp32: n 2^-24 of it for n keys.
  ds    a score is 128 products summed in fp32 in some order: 2^-17 of scale * sum_c |q_c k_c|, and two
        scalings, 2^-22 of it.
"""
import math

import numpy as np
import pytest

from oracle import cache64
from tests.test_cache_gpu import D, dev_lens, f64, make_cache, rnd

pytestmark = pytest.mark.gpu


def close(o, lse, ref, weight, n_keys, extra=0.0):
    """o and lse against `ref` where weights keep a relative `weight`."""
    o_ref, lse_ref, pv, size = ref
    ds = size * (2.0 ** -17 + 2.0 ** -22)
    tol = 2.0 ** -8 * np.abs(o_ref) + (weight + 2.0 ** -20 + n_keys * 2.0 ** -24 + 2 * ds[..., None]) * pv + extra + 1e-30
    worst = float((np.abs(f64(o) - o_ref) / tol).max())
    assert worst <= 1, worst
    assert (np.abs(f64(lse) - lse_ref) <= ds + 2.0 ** -20 * (1 + np.abs(lse_ref))).all()


def codes(rng, *shape, std=60.0):
    """E4M3 codes over their whole finite range."""
    import torch
    c = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(std))
    return c.clamp(-448, 448).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("Nk", [2, 3, 5, 40])
def test_weights_against_an_8_bit_cache_keep_eleven_bits(cuda_device, Nk):
    """Few keys of weights alike and values of both signs: outputs far below sum p |v|, in which the
    weights' rounding shows."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(Nk)
    B, H, block = 4, 16, 16
    q = rnd(rng, B, H, 1, D)
    k, v = codes(rng, B, H, Nk, D), codes(rng, B, H, Nk, D)
    ks = torch.full((B, H, -(-Nk // block)), 2.0 ** -8)
    vs = torch.ones_like(ks)
    scale = 1 / math.sqrt(D)
    ref = cache64.attend64(f64(q), f64(k) * 2.0 ** -8, f64(v), scale, True, None)
    o, lse = fa.decode_fp8(*(t.to(cuda_device) for t in (q, k, v, ks, vs)), block)
    assert fa.get_status() == 0
    close(o, lse, ref, 2.0 ** -11, Nk)
