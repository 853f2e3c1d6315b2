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


@pytest.mark.parametrize("Nk", [32, 300])
@pytest.mark.parametrize("spread", [8, 14, 18, 22, 26, 30, 40])
def test_weights_far_below_the_reference(cuda_device, spread, Nk):
    """A first block whose value scale is 2^spread times the others' but whose codes are zeros: it sets the
    reference of the weights, and the outputs come from the other blocks alone. A weight of 2^-k
    times the largest weight times scale keeps eleven bits to k = 25, and steps of 2^-36 below."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(spread + Nk)
    B, H, block = 2, 16, 16
    q = rnd(rng, B, H, 1, D)
    k, v = codes(rng, B, H, Nk, D), codes(rng, B, H, Nk, D)
    v[:, :, :block] = 0
    ks = torch.full((B, H, -(-Nk // block)), 2.0 ** -8)
    vs = torch.ones_like(ks)
    vs[:, :, 0] = 2.0 ** spread
    scale = 1 / math.sqrt(D)
    kr, sv = f64(k) * 2.0 ** -8, np.repeat(f64(vs), block, 2)[:, :, :Nk]
    ref = cache64.attend64(f64(q), kr, f64(v) * sv[..., None], scale, True, None)
    s = scale * np.einsum("bhkd,bhd->bhk", kr, f64(q)[:, :, 0])
    p = np.exp(s - ref[1])
    top = (p * sv).max(-1)[..., None, None]
    steps = 2.0 ** -36 * top * np.abs(f64(v)).sum(2, keepdims=True)
    for splits in (0, 1):
        o, lse = fa.decode_fp8(*(t.to(cuda_device) for t in (q, k, v, ks, vs)), block, num_splits=splits)
        assert fa.get_status() == 0
        close(o, lse, ref, 2.0 ** -11, Nk, steps)


@pytest.mark.parametrize("huge", [0, 12, 20, 24, 28])
def test_queries_with_one_huge_channel_are_exact(cuda_device, huge):
    """A channel 2^huge times as large as the others meets keys of zero there: the others, all within
    2^31 of it, enter exactly, in the attention and in its weights."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(huge)
    B, H, g, Nk, block = 2, 3, 4, 700, 64
    mag = np.exp2(rng.uniform(-1, 2, (B, H * g, 1, D))) * rng.choice([-1.0, 1.0], (B, H * g, 1, D))
    mag[..., 5] = 2.0 ** huge
    q = torch.from_numpy(mag.astype(np.float32)).bfloat16()
    k, v = codes(rng, B, H, Nk, D), codes(rng, B, H, Nk, D)
    k[..., 5] = 0
    ks = torch.full((B, H, -(-Nk // block)), 2.0 ** -7)
    vs = torch.ones_like(ks)
    scale = 1 / math.sqrt(D)
    kr = f64(k) * 2.0 ** -7
    ref = cache64.attend64(f64(q), kr, f64(v), scale, True, None)
    qd, kd, vd, ksd, vsd = (t.to(cuda_device) for t in (q, k, v, ks, vs))
    o, lse = fa.decode_fp8(qd, kd, vd, ksd, vsd, block)
    close(o, lse, ref, 2.0 ** -11, Nk)
    lse = torch.from_numpy(ref[1].astype(np.float32))
    acc = torch.zeros(B, H, Nk, device=cuda_device)
    add, size = cache64.weights64(f64(q), kr, f64(lse), scale, True, None)
    fa.cache_weights(qd, kd, lse.to(cuda_device), acc, k_scale=ksd, block=block)
    assert fa.get_status() == 0
    rel = size * (2.0 ** -17 + 2.0 ** -22) + 2.0 ** -22 * (float(np.abs(f64(lse)).max()) + 4) + 2.0 ** -22
    assert (np.abs(f64(acc) - add) <= (rel + g * 2.0 ** -23) * add + 1e-30).all()


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("Nq", [1, 3, 20])
def test_weights_of_rows_that_add_nothing_beside_keys_that_are_not_finite(cuda_device, fp8, Nq):
    """Rows with lse = -inf add nothing to a key that holds NaN or, in bf16, an infinity; nor do the rows
    that fill a tile up. A row that does see such a key adds what the formula gives."""
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nk, block = 3, 8, 2, 300, 64
    rng = np.random.default_rng(Nq + fp8)
    q = rnd(rng, B, Hq, Nq, D)
    q[..., 7] = q[..., 7].abs() + 0.5
    k, _, ks, _ = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    kr = cache64.dequantised(f64(k), None if ks is None else f64(ks), block)
    lse = torch.from_numpy(cache64.attend64(f64(q), kr, kr, 1 / math.sqrt(D), True, None)[1].astype(np.float32))
    lse[0] = float("-inf")                       # a slot of the batch that nothing runs in
    lse[1, :3] = float("-inf")                   # and one with a head left of its first group
    plain = kr.copy()
    for b, h, j, c, x in ((0, 0, 3, 7, "nan"), (0, 1, 299, 9, "nan"), (1, 0, 130, 1, "nan"), (2, 1, 40, 2, "nan"),
                          (0, 0, 5, 7, "inf"), (1, 1, 77, 7, "-inf"), (2, 0, 211, 7, "-inf")):
        if x == "nan" and fp8:
            k.view(torch.uint8)[b, h, j, c] = 0x7F
        elif not fp8:
            k[b, h, j, c] = float(x)
        else:
            continue
        kr[b, h, j, c], plain[b, h, j] = float(x), 0.0
    acc0 = torch.from_numpy(rng.uniform(0, 1, (B, H, Nk)).astype(np.float32))
    acc = acc0.to(cuda_device)
    with np.errstate(invalid="ignore"):
        add, _ = cache64.weights64(f64(q), kr, f64(lse), 1 / math.sqrt(D), True, None)
    _, size = cache64.weights64(f64(q), plain, f64(lse), 1 / math.sqrt(D), True, None)
    fa.cache_weights(q.to(cuda_device), k, lse.to(cuda_device), acc, k_scale=ks, block=block)
    assert fa.get_status() == 0
    want, got = f64(acc0) + add, f64(acc)
    assert np.array_equal(got[0], f64(acc0)[0])
    assert np.isnan(want[1, 0, 130]) and np.isnan(want[2, 1, 40]) and np.isfinite(want[0]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    rel = size * (2.0 ** -17 + 2.0 ** -22) + 2.0 ** -22 * (float(np.abs(f64(lse)[2]).max()) + 4) + 2.0 ** -22
    tol = rel * np.nan_to_num(add) + 2.0 ** -23 * (4 * Nq) * np.nan_to_num(want) + 1e-30
    assert (np.abs(np.nan_to_num(got) - np.nan_to_num(want)) <= tol).all()


@pytest.mark.parametrize("exponent", [100, 126, 127])
def test_store_into_a_block_of_the_largest_scale(cuda_device, exponent):
    """A scale from elsewhere may be any power of two: 2^127 has no normal reciprocal."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(exponent)
    ck, cv, ks, vs = make_cache(rng, 1, 2, 40, 32, True, cuda_device)
    ks.fill_(2.0 ** exponent), vs.fill_(2.0 ** exponent)
    k = (rnd(rng, 1, 2, 10, D).float().clamp(-1.9, 1.9) * 2.0 ** exponent).bfloat16()
    want = cache64.store64(f64(k), f64(ck), f64(ks), 32, [30])
    kd = k.to(cuda_device)
    fa.cache_store(kd, kd, ck, cv, ks, vs, 32, lens=dev_lens([30], cuda_device))
    assert fa.get_status() == 0
    assert np.array_equal(f64(ck), want[0]) and np.array_equal(f64(ks), want[1])
    assert (f64(ck)[0, :, 20:30] != 0).any()


@pytest.mark.parametrize("Nk", [2, 3, 5, 16])
def test_weights_against_a_bf16_cache_keep_sixteen_bits(cuda_device, Nk):
    """The same against listed blocks of a bf16 cache, where a weight enters as two bf16 numbers: one alone
    is off by up to 2^-8 of itself (and, emulated, past this bound 22 to 35 times)."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(Nk)
    B, H, block = 4, 16, 16
    q, k = rnd(rng, B, H, 1, D), rnd(rng, B, H, Nk, D, std=0.25)
    v = rnd(rng, B, H, Nk, D)
    scale = 1 / math.sqrt(D)
    ref = cache64.attend64(f64(q), f64(k), f64(v), scale, True, None)
    idx = torch.zeros(B, H, 1, 1, dtype=torch.int32)
    o, lse = fa.decode_blocks(*(t.to(cuda_device) for t in (q, k, v, idx)), block)
    assert fa.get_status() == 0
    close(o, lse, ref, 2.0 ** -16, Nk)


@pytest.mark.parametrize("fp8", [True, False])
def test_bounds_of_channels_with_nothing_but_nan(cuda_device, fp8):
    """Such a channel's minimum is the type's largest value and its maximum the lowest; others are not touched by it."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(31)
    k, _, _, _ = make_cache(rng, 1, 1, 64, 32, fp8, cuda_device)
    want = cache64.bounds64(f64(k), 32, None)
    if fp8:
        k.view(torch.uint8)[0, 0, 32:, 9] = 0x7F
    else:
        k[0, 0, 32:, 9] = float("nan")
    top = 448.0 if fp8 else float("inf")
    want[0, 0, 1, 0, 9], want[0, 0, 1, 1, 9] = top, -top
    assert np.array_equal(f64(fa.block_bounds(k, 32)), want)
