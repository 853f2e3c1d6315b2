"""The float64 restatement of the cache operators against independent facts."""
import numpy as np
import pytest

import oracle
from oracle import cache64


def test_e4m3_rounding_matches_torch():
    import torch
    bits = torch.arange(0, 1 << 16, dtype=torch.int32)
    x = (bits << 16).view(torch.float32)           # every bf16 value
    x = x[torch.isfinite(x)]
    ref = x.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache64.e4m3_round(x.double().numpy()), ref)


@pytest.mark.parametrize("amax", [0.0, 1e-42, 448.0, 448.1, 1.0, 0.875, 0.8751, 3.5, 3.500001, 3e38])
def test_scale_is_the_smallest_power_of_two_that_holds_amax(amax):
    s = cache64.scale_for(amax)
    assert np.log2(s) == int(np.log2(s)) and s >= 2.0 ** -100 and amax <= 448 * s
    assert s == 2.0 ** -100 or amax > 448 * s / 2


def test_attention_equals_the_decode_oracle_and_weights_its_column_sums():
    rng = np.random.default_rng(3)
    B, Hq, H, Nq, Nk, d = 2, 6, 2, 3, 50, 16
    q, k, v = rng.standard_normal((B, Hq, Nq, d)), rng.standard_normal((B, H, Nk, d)), rng.standard_normal((B, H, Nk, d))
    for causal in (True, False):
        o, lse, _, _ = cache64.attend64(q, k, v, 0.25, causal, None)
        o_ref, lse_ref = oracle.decode_fwd64(q, k, v, causal, 0.25)
        assert np.allclose(o, o_ref, atol=1e-12) and np.allclose(lse, lse_ref, atol=1e-12)
        add, _ = cache64.weights64(q, k, lse, 0.25, causal, None)
        assert np.allclose(add.sum(-1), Hq // H * Nq)          # every row's weights sum to one
        # all blocks listed: the same; a shorter length: the same as a shorter cache
        idx = np.broadcast_to(np.arange(4), (B, H, Nq, 4))
        o2, lse2, _, _ = cache64.attend64(q, k, v, 0.25, causal, None, idx, 16)
        assert np.allclose(o, o2) and np.allclose(lse, lse2)
        o3, lse3, _, _ = cache64.attend64(q, k, v, 0.25, causal, [37, 50])
        o4, lse4 = oracle.decode_fwd64(q[:1], k[:1, :, :37], v[:1, :, :37], causal, 0.25)
        assert np.allclose(o3[:1], o4) and np.allclose(lse3[:1], lse4)


def test_bounds_hold_every_score():
    rng = np.random.default_rng(4)
    k, q = rng.standard_normal((1, 1, 64, 8)), rng.standard_normal((1, 1, 1, 8))
    b = cache64.bounds64(k, 16, None)
    x = q[0, 0, 0]
    u = np.where(x >= 0, x * b[0, 0, :, 1], x * b[0, 0, :, 0]).sum(-1)
    assert (u >= (k[0, 0] @ x).reshape(4, 16).max(1) - 1e-12).all()
    top = cache64.select64(q, b, None, 2, 16, 64, None, 0, 0)[0, 0, 0]
    assert sorted(top) == list(top) and set(top) == set(np.argsort(-u, kind="stable")[:2])


def test_eviction_keeps_the_newest_and_the_heaviest_in_order():
    acc = np.array([[[3.0, 1.0, 3.0, np.nan, 0.5, 9.0, 0.0, 0.0]]])
    idx, lens = cache64.evict64(acc, 4, 2, None)
    assert idx[0, 0].tolist() == [0, 5, 6, 7] and lens == [4]
    idx, lens = cache64.evict64(acc, 4, 0, [5])
    assert idx[0, 0].tolist() == [0, 1, 2, 4] and lens == [4]     # NaN goes first
    idx, lens = cache64.evict64(acc, 4, 1, [2])
    assert idx[0, 0].tolist() == [0, 1, -1, -1] and lens == [2]
