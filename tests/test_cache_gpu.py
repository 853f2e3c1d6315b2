"""The cache operators on the GPU against the float64 restatement (oracle/cache64.py).

Tolerances, from the roundings that an operator makes:
  O     bf16 output: 2^-8 |o|; probabilities rounded before the P V product (8 bits kept, at
        most 2^-8 each): 2^-8 sum_j p_j |v_j|; scores' own error ds moves a probability by
        2 ds: 2 ds sum_j p_j |v_j|.
  ds    a score is 128 exact products summed in fp32 in some order: at most 128 * 2^-24 =
        2^-17 of scale * sum_c |q_c k_c|; then two scalings, 2^-22 of it.
  LSE   ds, and 2^-20 (1 + |lse|) for the exponentials (2^-22 each), the sum and the logarithm.
  acc   every weight is exp(S - lse): relative ds + 2^-22 (|S| + |lse| in fp32) + 2^-22; |S| is
        at most the size above; the sum over rows in fp32.
Stores, bounds, selections and evictions are compared for equality.
"""
import math

import numpy as np
import pytest

from oracle import cache64

pytestmark = pytest.mark.gpu

D = 128


def rnd(rng, *shape, std=1.0):
    import torch
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(std)).bfloat16()


def f64(t):
    return t.double().cpu().numpy()


def make_cache(rng, B, H, Nk, block, fp8, device, std=1.0, pow2=True):
    """A cache (k, v, ks, vs) on the device; 8-bit codes over their whole finite range."""
    import torch
    if not fp8:
        return rnd(rng, B, H, Nk, D, std=std).to(device), rnd(rng, B, H, Nk, D).to(device), None, None
    out = []
    nb = -(-Nk // block)
    for _ in range(2):
        c = torch.from_numpy(rng.standard_normal((B, H, Nk, D), dtype=np.float32) * 60).clamp(-448, 448)
        e = rng.integers(-8, -4, (B, H, nb)).astype(np.float32)
        s = np.exp2(e) if pow2 else np.exp2(e) * rng.uniform(0.6, 1.4, e.shape).astype(np.float32)
        out.append((c.to(torch.float8_e4m3fn).to(device), torch.from_numpy(s.astype(np.float32)).to(device)))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def dev_lens(lens, device):
    import torch
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device=device)


def poison(t, lens):
    """NaN behind every sequence's end."""
    import torch
    if lens is None:
        return
    for b, n in enumerate(lens):
        n = min(max(n, 0), t.shape[2])
        if t.dtype == torch.float8_e4m3fn:
            t.view(torch.uint8)[b, :, n:] = 0x7F
        else:
            t[b, :, n:] = float("nan")


def poison_scales(s, block, lens):
    """NaN and infinity in the scales of blocks behind every sequence's end."""
    if lens is None or s is None:
        return
    for b, n in enumerate(lens):
        j = -(-min(max(n, 0), 1 << 30) // block)
        s[b, :, j::2] = float("nan")
        s[b, :, j + 1::2] = float("inf")


def real(c, s, block, lens):
    """The cache's values with the NaN behind the ends taken out."""
    s = None if s is None else np.nan_to_num(f64(s), posinf=0.0)
    return np.nan_to_num(cache64.dequantised(np.nan_to_num(f64(c)), s, block))


def check_attend(o, lse, ref, label):
    o_ref, lse_ref, pv, size = ref
    o, lse = f64(o), f64(lse)
    ds = size * (2.0 ** -17 + 2.0 ** -22)
    tol = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -8 + 2 * ds[..., None]) * pv + 1e-30
    seen = lse_ref > -np.inf
    assert np.array_equal(np.isneginf(lse), ~seen), label
    assert np.all(o[~seen] == 0), label
    worst = np.abs(o - o_ref) / tol
    assert np.isfinite(o).all() and worst.max() <= 1, (label, float(worst.max()))
    tl = ds[seen] + 2.0 ** -20 * (1 + np.abs(lse_ref[seen]))
    assert (np.abs(lse[seen] - lse_ref[seen]) <= tl).all(), (label, float(np.abs(lse[seen] - lse_ref[seen]).max()))


# --------------------------------------------------------------------------------------------- store and bounds

STORES = [
    # B, Hkv, Nk, n_new, block, lens
    (1, 1, 1, 1, 16, None),
    (2, 2, 40, 1, 16, [40, 17]),
    (3, 1, 300, 1, 128, [1, 129, 300]),
    (2, 3, 257, 40, 32, [257, 33]),
    (2, 2, 200, 200, 64, None),
    (2, 1, 130, 131, 64, [130, 0]),      # more new tokens than the cache holds, and an empty sequence
    (2, 2, 500, 7, 64, [5, 1000]),       # a sequence shorter than the new tokens; a length past the end
    (5, 2, 384, 129, 16, [384, 383, 130, 129, 256]),
    (1, 2, 1000, 1000, 128, [999]),
    (4, 4, 5000, 4800, 64, [5000, 4990, 3001, 17]),   # prompts: the kernel of many tiles
    (4, 4, 4999, 4999, 16, None),
    (5, 4, 4900, 4700, 128, [4900, 4899, 0, 4701, 1]),
]


@pytest.mark.parametrize("case", STORES, ids=lambda c: "-".join(map(str, c[:5])))
def test_store_and_bounds(cuda_device, case):
    import torch
    import exact_io_aware_44_b200 as fa
    B, H, Nk, n_new, block, lens = case
    rng = np.random.default_rng(Nk * 7 + n_new)
    ck, cv, ks, vs = make_cache(rng, B, H, Nk, block, True, cuda_device)
    k, v = rnd(rng, B, H, n_new, D, std=3.0), rnd(rng, B, H, n_new, D, std=0.01)
    bounds = fa.block_bounds(ck, block, lens=None if lens is None else dev_lens([max(n - n_new, 0) for n in
                             cache64.clamp_lens(lens, B, Nk)], cuda_device))
    ref = [cache64.store64(f64(x), f64(c), f64(s), block, lens) for x, c, s in ((k, ck, ks), (v, cv, vs))]
    ld = dev_lens(lens, cuda_device)
    for _ in range(2):  # the same tokens again change nothing
        fa.cache_store(k.to(cuda_device), v.to(cuda_device), ck, cv, ks, vs, block, lens=ld)
        assert fa.get_status() == 0
        for got, want in zip((ck, ks, cv, vs), ref[0] + ref[1]):
            assert np.array_equal(f64(got), want)
    fa.block_bounds(ck, block, lens=ld, n_new=n_new, bounds=bounds)
    assert np.array_equal(f64(bounds), cache64.bounds64(f64(ck), block, lens))


def test_store_token_by_token_keeps_every_value_within_half_a_step(cuda_device):
    """Tokens of growing size appended one at a time: scales grow under older codes, which
    stay within E4M3's rounding of the block's final scale (two roundings at most: once as
    stored, once as subnormal of a larger scale)."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(5)
    B, H, Nk, block = 2, 2, 100, 32
    size = torch.from_numpy(np.exp2(rng.integers(-12, 12, (B, H, Nk, 1))).astype(np.float32))
    k = (rnd(rng, B, H, Nk, D).float() * size).bfloat16()
    ck, cv = (torch.zeros(B, H, Nk, D, dtype=torch.float8_e4m3fn, device=cuda_device) for _ in range(2))
    ks, vs = (torch.full((B, H, 4), 1e30, device=cuda_device) for _ in range(2))   # garbage: a first token sets it
    kd = k.to(cuda_device)
    for n in range(1, Nk + 1):
        x = kd[:, :, n - 1:n].contiguous()
        fa.cache_store(x, x, ck, cv, ks, vs, block, lens=dev_lens([n] * B, cuda_device))
    got = cache64.dequantised(f64(ck), f64(ks), block)
    amax = np.stack([np.abs(f64(k))[:, :, j * block:(j + 1) * block].max((2, 3)) for j in range(4)], -1)
    want = np.vectorize(cache64.scale_for)(amax)
    assert np.array_equal(f64(ks), want) and torch.equal(ck.view(torch.uint8), cv.view(torch.uint8))
    s = np.repeat(want, block, 2)[:, :, :Nk, None]
    assert (np.abs(got - f64(k)) <= 2.0 ** -4 * np.abs(f64(k)) + 2.0 ** -9 * s).all()


def test_store_of_values_that_are_not_finite(cuda_device):
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(6)
    k = rnd(rng, 1, 1, 20, D)
    k[0, 0, 3, 5], k[0, 0, 4, 6], k[0, 0, 5, 7] = float("inf"), float("-inf"), float("nan")
    k[0, 0, 16:] = 0
    ck, cv, ks, vs = make_cache(rng, 1, 1, 20, 16, True, cuda_device)
    ref = cache64.store64(f64(k), f64(ck), f64(ks), 16, None)
    kd = k.to(cuda_device)
    fa.cache_store(kd, kd, ck, cv, ks, vs, 16)
    assert np.array_equal(f64(ck), ref[0], equal_nan=True) and np.array_equal(f64(ks), ref[1])
    assert f64(ks)[0, 0, 1] == 2.0 ** -100 and np.isfinite(f64(ks)).all()
    b = fa.block_bounds(ck, 16)
    assert np.array_equal(f64(b), cache64.bounds64(f64(ck), 16, None))


@pytest.mark.parametrize("block", [16, 64, 128])
def test_store_into_scales_that_are_not_powers_of_two(cuda_device, block):
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(7 + block)
    ck, cv, ks, vs = make_cache(rng, 2, 2, 150, block, True, cuda_device, pow2=False)
    k = rnd(rng, 2, 2, 3, D)
    old_k, old_s = f64(ck), ks.clone()
    fa.cache_store(k.to(cuda_device), k.to(cuda_device), ck, cv, ks, vs, block, lens=dev_lens([150, 70], cuda_device))
    _, want = cache64.store64(f64(k), old_k, f64(old_s), block, [150, 70])
    assert np.array_equal(f64(ks), want)
    for b, n in enumerate((150, 70)):
        for h in range(2):
            s = np.repeat(want[b, h], block)[n - 3:n, None]
            x = (f64(k)[b, h].astype(np.float32) / s.astype(np.float32)).astype(np.float64)
            assert np.array_equal(f64(ck)[b, h, n - 3:n], cache64.e4m3_round(x))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
def test_bounds(cuda_device, fp8, block):
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(block + fp8)
    lens = [300, 0, 1, 129]
    k, _, _, _ = make_cache(rng, 4, 2, 300, block, fp8, cuda_device)
    poison(k, lens)
    got = fa.block_bounds(k, block, lens=dev_lens(lens, cuda_device))
    assert np.array_equal(f64(got), cache64.bounds64(f64(k), block, lens))
    part = torch.zeros_like(got)
    part.view(torch.uint8).fill_(0x11)
    before = f64(part)
    fa.block_bounds(k, block, lens=dev_lens(lens, cuda_device), n_new=2, bounds=part)
    want = cache64.bounds64(f64(k), block, lens)
    for b, n in enumerate(lens):
        for j in range(want.shape[2]):
            fresh = n > 0 and max(n - 2, 0) // block <= j <= (n - 1) // block
            assert np.array_equal(f64(part)[b, :, j], want[b, :, j] if fresh else before[b, :, j])


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("Nk", [5003, 12001])
def test_bounds_of_many_tokens(cuda_device, fp8, block, Nk):
    """Caches of which a warp takes 32 and 64 tokens at a time, whole and behind a long append."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(Nk + block + fp8)
    B, H, n_new = 5, 8, Nk - 900
    lens = [Nk, 0, 1, Nk - 77, 4097]
    k, _, _, _ = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    poison(k, lens)
    want = cache64.bounds64(f64(k), block, lens)
    got = fa.block_bounds(k, block, lens=dev_lens(lens, cuda_device))
    assert np.array_equal(f64(got), want)
    part = torch.ones_like(got, dtype=torch.float32).to(got.dtype)
    fa.block_bounds(k, block, lens=dev_lens(lens, cuda_device), n_new=n_new, bounds=part)
    for b, n in enumerate(lens):
        first, end = max(n - n_new, 0) // block, -(-n // block)
        assert np.array_equal(f64(part)[b, :, first:end], want[b, :, first:end])
        assert (f64(part)[b, :, :first] == 1).all() and (f64(part)[b, :, end:] == 1).all()


# --------------------------------------------------------------------------------------------- attention

ATTENDS = [
    # B, Hq, Hkv, Nq, Nk, block, lens
    (1, 1, 1, 1, 1, 16, None),
    (1, 8, 1, 1, 127, 16, None),
    (1, 8, 2, 1, 129, 32, None),
    (2, 8, 2, 1, 1000, 64, [1000, 3]),
    (4, 6, 2, 3, 700, 128, [700, 0, 2, 257]),      # an empty sequence, and one shorter than the queries
    (2, 16, 1, 1, 3000, 64, [2999, 128]),          # 16 rows a group
    (3, 24, 8, 5, 501, 16, [501, 250, 1]),         # 15 rows
    (2, 32, 4, 4, 900, 64, None),                  # 32 rows
    (1, 8, 1, 5, 900, 32, None),                   # 40 rows
    (1, 64, 1, 1, 640, 128, None),                 # a 64-head group
    (1, 4, 1, 40, 333, 64, [300]),                 # 160 rows, the causal edge spans 40 keys
    (5, 8, 2, 1, 4000, 64, [4000, 17, 2222, 1, 3999]),
    (40, 4, 4, 1, 260, 64, None),                  # many short sequences
    (5, 12, 2, 2, 600, 16, [600, -7, 599, 5000, 16]),   # lengths outside the cache count as the nearer end
    (70, 2, 1, 1, 300, 32, [300 - 4 * i for i in range(70)]),  # more sequences than a warp has lanes
    (3, 16, 4, 4, 1300, 64, [1, 1300, 1]),         # one-token sequences beside a long one
    (1, 1, 1, 17, 17, 16, None),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", ATTENDS, ids=lambda c: "-".join(map(str, c[:6])))
def test_decode_fp8(cuda_device, case, causal):
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nq, Nk, block, lens = case
    rng = np.random.default_rng(Nk + 13 * Nq + Hq)
    q = rnd(rng, B, Hq, Nq, D)
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, True, cuda_device, pow2=Nk % 2 == 0)
    poison(k, lens), poison(v, lens), poison_scales(ks, block, lens), poison_scales(vs, block, lens)
    scale = 1 / math.sqrt(D)
    ref = cache64.attend64(f64(q), real(k, ks, block, lens), real(v, vs, block, lens), scale, causal, lens)
    qd = q.to(cuda_device)
    for splits in (0, 1, 3):
        o, lse = fa.decode_fp8(qd, k, v, ks, vs, block, lens=dev_lens(lens, cuda_device), causal=causal,
                               num_splits=splits)
        assert fa.get_status() == 0
        check_attend(o, lse, ref, f"{case} splits={splits}")


def test_decode_fp8_scales_far_apart_and_growing_scores(cuda_device):
    """Blocks whose value scales differ by 2^20, and scores that grow along the cache, so that
    the running reference is raised again and again; queries of very different size."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(12)
    B, Hq, H, Nq, Nk, block = 2, 8, 2, 2, 2500, 16
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, True, cuda_device)
    nb = ks.shape[2]
    ks *= torch.linspace(0.05, 2.0, nb, device=cuda_device)
    vs *= torch.from_numpy(np.exp2(rng.integers(-10, 11, (B, H, nb))).astype(np.float32)).to(cuda_device)
    q = rnd(rng, B, Hq, Nq, D).float().abs()
    q *= torch.from_numpy(np.exp2(rng.integers(-6, 1, (B, Hq, Nq, 1))).astype(np.float32))
    q = q.bfloat16()
    ref = cache64.attend64(f64(q), real(k, ks, block, None), real(v, vs, block, None), 0.05, True, None)
    for splits in (0, 1, 7):
        o, lse = fa.decode_fp8(q.to(cuda_device), k, v, ks, vs, block, scale=0.05, num_splits=splits)
        check_attend(o, lse, ref, f"splits={splits}")


def test_decode_fp8_many_weak_keys_beside_a_strong_one(cuda_device):
    """One key far above 20000 others that hold a tenth of the weight together: none of it is
    lost to a narrow format."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(13)
    Nk, block = 20001, 64
    q = torch.ones(1, 4, 1, D).bfloat16()
    k = torch.zeros(1, 1, Nk, D)
    k[0, 0, 7777] = 1.0
    v = torch.ones(1, 1, Nk, D)
    v[0, 0, 7777] = -0.5
    scale = math.log(2e5) / D          # the strong key's weight is 2e5, the others' 1 each
    c = lambda t: t.to(torch.float8_e4m3fn).to(cuda_device)
    one = torch.ones(1, 1, -(-Nk // block), device=cuda_device)
    ref = cache64.attend64(f64(q), k.double().numpy(), v.double().numpy(), scale, True, None)
    for splits in (0, 1):
        o, lse = fa.decode_fp8(q.to(cuda_device), c(k), c(v), one, one, block, scale=scale, num_splits=splits)
        check_attend(o, lse, ref, f"splits={splits}")


def test_decode_fp8_repeats_bit_for_bit_and_writes_only_its_outputs(cuda_device):
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(14)
    B, Hq, H, Nq, Nk, block = 3, 12, 2, 1, 1500, 64
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, True, cuda_device)
    q = rnd(rng, B, Hq, Nq, D).to(cuda_device)
    n = q.numel()
    o_buf = torch.full((n + 4096,), 7.0, dtype=torch.bfloat16, device=cuda_device)
    l_buf = torch.full((B * Hq + 28 + 512,), 7.0, device=cuda_device)
    ws = torch.full((fa.decode_fp8_workspace_bytes(B, Hq, H, Nq, Nk, D, block),), 0xFF, dtype=torch.uint8,
                    device=cuda_device)
    lens = dev_lens([1500, 0, 77], cuda_device)
    o, lse = fa.decode_fp8(q, k, v, ks, vs, block, lens=lens, out=o_buf[:n].view_as(q),
                           lse=l_buf[:B * Hq].view(B, Hq, 1), workspace=ws)
    o2, lse2 = fa.decode_fp8(q, k, v, ks, vs, block, lens=lens)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (o_buf[n:] == 7).all() and (l_buf[B * Hq:] == 7).all()


# --------------------------------------------------------------------------------------------- selected blocks

SELECTS = [
    # B, Hq, Hkv, Nq, Nk, block, n_select, n_first, n_last, lens
    (1, 1, 1, 1, 1, 16, 1, 0, 1, None),
    (2, 8, 2, 1, 1000, 16, 8, 1, 1, [1000, 31]),
    (3, 12, 2, 3, 700, 32, 5, 1, 2, [700, 0, 2]),
    (1, 40, 2, 2, 640, 64, 3, 0, 0, None),          # 20 heads a group
    (2, 4, 4, 1, 9000, 16, 100, 2, 3, [9000, 4500]),  # 563 blocks
    (1, 4, 1, 1, 200, 128, 8, 1, 1, None),          # fewer blocks than the list
    (1, 3, 1, 2, 66000, 16, 1000, 1, 1, [65999]),   # 4125 blocks
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("case", SELECTS, ids=lambda c: "-".join(map(str, c[:9])))
def test_select_blocks(cuda_device, case, fp8, causal):
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nq, Nk, block, n_select, n_first, n_last, lens = case
    rng = np.random.default_rng(Nk + n_select)
    q = rnd(rng, B, Hq, Nq, D)
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    ld = dev_lens(lens, cuda_device)
    bounds = fa.block_bounds(k, block, lens=ld)
    # equal blocks: ties go to the lower index
    nb = bounds.shape[2]
    if nb > 6:
        bounds.view(torch.uint8)[:, :, 5] = bounds.view(torch.uint8)[:, :, 2]
        bounds.view(torch.uint8)[:, :, nb - 2] = bounds.view(torch.uint8)[:, :, 2]
        if fp8:
            ks[:, :, 5] = ks[:, :, nb - 2] = ks[:, :, 2]
    want = cache64.select64(f64(q), f64(bounds), f64(ks) if fp8 else None, n_select, block, Nk, lens, n_first, n_last,
                            causal)
    got = fa.select_blocks(q.to(cuda_device), bounds, n_select, block, Nk, k_scale=ks, lens=ld, n_first=n_first,
                           n_last=n_last, causal=causal)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n_select", [1, 2, 700, 2047, 2048, 2049, 4999, 5000, 5001])
def test_select_blocks_thousands_of_ties(cuda_device, n_select):
    """5000 blocks with two scores between them: the larger all first, then the lowest indices."""
    import torch
    import exact_io_aware_44_b200 as fa
    bounds = torch.zeros(1, 1, 5000, 2, D, dtype=torch.bfloat16, device=cuda_device)
    high = np.random.default_rng(n_select).permutation(5000)[:700]
    bounds[0, 0, torch.from_numpy(high).to(cuda_device)] = 1.0
    q = torch.ones(1, 1, 1, D, dtype=torch.bfloat16, device=cuda_device)
    got = fa.select_blocks(q, bounds, n_select, 16, 80000, n_first=0, n_last=0)[0, 0, 0].cpu().numpy()
    order = np.concatenate([np.sort(high), np.setdiff1d(np.arange(5000), high)])
    want = np.concatenate([np.sort(order[:n_select]), np.full(max(0, n_select - 5000), -1)])
    assert np.array_equal(got, want)


def test_select_blocks_all_equal_and_not_finite(cuda_device):
    """Bounds of zero: every score ties, the lowest indices win. NaN scores come last."""
    import torch
    import exact_io_aware_44_b200 as fa
    bounds = torch.zeros(1, 1, 50, 2, D, dtype=torch.bfloat16, device=cuda_device)
    q = torch.ones(1, 2, 1, D, dtype=torch.bfloat16, device=cuda_device)
    got = fa.select_blocks(q, bounds, 6, 16, 800, n_first=0, n_last=1)
    assert got[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 49]
    bounds[0, 0, :3] = float("nan")
    bounds[0, 0, 7] = float("inf")
    got = fa.select_blocks(q, bounds, 6, 16, 800, n_first=0, n_last=0)
    assert got[0, 0, 0].tolist() == [3, 4, 5, 6, 7, 8]


@pytest.mark.parametrize("g", [1, 4, 8, 9, 20])
@pytest.mark.parametrize("codes", ["all", "subnormal", "nan"])
@pytest.mark.parametrize("exponent", [-100, 0, 100])
def test_select_blocks_by_every_8_bit_code(cuda_device, g, codes, exponent):
    """Bounds over all codes, over the subnormal ones alone, and with a NaN in every seventh block
    (which then comes last), against queries near both ends of their range."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(g + 100 + exponent)
    nb, Nq, n_select = 333, 2, 40
    c = rng.integers(0, 8 if codes == "subnormal" else 0x7F, (1, 1, nb, 2, D), dtype=np.uint8)
    c |= rng.integers(0, 2, c.shape, dtype=np.uint8) << 7
    b = torch.from_numpy(c).view(torch.float8_e4m3fn)
    b = torch.stack([b.float().amin(3), b.float().amax(3)], 3).to(torch.float8_e4m3fn)
    if codes == "nan":
        for j in range(0, nb, 7):
            b.view(torch.uint8)[0, 0, j, j % 2, rng.integers(D)] = 0x7F | (j % 3 == 0) << 7
    q = (torch.from_numpy(rng.standard_normal((1, g, Nq, D), dtype=np.float32)) * 2.0 ** exponent).bfloat16()
    ks = torch.from_numpy(np.exp2(rng.integers(-2, 2, (1, 1, nb))).astype(np.float32))
    got = fa.select_blocks(q.to(cuda_device), b.to(cuda_device), n_select, 16, nb * 16, k_scale=ks.to(cuda_device),
                           n_first=0, n_last=0)
    want = cache64.select64(f64(q), f64(b), f64(ks), n_select, 16, nb * 16, None, 0, 0)
    assert np.array_equal(got.cpu().numpy(), want)


LISTS = [
    # B, Hq, Hkv, Nq, Nk, block, n_select, lens
    (1, 1, 1, 1, 1, 16, 1, None),
    (2, 8, 2, 1, 1000, 16, 9, [1000, 40]),
    (3, 12, 2, 3, 701, 32, 5, [701, 0, 2]),
    (1, 32, 1, 2, 640, 64, 4, None),                 # 32 heads a group
    (1, 40, 1, 1, 640, 128, 3, [600]),               # 40 heads a group
    (2, 16, 2, 4, 3000, 64, 20, [3000, 1111]),
    (16, 8, 2, 1, 500, 128, 2, None),
    (5, 4, 1, 1, 2000, 16, 100, [2000, 16, 1, 0, 777]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("case", LISTS, ids=lambda c: "-".join(map(str, c[:7])))
def test_decode_blocks(cuda_device, case, fp8, causal):
    """Lists in any order, with entries of -1 and past the cache (skipped) and one that is listed
    twice (counts twice); NaN behind the sequences' ends."""
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nq, Nk, block, n_select, lens = case
    rng = np.random.default_rng(Nk + n_select + Nq)
    q = rnd(rng, B, Hq, Nq, D)
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    poison(k, lens), poison(v, lens), poison_scales(ks, block, lens), poison_scales(vs, block, lens)
    nb = -(-Nk // block)
    idx = np.stack([rng.permutation(max(nb, n_select))[:n_select] for _ in range(B * H * Nq)])
    idx = idx.reshape(B, H, Nq, n_select)
    if n_select > 3:
        idx[..., 1], idx[..., 2] = -1, nb + 5
        idx[..., 3] = idx[..., 0]
    scale = 1 / math.sqrt(D)
    ref = cache64.attend64(f64(q), real(k, ks, block, lens), real(v, vs, block, lens), scale, causal, lens, idx, block)
    di = torch.from_numpy(idx.astype(np.int32)).to(cuda_device)
    for splits in (0, 1, 2):
        o, lse = fa.decode_blocks(q.to(cuda_device), k, v, di, block, k_scale=ks, v_scale=vs,
                                  lens=dev_lens(lens, cuda_device), causal=causal, num_splits=splits)
        assert fa.get_status() == 0
        check_attend(o, lse, ref, f"{case} fp8={fp8} splits={splits}")


def test_decode_blocks_with_nothing_listed(cuda_device):
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(15)
    k, v, _, _ = make_cache(rng, 2, 2, 256, 64, False, cuda_device)
    idx = torch.full((2, 2, 1, 3), -1, dtype=torch.int32, device=cuda_device)
    o, lse = fa.decode_blocks(rnd(rng, 2, 4, 1, D).to(cuda_device), k, v, idx, 64)
    assert (o == 0).all() and torch.isneginf(lse).all()


def test_decode_blocks_of_the_whole_cache_is_decode(cuda_device):
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(16)
    k, v, _, _ = make_cache(rng, 2, 2, 640, 64, False, cuda_device)
    q = rnd(rng, 2, 8, 1, D).to(cuda_device)
    idx = torch.arange(10, dtype=torch.int32, device=cuda_device).expand(2, 2, 1, 10).contiguous()
    o, lse = fa.decode_blocks(q, k, v, idx, 64)
    o2, lse2 = fa.decode(q, k, v)
    # both are within 2^-8 |o| + 2^-8 sum p |v| of the exact result
    assert (o.float() - o2.float()).abs().max() <= 4 * 2.0 ** -8 * v.float().abs().max()
    assert (lse - lse2).abs().max() <= 1e-4


# --------------------------------------------------------------------------------------------- weights

WEIGHTS = [
    # B, Hq, Hkv, Nq, Nk, block, lens
    (1, 1, 1, 1, 1, 16, None),
    (2, 8, 2, 1, 1000, 64, [1000, 40]),
    (3, 6, 2, 3, 301, 32, [301, 0, 2]),
    (1, 32, 1, 1, 640, 128, None),
    (1, 8, 1, 5, 400, 16, None),           # 40 rows
    (1, 4, 2, 130, 130, 64, None),         # a whole prompt
    (2, 3, 1, 77, 333, 64, [333, 200]),    # the end of a prompt behind a cached prefix
    (1, 2, 2, 300, 300, 128, [250]),       # queries whose position is before the sequence
    (12, 8, 8, 1, 2000, 64, None),
    (1, 40, 1, 1, 700, 64, [650]),         # 40 heads, one query
    (1, 36, 2, 7, 900, 16, [900]),         # 126 rows of heads with 7 queries each
    (2, 2, 1, 200, 600, 32, [600, 201]),   # rows of two heads in one tile
    (34, 2, 1, 2, 700, 64, [700 - 20 * i for i in range(34)]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: "-".join(map(str, c[:6])))
def test_cache_weights(cuda_device, case, fp8, causal):
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nq, Nk, block, lens = case
    rng = np.random.default_rng(Nk + Nq + fp8)
    q = rnd(rng, B, Hq, Nq, D)
    k, _, ks, _ = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    poison(k, lens), poison_scales(ks, block, lens)
    scale = 1 / math.sqrt(D)
    kr = real(k, ks, block, lens)
    _, lse, _, _ = cache64.attend64(f64(q), kr, kr, scale, causal, lens)
    lse = torch.from_numpy(lse.astype(np.float32))
    lse[:, 0, 0] = float("-inf")           # a row that adds nothing
    acc0 = torch.from_numpy(rng.uniform(0, 1, (B, H, Nk)).astype(np.float32))
    acc = acc0.to(cuda_device)
    add, size = cache64.weights64(f64(q), kr, f64(lse), scale, causal, lens)
    out = fa.cache_weights(q.to(cuda_device), k, lse.to(cuda_device), acc, k_scale=ks, block=block,
                           lens=dev_lens(lens, cuda_device), causal=causal)
    assert fa.get_status() == 0 and out is acc
    want = f64(acc0) + add
    big = float(np.abs(f64(lse)[np.isfinite(f64(lse))]).max()) if np.isfinite(f64(lse)).any() else 0.0
    rel = size * (2.0 ** -17 + 2.0 ** -22) + 2.0 ** -22 * (big + 4) + 2.0 ** -22
    rows = Hq // H * Nq
    tol = rel * add + 2.0 ** -23 * min(rows, 64) * want + 1e-30
    err = np.abs(f64(acc) - want)
    assert (err <= tol).all(), float((err / tol).max())
    for b, n in enumerate(cache64.clamp_lens(lens, B, Nk)):
        assert np.array_equal(f64(acc)[b, :, n:], f64(acc0)[b, :, n:])


@pytest.mark.parametrize("Nq", [1, 5, 200])
@pytest.mark.parametrize("fp8", [True, False])
def test_cache_weights_rows_that_add_nothing_may_hold_anything(cuda_device, fp8, Nq):
    """Padded queries: lse = -inf, NaN and infinity in q. The other rows' sums do not change by a bit."""
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nk, block = 2, 8, 2, 700, 64
    lens = [700, 333]
    rng = np.random.default_rng(Nq + fp8)
    q = rnd(rng, B, Hq, Nq, D)
    k, _, ks, _ = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    lse = torch.full((B, Hq, Nq), 6.0)
    lse[0, 1], lse[1, 4:], lse[0, 6, -1] = float("-inf"), float("-inf"), float("-inf")
    bad = q.clone()
    bad[0, 1], bad[1, 4:], bad[0, 6, -1] = float("nan"), float("inf"), float("nan")
    out = []
    for x in (q, bad):
        acc = torch.zeros(B, H, Nk, device=cuda_device)
        fa.cache_weights(x.to(cuda_device), k, lse.to(cuda_device), acc, k_scale=ks, block=block,
                         lens=dev_lens(lens, cuda_device))
        assert fa.get_status() == 0
        out.append(f64(acc))
    assert np.isfinite(out[0]).all() and (out[0][0, 0, :600] > 0).all()
    assert np.array_equal(out[0], out[1])


@pytest.mark.parametrize("fp8", [True, False])
def test_queries_that_see_no_key_may_hold_anything(cuda_device, fp8):
    """Queries in front of the sequence's first token hold NaN; the others' results do not change by a bit."""
    import torch
    import exact_io_aware_44_b200 as fa
    B, Hq, H, Nq, Nk, block = 3, 6, 2, 5, 300, 32
    lens = dev_lens([300, 3, 0], cuda_device)
    rng = np.random.default_rng(77 + fp8)
    q = rnd(rng, B, Hq, Nq, D)
    bad = q.clone()
    bad[1, :, :2], bad[2] = float("nan"), float("inf")
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    idx = torch.arange(10, dtype=torch.int32).expand(B, H, Nq, 10).contiguous().to(cuda_device)
    bounds = fa.block_bounds(k, block, lens)
    got = []
    for x in (q.to(cuda_device), bad.to(cuda_device)):
        got.append(list(fa.decode_blocks(x, k, v, idx, block, ks, vs, lens)))
        if fp8:
            got[-1] += fa.decode_fp8(x, k, v, ks, vs, block, lens)
        got[-1].append(fa.select_blocks(x, bounds, 4, block, Nk, ks, lens))
        assert fa.get_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[1][0][1, :, :2] == 0).all() and torch.isneginf(got[1][1][1, :, :2]).all()
    assert torch.isfinite(got[1][0].float()).all()


# --------------------------------------------------------------------------------------------- eviction

EVICTS = [
    # B, Hkv, Nk, keep, recent, block, lens, capacity of the new cache
    (1, 1, 1, 1, 0, 16, None, 1),
    (2, 2, 300, 50, 10, 16, [300, 40], 300),
    (3, 1, 500, 77, 77, 32, [500, 0, 78], 90),
    (2, 2, 1000, 333, 0, 64, None, 400),
    (1, 3, 200, 300, 5, 128, None, 200),         # keeps everything
    (2, 1, 5000, 1000, 100, 64, [5000, 1001], 1000),
    (1, 1, 40000, 129, 1, 128, None, 129),
    (1, 2, 50001, 5000, 33, 16, [50001], 5003),  # more keys than shared memory holds, rows that are not whole float4s
    (1, 1, 45000, 44000, 7, 64, None, 44000),
    (3, 2, 2503, 640, 64, 32, [2503, 700, 639], 2503),
]


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("case", EVICTS, ids=lambda c: "-".join(map(str, c[:6])))
def test_cache_evict(cuda_device, case, fp8):
    import torch
    import exact_io_aware_44_b200 as fa
    B, H, Nk, keep, recent, block, lens, cap = case
    rng = np.random.default_rng(Nk + keep + fp8)
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, fp8, cuda_device)
    acc = rng.uniform(0, 1, (B, H, Nk)).astype(np.float32)
    acc = np.round(acc * 40) / 40 if Nk > 100 else acc                      # many ties
    acc[rng.uniform(size=acc.shape) < 0.02] = np.nan
    acc[rng.uniform(size=acc.shape) < 0.02] = np.inf
    acc[rng.uniform(size=acc.shape) < 0.02] = -0.0
    acc = torch.from_numpy(acc).to(cuda_device)
    nb = -(-cap // block)
    out = [torch.empty(B, H, cap, D, dtype=k.dtype, device=cuda_device) for _ in range(2)]
    for t in out:
        t.view(torch.uint8).fill_(0x22)
    out += [torch.full((B, H, cap), 5.0, device=cuda_device),
            torch.empty(B, H, keep, dtype=torch.int32, device=cuda_device),
            torch.empty(B, dtype=torch.int32, device=cuda_device)]
    if fp8:
        out += [torch.full((B, H, nb), 5.0, device=cuda_device) for _ in range(2)]
    before = [f64(t) for t in out]
    got = fa.cache_evict(k, v, acc, keep, recent, k_scale=ks, v_scale=vs, block=block, lens=dev_lens(lens, cuda_device),
                         out=out)
    assert fa.get_status() == 0
    idx, new = cache64.evict64(f64(acc), keep, recent, lens)
    assert np.array_equal(got[3].cpu().numpy(), idx) and got[4].tolist() == new
    for b, m in enumerate(new):
        for h in range(H):
            at = idx[b, h, :m]
            assert np.array_equal(f64(got[2])[b, h, :m], f64(acc)[b, h, at], equal_nan=True)
            assert np.array_equal(f64(got[2])[b, h, m:], before[2][b, h, m:])
            for t, (src, s) in enumerate(((k, ks), (v, vs))):
                rows = f64(src)[b, h, at]
                if fp8:
                    of = f64(s)[b, h, at // block]
                    want = before[5 + t][b, h].copy()
                    for j in range(-(-m // block)):
                        want[j] = of[j * block:(j + 1) * block].max()
                    assert np.array_equal(f64(got[5 + t])[b, h], want)
                    rows = cache64.e4m3_round(rows * (of / np.repeat(want, block)[:m])[:, None])
                assert np.array_equal(f64(got[t])[b, h, :m], rows)
                assert np.array_equal(f64(got[t])[b, h, m:], before[t][b, h, m:])


# --------------------------------------------------------------------------------------------- together

def test_serving_loop_over_an_8_bit_cache(cuda_device):
    """Prompts stored, then decode steps (append, bounds, selection, attention, weights), an
    eviction in the middle, and steps on the new cache: each step against float64 on the
    cache's own values, on a stream of its own, with one workspace."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(21)
    B, Hq, H, Nk, block = 2, 8, 2, 512, 32
    dev, scale = cuda_device, 1 / math.sqrt(D)
    nb = Nk // block
    stream = torch.cuda.Stream(device=dev)
    stream.wait_stream(torch.cuda.current_stream())
    lens = [300, 211]
    kc, vc = (torch.zeros(B, H, Nk, D, dtype=torch.float8_e4m3fn, device=dev) for _ in range(2))
    ks, vs = (torch.ones(B, H, nb, device=dev) for _ in range(2))
    acc = torch.zeros(B, H, Nk, device=dev)
    n0 = max(lens)
    qp, kp, vp = rnd(rng, B, Hq, n0, D), rnd(rng, B, H, n0, D), rnd(rng, B, H, n0, D)
    with torch.cuda.stream(stream):
        ld = dev_lens(lens, dev)
        fa.cache_store(kp.to(dev), vp.to(dev), kc, vc, ks, vs, block, lens=ld)
        bounds = fa.block_bounds(kc, block, lens=ld)
        _, lse = fa.decode_fp8(qp.to(dev), kc, vc, ks, vs, block, lens=ld)
        fa.cache_weights(qp.to(dev), kc, lse, acc, k_scale=ks, block=block, lens=ld)
    want_acc = np.zeros((B, H, Nk))

    def values():
        return real(kc, ks, block, lens), real(vc, vs, block, lens)

    stream.synchronize()
    add, _ = cache64.weights64(f64(qp), values()[0], f64(lse), scale, True, lens)
    want_acc += add
    ws = torch.empty(max(fa.decode_blocks_workspace_bytes(True, B, Hq, H, 1, Nk, D, block, 6),
                         fa.select_blocks_workspace_bytes(B, Hq, H, 1, Nk, D, block)), dtype=torch.uint8, device=dev)
    for step in range(6):
        if step == 3:
            with torch.cuda.stream(stream):
                kc, vc, acc, idx, ld, ks, vs = fa.cache_evict(kc, vc, acc, 160, 32, k_scale=ks, v_scale=vs, block=block,
                                                              lens=dev_lens(lens, dev))
                bounds = fa.block_bounds(kc, block, lens=ld)
            stream.synchronize()
            lens = ld.tolist()
            assert lens == [160, 160]
            want_acc = np.stack([[np.concatenate([want_acc[b, h, idx[b, h].cpu().numpy()], np.zeros(Nk - 160)])
                                  for h in range(H)] for b in range(B)])
        lens = [n + 1 for n in lens]
        q, k, v = (rnd(rng, B, n, 1, D) for n in (Hq, H, H))
        with torch.cuda.stream(stream):
            qd, ld = q.to(dev), dev_lens(lens, dev)
            fa.cache_store(k.to(dev), v.to(dev), kc, vc, ks, vs, block, lens=ld)
            fa.block_bounds(kc, block, lens=ld, n_new=1, bounds=bounds)
            idx = fa.select_blocks(qd, bounds, 6, block, Nk, k_scale=ks, lens=ld, workspace=ws)
            o, lse = fa.decode_blocks(qd, kc, vc, idx, block, k_scale=ks, v_scale=vs, lens=ld, workspace=ws)
            of, lf = fa.decode_fp8(qd, kc, vc, ks, vs, block, lens=ld)
            fa.cache_weights(qd, kc, lf, acc, k_scale=ks, block=block, lens=ld)
        stream.synchronize()
        assert fa.get_status(stream) == 0
        kr, vr = values()
        assert np.array_equal(idx.cpu().numpy(),
                              cache64.select64(f64(q), cache64.bounds64(np.nan_to_num(f64(kc)), block, lens), f64(ks), 6,
                                               block, Nk, lens, 1, 1))
        check_attend(o, lse, cache64.attend64(f64(q), kr, vr, scale, True, lens, idx.cpu().numpy(), block), step)
        check_attend(of, lf, cache64.attend64(f64(q), kr, vr, scale, True, lens), step)
        add, _ = cache64.weights64(f64(q), kr, f64(lf), scale, True, lens)
        want_acc += add
        for b, n in enumerate(lens):
            assert np.allclose(f64(acc)[b, :, :n], want_acc[b, :, :n], rtol=1e-4, atol=1e-6)


@pytest.mark.parametrize("fp8", [True, False])
def test_decode_step_captured_and_replayed(cuda_device, fp8):
    """A whole step inside a CUDA graph: replays on new tokens and lengths copied into the captured
    buffers equal eager calls on copies of the same state."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(22 + fp8)
    dev, B, Hq, H, Nk, block, keep = cuda_device, 3, 12, 4, 700, 64, 200
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, fp8, dev)
    state = {"k": k, "v": v, "acc": torch.rand(B, H, Nk, device=dev), "q": rnd(rng, B, Hq, 2, D).to(dev),
             "nk": rnd(rng, B, H, 2, D).to(dev), "nv": rnd(rng, B, H, 2, D).to(dev),
             "lens": dev_lens([700, 2, 333], dev), "bounds": fa.block_bounds(k, block)}
    if fp8:
        state.update(ks=ks, vs=vs)
    nbytes = max(fa.decode_blocks_workspace_bytes(fp8, B, Hq, H, 2, Nk, D, block, 5),
                 fa.select_blocks_workspace_bytes(B, Hq, H, 2, Nk, D, block),
                 fa.decode_fp8_workspace_bytes(B, Hq, H, 2, Nk, D, block))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)

    def buffers():
        o = {"idx": torch.empty(B, H, 2, 5, dtype=torch.int32, device=dev), "o": torch.empty_like(state["q"]),
             "lse": torch.empty(B, Hq, 2, device=dev), "of": torch.empty_like(state["q"]),
             "lf": torch.empty(B, Hq, 2, device=dev),
             "ev": [torch.zeros_like(k), torch.zeros_like(v), torch.zeros(B, H, Nk, device=dev),
                    torch.empty(B, H, keep, dtype=torch.int32, device=dev), torch.empty(B, dtype=torch.int32, device=dev)]}
        if fp8:
            o["ev"] += [torch.ones_like(ks), torch.ones_like(vs)]
        return o

    def step(s, o):
        kw = dict(k_scale=s.get("ks"), lens=s["lens"])
        if fp8:
            fa.cache_store(s["nk"], s["nv"], s["k"], s["v"], s["ks"], s["vs"], block, lens=s["lens"])
        fa.block_bounds(s["k"], block, lens=s["lens"], n_new=2, bounds=s["bounds"])
        fa.select_blocks(s["q"], s["bounds"], 5, block, Nk, out=o["idx"], workspace=ws, **kw)
        fa.decode_blocks(s["q"], s["k"], s["v"], o["idx"], block, v_scale=s.get("vs"), out=o["o"], lse=o["lse"],
                         workspace=ws, **kw)
        if fp8:
            fa.decode_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], block, lens=s["lens"], out=o["of"], lse=o["lf"],
                          workspace=ws)
        fa.cache_weights(s["q"], s["k"], o["lse"], s["acc"], block=block, **kw)
        fa.cache_evict(s["k"], s["v"], s["acc"], keep, 20, v_scale=s.get("vs"), block=block, out=o["ev"], **kw)

    copy = lambda s: {n: t.clone() for n, t in s.items()}
    warm, out = copy(state), buffers()
    step(warm, out)
    assert fa.get_status() == 0
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream(device=dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        step(state, out)
    torch.cuda.current_stream().wait_stream(s)
    for lens in ([700, 2, 333], [64, 699, 1], [0, 128, 650]):
        state["lens"].copy_(dev_lens(lens, dev))
        state["q"].copy_(rnd(rng, B, Hq, 2, D).to(dev))
        state["nk"].copy_(rnd(rng, B, H, 2, D).to(dev))
        eager, eo = copy(state), buffers()
        for a, b in zip(eo["ev"], out["ev"]):
            a.copy_(b)
        g.replay()
        step(eager, eo)
        torch.cuda.synchronize()
        assert fa.get_status() == 0
        names = ["idx", "o", "lse"] + (["of", "lf"] if fp8 else [])
        pairs = [(out[n], eo[n]) for n in names] + list(zip(out["ev"], eo["ev"])) + [(state[n], eager[n]) for n in state]
        for a, b in pairs:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del g


def test_two_streams_at_once(cuda_device):
    """Calls in flight together on two streams, each with a workspace of its own."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(23)
    B, Hq, H, Nk, block = 4, 16, 4, 4000, 64
    k, v, ks, vs = make_cache(rng, B, H, Nk, block, True, cuda_device)
    q = [rnd(rng, B, Hq, 1, D).to(cuda_device) for _ in range(2)]
    want = [fa.decode_fp8(x, k, v, ks, vs, block) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=cuda_device) for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i in (0, 1):
            got[i].append(fa.decode_fp8(q[i], k, v, ks, vs, block, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_offsets_past_32_bits(cuda_device):
    """A cache of more than 2^32 bytes: the last head's keys lie past what 32 bits reach."""
    import torch
    import exact_io_aware_44_b200 as fa
    rng = np.random.default_rng(24)
    B, H, Nk, block = 1, 34, 1 << 20, 128           # 4.6 GB a tensor
    k = torch.zeros(B, H, Nk, D, dtype=torch.float8_e4m3fn, device=cuda_device)
    v = torch.zeros_like(k)
    s = torch.ones(B, H, Nk // block, device=cuda_device)
    tail = 300
    kt, vt = (torch.from_numpy(rng.standard_normal((tail, D), dtype=np.float32)).to(torch.float8_e4m3fn) for _ in range(2))
    k.view(torch.uint8)[0, -1, -tail:] = kt.view(torch.uint8).to(cuda_device)
    v.view(torch.uint8)[0, -1, -tail:] = vt.view(torch.uint8).to(cuda_device)
    q = rnd(rng, B, H, 1, D, std=4.0)
    n_sel = 4
    idx = torch.arange(Nk // block - n_sel, Nk // block, dtype=torch.int32, device=cuda_device)
    idx = idx.expand(B, H, 1, n_sel).contiguous()
    o, lse = fa.decode_blocks(q.to(cuda_device), k, v, idx, block, k_scale=s, v_scale=s)
    kk = np.zeros((1, 1, n_sel * block, D))
    vv = kk.copy()
    kk[0, 0, -tail:], vv[0, 0, -tail:] = f64(kt), f64(vt)
    ref = cache64.attend64(f64(q)[:, -1:], kk, vv, 1 / math.sqrt(D), True, None)
    check_attend(o[:, -1:], lse[:, -1:], ref, "selected")
    of, lf = fa.decode_fp8(q.to(cuda_device), k, v, s, s, block)
    full = math.log(math.exp(float(ref[1][0, 0, 0])) + Nk - n_sel * block)
    assert abs(float(lf[0, -1, 0]) - full) <= 2.0 ** -20 * (1 + full) + 1e-5
    acc = torch.zeros(B, H, Nk, device=cuda_device)
    fa.cache_weights(q.to(cuda_device), k, lf, acc, k_scale=s, block=block)
    assert abs(float(acc[0, -1].double().sum()) - 1) <= 1e-4
    new = rnd(rng, B, H, 1, D).to(cuda_device)
    fa.cache_store(new, new, k, v, s, s.clone(), block)
    assert np.array_equal(f64(k[0, -1, -1]), cache64.e4m3_round(f64(new)[0, -1, 0]))
    b = fa.block_bounds(k, block)
    assert np.array_equal(f64(b[0, -1, -1, 1]), f64(k[0, -1, -block:]).max(0))
    assert fa.get_status() == 0
