"""Refusals of the cache operators' Python entry points that name what is wrong, without a GPU."""
import pytest

import exact_io_aware_44_b200 as fa

D = 128


def caches(fp8, B=2, H=2, Nk=100, cap=40, keep=30, block=64):
    """A cache, its weights and scales, and an output tuple to evict into."""
    import torch
    dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k, v = (torch.zeros(B, H, Nk, D, dtype=dtype) for _ in range(2))
    s = [torch.ones(B, H, -(-Nk // block)) for _ in range(2)] if fp8 else [None, None]
    out = [torch.zeros(B, H, cap, D, dtype=dtype) for _ in range(2)]
    out += [torch.zeros(B, H, cap), torch.zeros(B, H, keep, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)]
    out += [torch.ones(B, H, -(-cap // block)) for _ in range(2)] if fp8 else []
    return k, v, torch.zeros(B, H, Nk), s, out


def evict(k, v, acc, s, out, lens=None):
    return fa.cache_evict(k, v, acc, 30, 5, k_scale=s[0], v_scale=s[1], lens=lens, out=out)


@pytest.mark.parametrize("fp8", [True, False])
def test_evict_refuses_outputs_that_overlap(fp8):
    import torch
    k, v, acc, s, out = caches(fp8)
    # a window into the cache that is cut, anywhere in it
    for src in (k, v):
        for at in (0, 16, k.numel() - out[0].numel()):
            bad = list(out)
            bad[1] = src.view(-1)[at:at + out[1].numel()].view(out[1].shape)
            with pytest.raises(ValueError, match="overlap"):
                evict(k, v, acc, s, bad)
    bad = list(out)
    bad[2] = acc.view(-1)[7:7 + out[2].numel()].view(out[2].shape)
    with pytest.raises(ValueError, match="overlap"):
        evict(k, v, acc, s, bad)
    # two outputs in one place
    bad = list(out)
    bad[1] = bad[0]
    with pytest.raises(ValueError, match="overlap"):
        evict(k, v, acc, s, bad)
    both = torch.zeros(2 * out[0].numel() - 16, dtype=out[0].dtype)
    bad[0], bad[1] = (both[at:at + out[0].numel()].view(out[0].shape) for at in (0, out[0].numel() - 16))
    with pytest.raises(ValueError, match="overlap"):
        evict(k, v, acc, s, bad)
    lens = torch.full((2,), 90, dtype=torch.int32)
    bad = list(out)
    bad[4] = lens
    with pytest.raises(ValueError, match="overlap"):
        evict(k, v, acc, s, bad, lens)


def test_evict_takes_inputs_and_outputs_side_by_side():
    """Neighbours in one buffer, and K and V that are the same, do not overlap: the call goes on to ask for a GPU."""
    import torch
    k, v, acc, s, out = caches(False)
    n, m = k.numel(), out[0].numel()
    buf = torch.zeros(n + 2 * m, dtype=torch.bfloat16)
    k = buf[m:m + n].view(k.shape)
    out[0], out[1] = buf[:m].view(out[0].shape), buf[m + n:].view(out[1].shape)
    with pytest.raises(ValueError, match="CUDA"):
        evict(k, k, acc, s, out)


def test_store_refuses_keys_and_values_in_one_place():
    """One tensor for both caches, or for both sets of scales, would be written twice at once."""
    import torch
    k, v, _, s, _ = caches(True)
    new = torch.zeros(2, 2, 1, D, dtype=torch.bfloat16)
    for args in ((k, k, *s), (k, v, s[0], s[0])):
        with pytest.raises(ValueError, match="same memory"):
            fa.cache_store(new, new, *args, 64)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_store(new, new, k, v, *s, 64)


def test_selection_names_the_counts_that_do_not_fit():
    """A list too short for the blocks that are always taken: the defaults take two."""
    import torch
    q = torch.zeros(2, 4, 1, D, dtype=torch.bfloat16)
    bounds = torch.zeros(2, 2, 7, 2, D, dtype=torch.bfloat16)
    for n_select, more in ((1, {}), (3, {"n_first": 2, "n_last": 2}), (4, {"n_first": -1}), (4, {"n_last": -2})):
        with pytest.raises(ValueError, match="n_first"):
            fa.select_blocks(q, bounds, n_select, 16, 100, **more)
    for n_select, more in ((1, {"n_last": 0}), (1, {"n_first": 0}), (2, {})):
        with pytest.raises(ValueError, match="CUDA"):
            fa.select_blocks(q, bounds, n_select, 16, 100, **more)


def test_counts_past_32_bits_are_refused():
    """The C entry points take 32-bit counts; a larger Python integer must not lose its upper bits on the way."""
    import torch
    big = 1 << 32
    q = torch.zeros(2, 4, 1, D, dtype=torch.bfloat16)
    k, v, acc, s, _ = caches(False)
    k8, v8, _, s8, _ = caches(True)
    bounds = torch.zeros(2, 2, 7, 2, D, dtype=torch.bfloat16)
    idx = torch.zeros(2, 2, 1, 3, dtype=torch.int32)
    calls = [
        lambda: fa.decode_fp8(q, k8, v8, *s8, 64, num_splits=big + 1),
        lambda: fa.decode_blocks(q, k, v, idx, 64, num_splits=big + 1),
        lambda: fa.block_bounds(k, 16, n_new=big + 1, bounds=bounds),
        lambda: fa.select_blocks(q, bounds, big + 1, 16, 100),
        lambda: fa.select_blocks(q, bounds, big + 9, 16, 100, n_first=big),
        lambda: fa.cache_evict(k, v, acc, big + 5),
        lambda: fa.cache_evict(k, v, acc, big + 5, big),
        lambda: fa.decode_fp8_workspace_bytes(big + 1, 4, 2, 1, 100, D, 64),
        lambda: fa.decode_fp8_workspace_bytes(1, 4, 2, 1, 100, D, 64, big),
        lambda: fa.select_blocks_workspace_bytes(1, 4, 2, 1, big + 100, D, 64),
        lambda: fa.decode_blocks_workspace_bytes(True, 1, 4, 2, 1, 100, D, 64, big + 2),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError, match="32 bits"):
            call()
            pytest.fail(f"call {i} was taken")
