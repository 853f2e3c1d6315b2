"""Refusals of the cache operators, without a GPU: the C entry points return a code before
any CUDA call, and the Python entry points raise on tensors that do not fit."""
import ctypes

import pytest

import exact_io_aware_44_b200 as fa

P = ctypes.c_void_p
OK = 0x1000


def ptr(x):
    return P(x) if x else None


def store(k=OK, v=OK, ck=OK, cv=OK, ks=OK, vs=OK, lens=0, B=1, Hkv=2, n_new=1, Nk=100, d=128, block=64):
    return fa.lib.fa_cache_store(ptr(k), ptr(v), ptr(ck), ptr(cv), ptr(ks), ptr(vs), ptr(lens), B, Hkv, n_new, Nk, d,
                                 block, None)


def attend(q=OK, k=OK, v=OK, ks=OK, vs=OK, o=OK, lse=OK, ws=OK, lens=0, B=1, Hq=4, Hkv=2, Nq=1, Nk=100, d=128, block=64,
           scale=0.1, splits=0):
    return fa.lib.fa_decode_fp8(ptr(q), ptr(k), ptr(v), ptr(ks), ptr(vs), ptr(o), ptr(lse), ptr(ws), ptr(lens), B, Hq, Hkv,
                                Nq, Nk, d, block, 1, scale, splits, None)


def blocks(q=OK, ks=OK, vs=OK, idx=OK, ws=OK, lens=0, fp8=1, n_select=4, block=64, scale=0.1, Hq=4, Hkv=2, d=128):
    return fa.lib.fa_decode_blocks(ptr(q), ptr(OK), ptr(OK), ptr(ks), ptr(vs), ptr(idx), ptr(OK), ptr(OK), ptr(ws),
                                   ptr(lens), fp8, 1, Hq, Hkv, 1, 100, d, block, n_select, 1, scale, 0, None)


def select(q=OK, bounds=OK, ks=OK, idx=OK, ws=OK, lens=0, fp8=1, n_select=4, n_first=1, n_last=1, block=64, Nq=1, d=128):
    return fa.lib.fa_select_blocks(ptr(q), ptr(bounds), ptr(ks), ptr(idx), ptr(ws), ptr(lens), fp8, 1, 4, 2, Nq, 100, d,
                                   block, n_select, n_first, n_last, 1, None)


def weights(q=OK, k=OK, ks=OK, lse=OK, acc=OK, lens=0, fp8=1, Hq=4, Hkv=2, block=64, scale=0.1, d=128):
    return fa.lib.fa_cache_weights(ptr(q), ptr(k), ptr(ks), ptr(lse), ptr(acc), ptr(lens), fp8, 1, Hq, Hkv, 1, 100, d,
                                   block, 1, scale, None)


def evict(k=OK, acc=OK, idx=OK, olens=OK, oks=OK, fp8=1, keep=10, recent=2, Nk=100, out_Nk=100, block=64, d=128):
    return fa.lib.fa_cache_evict(ptr(k), ptr(OK), ptr(OK), ptr(OK), ptr(acc), None, ptr(OK), ptr(OK), ptr(oks), ptr(OK),
                                 ptr(OK), ptr(idx), ptr(olens), fp8, 1, 2, Nk, d, block, keep, recent, out_Nk, None)


def bounds(k=OK, b=OK, lens=0, n_new=0, Nk=100, block=64, d=128):
    return fa.lib.fa_block_bounds(ptr(k), ptr(b), ptr(lens), 1, 1, 2, Nk, d, block, n_new, None)


@pytest.mark.parametrize("call", [store, attend, blocks, select, weights, evict, bounds])
def test_sizes_that_no_operator_takes(call):
    assert call(d=64) == -2
    assert call(block=48) == -2
    assert call(block=0) == -2
    assert call(block=256) == -2


def test_store_refusals():
    assert store(B=0) == -1 and store(Nk=0) == -1 and store(n_new=-1) == -1
    assert store(n_new=0, k=0) == 0
    assert store(ck=0) == -1 and store(ks=0) == -1
    assert store(k=0x1008) == -3 and store(lens=0x1002) == -3
    assert store(B=1 << 16, Hkv=1 << 10, Nk=1 << 10) == -2      # B * Hkv * Nk >= 2^31


def test_attention_refusals():
    assert attend(Hq=3) == -1 and attend(Nq=0) == -1 and attend(Nk=0) == -1
    assert attend(scale=0.0) == -1 and attend(scale=float("nan")) == -1 and attend(scale=float("inf")) == -1
    assert attend(ks=0) == -1 and attend(ws=0) == -1 and attend(o=0) == -1
    assert attend(q=0x1008) == -3 and attend(ws=0x1010) == -3 and attend(lens=0x1001) == -3 and attend(vs=0x1004) == -3
    assert fa.decode_fp8_workspace_bytes(1, 3, 2, 1, 100, 128, 64) == 0
    assert fa.decode_fp8_workspace_bytes(1, 4, 2, 1, 100, 128, 64) > 0
    assert blocks(idx=0) == -1 and blocks(n_select=0) == -1 and blocks(vs=0) == -1 and blocks(Hq=5) == -1
    assert blocks(idx=0x1004) == -3 and blocks(ws=0x1010) == -3
    assert blocks(scale=-1.0) == -1


def test_selection_refusals():
    assert select(n_select=0) == -1 and select(n_first=-1) == -1 and select(n_first=3, n_last=2) == -1
    assert select(ks=0) == -1 and select(Nq=0) == -1
    assert select(bounds=0x1004) == -3 and select(ws=0x1010) == -3 and select(idx=0x1004) == -3
    assert fa.select_blocks_workspace_bytes(2, 8, 2, 3, 1000, 128, 64) == 2 * 2 * 3 * 16 * 8


def test_weight_and_eviction_refusals():
    assert weights(Hq=5) == -1 and weights(scale=0.0) == -1 and weights(acc=0) == -1 and weights(ks=0) == -1
    assert weights(acc=0x1004) == -3 and weights(lens=0x1003) == -3
    assert evict(keep=0) == -1 and evict(recent=-1) == -1 and evict(recent=11) == -1
    assert evict(out_Nk=9) == -1                       # smaller than keep
    assert evict(keep=200, out_Nk=99) == -1            # smaller than the cache that is kept whole
    assert evict(oks=0) == -1 and evict(olens=0) == -1
    assert evict(acc=0x1004) == -3 and evict(olens=0x1001) == -3
    assert bounds(n_new=-1) == -1 and bounds(b=0) == -1 and bounds(k=0x1004) == -3


def test_well_formed_calls_reach_the_device_check():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these pointers must not be launched on")
    for call in (store, attend, blocks, select, weights, evict, bounds):
        assert call() == -6, call.__name__
    assert blocks(fp8=0, ks=0, vs=0) == -6 and weights(fp8=0, ks=0) == -6


def test_python_entry_points_check_their_tensors():
    import torch
    f8, bf = torch.float8_e4m3fn, torch.bfloat16
    B, Hq, H, Nk, d = 2, 4, 2, 100, 128
    q = torch.zeros(B, Hq, 1, d, dtype=bf)
    k8, kb = torch.zeros(B, H, Nk, d, dtype=f8), torch.zeros(B, H, Nk, d, dtype=bf)
    s = torch.ones(B, H, 2)
    new = torch.zeros(B, H, 1, d, dtype=bf)
    idx = torch.zeros(B, H, 1, 2, dtype=torch.int32)
    acc, lse = torch.zeros(B, H, Nk), torch.zeros(B, Hq, 1)
    bnd = torch.zeros(B, H, 2, 2, d, dtype=f8)
    bad = [
        lambda: fa.cache_store(new, new, kb, kb, s, s, 64),                       # a bf16 cache
        lambda: fa.cache_store(new.float(), new, k8, k8.clone(), s, s, 64),
        lambda: fa.cache_store(new, new, k8, k8.clone(), s[:, :, :1], s, 64),     # scales of another size
        lambda: fa.cache_store(new, new, k8, k8.clone(), s, s, 48),
        lambda: fa.decode_fp8(q, kb, kb, s, s, 64),
        lambda: fa.decode_fp8(q, k8, k8, s, s, 64, lens=torch.zeros(B)),          # lens not int32
        lambda: fa.decode_fp8(q, k8, k8, s, s, 64, lens=torch.zeros(3, dtype=torch.int32)),
        lambda: fa.decode_fp8(q.transpose(1, 2), k8, k8, s, s, 64),               # not contiguous
        lambda: fa.decode_fp8(q[:1], k8, k8, s, s, 64),
        lambda: fa.decode_blocks(q, k8, k8, idx, 64),                             # an 8-bit cache without scales
        lambda: fa.decode_blocks(q, kb, kb, idx, 64, k_scale=s, v_scale=s),       # a bf16 cache with scales
        lambda: fa.decode_blocks(q, kb, kb, idx.long(), 64),
        lambda: fa.select_blocks(q, bnd, 2, 64, Nk),                              # no k_scale
        lambda: fa.select_blocks(q, bnd, 2, 32, Nk, k_scale=s),                   # bounds of other blocks
        lambda: fa.cache_weights(q, kb, lse[:, :2], acc, block=64),
        lambda: fa.cache_weights(q, kb, lse, acc.double(), block=64),
        lambda: fa.cache_evict(kb, kb, acc, 0),
        lambda: fa.cache_evict(k8, k8, acc, 10),
        lambda: fa.cache_evict(kb, kb, acc, 10, out=[kb, kb, acc, idx, idx]),
        lambda: fa.block_bounds(k8, 64, n_new=1),
        lambda: fa.block_bounds(k8.transpose(1, 2), 64),
        # sound arguments, but on the CPU: there is no CPU path
        lambda: fa.decode_fp8(q, k8, k8.clone(), s, s, 64),
        lambda: fa.cache_weights(q, kb, lse, acc, block=64),
        lambda: fa.cache_evict(kb, kb.clone(), acc, 10),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError)):
            f()
            pytest.fail(f"call {i} was taken")


def test_listed_blocks_of_more_queries_than_row_distances_hold():
    assert fa.decode_blocks_workspace_bytes(1, 1, 1, 1, 1 << 24, 100, 128, 64, 1) == 0
    assert fa.decode_blocks_workspace_bytes(1, 1, 1, 1, (1 << 24) - 1, 100, 128, 64, 1) > 0
