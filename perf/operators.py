"""Cases of the cache operators: storing into an 8-bit cache, attention over it, sparse attention over selected
blocks, accumulated attention weights, and eviction. `run` computes them in plain torch operations, or through this
package's entry points where `own` is true.

Layouts: q [B, Hq, Nq, d] bf16; caches [B, Hkv, Nk, d] in bf16 or E4M3; scales [B, Hkv, ceil(Nk / block)] float32, one
per block of tokens and head; lens [B] int32, the tokens that each sequence holds (the Nq newest are the queries' own).
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
DEV = "cuda"
D = 128


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def _store(name, B, Hkv, Nk, n_new, block, ragged):
    return {"name": name, "op": "store", "B": B, "Hkv": Hkv, "Nk": Nk, "n_new": n_new, "block": block,
            "ragged": ragged}


def _attend(name, B, Hkv, g, Nq, Nk, block, ragged, causal=True):
    return {"name": name, "op": "attend", "B": B, "Hkv": Hkv, "g": g, "Nq": Nq, "Nk": Nk, "block": block,
            "ragged": ragged, "causal": causal}


def _sparse(name, B, Hkv, g, Nq, Nk, block, n_select, fp8, ragged):
    return {"name": name, "op": "sparse", "B": B, "Hkv": Hkv, "g": g, "Nq": Nq, "Nk": Nk, "block": block,
            "n_select": n_select, "fp8": fp8, "ragged": ragged}


def _weights(name, B, Hkv, g, Nq, Nk, block, fp8, ragged):
    return {"name": name, "op": "weights", "B": B, "Hkv": Hkv, "g": g, "Nq": Nq, "Nk": Nk, "block": block,
            "fp8": fp8, "ragged": ragged}


def _evict(name, B, Hkv, Nk, keep, recent, block, fp8, ragged):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "Nk": Nk, "keep": keep, "recent": recent,
            "block": block, "fp8": fp8, "ragged": ragged}


def listed():
    return [
        # one new token of each of 8 sequences appended while serving: pure latency
        _store("store-token", 8, 8, 4096, 1, 64, True),
        # a batch of whole prompts written into the cache after prefill
        _store("store-prompt", 4, 8, 8192, 8192, 128, False),
        # the first steps of one short chat: launch latency
        _attend("attend-short", 1, 8, 4, 1, 1000, 64, False),
        # a serving batch whose sequences have very different lengths, odd ones among them
        _attend("attend-ragged", 16, 8, 4, 1, 16384, 64, True),
        # a long-context batch, four drafted tokens verified at once: the cache read bounds it
        _attend("attend-long", 16, 8, 4, 4, 32768, 128, False),
        # three heads a group, five queries, small blocks, an odd capacity
        _attend("attend-odd", 3, 8, 3, 5, 5001, 16, True),
        # a decode step over a long 8-bit cache that reads an eighth of it
        _sparse("sparse-fp8", 16, 8, 4, 1, 32768, 64, 64, True, False),
        # two new tokens against a bf16 cache of odd capacity, ragged, small blocks, an eight-head group
        _sparse("sparse-bf16", 4, 4, 8, 2, 8191, 32, 48, False, True),
        # the weights that one decode step gives the keys of a long 8-bit cache
        _weights("weights-token", 16, 8, 4, 1, 32768, 64, True, False),
        # the weights that a whole prompt gives its own keys (bf16, causal)
        _weights("weights-prompt", 1, 8, 4, 4096, 4096, 64, False, False),
        # a bf16 cache of ragged sequences cut back to a quarter
        _evict("evict-bf16", 4, 8, 8192, 2048, 256, 64, False, True),
        # a long 8-bit cache cut back to a quarter
        _evict("evict-fp8", 16, 8, 32768, 8192, 512, 64, True, False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _drawn(rng):
    op = rng.choice(["store", "attend", "sparse", "weights", "evict"])
    block = rng.choice([16, 32, 64, 128])
    B, Hkv = _log(rng, 1, 16), rng.choice([1, 2, 4, 8])
    Nk = _log(rng, 40, 32768)
    ragged = rng.random() < 0.6
    if op == "store":
        Nk = _log(rng, 40, 8192)
        n_new = rng.choice([1, _log(rng, 1, Nk), Nk])
        return _store("", min(B, 4) if n_new > 64 else B, Hkv, Nk, n_new, block, ragged and n_new < Nk)
    g, Nq = rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([1, 1, 2, 3, 4])
    if op == "attend":
        return _attend("", B, Hkv, g, Nq, Nk, block, ragged, rng.random() < 0.8)
    if op == "sparse":
        blocks = -(-Nk // block)
        return _sparse("", B, Hkv, g, Nq, Nk, block, _log(rng, 3, max(4, min(64, blocks))), rng.random() < 0.5,
                       ragged)
    if op == "weights":
        if rng.random() < 0.5:
            return _weights("", B, Hkv, g, Nq, Nk, block, rng.random() < 0.6, ragged)
        Nq = _log(rng, 40, 2048)
        return _weights("", 1, Hkv, min(g, 4), Nq, Nq + rng.choice([0, _log(rng, 1, 2048)]), block, False, False)
    keep = _log(rng, 4, max(5, Nk // 2))
    return _evict("", B, Hkv, Nk, keep, rng.randint(0, keep // 2), block, rng.random() < 0.5, ragged)


def draw(rng):
    return {k: v for k, v in _drawn(rng).items() if k != "name"}


def _lens(case):
    """The sequences' lengths: all full, or spread from 1 (B > 1) to the capacity; they go by the case alone."""
    B, Nk = case["B"], case["Nk"]
    if not case["ragged"]:
        return [Nk] * B
    if B == 1:
        return [max(1, Nk - Nk // 7)]
    got = [1 + (Nk - 1) * b // (B - 1) for b in range(B)]
    return [got[(5 * b + 2) % B] if B % 5 else got[(3 * b + 1) % B] for b in range(B)] if B % 15 else got


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _quantise_full(x, block):
    """(codes, scales) of x [B, H, N, d]: a power-of-two scale for each block of tokens and head."""
    B, H, N, d = x.shape
    nb = -(-N // block)
    pad = torch.zeros(B, H, nb * block, d, dtype=x.dtype, device=x.device)
    pad[:, :, :N] = x
    s = _scale_of(pad.view(B, H, nb, block * d).abs().amax(-1).float())
    codes = (pad.view(B, H, nb, block, d).float() / s[..., None, None]).clamp(-448, 448).to(E4M3)
    return codes.view(B, H, nb * block, d)[:, :, :N].contiguous(), s.contiguous()


def _scale_of(amax):
    """The smallest power of two s >= 2^-100 with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1): amax / 448 = (m / 0.875) 2^(e - 9)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -100)).clamp(min=-100)
    return torch.ldexp(torch.ones_like(amax), e)


def _keys(gen, B, H, N):
    """Keys and values as caches hold them: some channels wider than others, tokens of different size."""
    wide = 0.5 + torch.rand(1, H, 1, D, generator=gen, device=DEV) * 1.5
    size = 0.5 + torch.rand(B, H, N, 1, generator=gen, device=DEV)
    k = (torch.randn(B, H, N, D, generator=gen, device=DEV) * wide * size).bfloat16()
    v = (torch.randn(B, H, N, D, generator=gen, device=DEV) * size).bfloat16()
    return k, v


def prepare(case, seed):
    gen = _gen(seed)
    op, B, Hkv, Nk, block = case["op"], case["B"], case["Hkv"], case["Nk"], case["block"]
    nb = -(-Nk // block)
    s = dict(case)
    s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV) if case["ragged"] else None
    k, v = _keys(gen, B, Hkv, Nk)
    if op == "store":
        # the cache before the call, with the tokens that it holds already, and the new ones
        s["new_k"], s["new_v"] = _keys(gen, B, Hkv, case["n_new"])
        s["k"], s["ks"] = _quantise_full(k, block)
        s["v"], s["vs"] = _quantise_full(v, block)
        kf = s["k"].float()
        if nb * block > Nk:
            kf = torch.cat([kf, kf[:, :, -1:].expand(B, Hkv, nb * block - Nk, D)], 2)
        kf = kf.view(B, Hkv, nb, block, D)
        s["bounds"] = torch.stack([kf.amin(3), kf.amax(3)], 3).to(E4M3)
        return s
    if op == "evict":
        # weights as a history of decode steps leaves them: a few large, most small
        s["acc"] = torch.randn(B, Hkv, Nk, generator=gen, device=DEV).mul_(2).exp_()
        if case["fp8"]:
            s["k"], s["ks"] = _quantise_full(k, block)
            s["v"], s["vs"] = _quantise_full(v, block)
        else:
            s["k"], s["v"] = k, v
        # a second cache of the same capacity to compact into
        s["out"] = [torch.zeros_like(s["k"]), torch.zeros_like(s["v"]), torch.zeros_like(s["acc"]),
                    torch.zeros(B, Hkv, case["keep"], dtype=torch.int32, device=DEV),
                    torch.zeros(B, dtype=torch.int32, device=DEV)]
        if case["fp8"]:
            s["out"] += [torch.zeros_like(s["ks"]), torch.zeros_like(s["vs"])]
        return s
    Hq, Nq = Hkv * case["g"], case["Nq"]
    q = torch.randn(B, Hq, Nq, D, generator=gen, device=DEV)
    if Nk >= 64:  # some keys that the queries look for
        at = torch.randint(0, Nk, (B, Hkv, 4), generator=gen, device=DEV)
        mean = q.view(B, Hkv, case["g"] * Nq, D).mean(2, keepdim=True)
        mean = mean / mean.norm(dim=-1, keepdim=True) * 16
        k.scatter_(2, at[..., None].expand(B, Hkv, 4, D), mean.expand(B, Hkv, 4, D).bfloat16())
    s["q"], s["scale"] = q.bfloat16(), 1.0 / math.sqrt(D)
    fp8 = op == "attend" or case["fp8"]
    if fp8:
        s["k"], s["ks"] = _quantise_full(k, block)
        s["v"], s["vs"] = _quantise_full(v, block)
    else:
        s["k"], s["v"], s["ks"], s["vs"] = k, v, None, None
    if op == "sparse":
        held = torch.arange(nb * block, device=DEV)[None] < torch.tensor(_lens(case), device=DEV)[:, None]
        kf = torch.zeros(B, Hkv, nb * block, D, device=DEV, dtype=torch.bfloat16)
        kf[:, :, :Nk] = s["k"].to(torch.bfloat16)
        kf, held = kf.view(B, Hkv, nb, block, D), held.view(B, 1, nb, block, 1)
        s["bounds"] = torch.stack([kf.masked_fill(~held, math.inf).amin(3), kf.masked_fill(~held, -math.inf).amax(3)], 3)
        s["bounds"] = s["bounds"].masked_fill(~held.any(3)[..., None, :].expand_as(s["bounds"]), 0).to(s["k"].dtype)
    if op == "weights":
        s["acc"] = torch.rand(B, Hkv, Nk, generator=gen, device=DEV)
        lse = [_scores(s, b, torch.float64)[1].float() for b in range(B)]
        s["lse"] = torch.stack(lse).view(B, Hq, Nq).contiguous()
    return s


def _scores(s, b, dtype):
    """Sequence b's scores [Hkv, g * Nq, Nk] (unseen keys at -inf) and their log-sum-exp."""
    B, Hq, Nq, d = s["q"].shape
    Hkv, Nk = s["k"].shape[1:3]
    k = s["k"][b].to(dtype)
    if s["ks"] is not None:
        k = k * s["ks"][b].to(dtype).repeat_interleave(s["block"], 1)[:, :Nk, None]
    n = Nk if s["lens"] is None else int(s["lens"][b])
    x = torch.matmul(s["q"][b].to(dtype).view(Hkv, -1, d), k.transpose(1, 2)) * s["scale"]
    last = (n - Nq + torch.arange(Nq, device=DEV)) if s.get("causal", True) else torch.full((Nq,), n - 1, device=DEV)
    seen = torch.arange(Nk, device=DEV)[None] <= last.repeat(Hq // Hkv)[:, None]
    x = x.masked_fill(~seen, -math.inf)
    return x, torch.logsumexp(x, -1)


# ---------------------------------------------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------------------------------------------

def _seen(s, rows):
    """[B, 1, rows, Nk]: which keys a group's rows (head-major, Nq queries each) see."""
    B, Nk, Nq = s["k"].shape[0], s["k"].shape[2], s["Nq"]
    n = torch.full((B,), Nk, dtype=torch.int32, device=DEV) if s["lens"] is None else s["lens"]
    i = torch.arange(rows, device=DEV) % Nq
    last = n[:, None] - Nq + i if s.get("causal", True) else (n[:, None] - 1).expand(B, rows)
    return (torch.arange(Nk, device=DEV) <= last[..., None])[:, None]


def _dequantised(codes, scales, block):
    x = codes.float()
    return x if scales is None else x * scales.repeat_interleave(block, 2)[:, :, :x.shape[2], None]


def _softmax_product(x, v):
    """softmax(x) v and the log-sum-exp; rows that see nothing give 0 and -inf."""
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = (x - m).exp()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / l
    return o.masked_fill(l == 0, 0.0), (m + l.log()).squeeze(-1)


def _run_store(s):
    if own:
        import exact_io_aware_44_b200 as fa
        fa.cache_store(s["new_k"], s["new_v"], s["k"], s["v"], s["ks"], s["vs"], s["block"], lens=s["lens"])
        fa.block_bounds(s["k"], s["block"], lens=s["lens"], n_new=s["n_new"], bounds=s["bounds"])
        return s["k"], s["v"], s["ks"], s["vs"], s["bounds"]
    B, Hkv, Nk, d = s["k"].shape
    block, n_new, nb = s["block"], s["n_new"], s["ks"].shape[2]
    n = torch.full((B,), Nk, dtype=torch.int64, device=DEV) if s["lens"] is None else s["lens"].long()
    start = n - n_new
    # the blocks that new tokens fall into, as a window of whole blocks
    touched = min((n_new + block - 2) // block + 1, nb)
    first = (start.clamp(min=0) // block).clamp(max=nb - touched)
    blocks = first[:, None] + torch.arange(touched, device=DEV)
    pos = (blocks[..., None] * block + torch.arange(block, device=DEV)).view(B, 1, -1, 1)
    held, new = pos < n.view(B, 1, 1, 1), (pos >= start.view(B, 1, 1, 1)) & (pos < n.view(B, 1, 1, 1))
    at = pos.clamp(max=Nk - 1).expand(B, Hkv, touched * block, d)
    from_new = (pos - start.view(B, 1, 1, 1)).clamp(0, n_new - 1).expand_as(at)
    rows = blocks[:, None].expand(B, Hkv, touched)
    shape = (B, Hkv, touched, block, d)
    any_new, any_old = new.view(B, 1, touched, block).any(-1), (held & ~new).view(B, 1, touched, block).any(-1)

    def one(codes, scales, x):
        old_codes = codes.view(torch.uint8).gather(2, at)
        old_scale = scales.gather(2, rows)
        x = x.float().gather(2, from_new).masked_fill(~new, 0.0)
        need = _scale_of(x.view(B, Hkv, touched, -1).abs().amax(-1))
        scale = torch.where(any_new, torch.where(any_old, torch.maximum(need, old_scale), need), old_scale)
        old = old_codes.view(E4M3).float().view(shape) * (old_scale / scale)[..., None, None]
        y = torch.where(new, (x.view(shape) / scale[..., None, None]).view_as(x), old.view_as(x))
        y = y.clamp(-448, 448).to(E4M3)
        # tokens behind the sequence's end stay as they are (duplicated positions hold the last token's own value)
        keep = (held & any_new.repeat_interleave(block, 2)[..., None] & (pos < Nk)).expand_as(at)
        out = torch.where(keep, y.view(torch.uint8), old_codes)
        last = codes.view(torch.uint8)[:, :, -1].clone()
        codes.view(torch.uint8).scatter_(2, at, out)
        inside = keep & (pos == Nk - 1)
        codes.view(torch.uint8)[:, :, -1] = torch.where(inside.any(2), (out * inside).sum(2).to(torch.uint8), last)
        scales.scatter_(2, rows, scale)
        return y.float()

    k = one(s["k"], s["ks"], s["new_k"])
    one(s["v"], s["vs"], s["new_v"])
    lo = k.masked_fill(~held, math.inf).view(shape).amin(3)
    hi = k.masked_fill(~held, -math.inf).view(shape).amax(3)
    b_at = rows[..., None, None].expand(B, Hkv, touched, 2, d)
    old = s["bounds"].view(torch.uint8).gather(2, b_at)
    fresh = torch.where(any_new[..., None, None], torch.stack([lo, hi], 3).clamp(-448, 448).to(E4M3).view(torch.uint8), old)
    s["bounds"].view(torch.uint8).scatter_(2, b_at, fresh)
    return s["k"], s["v"], s["ks"], s["vs"], s["bounds"]


def _run_attend(s):
    if own:
        import exact_io_aware_44_b200 as fa
        return fa.decode_fp8(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["block"], lens=s["lens"], causal=s["causal"],
                             scale=s["scale"])
    B, Hq, Nq, d = s["q"].shape
    Hkv = s["Hkv"]
    q = s["q"].float().view(B, Hkv, -1, d)
    x = torch.matmul(q, _dequantised(s["k"], s["ks"], s["block"]).transpose(2, 3)) * s["scale"]
    x = x.masked_fill(~_seen(s, q.shape[2]), -math.inf)
    o, lse = _softmax_product(x, _dequantised(s["v"], s["vs"], s["block"]))
    return o.view(B, Hq, Nq, d).bfloat16(), lse.view(B, Hq, Nq)


def _run_sparse(s):
    if own:
        import exact_io_aware_44_b200 as fa
        idx = fa.select_blocks(s["q"], s["bounds"], s["n_select"], s["block"], s["Nk"], k_scale=s["ks"],
                               lens=s["lens"], n_first=1, n_last=1)
        o, lse = fa.decode_blocks(s["q"], s["k"], s["v"], idx, s["block"], k_scale=s["ks"], v_scale=s["vs"],
                                  lens=s["lens"], scale=s["scale"])
        return idx, o, lse
    B, Hq, Nq, d = s["q"].shape
    Hkv, Nk, block, n_select, g = s["Hkv"], s["Nk"], s["block"], s["n_select"], s["g"]
    nb = s["bounds"].shape[2]
    # the bound of every block for every query: in 64 bits, since a choice hangs on it
    q = s["q"].double().view(B, Hkv, g * Nq, d)
    lo, hi = s["bounds"].double().unbind(3)
    u = torch.matmul(q.clamp(min=0), hi.transpose(2, 3)) + torch.matmul(q.clamp(max=0), lo.transpose(2, 3))
    if s["ks"] is not None:
        u = u * s["ks"].double()[:, :, None]
    u = u.view(B, Hkv, g, Nq, nb).amax(2)
    n = torch.full((B,), Nk, dtype=torch.int32, device=DEV) if s["lens"] is None else s["lens"]
    last = (n[:, None] - Nq + torch.arange(Nq, device=DEV)).view(B, 1, Nq, 1)
    blk = torch.arange(nb, device=DEV)
    count = torch.where(last >= 0, last // block + 1, 0)
    u = u.masked_fill((blk < 1) | (blk >= count - 1), math.inf).masked_fill(blk >= count, -math.inf)
    order = u.sort(dim=-1, descending=True, stable=True).indices[..., :n_select]
    order = torch.where(torch.arange(order.shape[-1], device=DEV) < count, order, nb).sort(-1).values
    idx = torch.full((B, Hkv, Nq, n_select), -1, dtype=torch.int32, device=DEV)
    idx[..., :order.shape[-1]] = torch.where(order < nb, order, -1)
    # attention of each query's rows over its own blocks' keys
    pos = idx.long()[..., None] * block + torch.arange(block, device=DEV)
    seen = (idx >= 0)[..., None] & (pos <= last[..., None])
    at = pos.clamp(0, Nk - 1).view(B, Hkv, -1, 1).expand(B, Hkv, Nq * n_select * block, d)
    k, v = (t.view(torch.uint8).gather(2, at).view(E4M3) if s["fp8"] else t.gather(2, at) for t in (s["k"], s["v"]))
    k, v = k.float(), v.float()
    if s["fp8"]:
        of = idx.long().clamp(min=0).view(B, Hkv, -1)
        k = k * s["ks"].gather(2, of).repeat_interleave(block, 2)[..., None]
        v = v * s["vs"].gather(2, of).repeat_interleave(block, 2)[..., None]
    k, v = (t.view(B, Hkv, Nq, n_select * block, d) for t in (k, v))
    qi = s["q"].float().view(B, Hkv, g, Nq, d).transpose(2, 3)
    x = torch.matmul(qi, k.transpose(3, 4)) * s["scale"]
    x = x.masked_fill(~seen.view(B, Hkv, Nq, 1, -1), -math.inf)
    o, lse = _softmax_product(x, v)
    return idx, o.transpose(2, 3).reshape(B, Hq, Nq, d).bfloat16(), lse.transpose(2, 3).reshape(B, Hq, Nq)


def _run_weights(s):
    if own:
        import exact_io_aware_44_b200 as fa
        return fa.cache_weights(s["q"], s["k"], s["lse"], s["acc"], k_scale=s["ks"], block=s["block"], lens=s["lens"],
                                scale=s["scale"])
    B, Hq, Nq, d = s["q"].shape
    Hkv = s["Hkv"]
    q = s["q"].float().view(B, Hkv, -1, d)
    x = torch.matmul(q, _dequantised(s["k"], s["ks"], s["block"]).transpose(2, 3)) * s["scale"]
    p = (x - s["lse"].view(B, Hkv, -1, 1)).exp().masked_fill(~_seen(s, q.shape[2]), 0.0)
    return s["acc"].add_(p.sum(2))


def _run_evict(s):
    if own:
        import exact_io_aware_44_b200 as fa
        return fa.cache_evict(s["k"], s["v"], s["acc"], s["keep"], s["recent"], k_scale=s.get("ks"),
                              v_scale=s.get("vs"), block=s["block"], lens=s["lens"], out=s["out"])
    B, Hkv, Nk, d = s["k"].shape
    keep, block = s["keep"], s["block"]
    out_k, out_v, out_acc, out_idx, out_lens = s["out"][:5]
    n = torch.full((B,), Nk, dtype=torch.int32, device=DEV) if s["lens"] is None else s["lens"]
    count = n.clamp(max=keep)
    recent = count.clamp(max=s["recent"])
    j = torch.arange(Nk, device=DEV)
    key = s["acc"].masked_fill((j >= (n - recent)[:, None])[:, None], math.inf)
    key = key.masked_fill((j >= n[:, None])[:, None], -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    live = torch.arange(keep, device=DEV) < count[:, None, None]
    kept = torch.where(live[..., :order.shape[-1]], order, Nk).sort(-1).values
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=Nk)
    out_idx.copy_(torch.where(kept < Nk, kept, -1))
    out_lens.copy_(count)
    kept, live = kept.clamp(max=Nk - 1)[..., :Nk], live.expand(B, Hkv, keep)[..., :Nk]
    m = kept.shape[-1]
    out_acc[..., :m] = torch.where(live, s["acc"].gather(2, kept), out_acc[..., :m])
    at = kept[..., None].expand(B, Hkv, m, d)
    if not s["fp8"]:
        for src, dst in ((s["k"], out_k), (s["v"], out_v)):
            dst[:, :, :m] = torch.where(live[..., None], src.gather(2, at), dst[:, :, :m])
        return s["out"]
    nb = -(-m // block)
    for src, dst, scales, dst_scales in ((s["k"], out_k, s["ks"], s["out"][5]), (s["v"], out_v, s["vs"], s["out"][6])):
        of = scales.gather(2, kept // block)
        padded = torch.zeros(B, Hkv, nb * block, device=DEV)
        padded[..., :m] = of.masked_fill(~live, 0.0)
        new = padded.view(B, Hkv, nb, block).amax(-1)
        dst_scales[..., :nb] = torch.where(new > 0, new, dst_scales[..., :nb])
        ratio = (of / new.repeat_interleave(block, 2)[..., :m])[..., None]
        y = (src.view(torch.uint8).gather(2, at).view(E4M3).float() * ratio).to(E4M3)
        into = dst.view(torch.uint8)
        into[:, :, :m] = torch.where(live[..., None], y.view(torch.uint8), into[:, :, :m])
    return s["out"]


def run(state):
    return {"store": _run_store, "attend": _run_attend, "sparse": _run_sparse, "weights": _run_weights,
            "evict": _run_evict}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    op, B, Hkv, Nk, block = case["op"], case["B"], case["Hkv"], case["Nk"], case["block"]
    lens = _lens(case)
    if op == "store":
        new = sum(min(n, case["n_new"]) for n in lens) * Hkv
        # new K and V in, their codes and scales out, and the bounds of their blocks
        blocks = max(1, new // block)
        return {"bytes": new * D * 2 * 3 + blocks * (8 + 2 * D), "flops": new * D * 4}
    if op == "evict":
        kept = sum(min(n, case["keep"]) for n in lens) * Hkv
        elem = 1 if case["fp8"] else 2
        return {"bytes": sum(lens) * Hkv * 4 + kept * (2 * 2 * D * elem + 8), "flops": kept * D * 2}
    Nq, g = case["Nq"], case["g"]
    rows = B * Hkv * g * Nq
    if op == "attend":
        pairs = sum(n * Nq for n in lens) * Hkv * g
        return {"bytes": sum(lens) * Hkv * (2 * D + 8 / block) + rows * (4 * D + 4), "flops": 4 * D * pairs}
    elem = 1 if case["fp8"] else 2
    if op == "weights":
        pairs = sum(max(0, n * Nq - Nq * (Nq - 1) // 2) for n in lens) * Hkv * g
        return {"bytes": sum(lens) * Hkv * (D * elem + 8) + rows * (2 * D + 4), "flops": 2 * D * pairs}
    blocks = sum(-(-n // block) for n in lens) * Hkv
    taken = sum(min(n, case["n_select"] * block) * Nq for n in lens) * Hkv
    return {"bytes": blocks * 2 * D * elem + taken * 2 * D * elem + rows * (4 * D + 4),
            "flops": blocks * g * Nq * 2 * D + taken * g * 4 * D}


# ---------------------------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _e4m3_64(x):
    """x (float64) rounded to the nearest E4M3 value, ties to even, saturating: by the grid's own spacing."""
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6.0)
    step = torch.exp2(exponent - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_scale(amax):
    if amax <= 0:
        return 2.0 ** -100
    e = math.ceil(math.log2(amax / 448.0))
    while 448.0 * 2.0 ** (e - 1) >= amax:
        e -= 1
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** max(e, -100)


def exact(case, seed):
    s = prepare(case, seed)
    op, B, Hkv, Nk, block = case["op"], case["B"], case["Hkv"], case["Nk"], case["block"]
    lens, f64 = _lens(case), torch.float64
    if op == "store":
        out = {}
        k64 = None
        for name, x in (("k", s["new_k"]), ("v", s["new_v"])):
            codes, scales = s[name].to(f64), s[name + "s"].to(f64)
            for b, n in enumerate(lens):
                start, x64 = n - case["n_new"], x[b].to(f64)
                for j in range(max(start, 0) // block, -(-n // block)):
                    p0, p1 = j * block, min((j + 1) * block, n)
                    fresh = x64[:, max(p0, start) - start:p1 - start]
                    peak = fresh.abs().amax((1, 2)).tolist()
                    scale = torch.tensor([_exact_scale(a) for a in peak], dtype=f64, device=DEV)
                    if p0 < start:
                        scale = torch.maximum(scale, scales[b, :, j])
                        codes[b, :, p0:start] = _e4m3_64(codes[b, :, p0:start] * (scales[b, :, j] / scale)[:, None, None])
                    codes[b, :, max(p0, start):p1] = _e4m3_64(fresh / scale[:, None, None])
                    scales[b, :, j] = scale
            out[name], out[name + "s"] = codes, scales
            k64 = codes if name == "k" else k64
        bounds = s["bounds"].to(f64)
        for b, n in enumerate(lens):
            for j in range(max(n - case["n_new"], 0) // block, -(-n // block)):
                held = k64[b, :, j * block:min((j + 1) * block, n)]
                bounds[b, :, j, 0], bounds[b, :, j, 1] = held.amin(1), held.amax(1)
        return out["k"], out["v"], out["ks"], out["vs"], bounds
    if op == "evict":
        keep, out = case["keep"], [t.to(f64) for t in s["out"]]
        out[3].fill_(-1)
        j = torch.arange(Nk, device=DEV)
        for b, n in enumerate(lens):
            m = min(n, keep)
            r = min(case["recent"], m)
            out[4][b] = m
            for h in range(Hkv):
                acc = s["acc"][b, h, :n - r].to(f64)
                top = torch.sort(-acc, stable=True).indices[:m - r]
                kept = torch.cat([top.sort().values, j[n - r:n]])
                out[3][b, h, :m], out[2][b, h, :m] = kept.to(f64), s["acc"][b, h, kept].to(f64)
                for c, name in ((0, "k"), (1, "v")):
                    rows = s[name][b, h].to(f64)[kept]
                    if case["fp8"]:
                        of = s[name + "s"][b, h].to(f64)[kept // block]
                        groups = torch.nn.functional.pad(of, (0, -m % block)).view(-1, block).amax(1)
                        out[5 + c][b, h, :len(groups)] = groups
                        rows = _e4m3_64(rows * (of / groups.repeat_interleave(block)[:m])[:, None])
                    out[c][b, h, :m] = rows
        out[3], out[4] = out[3].long(), out[4].long()
        return out
    Hq, Nq, g = Hkv * case["g"], case["Nq"], case["g"]
    if op == "weights":
        if B * Hq * Nq * Nk > 1 << 32:
            return None
        acc = s["acc"].to(f64)
        for b in range(B):
            for h in range(Hkv):
                one = {**s, "q": s["q"][b:b + 1, h * g:(h + 1) * g], "k": s["k"][b:b + 1, h:h + 1],
                       "ks": None if s["ks"] is None else s["ks"][b:b + 1, h:h + 1],
                       "lens": None if s["lens"] is None else s["lens"][b:b + 1]}
                x = _scores(one, 0, f64)[0][0]
                l = s["lse"][b, h * g:(h + 1) * g].to(f64).reshape(-1, 1)
                acc[b, h] += torch.where(x == -math.inf, 0.0, torch.exp(x - l)).sum(0)
        return acc
    o = torch.zeros(B, Hq, Nq, D, dtype=f64, device=DEV)
    lse = torch.full((B, Hq, Nq), -math.inf, dtype=f64, device=DEV)
    if op == "attend":
        for b, n in enumerate(lens):
            x, l = _scores(s, b, f64)
            v = s["v"][b].to(f64) * s["vs"][b].to(f64).repeat_interleave(block, 1)[:, :Nk, None]
            p = torch.where(l[..., None] == -math.inf, 0.0, torch.exp(x - l[..., None]))
            o[b], lse[b] = torch.matmul(p, v).view(Hq, Nq, D), l.view(Hq, Nq)
        return o, lse
    idx = torch.full((B, Hkv, Nq, case["n_select"]), -1, dtype=torch.int64, device=DEV)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            lo, hi = s["bounds"][b, h].to(f64).unbind(1)
            ks = torch.ones(lo.shape[0], dtype=f64, device=DEV) if s["ks"] is None else s["ks"][b, h].to(f64)
            vs = torch.ones(lo.shape[0], dtype=f64, device=DEV) if s["vs"] is None else s["vs"][b, h].to(f64)
            for i in range(Nq):
                last = n - Nq + i
                if last < 0:
                    continue
                count = last // block + 1
                q = s["q"][b, h * g:(h + 1) * g, i].to(f64)
                u = torch.stack([(torch.where(r >= 0, r * hi[:count], r * lo[:count])).sum(1) * ks[:count] for r in q]).amax(0)
                u[0], u[count - 1] = math.inf, math.inf
                top = torch.sort(-u, stable=True).indices[:case["n_select"]].sort().values
                idx[b, h, i, :len(top)] = top
                at = (top[:, None] * block + torch.arange(block, device=DEV)).flatten()
                at = at[at <= last]
                x = torch.matmul(q, (s["k"][b, h].view(torch.uint8)[at].view(E4M3) if s["fp8"] else s["k"][b, h][at]).to(f64).T)
                x = x * ks[at // block] * s["scale"]
                l = torch.logsumexp(x, -1)
                v = (s["v"][b, h].view(torch.uint8)[at].view(E4M3) if s["fp8"] else s["v"][b, h][at]).to(f64) * vs[at // block][:, None]
                o[b, h * g:(h + 1) * g, i], lse[b, h * g:(h + 1) * g, i] = torch.matmul(torch.exp(x - l[:, None]), v), l
    return idx, o, lse
