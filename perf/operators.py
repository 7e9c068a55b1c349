"""The operators of the 4-bit key/value cache, as they are measured: append, load, pool, attend and evict.

``run`` computes them in a plain form (elementary torch operations in fp32, the gate's scores in fp64), or, where the
module's ``own`` is true, through the framework's ``kv4_*`` calls. The cache is the framework's: uint8
[batch, heads_kv, capacity / 64, 9216], one 64-token tile of one kv head in 9216 bytes:

  bytes 0..4095     key codes, 64 bytes a token: word w (4 bytes) holds channels 8w .. 8w+7, channel 8w + 2j in nibble j
                    and channel 8w + 2j + 1 in nibble j + 4
  bytes 4096..4607  key parameters, four uint16 a token, one for each 32 channels: scale code << 7 | zero point
  bytes 4608..9215  the same for the values, but a token whose index has bit 2 set holds channels 64..127 first

A value is scale * (code - zero); the scale is the fp16 number whose bits are the parameter's bits 7..14.
"""
import math

import torch

own = False

D, TILE, HALF = 128, 64, 4608
TILE_BYTES = 2 * HALF
TOP = 28800.0  # larger magnitudes are stored as this one


# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one new token for each of 64 requests: the append of a decode step
        {"name": "append decode", "op": "append", "batch": 64, "length": 16384, "n": 1, "ragged": True, "heads_kv": 8, "acc": True},
        # a whole prompt of the 128K workload goes into the cache
        {"name": "append prompt", "op": "append", "batch": 1, "length": 131072, "n": 131072, "ragged": False, "heads_kv": 8, "acc": False},
        # block means of the 128K workload's cache, for its gate
        {"name": "pool 128k", "op": "pool", "batch": 1, "length": 131072, "ragged": False, "heads_kv": 8, "block": 4096},
        # a ragged batch with small blocks, lengths that are no multiple of anything
        {"name": "pool batch", "op": "pool", "batch": 16, "length": 32749, "ragged": True, "heads_kv": 1, "block": 512},
        # the smallest decode step: one request, one head, every key
        {"name": "decode 4k", "op": "attend", "batch": 1, "length": 4096, "n": 1, "ragged": False, "heads_q": 1, "heads_kv": 1, "block": 0, "topk": 0, "acc": False},
        # one long request, every key, with the weights that eviction goes by
        {"name": "decode 128k acc", "op": "attend", "batch": 1, "length": 131072, "n": 1, "ragged": False, "heads_q": 32, "heads_kv": 8, "block": 0, "topk": 0, "acc": True},
        # a serving batch of ragged lengths, every key
        {"name": "decode batch", "op": "attend", "batch": 64, "length": 16381, "n": 1, "ragged": True, "heads_q": 32, "heads_kv": 8, "block": 0, "topk": 0, "acc": False},
        # the 1M workload's decode step: twelve blocks of 4096 tokens for each head
        {"name": "decode 1m top-12", "op": "attend", "batch": 1, "length": 1048575, "n": 1, "ragged": False, "heads_q": 32, "heads_kv": 8, "block": 4096, "topk": 12, "acc": False},
        # several long requests with block selection and accumulated weights
        {"name": "decode batch top-12", "op": "attend", "batch": 8, "length": 131072, "n": 1, "ragged": True, "heads_q": 32, "heads_kv": 8, "block": 4096, "topk": 12, "acc": True},
        # a chunk of a prompt against the cache, with the weights of its queries
        {"name": "chunk 512 at 32k", "op": "attend", "batch": 1, "length": 32768, "n": 512, "ragged": False, "heads_q": 32, "heads_kv": 8, "block": 0, "topk": 0, "acc": True},
        # after a prompt: 128K tokens go down to the 8192 heaviest
        {"name": "evict prompt", "op": "evict", "batch": 1, "length": 131072, "ragged": False, "heads_kv": 8, "budget": 8192, "recent": 1024},
        # during decoding: caches that have grown over their budget
        {"name": "evict batch", "op": "evict", "batch": 32, "length": 4608, "ragged": True, "heads_kv": 8, "budget": 4096, "recent": 256},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    most = max(_size(c) for c in listed())
    while True:
        c = {"op": rng.choice(["append", "pool", "attend", "attend", "attend", "evict"]), "batch": _log(rng, 1, 64), "length": _log(rng, 300, 200000), "ragged": rng.random() < 0.5}
        c["heads_kv"] = rng.choice([1, 2, 4, 8])
        if c["op"] == "append":
            c |= {"n": 1 if rng.random() < 0.4 else min(c["length"], _log(rng, 2, 60000)), "acc": rng.random() < 0.5}
        elif c["op"] == "pool":
            c |= {"block": 128 * rng.choice([1, 2, 4, 5, 8, 16, 32])}
        elif c["op"] == "attend":
            sparse = rng.random() < 0.5
            c |= {"n": 1 if rng.random() < 0.6 else min(c["length"], _log(rng, 2, 600)), "heads_q": c["heads_kv"] * rng.choice([1, 2, 3, 4, 8])}
            c |= {"block": 128 * rng.choice([1, 4, 8, 16, 32]) if sparse else 0, "topk": rng.randint(1, 16) if sparse else 0, "acc": rng.random() < 0.5}
        else:
            c["budget"] = max(2, int(c["length"] * rng.uniform(0.02, 0.95)))
            c["recent"] = rng.randint(0, c["budget"] // 2)
        tokens = c["batch"] * c["length"] * c["heads_kv"]
        scores = tokens * c.get("n", 1) * c.get("heads_q", 1) // c["heads_kv"]
        if tokens <= 1 << 21 and scores <= 1 << 29 and 0 < _size(c) <= most:
            return c


def _lengths(case):
    """Tokens in the cache, one number for each sequence: the same for every seed, so that work() knows them."""
    L = case["length"]
    if not case["ragged"]:
        return [L] * case["batch"]
    return [max(1, int(L * (0.125 + 0.875 * ((0.5 + 0.6180339887 * b) % 1.0)))) for b in range(case["batch"])]


def _news(case):
    """Tokens of this call (the last of each sequence), one number for each sequence."""
    n, lens = case["n"], _lengths(case)
    if n == 1 or not case["ragged"]:
        return [min(n, L) for L in lens]
    return [max(1, min(L, int(n * (0.25 + 0.75 * ((0.3 + 0.6180339887 * b) % 1.0))))) for b, L in enumerate(lens)]


def work(case):
    """Bytes read and written once, and the products' FLOPs."""
    lens, hkv = _lengths(case), case["heads_kv"]
    row = 144  # a token of one kv head: 2 * (64 bytes of codes + 8 of parameters)
    if case["op"] == "append":
        new = sum(_news(case)) * hkv
        return {"bytes": new * (512 + row + 512 + (4 if case["acc"] else 0)), "flops": 0}  # the new rows are read back as values
    if case["op"] == "pool":
        B = case["block"]
        return {"bytes": sum(L // B * (B * row // 2 + 512) for L in lens) * hkv, "flops": sum(L // B * B for L in lens) * hkv * D}
    if case["op"] == "evict":
        kept = sum(min(L, case["budget"]) for L in lens) * hkv
        return {"bytes": sum(lens) * hkv * 4 + kept * (2 * row + 8 + 512), "flops": 0}
    hq, n, G = case["heads_q"], _news(case), case["heads_q"] // hkv
    read = pairs = gated = 0.0
    for L, m in zip(lens, n):
        if case["topk"] == 0:
            read, pairs = read + L, pairs + m * (L - (m - 1) / 2)
            continue
        B, past = case["block"], (L - 1) // case["block"]
        k = min(case["topk"] - 1, past)
        # blocks that at least one of the rows of a kv head reads, when each row picks k of the past ones
        read += min(L, past * B * (1 - (1 - k / max(past, 1)) ** (m * G)) + min(L, (L - 1) % B + m))
        pairs += m * (k * B + (B if past else L) / 2)
        gated += past
    rows = sum(n)
    return {
        "bytes": read * hkv * (row + (8 if case["acc"] else 0)) + rows * hq * (512 + 4) + gated * hkv * 512,
        "flops": 4 * D * hq * pairs,
    }


def _size(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


# ------------------------------------------------------------------ the cache, in elementary operations


def _quantise(x):
    """x [..., 128] -> codes uint8 [..., 128], parameters int32 [..., 4]: 4-bit codes with a scale of four significant bits and a zero point for 32 channels."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=TOP, neginf=-TOP).clamp(-TOP, TOP).unflatten(-1, (4, 32))
    low, high = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    step = (high - low) / torch.full_like(low, 15.0)  # a quotient, not a product with 1/15
    bits = step.view(torch.int32)
    normal = ((bits + 0x7FFFF + ((bits >> 20) & 1)) >> 20) - (112 << 3)  # three bits of mantissa, to the nearest, ties to even
    small = torch.round(step * 2.0**17).to(torch.int32)  # below 2^-14: multiples of 2^-17
    code = torch.where(step >= 2.0**-14, normal, small).clamp(1, 0xD7)
    s = _scale(code << 7)
    zero = torch.floor(-low / s + 0.5).clamp(0, 15)
    c = (torch.floor(x / s[..., None] + 0.5) + zero[..., None]).clamp(0, 15)
    return c.to(torch.uint8).flatten(-2), (code << 7) | zero.to(torch.int32)


def _scale(par):
    return (par & 0x7F80).to(torch.int16).view(torch.float16).float()


def _swap(x):
    """Halves of the values' bytes, swapped for tokens whose index has bit 2 set: x [..., 64, 64]."""
    at = torch.arange(TILE, device=x.device)
    return torch.where(((at & 4) != 0)[:, None], x.roll(32, -1), x)


def _pack(codes, par, swapped):
    """Codes [..., 64, 128] and parameters [..., 64, 4] of tiles -> bytes [..., 4608]."""
    n = codes.unflatten(-1, (16, 4, 2)).transpose(-1, -2).flatten(-2)  # nibbles of each word
    b = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(-2)
    b = _swap(b) if swapped else b
    p = torch.stack((par & 255, par >> 8), -1).to(torch.uint8)
    return torch.cat((b.flatten(-2), p.flatten(-3)), -1)


def _values(half, swapped):
    """Bytes [..., tiles, 4608] -> fp32 values [..., tiles * 64, 128]."""
    b = half[..., : TILE * 64].unflatten(-1, (TILE, 64))
    b = _swap(b) if swapped else b
    n = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (16, 2, 4)).transpose(-1, -2).flatten(-3)
    p = half[..., TILE * 64 :].unflatten(-1, (TILE, 4, 2)).to(torch.int32)
    p = p[..., 0] | (p[..., 1] << 8)
    x = _scale(p)[..., None] * (n.unflatten(-1, (4, 32)).float() - (p & 15).float()[..., None])
    return x.flatten(-2).flatten(-3, -2)


def _keys(kv4):
    return _values(kv4[..., :HALF], False)


def _vals(kv4):
    return _values(kv4[..., HALF:], True)


# ------------------------------------------------------------------ what a user's program has in hand


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    lens, hkv, batch = _lengths(case), case["heads_kv"], case["batch"]
    tiles = -(-max(lens) // TILE)
    S = tiles * TILE
    s = {"op": case["op"], "lengths": torch.tensor(lens, dtype=torch.int32, device=dev), "longest": max(lens), "heads_kv": hkv}

    def rand(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32)

    if case["op"] == "append":
        n = _news(case)
        s["k"], s["v"] = (rand(sum(n), hkv, D).to(torch.bfloat16) for _ in "kv")
        s["start"] = s["lengths"] - torch.tensor(n, dtype=torch.int32, device=dev)
        s["cu"] = torch.tensor([sum(n[:b]) for b in range(batch + 1)], dtype=torch.int32, device=dev)
        s["n"] = max(n)
        s["kv4"] = torch.zeros((batch, hkv, tiles, TILE_BYTES), dtype=torch.uint8, device=dev)
        s["acc"] = torch.ones((batch, hkv, S), device=dev) if case["acc"] else None
        return s
    # keys that share a mean within a block, as the workloads' keys do; quantised a part at a time
    s["kv4"] = torch.empty((batch, hkv, tiles, TILE_BYTES), dtype=torch.uint8, device=dev)
    block = case.get("block") or 4096
    mean = rand(batch, hkv, -(-S // block), D)
    mean *= 0.5 * math.sqrt(D) / mean.norm(dim=-1, keepdim=True)
    part = max(1, (1 << 19) // (TILE * hkv))
    for b in range(batch):
        for t in range(0, tiles, part):
            u = min(tiles, t + part)
            k = rand(hkv, (u - t) * TILE, D) + mean[b, :, torch.arange(t * TILE, u * TILE, device=dev) // block]
            v = rand(hkv, (u - t) * TILE, D)
            k, v = (_quantise(x.to(torch.bfloat16).unflatten(1, (u - t, TILE))) for x in (k, v))
            s["kv4"][b, :, t:u] = torch.cat((_pack(*k, False), _pack(*v, True)), -1)
    if case["op"] == "pool":
        s["block"] = block
    elif case["op"] == "attend":
        n = _news(case)
        s |= {"block": case["block"], "topk": case["topk"], "n": max(n)}
        s["q"] = rand(sum(n), case["heads_q"], D).to(torch.bfloat16)
        s["cu"] = torch.tensor([sum(n[:b]) for b in range(batch + 1)], dtype=torch.int32, device=dev)
        s["acc"] = rand(batch, hkv, S).square() * 0.05 if case["acc"] else None
        s["kmean"] = None
        if case["topk"]:
            s["kmean"] = torch.stack([_means(s["kv4"][b], lens[b], block) for b in range(batch)])
    else:
        # weights as they accumulate: a few heavy tokens, many light ones, and some that nothing has attended yet
        s["acc"] = torch.exp(2.0 * rand(batch, hkv, S)) * (torch.rand((batch, hkv, S), generator=g, device=dev) > 0.1)
        s |= {"budget": case["budget"], "recent": case["recent"]}
        room = -(-case["budget"] // TILE)
        s["dst"] = torch.zeros((batch, hkv, room, TILE_BYTES), dtype=torch.uint8, device=dev)
        s["dst_acc"] = torch.zeros((batch, hkv, room * TILE), device=dev)
    return s


def _means(kv4, length, block):
    """Means of the complete blocks of one sequence (fp32 sums of a part at a time), the others zero: [heads_kv, blocks, 128]."""
    k = _keys(kv4)
    m = torch.zeros((kv4.shape[0], k.shape[1] // block, D), device=kv4.device)
    full = length // block
    m[:, :full] = k[:, : full * block].unflatten(1, (full, block)).mean(2) if full else 0
    return m


# ------------------------------------------------------------------ one pass


def run(s):
    return {"append": _append, "pool": _pool, "attend": _attend, "evict": _evict}[s["op"]](s)


def _append(s):
    if own:
        import block_sparse_long_fwd_b200 as moba

        moba.kv4_append(s["k"], s["v"], s["kv4"], s["start"], cu=s["cu"], acc=s["acc"])
        k, v = moba.kv4_load(s["kv4"], s["lengths"], s["n"], first=s["start"])
    else:
        kv4 = s["kv4"]
        t = torch.arange(s["k"].shape[0], device=kv4.device)
        b = torch.bucketize(t, s["cu"][1:].long(), right=True)
        at = s["start"][b] + t - s["cu"][b]  # the new tokens' places
        for_k, for_v = _quantise(s["k"]), _quantise(s["v"])
        _put(kv4[..., :HALF], b, at, for_k, False)
        _put(kv4[..., HALF:], b, at, for_v, True)
        if s["acc"] is not None:
            s["acc"][b, :, at] = 0.0
        k, v = _load(kv4, s["lengths"], s["n"], s["start"])
    return (k, v) if s["acc"] is None else (k, v, s["acc"])


def _put(half, b, at, stored, swapped):
    """Rows of tokens into their tiles: codes [T, heads, 128] and parameters [T, heads, 4] at sequence b, place `at`."""
    codes, par = stored
    n = codes.unflatten(-1, (16, 4, 2)).transpose(-1, -2).flatten(-2)
    rows = (n[..., 0::2] | (n[..., 1::2] << 4)).flatten(-2)
    if swapped:
        rows = torch.where(((at & 4) != 0)[:, None, None], rows.roll(32, -1), rows)
    p = torch.stack((par & 255, par >> 8), -1).to(torch.uint8).flatten(-2)
    half[..., : TILE * 64].unflatten(-1, (TILE, 64))[b, :, at // TILE, at % TILE] = rows
    half[..., TILE * 64 :].unflatten(-1, (TILE, 8))[b, :, at // TILE, at % TILE] = p


def _load(kv4, lengths, n, first):
    """Values of tokens first .. first + n - 1 of each sequence, zero from its length on: bf16 [batch, n, heads_kv, 128]."""
    at = first.long()[:, None] + torch.arange(n, device=kv4.device)
    inside = (at < lengths[:, None])[:, :, None, None]
    at = at.clamp(max=kv4.shape[2] * TILE - 1)
    return tuple(_row_values(half, at, swapped).where(inside, 0.0).to(torch.bfloat16) for half, swapped in ((kv4[..., :HALF], False), (kv4[..., HALF:], True)))


def _row_values(half, at, swapped):
    b = torch.arange(half.shape[0], device=half.device)[:, None]
    rows = half[..., : TILE * 64].unflatten(-1, (TILE, 64))[b, :, at // TILE, at % TILE]
    p = half[..., TILE * 64 :].unflatten(-1, (TILE, 4, 2))[b, :, at // TILE, at % TILE].to(torch.int32)
    if swapped:
        rows = torch.where(((at & 4) != 0)[:, :, None, None], rows.roll(32, -1), rows)
    n = torch.stack((rows & 15, rows >> 4), -1).flatten(-2).unflatten(-1, (16, 2, 4)).transpose(-1, -2).flatten(-3)
    p = p[..., 0] | (p[..., 1] << 8)
    return (_scale(p)[..., None] * (n.unflatten(-1, (4, 32)).float() - (p & 15).float()[..., None])).flatten(-2)


def _pool(s):
    if own:
        import block_sparse_long_fwd_b200 as moba

        return moba.kv4_pool(s["kv4"], s["lengths"], s["block"])
    k, B = _keys(s["kv4"]), s["block"]
    blocks = k.shape[2] // B
    m = k[:, :, : blocks * B].unflatten(2, (blocks, B)).mean(3)
    complete = torch.arange(blocks, device=k.device) < (s["lengths"] // B)[:, None]
    return m.where(complete[:, None, :, None], 0.0)


def _attend(s):
    if own:
        import block_sparse_long_fwd_b200 as moba

        more = {"kmean": s["kmean"], "block_size": s["block"], "topk": s["topk"]} if s["topk"] else {}
        out, lse = moba.kv4_attend(s["q"], s["kv4"], s["lengths"], cu=s["cu"], acc=s["acc"], **more)
    else:
        kv4, hkv, n = s["kv4"], s["heads_kv"], s["n"]
        batch, S = kv4.shape[0], kv4.shape[2] * TILE
        hq = s["q"].shape[1]
        G = hq // hkv
        cu = s["cu"].long()
        new = cu[1:] - cu[:-1]
        i = torch.arange(n, device=kv4.device)
        here = i < new[:, None]  # [batch, n]: a query, or padding
        q = s["q"].float()[(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)]
        q = q.unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4)  # [batch, heads_kv, G, n, 128]
        at = s["lengths"][:, None] - new[:, None] + i  # the queries' places
        key = torch.arange(S, device=kv4.device)
        seen = (key <= at[..., None])[:, None, None] & here[:, None, None, :, None]
        if s["topk"]:
            seen = seen & _chosen(q, s["kmean"], at, s["block"], s["topk"], S)
        z = torch.matmul(q.flatten(2, 3), _keys(kv4).transpose(-1, -2)).unflatten(2, (G, n)) * (1.0 / math.sqrt(D))
        z = z.masked_fill(~seen, -math.inf)
        top = z.amax(-1, keepdim=True).clamp(min=-1e30)
        e = torch.exp(z - top)
        total = e.sum(-1, keepdim=True)
        p = e / total.where(total > 0, 1.0)
        o = torch.matmul(p.flatten(2, 3), _vals(kv4)).unflatten(2, (G, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)
        lse = (top + torch.log(total)).squeeze(-1).flatten(1, 2).permute(1, 0, 2)
        out, lse = o[here].to(torch.bfloat16), lse[:, here]
        if s["acc"] is not None:
            s["acc"] += p.sum((2, 3))
    return (out, lse) if s["acc"] is None else (out, lse, s["acc"])


def _chosen(q, kmean, at, block, topk, S):
    """Keys of each query's blocks: its own, and the topk - 1 past blocks of the highest score q . mean (fp64), ties to the lower index."""
    score = torch.matmul(q.flatten(2, 3).double(), kmean.double().transpose(-1, -2)).unflatten(2, q.shape[2:4])
    blocks = -(-S // block)
    mine = (at // block)[:, None, None, :, None]
    score = torch.nn.functional.pad(score, (0, blocks - score.shape[-1]), value=-math.inf)
    score = score.masked_fill(torch.arange(blocks, device=q.device) >= mine, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., : topk - 1]
    pick = torch.zeros(score.shape, dtype=torch.bool, device=q.device).scatter(-1, order, True) & (score > -math.inf)
    pick = pick | (torch.arange(blocks, device=q.device) == mine)
    return pick.repeat_interleave(block, dim=-1)[..., :S]


def _evict(s):
    kv4, budget = s["kv4"], s["budget"]
    if own:
        import block_sparse_long_fwd_b200 as moba

        lengths, kept = moba.kv4_evict(kv4, s["acc"], s["lengths"], budget, s["recent"], s["dst"], s["dst_acc"])
        k, v = moba.kv4_load(s["dst"], lengths, budget)
        return lengths, kept, s["dst_acc"], k, v
    S = kv4.shape[2] * TILE
    at, L = torch.arange(S, device=kv4.device), s["lengths"].long()[:, None, None]
    w = s["acc"].masked_fill(at >= L, -math.inf).masked_fill((at >= L - s["recent"]) & (at < L), math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., : min(budget, S)]
    order = order.masked_fill(order >= L, S).sort(-1).values
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=S)
    there = order < L
    kept, src = order.where(there, -1).int(), order.clamp(max=S - 1)
    dst, to = s["dst"], torch.arange(budget, device=kv4.device)
    b, h = torch.arange(kv4.shape[0], device=kv4.device)[:, None, None], torch.arange(kv4.shape[1], device=kv4.device)[:, None]
    _move(kv4[..., :HALF], dst[..., :HALF], b, h, src, to, there, False)
    _move(kv4[..., HALF:], dst[..., HALF:], b, h, src, to, there, True)
    s["dst_acc"][..., :budget] = torch.gather(s["acc"], -1, src).where(there, s["dst_acc"][..., :budget])
    lengths = s["lengths"].clamp(max=budget)
    k, v = _load(dst, lengths, budget, torch.zeros_like(lengths))
    return lengths, kept, s["dst_acc"], k, v


def _move(half, dst, b, h, src, to, there, swapped):
    rows = half[..., : TILE * 64].unflatten(-1, (TILE, 64))[b, h, src // TILE, src % TILE]
    p = half[..., TILE * 64 :].unflatten(-1, (TILE, 8))[b, h, src // TILE, src % TILE]
    if swapped:
        rows = torch.where((((src ^ to) & 4) != 0)[..., None], rows.roll(32, -1), rows)
    for_rows, for_p = dst[..., : TILE * 64].unflatten(-1, (TILE, 64)), dst[..., TILE * 64 :].unflatten(-1, (TILE, 8))
    old = for_rows[b, h, to // TILE, to % TILE], for_p[b, h, to // TILE, to % TILE]
    for_rows[b, h, to // TILE, to % TILE] = rows.where(there[..., None], old[0])
    for_p[b, h, to // TILE, to % TILE] = p.where(there[..., None], old[1])


# ------------------------------------------------------------------ in 64 bits, from the definition


def _table(half, swapped):
    """fp64 values of one kv head's bytes [tiles, 4608]: each channel's nibble looked up by its place."""
    c = torch.arange(D, device=half.device)
    word, within = c // 8, c % 8
    nibble = within // 2 + 4 * (within % 2)
    byte = 4 * word + nibble // 2
    token = torch.arange(TILE, device=half.device)[:, None]
    place = byte ^ torch.where((token & 4) != 0, 32, 0) if swapped else byte.expand(TILE, D)
    code = (half[:, (64 * token + place).reshape(-1)].view(-1, TILE, D).to(torch.int16) >> (4 * (nibble % 2)).to(torch.int16)) & 15
    low, high = (half[:, (64 * TILE + 8 * token + 2 * (c // 32) + e).reshape(-1)].view(-1, TILE, D).to(torch.int16) for e in (0, 1))
    exponent, mantissa, zero = high >> 2, ((high & 3) << 1) | (low >> 7), low & 15
    scale = torch.where(exponent > 0, (1.0 + mantissa.double() / 8) * torch.exp2(exponent.double() - 15), mantissa.double() * 2.0**-17)
    return ((code - zero).double() * scale).flatten(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    lens, hkv = _lengths(case), case["heads_kv"]
    if case["op"] == "append":
        n = _news(case)
        res = []
        for x in (s["k"], s["v"]):
            got = torch.zeros((case["batch"], max(n), hkv, D), dtype=torch.float64, device=x.device)
            for b in range(case["batch"]):
                got[b, : n[b]] = _rounded(x[sum(n[:b]) : sum(n[: b + 1])].double())
            res.append(got)
        if s["acc"] is not None:
            acc = s["acc"].double()
            for b in range(case["batch"]):
                acc[b, :, lens[b] - n[b] : lens[b]] = 0
            res.append(acc)
        return tuple(res)
    if case["op"] == "pool":
        B = case["block"]
        m = torch.zeros((case["batch"], hkv, s["kv4"].shape[2] * TILE // B, D), dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            for h in range(hkv):
                k = _table(s["kv4"][b, h, :, :HALF], False)
                for j in range(lens[b] // B):
                    m[b, h, j] = k[j * B : (j + 1) * B].mean(0)
        return m
    if case["op"] == "evict":
        return _exact_evict(case, s, lens)
    return _exact_attend(case, s, lens)


def _rounded(x):
    """The values that rows x (fp64) are stored as."""
    x = x.clamp(-TOP, TOP).unflatten(-1, (4, 32))
    low, high = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    step = (high - low) / 15
    unit = torch.exp2(torch.floor(torch.log2(step.clamp(min=2.0**-14))) - 3)  # scales have four significant bits
    scale = (torch.round(step / unit) * unit).clamp(2.0**-17, 3840.0)
    zero = torch.floor(-low / scale + 0.5).clamp(0, 15)
    return (((torch.floor(x / scale + 0.5) + zero).clamp(0, 15) - zero) * scale).flatten(-2)


def _exact_attend(case, s, lens):
    hkv, n, hq = case["heads_kv"], _news(case), case["heads_q"]
    G = hq // hkv
    out = torch.zeros((sum(n), hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((hq, sum(n)), dtype=torch.float64, device="cuda")
    acc = s["acc"].double() if s["acc"] is not None else None
    for b in range(case["batch"]):
        t0, L, m = sum(n[:b]), lens[b], n[b]
        place = torch.arange(L - m, L, device="cuda")
        for h in range(hkv):
            tiles = -(-L // TILE)
            k, v = _table(s["kv4"][b, h, :tiles, :HALF], False)[:L], _table(s["kv4"][b, h, :tiles, HALF:], True)[:L]
            for u in range(0, m, 64):
                p = place[u : u + 64]
                rows = slice(t0 + u, t0 + u + len(p))
                q = s["q"][rows, h * G : (h + 1) * G].double()
                z = torch.einsum("tgd,sd->tgs", q, k) / math.sqrt(D)
                off = (torch.arange(L, device="cuda") > p[:, None])[:, None].expand_as(z)
                if case["topk"]:
                    B = case["block"]
                    mine = p // B
                    score = torch.einsum("tgd,jd->tgj", q, s["kmean"][b, h].double())
                    j = torch.arange(score.shape[-1], device="cuda")
                    score = score.masked_fill(j >= mine[:, None, None], -math.inf)
                    # a block's rank: blocks with a higher score, or the same score and a lower index
                    higher = (score[..., None, :] > score[..., None]) | ((score[..., None, :] == score[..., None]) & (j < j[:, None]))
                    pick = (higher.sum(-1) < case["topk"] - 1) & (score > -math.inf)
                    pick = torch.nn.functional.pad(pick, (0, -(-L // B) - pick.shape[-1])) if pick.shape[-1] < -(-L // B) else pick
                    pick = pick | (torch.arange(pick.shape[-1], device="cuda") == mine[:, None, None])
                    off = off | ~pick[..., torch.arange(L, device="cuda") // B]
                z = z.masked_fill(off, -math.inf)
                r = torch.logsumexp(z, -1)
                w = torch.exp(z - r[..., None])
                out[rows, h * G : (h + 1) * G] = torch.einsum("tgs,sd->tgd", w, v)
                lse[h * G : (h + 1) * G, rows] = r.T
                if acc is not None:
                    acc[b, h, :L] += w.sum((0, 1))
    return (out, lse) if acc is None else (out, lse, acc)


def _exact_evict(case, s, lens):
    import numpy as np

    budget, recent, hkv = case["budget"], case["recent"], case["heads_kv"]
    room = s["dst_acc"].shape[-1]
    kept = np.full((case["batch"], hkv, budget), -1, dtype=np.int32)
    acc = torch.zeros((case["batch"], hkv, room), dtype=torch.float64, device="cuda")
    k, v = (torch.zeros((case["batch"], budget, hkv, D), dtype=torch.float64, device="cuda") for _ in "kv")
    weights = s["acc"].cpu().numpy()
    for b, L in enumerate(lens):
        for h in range(hkv):
            old = np.arange(max(0, L - recent))
            if L > budget:  # the heaviest of the older tokens, the first of equals
                old = np.sort(old[np.lexsort((old, -weights[b, h, : len(old)]))][: budget - min(recent, L)])
            at = np.concatenate((old, np.arange(max(0, L - recent), L)))
            kept[b, h, : len(at)] = at
            i = torch.from_numpy(at).cuda()
            acc[b, h, : len(at)] = s["acc"][b, h, i].double()
            k[b, : len(at), h] = _table(s["kv4"][b, h, :, :HALF], False)[i]
            v[b, : len(at), h] = _table(s["kv4"][b, h, :, HALF:], True)[i]
    return torch.tensor([min(L, budget) for L in lens], dtype=torch.int32), kept, acc, k, v
