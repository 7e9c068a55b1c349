"""The 4-bit key/value cache in numpy, from its definition: the stored values,
the bytes of the layout (include/moba.h, csrc/kv4.cuh), attention, pooling and
eviction in fp64. Shares no code with the library or its binding."""
import numpy as np

TILE, TILE_BYTES, HALF, D = 64, 9216, 4608, 128
TOP = 28800.0


def scales():
    """Every scale, by its code 0 .. 0xD7: fp16 numbers with three bits of mantissa."""
    code = np.arange(0xD8)
    e, m = code >> 3, code & 7
    return np.where(e > 0, (1 + m / 8.0) * 2.0 ** (e - 15.0), m * 2.0**-17)


def quantise(x):
    """x [..., 128] -> (codes, zero points, scale codes); the last two [..., 4]."""
    x = np.asarray(x, dtype=np.float64)
    x = np.clip(np.where(np.isnan(x), 0.0, x), -TOP, TOP).reshape(*x.shape[:-1], 4, 32)
    lo, hi = np.minimum(x.min(-1), 0.0), np.maximum(x.max(-1), 0.0)
    step = (hi - lo) / 15.0
    table = scales()[1:]
    # the nearest scale; of two equally near ones the one with an even code
    at = np.searchsorted(table, step).clip(1, len(table) - 1)
    below, above = table[at - 1], table[at]
    up = (step - below > above - step) | ((step - below == above - step) & ((at + 1) % 2 == 0))
    code = np.where(up, at + 1, at)
    s = scales()[code]
    zero = np.clip(np.floor(-lo / s + 0.5), 0, 15)
    c = np.clip(np.floor(x / s[..., None] + 0.5) + zero[..., None], 0, 15)
    return c.astype(np.int64).reshape(*x.shape[:-2], D), zero.astype(np.int64), code


def values(c, zero, code):
    return ((c.reshape(*c.shape[:-1], 4, 32) - zero[..., None]) * scales()[code][..., None]).reshape(c.shape)


def stored(x):
    """What rows x [..., 128] are stored as, in fp64."""
    return values(*quantise(x))


def _place(tok, ch, is_v):
    """(byte within a half, shift) of a channel's code."""
    word, j = ch // 8, ch % 8
    nibble = j // 2 + 4 * (j % 2)
    byte = 4 * word + nibble // 2
    if is_v and tok & 4:
        byte ^= 32
    return tok * 64 + byte, 4 * (nibble % 2)


def _places(is_v):
    p = np.array([[_place(t, c, is_v) for c in range(D)] for t in range(TILE)])
    return p[..., 0], p[..., 1]


def pack(k, v):
    """Rows k, v [heads, tokens, 128] of one sequence, tokens a multiple of 64 -> uint8 [heads, tiles, 9216]."""
    heads, n = k.shape[:2]
    out = np.zeros((heads, n // TILE, TILE_BYTES), dtype=np.uint8)
    for s, x in enumerate((k, v)):
        c, zero, code = (a.reshape(heads, n // TILE, TILE, -1) for a in quantise(x))
        half = out[..., s * HALF:(s + 1) * HALF]
        byte, shift = _places(s == 1)
        for odd in (0, 4):
            pick = shift[0] == odd
            half[..., byte[:, pick].reshape(-1)] |= (c[..., pick] << odd).astype(np.uint8).reshape(heads, -1, TILE * 64)
        par = (code << 7) | zero
        half[..., 4096::2] = (par & 255).astype(np.uint8).reshape(heads, -1, 256)
        half[..., 4097::2] = (par >> 8).astype(np.uint8).reshape(heads, -1, 256)
    return out


def unpack(tiles):
    """uint8 [heads, tiles, 9216] -> k, v in fp64 [heads, tokens, 128]."""
    res = []
    for s in (0, 1):
        half = tiles[..., s * HALF:(s + 1) * HALF].astype(np.int64)
        byte, shift = _places(s == 1)
        c = (half[..., byte.reshape(-1)] >> shift.reshape(-1)) & 15
        par = half[..., 4096::2] | half[..., 4097::2] << 8
        shape = (tiles.shape[0], -1)
        res.append(values(c.reshape(*shape, D), (par & 15).reshape(*shape, 4), (par >> 7).reshape(*shape, 4)))
    return res


def means(k, length, block, blocks):
    """k [heads, tokens, 128] -> [heads, blocks, 128], zero for blocks that are not complete."""
    m = np.zeros((k.shape[0], blocks, D))
    for j in range(length // block):
        m[:, j] = k[:, j * block:(j + 1) * block].mean(1)
    return m


def seen(q, length, n, kmean=None, block=0, topk=0):
    """Keys each row attends: bool [n, G, length] for q [n, G, 128] of one kv head."""
    pos = length - n + np.arange(n)
    key = np.arange(length)
    mask = np.broadcast_to((key <= pos[:, None])[:, None], (n, q.shape[1], length)).copy()
    if kmean is None:
        return mask
    for i in range(n):
        if pos[i] < 0:
            continue
        own = pos[i] // block
        for g in range(q.shape[1]):
            score = kmean[:own].astype(np.float64) @ q[i, g]
            order = sorted(range(own), key=lambda j: (-score[j], j))[:topk - 1]
            mask[i, g] &= np.isin(key // block, order + [own])
    return mask


def attend(q, k, v, mask):
    """One kv head: q [n, G, 128], k, v [length, 128], mask [n, G, length] -> out, lse, weights [length], and the
    scores' and values' sizes that the tolerances are made of."""
    z = np.einsum("ngd,sd->ngs", q, k) / np.sqrt(D)
    size = np.einsum("ngd,sd->ngs", np.abs(q), np.abs(k)) / np.sqrt(D)
    z = np.where(mask, z, -np.inf)
    top = np.maximum(z.max(-1, keepdims=True, initial=-np.inf), -1e300)
    e = np.exp(z - top)
    total = e.sum(-1, keepdims=True)
    w = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[..., 0]
    out = np.einsum("ngs,sd->ngd", w, v)
    return {"out": out, "lse": lse, "weights": w.sum((0, 1)), "size": float(np.where(mask, size, 0).max(initial=0.0)),
            "spread": np.einsum("ngs,sd->ngd", w, np.abs(v))}


def evict(acc, length, budget, recent):
    """Indexes that stay, ascending."""
    if length <= budget:
        return np.arange(length)
    older = np.arange(length - recent)
    w = np.where(np.isnan(acc[:len(older)]), -np.inf, acc[:len(older)])
    nan = np.isnan(acc[:len(older)])
    order = sorted(older, key=lambda i: (nan[i], -w[i], i))[:budget - recent]
    return np.concatenate((np.sort(np.array(order, dtype=np.int64)), np.arange(length - recent, length)))
