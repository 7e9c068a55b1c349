"""The 4-bit key/value cache on the GPU against its numpy definition in fp64.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32 at 1):
  scores   128 exact products summed in fp32, in an order and rounding of the tensor core's choosing: at most
           d = 140 * 2u * max sum |q k| / sqrt(128), the few roundings of the scale included;
  weights  relative r = 2 d + 2^-21 (the exponential's and its argument's) + N u (the sum over N keys);
  out      2^-8 |out| (its rounding to bf16) + (r + 2^-11 + N u) * sum w |v| (weights enter the products as fp16);
           fp16 weights end at 2^-37 of the largest: + N * 2^-37 max |v|;
  lse      d + 2^-21 + N u + 4 u |lse|;
  acc      2 r times the weights + (rows + 2) u |acc|.
What is stored, loaded, pooled over few bits and moved is compared bit for bit.
"""
import numpy as np
import pytest

import kv4_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

import block_sparse_long_fwd_b200 as moba  # noqa: E402

U = 2.0**-24


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def ok():
    torch.cuda.synchronize()
    assert moba.device_status() == moba.MOBA_OK


def random_cache(lengths, hkv, capacity, seed, offset=0.5):
    """A cache filled by the reference, with its values: (kv4 on the GPU, [k, v of each sequence])."""
    rng = np.random.default_rng(seed)
    tiles, vals = [], []
    for _ in lengths:
        mu = rng.standard_normal((hkv, 1, 128)) * offset
        k = f64(bf16(rng.standard_normal((hkv, capacity, 128)) + mu))
        v = f64(bf16(rng.standard_normal((hkv, capacity, 128))))
        t = ref.pack(k, v)
        tiles.append(t)
        vals.append(ref.unpack(t))
    return torch.from_numpy(np.stack(tiles)).cuda(), vals


# ------------------------------------------------------------------ append and load


@pytest.mark.parametrize("hkv,starts,news", [
    (1, [0], [1]), (1, [0], [64]), (2, [0], [131]), (3, [63], [2]), (8, [5, 0, 127, 64], [1, 1, 1, 1]),
    (2, [0, 100, 3], [65, 0, 200]), (1, [0, 7], [0, 0]),
])
@pytest.mark.parametrize("with_acc", [False, True])
def test_append_stores_the_defined_bytes_and_nothing_else(hkv, starts, news, with_acc):
    rng = np.random.default_rng(3)
    batch, cap, T = len(news), 320, sum(news)
    k, v = (bf16(rng.standard_normal((T + 5, hkv, 128)) * 2 + 0.3) for _ in "kv")
    cu = np.concatenate(([0], np.cumsum(news)))
    before = rng.integers(0, 256, (batch, hkv, cap // 64, 9216)).astype(np.uint8)
    kv4 = torch.from_numpy(before.copy()).cuda()
    acc = torch.ones(batch, hkv, cap, device="cuda") if with_acc else None
    # five rows lie behind the last sequence
    moba.kv4_append(k.cuda(), v.cuda(), kv4, ints(starts), cu=ints(cu), acc=acc)
    ok()
    want, want_acc = before.copy(), np.ones((batch, hkv, cap))
    for b in range(batch):
        rows = np.zeros((2, hkv, cap, 128))
        at = slice(starts[b], starts[b] + news[b])
        for s, x in enumerate((k, v)):
            rows[s][:, at] = f64(x)[cu[b]:cu[b + 1]].transpose(1, 0, 2)
        new = ref.pack(rows[0], rows[1])
        for t in range(at.start, at.stop):
            tile, i = t // 64, t % 64
            for off in (0, 4608):
                for a, z in ((off + 64 * i, 64), (off + 4096 + 8 * i, 8)):
                    want[b, :, tile, a:a + z] = new[:, tile, a:a + z]
        want_acc[b, :, at] = 0
    assert np.array_equal(kv4.cpu().numpy(), want)
    if with_acc:
        assert np.array_equal(acc.cpu().numpy(), want_acc)


def test_append_of_awkward_values():
    # NaN, infinities, more than the largest stored value, subnormals, a span of one bf16 step, scales on both
    # sides of a tie (255 and 272 are 17 and 18.13 times 15)
    rng = np.random.default_rng(9)
    x = f64(bf16(rng.standard_normal((64, 1, 128)) * np.exp2(rng.integers(-30, 16, (64, 1, 4))).repeat(32, -1)))
    x[0, 0, :8] = [np.nan, np.inf, -np.inf, 3e38, -3e38, 1e-40, -1e-40, 0]
    x[1] = 0.0
    x[2] = 7.0
    x[3] = -7.0
    x[4] = np.resize(np.array([0.0, 255.0, 8.5, 25.5, 17.0]), 128)
    x[5] = np.resize(np.array([-1.0, 1.0, 0.5, -0.5]) * 2.0**-15, 128)
    x[6] = np.resize(np.arange(-9, 10) * 4.5, 128)
    x[7] = np.nan
    kv4 = moba.kv4_cache(1, 1, 64)
    moba.kv4_append(bf16(x).cuda(), bf16(-x).cuda(), kv4, ints([0]))
    k, v = moba.kv4_load(kv4, ints([64]), 64)
    ok()
    assert np.array_equal(f64(k)[0, :, 0], ref.stored(f64(bf16(x)))[:, 0])
    assert np.array_equal(f64(v)[0, :, 0], ref.stored(f64(bf16(-x)))[:, 0])


def test_append_without_offsets_takes_the_same_number_for_each():
    rng = np.random.default_rng(4)
    k, v = (bf16(rng.standard_normal((6, 2, 128))) for _ in "kv")
    kv4 = moba.kv4_cache(3, 2, 64)
    moba.kv4_append(k.cuda(), v.cuda(), kv4, ints([0, 10, 62]))
    got = moba.kv4_load(kv4, ints([2, 12, 64]), 2, first=ints([0, 10, 62]))
    ok()
    for x, y in zip((k, v), got):
        assert np.array_equal(f64(y), ref.stored(f64(x)).reshape(3, 2, 2, 128))


def test_tokens_without_room_are_skipped_and_reported():
    kv4 = moba.kv4_cache(2, 1, 64)
    x = torch.ones(4, 1, 128, dtype=torch.bfloat16, device="cuda")
    moba.kv4_append(x, x, kv4, ints([63, 0]))
    assert moba.device_status() == moba.MOBA_ERR_DEVICE_CHECK
    moba.kv4_append(x, x, kv4, ints([-1, 3]))
    assert moba.device_status() == moba.MOBA_ERR_DEVICE_CHECK
    k, _ = moba.kv4_load(kv4, ints([64, 64]), 64)
    ok()
    want = np.zeros((2, 64))
    want[0, [63, 0]] = want[1, [0, 1, 3, 4]] = 1
    assert np.array_equal(f64(k)[:, :, 0].max(-1) > 0.5, want > 0)


@pytest.mark.parametrize("n,first", [(1, None), (70, None), (33, [0, 60, 250]), (256, [-3, 255, 100])])
def test_load_gives_zero_outside_the_sequence(n, first):
    lengths = [0, 77, 256]
    kv4, vals = random_cache(lengths, 2, 256, 7)
    k, v = moba.kv4_load(kv4, ints(lengths), n, first=None if first is None else ints(first))
    ok()
    for b, L in enumerate(lengths):
        at = (first[b] if first else 0) + np.arange(n)
        inside = (at >= 0) & (at < L)
        for got, x in zip((k, v), vals[b]):
            want = np.where(inside[:, None, None], x.transpose(1, 0, 2)[at.clip(0, 255)], 0)
            assert np.array_equal(f64(got[b]), want)


# ------------------------------------------------------------------ pool


@pytest.mark.parametrize("hkv,lengths,block", [
    (1, [128], 128), (1, [127], 128), (2, [0, 1000, 128 * 7, 1024], 128), (3, [1000, 1023], 256), (1, [1024], 1024),
    (2, [1024, 700], 384),
])
def test_pool_gives_the_means_of_complete_blocks(hkv, lengths, block):
    cap = 1024
    kv4, vals = random_cache(lengths, hkv, cap, 11)
    m = moba.kv4_pool(kv4, ints(lengths), block)
    ok()
    assert m.shape == (len(lengths), hkv, cap // block, 128)
    for b, L in enumerate(lengths):
        want = ref.means(vals[b][0], L, block, cap // block)
        # one rounding of the mean, and of each of at most `block` partial sums of at most sum |k|
        size = ref.means(np.abs(vals[b][0]), L, block, cap // block)
        assert (np.abs(f64(m[b]) - want) <= (block + 1) * U * size).all()
        assert (f64(m[b])[:, L // block:] == 0).all()


@pytest.mark.parametrize("block", [1536, 4096, 8192])
def test_pool_of_large_blocks_by_several_ctas(block):
    hkv, cap, lengths = 2, 8192, [8192, 5000]
    kv4, vals = random_cache(lengths, hkv, cap, 12)
    m = moba.kv4_pool(kv4, ints(lengths), block)
    ok()
    for b, L in enumerate(lengths):
        want, size = (ref.means(x, L, block, cap // block) for x in (vals[b][0], np.abs(vals[b][0])))
        assert (np.abs(f64(m[b]) - want) <= (block + 1) * U * size).all()
        assert (f64(m[b])[:, L // block:] == 0).all()


@pytest.mark.parametrize("block,blocks", [(128, 1), (128, 2), (128, 3), (128, 5), (256, 1), (256, 3), (512, 1)])
def test_pool_writes_the_means_and_nothing_behind_them(block, blocks):
    # a CTA takes several small blocks: the last one may have fewer
    cap, hkv = block * blocks + 64, 2
    lengths = [cap, block * blocks - 1]
    kv4, vals = random_cache(lengths, hkv, cap, 13)
    buf = torch.full((2 * hkv * blocks + 4, 128), 7.0, device="cuda")
    m = moba.kv4_pool(kv4, ints(lengths), block, kmean=buf[:2 * hkv * blocks].view(2, hkv, blocks, 128))
    ok()
    assert (buf[2 * hkv * blocks:] == 7).all()
    for b, L in enumerate(lengths):
        want, size = (ref.means(x, L, block, blocks) for x in (vals[b][0], np.abs(vals[b][0])))
        assert (np.abs(f64(m[b]) - want) <= (block + 1) * U * size).all()
        assert (f64(m[b])[:, L // block:] == 0).all()


def test_pool_of_less_than_a_block_is_empty():
    kv4, _ = random_cache([64], 1, 64, 1)
    assert moba.kv4_pool(kv4, ints([64]), 128).shape == (1, 1, 0, 128)


# ------------------------------------------------------------------ attend


def check_attend(got, q, vals, lengths, news, hkv, sparse=None, kmean=None, rows=None):
    """got = (out, lse, acc or None, acc before); q [T, Hq, 128] fp64."""
    out, lse, acc, acc0 = got
    out, lse = f64(out), f64(lse)
    G = q.shape[1] // hkv
    t = 0
    for b, (L, n) in enumerate(zip(lengths, news)):
        for h in range(hkv):
            qq = q[t:t + n, h * G:(h + 1) * G]
            k, v = (x[h, :L] for x in vals[b])
            mask = ref.seen(qq, L, n, None if kmean is None else kmean[b, h], *(sparse or ()))
            r = ref.attend(qq, k, v, mask)
            d = 140 * 2 * U * r["size"]
            w = 2 * d + 2.0**-21 + L * U
            top = np.abs(v).max(initial=0.0)
            tol = 2.0**-8 * np.abs(r["out"]) + (w + 2.0**-11 + L * U) * r["spread"] + L * 2.0**-37 * top
            o = out[t:t + n, h * G:(h + 1) * G]
            off = np.abs(o - r["out"])
            assert bool((off <= tol).all()), (b, h, off.max(), (off / tol).max())
            e = lse[h * G:(h + 1) * G, t:t + n].T
            none = ~mask.any(-1)
            r["lse"][none] = 0
            assert (e[none] == -np.inf).all() and (o[none] == 0).all()
            e = np.where(none, 0, e)
            off, tol = np.abs(e - r["lse"])[~none], (d + 2.0**-21 + L * U + 4 * U * np.abs(r["lse"]))[~none]
            assert bool((off <= tol).all()), (b, h, off.max(), (off / tol).max())
            if acc is not None:
                a, a0 = f64(acc[b, h]), f64(acc0[b, h])
                want = a0[:L] + r["weights"]
                off, tol = np.abs(a[:L] - want), 2 * w * r["weights"] + (n * G + 2) * U * want
                assert bool((off <= tol).all()), (b, h, off.max(), (off / tol).max())
                assert np.array_equal(a[L:], a0[L:])
        t += n


def attend_case(hkv, G, lengths, news, sparse=None, acc=True, seed=0, cap=None, qscale=1.0, pad=3, distinct=None):
    """distinct: so many different sequences, one after the other again and again."""
    rng = np.random.default_rng(seed + 100)
    cap = cap or -(-max(max(lengths), 1) // 64) * 64 + 64
    kv4, vals = random_cache(lengths[:distinct], hkv, cap, seed)
    if distinct:
        at = np.arange(len(lengths)) % distinct
        kv4, vals = kv4[torch.from_numpy(at).cuda()], [vals[i] for i in at]
    T = sum(news)
    q = bf16(rng.standard_normal((T + pad, hkv * G, 128)) * qscale)
    kmean = moba.kv4_pool(kv4, ints(lengths), sparse[0]) if sparse else None
    a0 = torch.from_numpy(rng.random((len(lengths), hkv, cap)).astype(np.float32)).cuda() if acc else None
    a = a0.clone() if acc else None
    out = torch.full((T + pad, hkv * G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hkv * G, T + pad), 7.0, device="cuda")
    cu = ints(np.concatenate(([0], np.cumsum(news))))
    more = {"kmean": kmean, "block_size": sparse[0], "topk": sparse[1]} if sparse else {}
    moba.kv4_attend(q.cuda(), kv4, ints(lengths), cu=cu, acc=a, out=out, lse=lse, **more)
    ok()
    # rows behind the last sequence are left alone
    assert (out[T:] == 7).all() and (lse[:, T:] == 7).all()
    check_attend((out[:T], lse[:, :T], a, a0), f64(q)[:T], vals, lengths, news, hkv, sparse,
                 f64(kmean) if sparse else None)


DENSE = [
    # hkv, G, lengths, new tokens
    (1, 1, [1], [1]),
    (1, 1, [64], [1]),
    (1, 1, [65], [1]),
    (2, 4, [63], [1]),
    (1, 1, [4096], [1]),
    (2, 4, [1000], [1]),
    (8, 4, [130, 1, 700, 64, 65], [1, 1, 1, 1, 1]),
    (1, 8, [777], [1]),
    (1, 16, [777], [1]),
    (2, 3, [500, 129], [1, 1]),
    (1, 5, [321], [7]),
    (2, 4, [300, 64, 1, 200], [2, 64, 1, 0]),   # a sequence without queries
    (1, 2, [0, 90], [0, 1]),                    # an empty one
    (1, 2, [3, 90], [5, 2]),                    # more queries than tokens: rows without keys
    (1, 1, [2000], [300]),
    (2, 4, [700], [129]),
    (1, 40, [200], [9]),
    (2, 4, [1500, 900], [200, 77]),             # many rows: units of 256, the last of them short
    (1, 8, [128], [128]),                       # a whole prompt
    (1, 1, [5000], [257]),                      # a single row in the second tile
    (1, 1, [4100], [128]),
    (1, 3, [77, 300, 0, 64], [90, 100, 70, 64]),  # more queries than tokens
    (1, 70, [1000, 130], [1, 1]),               # one token, many heads of a kv head
]


@pytest.mark.parametrize("hkv,G,lengths,news", DENSE)
@pytest.mark.parametrize("acc", [False, True])
def test_attention_over_every_key(hkv, G, lengths, news, acc):
    attend_case(hkv, G, lengths, news, acc=acc, seed=len(lengths) + G)


def test_many_short_sequences_with_empty_ones_between():
    # far more units than CTAs, most of them without tiles: every range walks over several, and past the kept ones
    rng = np.random.default_rng(2)
    lengths = [int(x) for x in np.where(rng.random(700) < 0.3, rng.integers(1, 90, 700), 0)]
    attend_case(1, 2, lengths, [1 if L else 0 for L in lengths], acc=False, seed=1, cap=128)
    attend_case(1, 2, lengths, [1] * 700, acc=False, seed=1, cap=128)  # a query without keys for each empty one


def test_more_sequences_than_a_cta_copies():
    # the offsets and lengths of 9000 sequences do not fit beside the pieces: they are read where they lie
    attend_case(1, 2, [1 + 7 * i % 64 for i in range(9000)], [1] * 9000, acc=False, seed=4, cap=64, distinct=16)


def test_many_sequences_with_many_rows_each():
    # a CTA of the kernel for many rows walks over more units than it keeps beside it
    attend_case(1, 7, [20 + i % 45 for i in range(2600)], [7 + i % 2 for i in range(2600)], seed=5, cap=64, distinct=16)


SPARSE = [
    # hkv, G, lengths, new tokens, block, topk
    (1, 1, [1], [1], 128, 2),
    (1, 1, [128], [1], 128, 1),
    (1, 1, [129], [1], 128, 2),
    (2, 4, [2000], [1], 128, 4),
    (1, 2, [1300, 100, 640, 641], [1, 1, 1, 1], 128, 3),
    (2, 4, [1500], [9], 256, 3),
    (1, 3, [900, 1025], [200, 3], 128, 2),
    (1, 1, [4000], [1], 128, 17),
    (1, 8, [3000], [2], 384, 3),
    (1, 16, [1100], [5], 128, 3),
    (1, 4, [700, 0, 3], [3, 0, 4], 128, 2),
    (1, 2, [600], [1], 128, 1),
    # many rows: masks a row and block, units of 256 rows over several blocks of picks
    (2, 4, [1500], [200], 256, 3),
    (1, 8, [700, 0, 3, 1300, 260], [90, 70, 80, 64, 0], 128, 2),
    (2, 3, [1100, 1000], [300, 1], 384, 2),
    (1, 1, [2000], [513], 128, 4),
    (1, 40, [300], [9], 128, 1),
    (1, 2, [40000], [3], 128, 5),               # more past blocks than a warp keeps in registers
    (2, 1, [50 + i % 400 for i in range(300)], [1] * 300, 128, 2),  # more sequences than the gate copies
]


@pytest.mark.parametrize("hkv,G,lengths,news,block,topk", SPARSE)
@pytest.mark.parametrize("acc", [False, True])
def test_attention_over_chosen_blocks(hkv, G, lengths, news, block, topk, acc):
    attend_case(hkv, G, lengths, news, sparse=(block, topk), acc=acc, seed=block + topk)


@pytest.mark.parametrize("acc", [False, True])
def test_many_rows_that_choose_a_small_part_of_a_large_cache(acc):
    attend_case(1, 4, [900, 130], [100, 60], sparse=(128, 1), acc=acc, seed=6, cap=16384)


@pytest.mark.parametrize("qscale", [1e-4, 30.0])
def test_attention_of_small_and_large_scores(qscale):
    # at 30 the softmax sits on a few keys and the running maximum moves far; the tolerances grow with the scores
    attend_case(2, 4, [3000], [1], qscale=qscale, seed=3)
    attend_case(1, 2, [1000], [40], qscale=qscale, seed=4)


@pytest.mark.parametrize("kscale,vscale", [(2.0**-9, 2.0**-9), (1.0, 5000.0), (6000.0, 1.0), (2000.0, 2.0**-12)])
def test_attention_over_keys_and_values_of_every_size(kscale, vscale):
    # scales from the smallest to the largest: nothing overflows or flushes on the way to the products. One channel
    # in 32 is twenty times the others (a zero point at either end of its range)
    rng = np.random.default_rng(17)
    L, hkv, G = 500, 2, 4
    x = rng.standard_normal((2, hkv, 512, 128))
    x[..., ::32] *= np.where(rng.random((2, hkv, 512, 4)) < 0.5, 20, 1)
    k, v = x[0] * kscale, x[1] * vscale
    tiles = ref.pack(f64(bf16(k)), f64(bf16(v)))
    q = bf16(rng.standard_normal((1, hkv * G, 128)) / kscale)
    a = torch.zeros(1, hkv, 512, device="cuda")
    out, lse = moba.kv4_attend(q.cuda(), torch.from_numpy(tiles[None]).cuda(), ints([L]), acc=a)
    ok()
    check_attend((out, lse, a, torch.zeros_like(a)), f64(q), [ref.unpack(tiles)], [L], [1], hkv)


def test_equal_scores_go_to_the_lower_block():
    # blocks 1, 3 and 4 are equal and best; topk 3 takes 1 and 3 beside the own block
    hkv, cap, B = 1, 1024, 128
    k = np.zeros((hkv, cap, 128))
    for j, x in enumerate([0.0, 1.0, 0.5, 1.0, 1.0, 0.25]):
        k[:, j * B:(j + 1) * B] = x
    v = np.zeros((hkv, cap, 128))
    v[0] = (np.arange(cap) // B)[:, None] == np.arange(128)
    kv4 = torch.from_numpy(ref.pack(k, v)[None]).cuda()
    q = torch.ones(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    length = ints([6 * B + 1])
    out, _ = moba.kv4_attend(q, kv4, length, kmean=moba.kv4_pool(kv4, length, B), block_size=B, topk=3)
    ok()
    assert set(np.nonzero(f64(out)[0, 0] > 0)[0]) == {1, 3, 6}


def test_zero_scores_of_either_sign_are_equal():
    # a query of zeros scores -0 against a mean of negative numbers: a tie all the same
    cap, B = 1024, 128
    k = np.ones((1, cap, 128))
    k[:, :2 * B] = -1
    v = np.zeros((1, cap, 128))
    v[0] = (np.arange(cap) // B)[:, None] == np.arange(128)
    kv4 = torch.from_numpy(ref.pack(k, v)[None]).cuda()
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    length = ints([6 * B + 1])
    out, _ = moba.kv4_attend(q, kv4, length, kmean=moba.kv4_pool(kv4, length, B), block_size=B, topk=3)
    ok()
    assert set(np.nonzero(f64(out)[0, 0] > 0)[0]) == {0, 1, 6}


def test_garbage_behind_the_last_token_is_not_read_into_results():
    # what lies behind the length, codes and parameters, may be anything
    hkv, L, cap = 2, 333, 512
    kv4, vals = random_cache([L], hkv, cap, 5)
    q = bf16(np.random.default_rng(1).standard_normal((1, 8, 128))).cuda()
    want = moba.kv4_attend(q, kv4, ints([L]))
    dirty = kv4.clone()
    for tile in range(cap // 64):
        for i in range(64):
            if tile * 64 + i >= L:
                for off in (0, 4608):
                    dirty[:, :, tile, off + 64 * i:off + 64 * i + 64] = 0xFF
                    dirty[:, :, tile, off + 4096 + 8 * i:off + 4096 + 8 * i + 8] = 0xFF
    got = moba.kv4_attend(q, dirty, ints([L]))
    a, b = (torch.zeros(1, hkv, cap, device="cuda") for _ in "ab")
    moba.kv4_attend(q, kv4, ints([L]), acc=a)
    moba.kv4_attend(q, dirty, ints([L]), acc=b)
    ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 9, 100])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(n, bad):
    hkv, L = 2, 700
    kv4, _ = random_cache([L], hkv, 704, 5)
    q = bf16(np.random.default_rng(1).standard_normal((n, 4, 128))).cuda()
    want = moba.kv4_attend(q, kv4, ints([L]))
    dirty = q.clone()
    dirty[n // 2, 1, 5] = bad
    got = moba.kv4_attend(dirty, kv4, ints([L]))
    ok()
    other = torch.ones(n, 4, dtype=torch.bool, device="cuda")
    other[n // 2, 1] = False
    assert torch.equal(got[0][other], want[0][other]) and torch.equal(got[1].T[other], want[1].T[other])
    assert got[0][~other].isnan().all() and got[1].T[~other].isnan().all()


def test_tensors_of_another_kind_are_refused():
    kv4, _ = random_cache([64], 2, 128, 5)
    q, acc, L = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, 128, device="cuda"), ints([64])
    k = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
    moba.kv4_attend(q, kv4, L, acc=acc)
    for call in (
        lambda: moba.kv4_attend(q.half(), kv4, L), lambda: moba.kv4_attend(q.transpose(0, 1), kv4, L),
        lambda: moba.kv4_attend(q[..., :64], kv4, L), lambda: moba.kv4_attend(q, kv4[:, :, ::2], L),
        lambda: moba.kv4_attend(q, kv4, L.long()), lambda: moba.kv4_attend(q, kv4, L.cpu()),
        lambda: moba.kv4_attend(q, kv4, L, acc=acc[..., :64]), lambda: moba.kv4_attend(q, kv4, L, acc=acc.double()),
        lambda: moba.kv4_attend(q, kv4, L, cu=ints([0, 1, 1])), lambda: moba.kv4_attend(q, kv4, L, topk=3),
        lambda: moba.kv4_attend(q, kv4, L, kmean=torch.zeros(1, 2, 1, 128, device="cuda")),
        lambda: moba.kv4_attend(q, kv4, L, kmean=torch.zeros(1, 1, 1, 128, device="cuda"), block_size=128, topk=2),
        lambda: moba.kv4_append(k, k[:, :1], kv4, L), lambda: moba.kv4_append(k.float(), k.float(), kv4, L),
        lambda: moba.kv4_append(k, k, kv4, ints([0, 0])), lambda: moba.kv4_load(kv4, L, 129), lambda: moba.kv4_load(kv4, L, -1),
        lambda: moba.kv4_pool(kv4, L, 0), lambda: moba.kv4_pool(kv4.view(torch.int8), L, 128),
        lambda: moba.kv4_evict(kv4, acc, L, 200, 0, moba.kv4_cache(1, 2, 128), acc.clone()),
        lambda: moba.kv4_evict(kv4, acc, L, 64, 65, moba.kv4_cache(1, 2, 128), acc.clone()),
        lambda: moba.kv4_evict(kv4, acc, L, 64, 0, moba.kv4_cache(1, 1, 128), acc.clone()),
    ):
        with pytest.raises((ValueError, moba.MobaError)):
            call()
    with pytest.raises(moba.MobaError):
        moba.kv4_pool(kv4, L, 100)
    with pytest.raises(moba.MobaError):
        moba.kv4_evict(kv4, acc, L, 64, 0, kv4, acc.clone())
    ok()


def test_more_pairs_than_are_counted_are_refused():
    # a million tokens against room for 2^30: refused before anything is launched or read
    x = torch.zeros(64, device="cuda").data_ptr()
    rc = moba.lib().moba_kv4_attend(x, 1 << 20, None, x, x, None, 1, 1, 1, 128, 1 << 30, 0, 0, None, x, x, 0)
    assert rc == moba.MOBA_ERR_UNSUPPORTED and "chunks" in moba.last_error()
    ok()


def test_a_length_beyond_the_capacity_is_cut_and_reported():
    kv4, vals = random_cache([128], 1, 128, 5)
    q = bf16(np.random.default_rng(1).standard_normal((1, 2, 128))).cuda()
    want = moba.kv4_attend(q, kv4, ints([128]))
    ok()
    got = moba.kv4_attend(q, kv4, ints([1000]))
    assert moba.device_status() == moba.MOBA_ERR_DEVICE_CHECK
    assert torch.equal(got[0], want[0])
    ok()


def test_the_same_call_gives_the_same_bits():
    lengths = [5000, 33, 2000]
    kv4, _ = random_cache(lengths, 2, 5056, 2)
    q = bf16(np.random.default_rng(1).standard_normal((6, 8, 128))).cuda()
    runs = []
    for _ in range(3):
        acc = torch.zeros(3, 2, 5056, device="cuda")
        runs.append((*moba.kv4_attend(q, kv4, ints(lengths), acc=acc), acc))
    ok()
    for r in runs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(r, runs[0]))


# ------------------------------------------------------------------ evict


def evict_case(hkv, lengths, budget, recent, acc, cap, dcap, seed=0):
    kv4, vals = random_cache(lengths, hkv, cap, seed)
    dst = torch.full((len(lengths), hkv, dcap // 64, 9216), 0xAB, dtype=torch.uint8, device="cuda")
    dst_acc = torch.full((len(lengths), hkv, dcap), 5.0, device="cuda")
    acc = torch.from_numpy(acc.astype(np.float32)).cuda()
    new, kept = moba.kv4_evict(kv4, acc, ints(lengths), budget, recent, dst, dst_acc)
    k, v = moba.kv4_load(dst, new, min(budget, dcap))
    ok()
    assert new.tolist() == [min(L, budget) for L in lengths]
    for b, L in enumerate(lengths):
        for h in range(hkv):
            a = acc[b, h].double().cpu().numpy()
            want = ref.evict(a, L, budget, recent)
            n = len(want)
            assert np.array_equal(kept[b, h, :n].cpu().numpy(), want) and (kept[b, h, n:] == -1).all()
            assert np.array_equal(f64(k[b, :n, h]), vals[b][0][h, want])
            assert np.array_equal(f64(v[b, :n, h]), vals[b][1][h, want])
            assert np.array_equal(f64(dst_acc[b, h, :n]), a[want], equal_nan=True)
            assert (dst_acc[b, h, n:] == 5).all()
            raw = dst[b, h].cpu().numpy()
            for t in range(n, dcap):  # places behind the kept tokens are left alone
                for off in (0, 4608):
                    i = t % 64
                    assert (raw[t // 64, off + 64 * i:off + 64 * i + 64] == 0xAB).all()
                    assert (raw[t // 64, off + 4096 + 8 * i:off + 4096 + 8 * i + 8] == 0xAB).all()


@pytest.mark.parametrize("hkv,lengths,budget,recent", [
    (1, [1], 1, 0), (1, [2], 1, 0), (1, [2], 1, 1), (1, [64], 64, 3), (1, [65], 64, 64), (2, [500, 0, 100, 101], 100, 10),
    (1, [5000], 37, 0), (1, [5000], 4999, 1), (3, [1025, 2049], 1000, 1000), (1, [4000], 3, 2),
])
def test_evict_keeps_the_heaviest_and_the_last(hkv, lengths, budget, recent):
    cap = -(-max(lengths) // 64) * 64
    rng = np.random.default_rng(budget)
    acc = np.exp(2 * rng.standard_normal((len(lengths), hkv, cap))) * (rng.random((len(lengths), hkv, cap)) > 0.1)
    evict_case(hkv, lengths, budget, recent, acc, cap, -(-budget // 64) * 64 + 64)


@pytest.mark.parametrize("kind", ["equal", "few", "zero", "signed", "special", "close"])
def test_evict_of_awkward_weights(kind):
    cap, rng = 2048, np.random.default_rng(8)
    acc = {"equal": lambda: np.full((1, 2, cap), 0.25), "few": lambda: rng.integers(0, 3, (1, 2, cap)) / 2.0,
           "zero": lambda: np.where(rng.random((1, 2, cap)) < 0.5, 0.0, -0.0),
           "signed": lambda: rng.standard_normal((1, 2, cap)),
           "special": lambda: rng.choice([np.nan, np.inf, -np.inf, 0.0, 1e-45, 1.0], (1, 2, cap)),
           "close": lambda: 1.0 + rng.integers(0, 4, (1, 2, cap)) * 2.0**-23}[kind]()
    evict_case(2, [2000], 700, 33, acc, cap, 704, seed=1)


@pytest.mark.parametrize("hkv,length,budget,recent,distinct", [
    (1, 300000, 5000, 100, 1 << 20), (1, 300000, 299000, 0, 1 << 20), (1, 280001, 70000, 64, 50), (160, 33000, 900, 10, 1 << 20),
])
def test_evict_from_long_caches(hkv, length, budget, recent, distinct):
    # parts longer than one sweep of a CTA, read again in each pass; whatever the cache holds is moved as it is
    cap, dcap = -(-length // 64) * 64, -(-budget // 64) * 64
    g = torch.Generator(device="cuda").manual_seed(7)
    kv4 = torch.randint(0, 256, (1, hkv, cap // 64, 9216), dtype=torch.uint8, device="cuda", generator=g)
    acc = torch.randint(0, distinct, (1, hkv, cap), device="cuda", generator=g).float()
    dst, dst_acc = moba.kv4_cache(1, hkv, dcap), torch.zeros(1, hkv, dcap, device="cuda")
    new, kept = moba.kv4_evict(kv4, acc, ints([length]), budget, recent, dst, dst_acc)
    ok()
    assert new.tolist() == [budget]
    for h in range(0, hkv, 40):
        want = ref.evict(f64(acc[0, h]), length, budget, recent)
        assert np.array_equal(kept[0, h].cpu().numpy(), want)
        assert np.array_equal(dst_acc[0, h, :budget].cpu().numpy(), acc[0, h].cpu().numpy()[want])
        src, to = kv4[0, h].cpu().numpy(), dst[0, h].cpu().numpy()
        for new_at, old_at in [(i, want[i]) for i in (0, 1, budget // 2, budget - 1)]:
            for off in (0, 4096):  # keys: codes and parameters (the values' codes change places with the token's index)
                n = 64 if off == 0 else 8
                a, b = off + n * (old_at % 64), off + n * (new_at % 64)
                assert np.array_equal(src[old_at // 64, a:a + n], to[new_at // 64, b:b + n])


# ------------------------------------------------------------------ together, streams, graphs


def test_a_request_from_prompt_to_eviction():
    """A prompt is stored, attended, decoded with weights, evicted, and decoded on: every step against fp64."""
    rng = np.random.default_rng(21)
    batch, hkv, G, cap, B, topk = 2, 2, 2, 1024, 128, 3
    prompts = [700, 451]
    cu = np.concatenate(([0], np.cumsum(prompts)))
    kv4, acc = moba.kv4_cache(batch, hkv, cap), torch.zeros(batch, hkv, cap, device="cuda")
    k, v = (bf16(rng.standard_normal((sum(prompts), hkv, 128))) for _ in "kv")
    lengths = ints([0, 0])
    moba.kv4_append(k.cuda(), v.cuda(), kv4, lengths, cu=ints(cu), acc=acc)
    lengths = lengths + ints(prompts)
    vals = [[ref.stored(f64(x)[cu[b]:cu[b + 1]].transpose(1, 0, 2)) for x in (k, v)] for b in range(batch)]
    q = bf16(rng.standard_normal((16 * batch, hkv * G, 128)))  # the prompts' last 16 tokens
    a0 = acc.clone()
    out, lse = moba.kv4_attend(q.cuda(), kv4, lengths, acc=acc)
    ok()
    check_attend((out, lse, acc, a0), f64(q), vals, prompts, [16, 16], hkv)

    def step(kv4, acc, lengths, vals, sparse):
        k, v = (bf16(rng.standard_normal((batch, hkv, 128))) for _ in "kv")
        q = bf16(rng.standard_normal((batch, hkv * G, 128)))
        moba.kv4_append(k.cuda(), v.cuda(), kv4, lengths, acc=acc)
        lengths = lengths + 1
        vals = [[np.concatenate((x, ref.stored(f64(y)[b][:, None])), 1) for x, y in zip(vals[b], (k, v))]
                for b in range(batch)]
        kmean = moba.kv4_pool(kv4, lengths, B) if sparse else None
        a0 = acc.clone()
        more = {"kmean": kmean, "block_size": B, "topk": topk} if sparse else {}
        out, lse = moba.kv4_attend(q.cuda(), kv4, lengths, acc=acc, **more)
        ok()
        check_attend((out, lse, acc, a0), f64(q), vals, lengths.tolist(), [1, 1], hkv, (B, topk) if sparse else None,
                     f64(kmean) if sparse else None)
        return lengths, vals

    for i in range(4):
        lengths, vals = step(kv4, acc, lengths, vals, i % 2 == 0)
    weights = f64(acc)
    dst, dst_acc = moba.kv4_cache(batch, hkv, 512), torch.zeros(batch, hkv, 512, device="cuda")
    old = lengths.tolist()
    lengths, kept = moba.kv4_evict(kv4, acc, lengths, 400, 32, dst, dst_acc)
    ok()
    new = []
    for b in range(batch):
        at = [ref.evict(weights[b, h], old[b], 400, 32) for h in range(hkv)]
        assert all(np.array_equal(kept[b, h].cpu().numpy(), at[h]) for h in range(hkv))
        new.append([np.stack([x[h, at[h]] for h in range(hkv)]) for x in vals[b]])
    for i in range(3):
        lengths, new = step(dst, dst_acc, lengths, new, i % 2 == 0)
    # and the cache read back serves the framework's bf16 attention
    k, v = moba.kv4_load(dst, lengths, 403)
    q = bf16(rng.standard_normal((3, hkv * G, 128))).cuda()
    o1, e1 = moba.fwd_chunk(q, k[0], v[0], 128, 64)
    o2, e2 = moba.kv4_attend(torch.cat((q, q)), dst, lengths)
    ok()
    assert (o1 - o2[:3]).abs().max() <= 2e-2 and (e1 - e2[:, :3]).abs().max() <= 1e-3


def test_calls_on_other_streams():
    lengths = [900, 1500]
    kv4, vals = random_cache(lengths, 2, 1536, 2)
    q = bf16(np.random.default_rng(1).standard_normal((2, 8, 128))).cuda()
    lens = ints(lengths)
    want = moba.kv4_attend(q, kv4, lens)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in (a, b):
            with torch.cuda.stream(s):
                got.append(moba.kv4_attend(q, kv4, lens))
    got.append(moba.kv4_attend(q, kv4, lens, stream=a))
    ok()
    for o, e in got:
        assert torch.equal(o, want[0]) and torch.equal(e, want[1])


def pool_of(x):
    """The stream whose memory a tensor lies in."""
    at = x.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's memory")


def stream_calls():
    kv4, _ = random_cache([256, 200], 2, 256, 2)
    L, acc = ints([256, 200]), torch.zeros(2, 2, 256, device="cuda")
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(300, 2, 128, dtype=torch.bfloat16, device="cuda")
    dst, dst_acc = moba.kv4_cache(2, 2, 128), torch.zeros(2, 2, 128, device="cuda")
    out, lse = moba.fwd(p, p, p, 128, 2)
    return {
        "load": lambda s: moba.kv4_load(kv4, L, 256, stream=s),
        "pool": lambda s: [moba.kv4_pool(kv4, L, 128, stream=s)],
        "attend": lambda s: moba.kv4_attend(q, kv4, L, acc=acc, stream=s),
        "evict": lambda s: moba.kv4_evict(kv4, acc, L, 100, 10, dst, dst_acc, stream=s),
        "fwd": lambda s: moba.fwd(p, p, p, 128, 2, stream=s),
        "fwd_chunk": lambda s: moba.fwd_chunk(p[200:], p, p, 128, 2, stream=s),
        "fwd_varlen": lambda s: moba.fwd_varlen(p, p, p, [0, 100, 300], 128, 2, stream=s),
        "bwd": lambda s: moba.bwd(p, p, p, out, lse, p, 128, 2, stream=s),
        "key means": lambda s: [moba.pool(p, 128, stream=s)],
        "gate": lambda s: [moba.gate(p, moba.pool(p, 128), 2, 128, 2, stream=s)],
    }


@pytest.mark.parametrize("name", ["load", "pool", "attend", "evict", "fwd", "fwd_chunk", "fwd_varlen", "bwd", "key means", "gate"])
def test_outputs_lie_in_the_memory_of_the_stream_that_writes_them(name):
    call = stream_calls()[name]
    here, side = torch.cuda.current_stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    assert all(pool_of(x) == here.cuda_stream for x in call(None))
    assert all(pool_of(x) == side.cuda_stream for x in call(side))
    handle = type("handle", (), {"cuda_stream": side.cuda_stream})  # a stream of another library
    assert all(pool_of(x) == side.cuda_stream for x in call(handle))
    ok()


@pytest.mark.parametrize("cycles", [200_000_000, 2_000_000_000])
def test_tensors_dropped_after_a_call_on_another_stream_are_not_handed_out_at_once(cycles):
    kv4, _ = random_cache([1000], 2, 1024, 2)
    L = ints([1000])
    side = torch.cuda.Stream()
    want = moba.kv4_load(kv4, L, 1000)
    at, size = kv4.data_ptr(), kv4.shape
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(cycles)  # a tenth of a second of work, or one, before the call
    got = moba.kv4_load(kv4, L, 1000, stream=side)
    del kv4
    taken = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
    waiting = not side.query()  # the host has not slept itself
    assert not waiting or at not in {x.data_ptr() for x in taken}
    here = torch.cuda.current_stream()
    here.wait_stream(side)
    torch.cuda._sleep(cycles)
    copy = [x.clone() for x in got]  # read here, later
    places, shape = {x.data_ptr() for x in got}, got[0].shape
    del got
    with torch.cuda.stream(side):
        taken = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    waiting = not here.query()
    assert not waiting or not places & {x.data_ptr() for x in taken}
    ok()
    assert all(torch.equal(x, y) for x, y in zip(copy, want))


@pytest.mark.parametrize("sparse", [False, True])
def test_a_captured_decode_step_takes_the_lengths_of_its_replay(sparse):
    rng = np.random.default_rng(6)
    hkv, G, cap, B = 2, 4, 1024, 128
    kv4, vals = random_cache([600, 300], hkv, cap, 2)
    lengths, acc = ints([600, 300]), torch.zeros(2, hkv, cap, device="cuda")
    k, v = (torch.zeros(2, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q = torch.zeros(2, hkv * G, 128, dtype=torch.bfloat16, device="cuda")
    kmean = moba.kv4_pool(kv4, lengths, B)
    out, lse = torch.empty_like(q), torch.empty(hkv * G, 2, device="cuda")
    more = {"kmean": kmean, "block_size": B, "topk": 3} if sparse else {}

    def step():
        moba.kv4_append(k, v, kv4, lengths, acc=acc)
        lengths.add_(1)
        moba.kv4_pool(kv4, lengths, B, kmean=kmean)
        moba.kv4_attend(q, kv4, lengths, acc=acc, out=out, lse=lse, **more)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    lengths.copy_(ints([600, 300]))
    acc.zero_()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    for g in (g1, g2):  # two captured graphs of the same step, replayed in turn
        with torch.cuda.graph(g):
            step()
    n = [600, 300]
    for i in range(6):
        x = [bf16(rng.standard_normal((2, hkv, 128))) for _ in "kv"]
        y = bf16(rng.standard_normal((2, hkv * G, 128)))
        k.copy_(x[0]), v.copy_(x[1]), q.copy_(y)
        a0 = acc.clone()
        (g1, g2)[i % 2].replay()
        ok()
        for b in range(2):
            for s in range(2):
                vals[b][s][:, n[b]] = ref.stored(f64(x[s])[b])
            a0[b, :, n[b]] = 0
        n = [n[0] + 1, n[1] + 1]
        assert lengths.tolist() == n
        check_attend((out, lse, acc, a0), f64(y), vals, n, [1, 1], hkv, (B, 3) if sparse else None,
                     f64(kmean) if sparse else None)


def test_failed_scratch_allocation_returns_oom(monkeypatch):
    kv4, _ = random_cache([64], 1, 64, 1)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    monkeypatch.setenv("MOBA_TEST_SCRATCH_PAD", str(1 << 46))
    with pytest.raises(moba.MobaError) as e:
        moba.kv4_attend(q, kv4, ints([64]))
    assert e.value.code == moba.MOBA_ERR_OOM
    monkeypatch.delenv("MOBA_TEST_SCRATCH_PAD")
    moba.kv4_attend(q, kv4, ints([64]))
    ok()


def test_calls_without_rows_do_nothing():
    kv4, _ = random_cache([64], 1, 64, 1)
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    moba.kv4_append(none, none, kv4, ints([0]))
    out, lse = moba.kv4_attend(none, kv4, ints([64]))
    k, v = moba.kv4_load(kv4, ints([64]), 0)
    ok()
    assert out.shape == (0, 1, 128) and lse.shape == (1, 0) and k.shape == (1, 0, 1, 128)


def test_offsets_beyond_32_bits():
    # the last head's tiles start beyond 2^32 bytes
    hkv, cap = 8, 64 * 70000
    kv4 = torch.zeros(1, hkv, cap // 64, 9216, dtype=torch.uint8, device="cuda")
    assert kv4.numel() > 1 << 32
    rng = np.random.default_rng(2)
    L = cap - 5
    new = bf16(rng.standard_normal((300, hkv, 128)))
    acc = torch.zeros(1, hkv, cap, device="cuda")
    moba.kv4_append(new.cuda(), new.flip(0).cuda(), kv4, ints([L - 300]))
    k, v = moba.kv4_load(kv4, ints([L]), 300, first=ints([L - 300]))
    ok()
    assert np.array_equal(f64(k)[0], ref.stored(f64(new))) and np.array_equal(f64(v)[0], ref.stored(f64(new))[::-1])
    # zero keys score 0 against every query: their weights are equal, and their values zero
    q = bf16(rng.standard_normal((1, hkv * 2, 128)))
    out, lse = moba.kv4_attend(q.cuda(), kv4, ints([L]), acc=acc)
    ok()
    for h in range(hkv):
        kk, vv = f64(k)[0, :, h], f64(v)[0, :, h]
        z = f64(q)[0, 2 * h:2 * h + 2] @ kk.T / np.sqrt(128)
        total = np.exp(z).sum(-1) + (L - 300)
        want = np.exp(z) @ vv / total[:, None]
        # L sums of equal size: fp32 sums of at most L / 2^10 terms in a chain
        assert np.abs(f64(lse)[2 * h:2 * h + 2, 0] - np.log(total)).max() <= 2.0**-12
        assert (np.abs(f64(out)[0, 2 * h:2 * h + 2] - want) <= 2.0**-7 * np.abs(want) + 2.0**-10 * np.abs(vv).max() * 300 / L).all()
    assert abs(f64(acc)[0].sum(-1) - 2).max() <= 2.0**-8


FEW = [(hkv, G, lengths, news, None) for hkv, G, lengths, news in DENSE]
FEW += [(hkv, G, lengths, news, (block, topk)) for hkv, G, lengths, news, block, topk in SPARSE]
FEW = [c for c in FEW if sum(c[3]) * c[1] <= 8 * len(c[3])]  # at most eight rows a sequence and kv head, on average
FEW += [
    # one sequence of many rows among short ones: its rows pass by eight at a time
    (2, 4, [300, 64, 1, 200, 700, 90, 640, 513], [9, 1, 1, 1, 1, 1, 1, 1], None),
    (1, 8, [600, 64, 1300], [3, 0, 0], None),
    (1, 3, [130, 2000, 1, 0, 65, 64, 63, 128, 500], [1, 16, 1, 0, 1, 1, 1, 1, 1], None),
    (2, 4, [300, 64, 1, 200, 700, 1900, 640, 513], [9, 1, 1, 1, 1, 1, 1, 1], (128, 2)),
    (1, 8, [1600, 64, 1300], [3, 0, 0], (256, 2)),
    (1, 3, [130, 2000, 1, 0, 65, 1064, 63, 128, 500], [1, 16, 1, 0, 1, 1, 1, 1, 1], (128, 3)),
    (1, 1, [5, 4000], [0, 16], (128, 1)),
    (1, 2, [9000, 100], [2, 5], (128, 4)),
]


@pytest.mark.parametrize("hkv,G,lengths,news,sparse", FEW)
def test_weights_of_few_rows_whose_scores_are_not_kept(hkv, G, lengths, news, sparse, monkeypatch):
    # where the scores would fill too much scratch they are computed again, key by key
    monkeypatch.setenv("MOBA_TEST_KEPT_SCORES", "0")
    attend_case(hkv, G, lengths, news, sparse=sparse, seed=len(lengths) + G)


@pytest.mark.parametrize("hkv,G,lengths,news,sparse", FEW[-8:])
def test_weights_of_a_sequence_with_many_rows_among_short_ones(hkv, G, lengths, news, sparse):
    attend_case(hkv, G, lengths, news, sparse=sparse, seed=len(lengths) + G)


@pytest.mark.parametrize("sparse", [None, (128, 2)])
@pytest.mark.parametrize("n,kept", [(1, True), (1, False), (9, True), (100, True)])
def test_garbage_behind_the_last_token_changes_nothing(n, kept, sparse, monkeypatch):
    # for each of the kernels, with and without chosen blocks, and their weights
    hkv, G, cap, lengths = 2, 4, 1024, [333, 700, 448]
    if not kept:
        monkeypatch.setenv("MOBA_TEST_KEPT_SCORES", "0")
    kv4, _ = random_cache(lengths, hkv, cap, 5)
    dirty = kv4.clone()
    for b, L in enumerate(lengths):
        dirty[b, :, -(-L // 64):] = 0xFF
        if L % 64:
            for off in (0, 4608):
                dirty[b, :, L // 64, off + 64 * (L % 64):off + 4096] = 0xFF
                dirty[b, :, L // 64, off + 4096 + 8 * (L % 64):off + 4608] = 0xFF
    q = bf16(np.random.default_rng(1).standard_normal((3 * n, hkv * G, 128))).cuda()
    got = []
    for cache in (kv4, dirty):
        more = {}
        if sparse:
            more = {"kmean": moba.kv4_pool(cache, ints(lengths), sparse[0]), "block_size": sparse[0], "topk": sparse[1]}
        acc = torch.zeros(3, hkv, cap, device="cuda")
        got.append((*moba.kv4_attend(q, cache, ints(lengths), acc=acc, **more), acc, *moba.kv4_load(cache, ints(lengths), cap)))
    ok()
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert got[1][0].isfinite().all() and got[1][1].isfinite().all()


def test_append_of_spans_that_fp32_does_not_hold():
    # 255 is 17 times 15, half way between the scales 16 and 18, of which 16 is even; a least value a little below zero
    # makes the span larger, by less than fp32 shows, and the nearest scale the upper one
    x = np.zeros((64, 1, 128))
    for i in range(64):
        for g in range(4):
            top = 255.0 * 2.0 ** (g * 2 - 20 + i % 32)
            top = top if top <= 28800 else 255.0
            x[i, 0, 32 * g:32 * g + 8] = np.array([top, -top * 2.0 ** -(17 + i % 24), 0.3 * top, 0.94 * top, 0.97 * top,
                                                   top / 2, 0, 0]) * (1 if i < 32 else -1)
    kv4 = moba.kv4_cache(1, 1, 64)
    moba.kv4_append(bf16(x).cuda(), bf16(-x).cuda(), kv4, ints([0]))
    k, v = moba.kv4_load(kv4, ints([64]), 64)
    ok()
    assert np.array_equal(f64(k)[0, :, 0], ref.stored(f64(bf16(x)))[:, 0])
    assert np.array_equal(f64(v)[0, :, 0], ref.stored(f64(bf16(-x)))[:, 0])


@pytest.mark.parametrize("n,sparse", [(1, None), (9, None), (100, None), (1, (128, 2)), (9, (128, 2)), (100, (128, 2))])
def test_results_in_the_place_of_the_queries(n, sparse):
    lengths = [700, 333]
    kv4, _ = random_cache(lengths, 2, 704, 5)
    kmean = moba.kv4_pool(kv4, ints(lengths), 128)
    more = {"kmean": kmean, "block_size": sparse[0], "topk": sparse[1]} if sparse else {}
    q = bf16(np.random.default_rng(1).standard_normal((2 * n, 8, 128))).cuda()
    want = moba.kv4_attend(q, kv4, ints(lengths), **more)
    buf = torch.cat((q, q[:1]))
    acc = torch.zeros(2, 2, 704, device="cuda")
    with pytest.raises(ValueError):  # the weights' kernels read the queries again
        moba.kv4_attend(buf[:2 * n], kv4, ints(lengths), out=buf[:2 * n], acc=acc, **more)
    with pytest.raises(ValueError):
        moba.kv4_attend(buf[:2 * n], kv4, ints(lengths), out=buf[1:], **more)
    got = moba.kv4_attend(buf[:2 * n], kv4, ints(lengths), out=buf[:2 * n], **more)
    ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (acc == 0).all()


def scores_of_size(size, n, sparse):
    """A call whose scores are some `size` in magnitude: (out, lse, growth of acc, z, d, values), in fp64."""
    hkv, G, L, cap = 1, 4, 700, 704
    rng = np.random.default_rng(5)
    k, v = (f64(bf16(rng.standard_normal((hkv, cap, 128)))) for _ in "kv")
    q = rng.standard_normal((n, hkv * G, 128)) * abs(size)
    if size < 0:  # every score is negative
        k, q = np.abs(k) + 1, -np.abs(q)
    tiles, q = ref.pack(k, v), bf16(q)
    k, v = ref.unpack(tiles)
    kv4, lens, a0 = torch.from_numpy(tiles[None]).cuda(), ints([L]), torch.rand(1, hkv, cap, device="cuda")
    acc, more = a0.clone(), {}
    if sparse:
        more = {"kmean": moba.kv4_pool(kv4, lens, sparse[0]), "block_size": sparse[0], "topk": sparse[1]}
    out, lse = moba.kv4_attend(q.cuda(), kv4, lens, acc=acc, **more)
    ok()
    q = f64(q)
    mask = ref.seen(q, L, n, f64(more["kmean"])[0, 0] if sparse else None, *(sparse or ()))
    z = np.where(mask, np.einsum("ngd,sd->ngs", q, k[0, :L]) / np.sqrt(128), -np.inf)
    d = 140 * 2 * U * np.einsum("ngd,sd->ngs", np.abs(q), np.abs(k[0, :L])).max(-1) / np.sqrt(128)
    return f64(out), f64(lse).T, (f64(acc) - f64(a0))[0, 0], z, d, v[0, :L]


SIZES = [1e5, 1e7, 3e7, 1e9, 1e20, 1e36, -1e31]


@pytest.mark.parametrize("sparse", [None, (128, 3)])
@pytest.mark.parametrize("n", [1, 9, 100])
@pytest.mark.parametrize("size", SIZES)
def test_scores_of_any_size_give_finite_results(size, n, sparse):
    """Scores far beyond what fp32 holds to a whole: the result is the value of the best key, or lies between those of
    the keys that the scores' error (d, as above) does not tell apart from it; the others weigh less than e^-30 each."""
    out, lse, _, z, d, v = scores_of_size(size, n, sparse)
    near = z >= (z.max(-1) - 2 * d - 30)[..., None]
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    assert (np.abs(lse - z.max(-1)) <= d + np.log(len(v)) + 4 * U * np.abs(lse)).all()
    for i in range(n):
        for g in range(out.shape[1]):
            some = v[near[i, g]]
            # rounded to bf16, the weights to fp16 (the sum of them is not): 2^-8 and 2^-10, and 700 times e^-30
            tol = (2.0**-8 + 2.0**-10) * np.abs(some).max(0) + 2.0**-30
            assert (out[i, g] >= some.min(0) - tol).all() and (out[i, g] <= some.max(0) + tol).all()


@pytest.mark.parametrize("sparse", [None, (128, 3)])
@pytest.mark.parametrize("n,kept", [(1, True), (1, False), (9, True), (100, True)])
@pytest.mark.parametrize("size", SIZES)
def test_weights_of_scores_of_any_size(size, n, kept, sparse, monkeypatch):
    # a row gives a key a weight of one at most, and none to the keys far from its best
    if not kept:
        monkeypatch.setenv("MOBA_TEST_KEPT_SCORES", "0")
    _, _, grown, z, d, v = scores_of_size(size, n, sparse)
    L, rows = len(v), n * z.shape[1]
    most = (z >= (z.max(-1) - 2 * d - 30)[..., None]).sum((0, 1))
    # one rounding of fp32 for each row, at magnitudes of rows + 1, and L times e^-30
    assert np.isfinite(grown).all() and (grown[L:] == 0).all()
    assert (grown[:L] >= -2 * U).all() and (grown[:L] <= most + (rows + 2) * (rows + 1) * U + 2.0**-30).all()


@pytest.mark.parametrize("n,kept", [(2, True), (2, False), (9, True), (100, True)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_the_weights_of_its_own_keys_alone(n, kept, bad, monkeypatch):
    hkv, G, L, cap = 2, 4, 700, 768
    if not kept:
        monkeypatch.setenv("MOBA_TEST_KEPT_SCORES", "0")
    kv4, _ = random_cache([L], hkv, cap, 5)
    q = bf16(np.random.default_rng(1).standard_normal((n, hkv * G, 128))).cuda()
    dirty = q.clone()
    row = n // 2 - 1
    dirty[row, 1, 5] = bad
    kmean = moba.kv4_pool(kv4, ints([L]), 128)
    for more in ({}, {"kmean": kmean, "block_size": 128, "topk": 2}):
        a, b = (torch.zeros(1, hkv, cap, device="cuda") for _ in "ab")
        moba.kv4_attend(q, kv4, ints([L]), acc=a, **more)
        moba.kv4_attend(dirty, kv4, ints([L]), acc=b, **more)
        ok()
        own = L - n + row  # the row's position
        assert torch.equal(a[:, 1], b[:, 1]) and torch.equal(a[0, 0, own + 1:], b[0, 0, own + 1:])
        spoilt = ~b[0, 0, :own + 1].isfinite()
        if not more:
            assert spoilt.all() if bad != bad else spoilt.any()
        else:  # its own block, and one other
            blocks = spoilt.nonzero()[:, 0].div(128, rounding_mode="floor").unique().tolist()
            assert own // 128 in blocks and len(blocks) <= 2


@pytest.mark.parametrize("sparse", [None, (128, 2)])
@pytest.mark.parametrize("news", [[1, 1, 1], [9, 3, 11], [100, 0, 70]])
def test_rows_before_the_first_sequence_are_left_alone(news, sparse):
    hkv, G, cap, lengths, lead, pad = 2, 4, 768, [700, 333, 130], 5, 2
    kv4, vals = random_cache(lengths, hkv, cap, 5)
    T = sum(news)
    cu = ints(lead + np.concatenate(([0], np.cumsum(news))))
    q = bf16(np.random.default_rng(1).standard_normal((lead + T + pad, hkv * G, 128)))
    kmean = moba.kv4_pool(kv4, ints(lengths), sparse[0]) if sparse else None
    more = {"kmean": kmean, "block_size": sparse[0], "topk": sparse[1]} if sparse else {}
    out = torch.full((lead + T + pad, hkv * G, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hkv * G, lead + T + pad), 7.0, device="cuda")
    acc = torch.zeros(3, hkv, cap, device="cuda")
    moba.kv4_attend(q.cuda(), kv4, ints(lengths), cu=cu, acc=acc, out=out, lse=lse, **more)
    k = bf16(np.random.default_rng(2).standard_normal((lead + T + pad, hkv, 128)))
    store = moba.kv4_cache(3, hkv, 128)
    moba.kv4_append(k.cuda(), k.cuda(), store, ints([0, 7, 20]), cu=cu)
    loaded, _ = moba.kv4_load(store, ints([128] * 3), 128)
    ok()
    rest = torch.ones(lead + T + pad, dtype=torch.bool, device="cuda")
    rest[lead:lead + T] = False
    assert (out[rest] == 7).all() and (lse[:, rest] == 7).all()
    check_attend((out[lead:lead + T], lse[:, lead:lead + T], acc, torch.zeros_like(acc)), f64(q)[lead:lead + T], vals,
                 lengths, news, hkv, sparse, f64(kmean) if sparse else None)
    want, at = np.zeros((3, 128, hkv, 128)), lead
    for b, (start, n) in enumerate(zip([0, 7, 20], news)):
        want[b, start:start + n] = ref.stored(f64(k)[at:at + n])
        at += n
    assert np.array_equal(f64(loaded), want)


@pytest.mark.parametrize("cu", [[0, 1, 500], [0, 2, 1], [-3, 1, 2], [0, 2, 1, 2]])
def test_offsets_outside_the_rows_are_read_as_no_query_and_reported(cu):
    batch = len(cu) - 1
    kv4, vals = random_cache([300] * batch, 1, 320, 5)
    for G in (1, 40):
        q = bf16(np.random.default_rng(1).standard_normal((2, G, 128))).cuda()
        acc = torch.zeros(batch, 1, 320, device="cuda")
        moba.kv4_attend(q, kv4, ints([300] * batch), cu=ints(cu), acc=acc)
        assert moba.device_status() == moba.MOBA_ERR_DEVICE_CHECK
        want = moba.kv4_attend(q[:1], kv4[:1], ints([300]))  # and the next call is as ever
        ok()
        check_attend((*want, None, None), f64(q)[:1], vals[:1], [300], [1], 1)


def test_calls_from_two_threads_at_once():
    import threading

    lengths = [900, 1500]
    kv4, _ = random_cache(lengths, 2, 1536, 2)
    lens, kmean = ints(lengths), moba.kv4_pool(kv4, ints(lengths), 128)
    cases = []
    for i, n in enumerate((1, 40)):
        q = bf16(np.random.default_rng(i).standard_normal((2 * n, 8, 128))).cuda()
        more = {"kmean": kmean, "block_size": 128, "topk": 3} if i else {}
        acc = torch.zeros(2, 2, 1536, device="cuda")
        cases.append((q, more, (*moba.kv4_attend(q, kv4, lens, acc=acc, **more), acc)))
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        q, more, _ = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                acc = torch.zeros(2, 2, 1536, device="cuda")
                got[i].append((*moba.kv4_attend(q, kv4, lens, acc=acc, **more), acc))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    for i in (0, 1):
        assert len(got[i]) == 50
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, cases[i][2]))


def test_captured_eviction_takes_the_weights_and_lengths_of_its_replay():
    hkv, cap, rng = 2, 1024, np.random.default_rng(3)
    kv4, vals = random_cache([1000, 700], hkv, cap, 2)
    lengths, acc = ints([1000, 700]), torch.zeros(2, hkv, cap, device="cuda")
    dst, dst_acc = moba.kv4_cache(2, hkv, 320), torch.zeros(2, hkv, 320, device="cuda")
    moba.kv4_evict(kv4, acc, lengths, 300, 20, dst, dst_acc)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new, kept = moba.kv4_evict(kv4, acc, lengths, 300, 20, dst, dst_acc)
        k, _ = moba.kv4_load(dst, new, 300)
    for now in ([1000, 700], [640, 0], [299, 301]):
        a = rng.random((2, hkv, cap)).astype(np.float32)
        acc.copy_(torch.from_numpy(a))
        lengths.copy_(ints(now))
        g.replay()
        ok()
        assert new.tolist() == [min(L, 300) for L in now]
        for b, L in enumerate(now):
            for h in range(hkv):
                want = ref.evict(a[b, h].astype(np.float64), L, 300, 20)
                assert np.array_equal(kept[b, h, :len(want)].cpu().numpy(), want) and (kept[b, h, len(want):] == -1).all()
                assert np.array_equal(f64(k[b, :len(want), h]), vals[b][0][h, want]) and (k[b, len(want):] == 0).all()


@pytest.mark.parametrize("n", [9, 100])
@pytest.mark.parametrize("kscale,vscale", [(2.0**-9, 2.0**-9), (1.0, 5000.0), (6000.0, 1.0), (2000.0, 2.0**-12), (2.0**-6, 1.0)])
def test_many_rows_over_keys_and_values_of_every_size(n, kscale, vscale):
    # queries as large as the keys are small, row by row: a unit holds small and large ones (some 64 and more) side by side
    rng = np.random.default_rng(23)
    L, hkv, G, cap = 600, 2, 4, 640
    k, v = rng.standard_normal((hkv, cap, 128)) * kscale, rng.standard_normal((hkv, cap, 128)) * vscale
    tiles = ref.pack(f64(bf16(k)), f64(bf16(v)))
    size = np.where(rng.random((n, hkv * G, 1)) < 0.5, 1.0, 2.0 ** rng.integers(-6, 3, (n, hkv * G, 1)))
    q = bf16(rng.standard_normal((n, hkv * G, 128)) / kscale * size)
    a = torch.zeros(1, hkv, cap, device="cuda")
    out, lse = moba.kv4_attend(q.cuda(), torch.from_numpy(tiles[None]).cuda(), ints([L]), acc=a)
    ok()
    check_attend((out, lse, a, torch.zeros_like(a)), f64(q), [ref.unpack(tiles)], [L], [n], hkv)


def test_a_captured_call_on_a_given_stream():
    # the captured stream itself, and one that is forked from it and joined again
    lengths = [900, 1500]
    kv4, _ = random_cache(lengths, 2, 1536, 2)
    lens = ints(lengths)
    q = bf16(np.random.default_rng(1).standard_normal((2, 8, 128))).cuda()
    want = moba.kv4_attend(q, kv4, lens)
    whole = moba.kv4_load(kv4, lens, 1500)
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        x = q * 1
        a = moba.kv4_attend(x, kv4, lens, stream=main)
        side.wait_stream(main)
        b = moba.kv4_attend(x, kv4, lens, stream=side)
        c = moba.kv4_load(kv4, lens, 1500, stream=side)
        del x
        main.wait_stream(side)
        taken = [torch.full_like(q, 3.0) for _ in range(4)]  # nothing of this takes a place that is still read
    for _ in range(3):
        g.replay()
        ok()
        for got, to in ((a, want), (b, want), (c, whole)):
            assert all(torch.equal(x, y) for x, y in zip(got, to))
        assert all((t == 3).all() for t in taken)
