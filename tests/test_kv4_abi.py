"""What the 4-bit cache's entry points refuse, before any launch (no GPU)."""
import pytest
import torch

import block_sparse_long_fwd_b200 as moba
from block_sparse_long_fwd_b200 import build as moba_build

F = 0x100000  # aligned, never dereferenced: checks fail first
BAD, UNSUP = moba.MOBA_ERR_INVALID_ARG, moba.MOBA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    moba_build.build()
    return moba.lib()


ORDER = {
    "append": "k v total cu start batch heads_kv head_dim capacity kv4 acc",
    "load": "kv4 lengths first batch heads_kv head_dim capacity n k v",
    "pool": "kv4 lengths batch heads_kv head_dim capacity block_size kmean",
    "attend": "q total cu kv4 lengths kmean batch heads_q heads_kv head_dim capacity block_size topk acc out lse",
    "evict": "kv4 acc lengths batch heads_kv head_dim capacity budget recent dst_kv4 dst_acc dst_capacity kept new_lengths",
}
GOOD = {"k": F, "v": F, "q": F, "total": 4, "cu": F, "start": F, "lengths": F, "first": F, "batch": 2, "heads_q": 4,
        "heads_kv": 2, "head_dim": 128, "capacity": 1024, "n": 16, "kv4": F, "acc": F, "kmean": F, "block_size": 128,
        "topk": 3, "out": F, "lse": F, "budget": 100, "recent": 10, "dst_kv4": F + (1 << 24), "dst_acc": F + (1 << 26),
        "dst_capacity": 128, "kept": F, "new_lengths": F + 4096}


def call(lib, op, **change):
    args = {**GOOD, **change}
    return getattr(lib, "moba_kv4_" + op)(*[args[n] for n in ORDER[op].split()], None)


EVERY = list(ORDER)


@pytest.mark.parametrize("op", EVERY)
@pytest.mark.parametrize("change,code", [
    ({"kv4": None}, BAD), ({"kv4": F + 8}, BAD), ({"batch": 0}, BAD), ({"heads_kv": 0}, BAD), ({"head_dim": 64}, BAD),
    ({"capacity": 0}, BAD), ({"capacity": 100}, BAD), ({"capacity": -64}, BAD), ({"capacity": 1 << 31}, UNSUP),
    ({"batch": 65536, "total": 65536}, UNSUP),
])
def test_a_bad_cache_is_refused(lib, op, change, code):
    assert call(lib, op, **change) == code
    assert moba.last_error()


@pytest.mark.parametrize("op,change,code,what", [
    ("append", {"k": None}, BAD, "null"), ("append", {"v": F + 2}, BAD, "aligned"), ("append", {"start": None}, BAD, "null"),
    ("append", {"total": -1}, BAD, "total"), ("append", {"cu": None, "total": 5}, BAD, "multiple of batch"),
    ("append", {"start": F + 2}, BAD, "aligned"),
    ("load", {"lengths": None}, BAD, "null"), ("load", {"n": -1}, BAD, "n must"), ("load", {"n": 1025}, BAD, "n must"),
    ("load", {"v": F + 8}, BAD, "aligned"), ("load", {"first": F + 1}, BAD, "aligned"),
    ("pool", {"block_size": 100}, BAD, "block_size"), ("pool", {"block_size": 0}, BAD, "block_size"),
    ("pool", {"kmean": None}, BAD, "null"), ("pool", {"kmean": F + 4}, BAD, "aligned"),
    ("attend", {"q": None}, BAD, "null"), ("attend", {"heads_q": 3}, BAD, "multiple"), ("attend", {"heads_q": 0}, BAD, "multiple"),
    ("attend", {"cu": None, "total": 5}, BAD, "multiple of batch"), ("attend", {"total": 1 << 30}, BAD, "total"),
    ("attend", {"block_size": 64}, BAD, "block_size"), ("attend", {"topk": 0}, BAD, "topk"),
    ("attend", {"capacity": 1 << 20, "topk": 66}, UNSUP, "topk"),
    ("attend", {"capacity": 1 << 22}, UNSUP, "blocks"),
    ("attend", {"out": F + 8}, BAD, "aligned"), ("attend", {"lse": F + 2}, BAD, "aligned"), ("attend", {"kmean": F + 8}, BAD, "aligned"),
    ("evict", {"acc": None}, BAD, "null"), ("evict", {"budget": 0}, BAD, "budget"), ("evict", {"budget": 129}, BAD, "budget"),
    ("evict", {"recent": 101}, BAD, "recent"), ("evict", {"recent": -1}, BAD, "recent"), ("evict", {"dst_capacity": 100}, BAD, "capacity"),
    ("evict", {"dst_kv4": F}, BAD, "overlap"), ("evict", {"dst_kv4": F + 4 * 16 * 9216 - 16}, BAD, "overlap"),
    ("evict", {"dst_acc": F + 4}, BAD, "overlap"), ("evict", {"new_lengths": F}, BAD, "overlap"),
])
def test_bad_arguments_are_refused_with_a_message(lib, op, change, code, what):
    assert call(lib, op, **change) == code
    assert what in moba.last_error()


@pytest.mark.parametrize("op", EVERY)
def test_good_arguments_pass_the_checks(lib, op):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the pointers would be used")
    assert call(lib, op) == moba.MOBA_ERR_CUDA


def test_the_binding_refuses_tensors_of_another_kind():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(1, 2, 1, moba.KV4_TILE_BYTES, dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        moba.kv4_append(x, x, cache, i)
    with pytest.raises(ValueError):
        moba.kv4_attend(x, cache, i)
    with pytest.raises(ValueError):
        moba.kv4_load(cache, i, 1)
    with pytest.raises(ValueError):
        moba.kv4_pool(cache, i, 128)
    with pytest.raises(ValueError):
        moba.kv4_evict(cache, torch.zeros(1, 2, 64), i, 1, 0, cache, torch.zeros(1, 2, 64))
    assert moba.kv4_cache(2, 3, 65, device="cpu").shape == (2, 3, 2, 9216)


@pytest.mark.parametrize("total,heads_q", [(1 << 62, 4), ((1 << 62) + 2, 4), (1 << 61, 8), ((1 << 31) + 2, 2), ((1 << 63) - 1, 2)])
def test_rows_whose_number_wraps_are_refused(lib, total, heads_q):
    # total * heads_q is a small number, or a negative one, in 64 bits
    assert call(lib, "attend", total=total, heads_q=heads_q) == BAD
    assert "total" in moba.last_error()
