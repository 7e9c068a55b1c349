"""B200 (sm_100a) MoBA causal prefill forward pass: thin Python binding.

Every step of the forward pass (key mean-pool, gate + top-k, router, block
attention, log-sum-exp merge) runs in the CUDA kernels of the C-ABI library
``libmoba_b200.so`` declared in ``include/moba.h``. This module only passes
pointers, sizes and the current torch stream to it; PyTorch supplies device
memory and streams. There is no CPU fallback: when the library is missing the
calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoba_b200.so")

MOBA_OK = 0
MOBA_ERR_INVALID_ARG = 1
MOBA_ERR_UNSUPPORTED = 2
MOBA_ERR_OOM = 3
MOBA_ERR_CUDA = 4
MOBA_ERR_DEVICE_TIMEOUT = 5
MOBA_ERR_DEVICE_CHECK = 6
HEAD_DIM = 128
MAX_TOPK = 64
KV4_TILE = 64
KV4_TILE_BYTES = 9216

# every entry point the header declares, with its ctypes signature
_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
SIGNATURES = {
    "moba_fwd": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moba_fwd_chunk": (_i32, [_vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moba_fwd_chunk_means": (_i32, [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moba_fwd_varlen": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moba_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp]),
    "moba_fwd_host": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moba_pool": (_i32, [_vp, _i64, _i32, _i32, _i32, _vp, _vp]),
    "moba_gate": (_i32, [_vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp]),
    "moba_fwd_noalloc": (_i32, [_vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moba_kv4_append": (_i32, [_vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _i64, _vp, _vp, _vp]),
    "moba_kv4_load": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i64, _i64, _vp, _vp, _vp]),
    "moba_kv4_pool": (_i32, [_vp, _vp, _i32, _i32, _i32, _i64, _i32, _vp, _vp]),
    "moba_kv4_attend": (_i32, [_vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _i32, _i32, _vp, _vp, _vp,
                               _vp]),
    "moba_kv4_evict": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp]),
    "moba_profile_begin": (_i32, []),
    "moba_profile_end": (_i32, [_vp, _vp, _vp]),
    "moba_last_error": (ctypes.c_char_p, []),
    "moba_device_status": (_i32, [_vp]),
    "moba_selftest_bounded_wait": (_i32, [_i32, _vp]),
    "moba_selftest_bounded_wait_async": (_i32, [_i32, _vp]),
    "moba_selftest_device_check": (_i32, [_vp]),
}


class MobaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"moba status {code}: {msg}")
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library. Raises when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_sparse_long_fwd_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    return lib().moba_last_error().decode()


def _check(rc: int) -> None:
    if rc != MOBA_OK:
        raise MobaError(rc, last_error())


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _lend(stream, *tensors):
    """The stream as torch knows it. The caller's tensors that it will use may be dropped right after the call: their
    memory is handed out again only behind the stream's work.
    """
    given = [x for x in tensors if x is not None and x.is_cuda]  # the calls refuse the others themselves
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=given[0].device)
    for x in given:
        x.record_stream(stream)
    return stream


def _empty(like: torch.Tensor, stream, shape, dtype) -> torch.Tensor:
    """Memory for an output, of the stream that writes it (None: the current one): another stream's could still be in
    use there. Where the caller's current stream reads the result, that is waited for too before it is handed out again.
    """
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    current = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(stream):
        x = like.new_empty(shape, dtype=dtype)
    if current != stream:
        x.record_stream(current)
    return x


def _dev_bf16(x: torch.Tensor, name: str) -> torch.Tensor:
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    return x


def nblocks(seqlen: int, block_size: int) -> int:
    return (seqlen + block_size - 1) // block_size


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_size: int, topk: int, out=None, lse=None,
        stream=None):
    """MoBA forward. q [S,Hq,128], k/v [S,Hkv,128] bf16 on the GPU.

    Returns (out [S,Hq,128] bf16, lse [Hq,S] fp32), queued on ``stream``
    (default: the current torch stream).
    """
    _dev_bf16(q, "q"), _dev_bf16(k, "k"), _dev_bf16(v, "v")
    S, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (S, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [S, heads_kv, head_dim] matching q")
    if stream is not None:
        stream = _lend(stream, q, k, v, out, lse)
    if out is None:
        out = _empty(q, stream, q.shape, q.dtype)
    if lse is None:
        lse = _empty(q, stream, (Hq, S), torch.float32)
    _check(lib().moba_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), S, Hq, Hkv, d, block_size, topk,
                          out.data_ptr(), lse.data_ptr(), _stream(stream)))
    return out, lse


def fwd_chunk(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_size: int, topk: int, out=None, lse=None,
              stream=None, kmean=None):
    """MoBA forward for the last n = q.shape[0] tokens of a sequence of
    S = k.shape[0] tokens (chunked prefill; n = 1 is a decode step).

    q [n,Hq,128] holds the queries of tokens S-n .. S-1; k/v [S,Hkv,128] the
    keys and values of all S tokens. Returns (out [n,Hq,128] bf16,
    lse [Hq,n] fp32), equal to those rows of ``fwd`` on the whole sequence.
    """
    _dev_bf16(q, "q"), _dev_bf16(k, "k"), _dev_bf16(v, "v")
    n, Hq, d = q.shape
    S, Hkv = k.shape[0], k.shape[1]
    if v.shape != k.shape or k.shape[2] != d or not 1 <= n <= S:
        raise ValueError("q must be [n, heads_q, head_dim] with 1 <= n <= S; k and v [S, heads_kv, head_dim]")
    if stream is not None:
        stream = _lend(stream, q, k, v, kmean, out, lse)
    if out is None:
        out = _empty(q, stream, q.shape, q.dtype)
    if lse is None:
        lse = _empty(q, stream, (Hq, n), torch.float32)
    if kmean is not None:
        # block means from pool() for these k and block_size, kept by the caller
        if kmean.dtype != torch.float32 or not kmean.is_cuda or not kmean.is_contiguous():
            raise ValueError("kmean must be a contiguous fp32 CUDA tensor from pool()")
        _check(lib().moba_fwd_chunk_means(q.data_ptr(), k.data_ptr(), v.data_ptr(), kmean.data_ptr(), S, S - n, Hq,
                                          Hkv, d, block_size, topk, out.data_ptr(), lse.data_ptr(), _stream(stream)))
        return out, lse
    _check(lib().moba_fwd_chunk(q.data_ptr(), k.data_ptr(), v.data_ptr(), S, S - n, Hq, Hkv, d, block_size, topk,
                                out.data_ptr(), lse.data_ptr(), _stream(stream)))
    return out, lse


def fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens, block_size: int, topk: int, out=None,
               lse=None, stream=None):
    """MoBA forward over a packed batch of independent sequences.

    q [T,Hq,128], k/v [T,Hkv,128] bf16 on the GPU hold the sequences one after
    another; ``cu_seqlens`` (a sequence of ints or a CPU tensor, length
    batch + 1, starting at 0) gives their offsets. Returns (out [T,Hq,128]
    bf16, lse [Hq,T] fp32); sequence b's rows equal ``fwd`` on its tokens.
    """
    _dev_bf16(q, "q"), _dev_bf16(k, "k"), _dev_bf16(v, "v")
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (T, Hkv, d) or v.shape != k.shape:
        raise ValueError("k and v must be [T, heads_kv, head_dim] matching q")
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int64, device="cpu").contiguous()
    if cu.dim() != 1 or cu.numel() < 2 or int(cu[-1]) != T:
        raise ValueError("cu_seqlens must be 1-D with batch + 1 entries ending at q.shape[0]")
    if stream is not None:
        stream = _lend(stream, q, k, v, out, lse)
    if out is None:
        out = _empty(q, stream, q.shape, q.dtype)
    if lse is None:
        lse = _empty(q, stream, (Hq, T), torch.float32)
    _check(lib().moba_fwd_varlen(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu.data_ptr(), cu.numel() - 1, Hq, Hkv, d,
                                 block_size, topk, out.data_ptr(), lse.data_ptr(), _stream(stream)))
    return out, lse


def bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
        dout: torch.Tensor, block_size: int, topk: int, stream=None):
    """Gradient of ``fwd`` with the gate's choice held fixed.

    q [S,Hq,128], k/v [S,Hkv,128], out and dout [S,Hq,128] bf16 and lse
    [Hq,S] fp32 (``fwd``'s outputs) on the GPU. Returns (dq, dk, dv) bf16.
    """
    for name, x in (("q", q), ("k", k), ("v", v), ("out", out), ("dout", dout)):
        _dev_bf16(x, name)
    S, Hq, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (S, Hkv, d) or v.shape != k.shape or out.shape != q.shape or dout.shape != q.shape:
        raise ValueError("k, v must be [S, heads_kv, head_dim]; out and dout [S, heads_q, head_dim]")
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous() or lse.shape != (Hq, S):
        raise ValueError("lse must be a contiguous fp32 CUDA tensor [heads_q, S]")
    if stream is not None:
        stream = _lend(stream, q, k, v, out, lse, dout)
    dq, dk, dv = (_empty(x, stream, x.shape, x.dtype) for x in (q, k, v))
    _check(lib().moba_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                          S, Hq, Hkv, d, block_size, topk, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                          _stream(stream)))
    return dq, dk, dv


STAGES = ("pool", "gate", "route", "attention", "merge", "bwd_prep", "bwd_dq", "bwd_dkdv")


def profile_begin() -> None:
    """Start per-stage device timing of the forward calls from this thread."""
    _check(lib().moba_profile_begin())


def profile_end():
    """Stop timing; returns ({stage: total ms}, kernel launches, forward calls)."""
    ms = (ctypes.c_float * len(STAGES))()
    n, c = ctypes.c_int(0), ctypes.c_int(0)
    _check(lib().moba_profile_end(ms, ctypes.byref(n), ctypes.byref(c)))
    return dict(zip(STAGES, list(ms))), n.value, c.value


def fwd_host(q, k, v, block_size: int, topk: int, out=None, lse=None, stream=None):
    """MoBA forward on HOST tensors (bf16 torch CPU tensors, pinned for speed).

    The library copies inputs to the device, runs the pass, copies out/lse
    back and synchronises the stream.
    """
    S, Hq, d = q.shape
    Hkv = k.shape[1]
    for name, x in (("q", q), ("k", k), ("v", v)):
        if x.is_cuda or x.dtype != torch.bfloat16 or not x.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CPU tensor")
    if out is None:
        out = torch.empty((S, Hq, d), dtype=torch.bfloat16, pin_memory=q.is_pinned())
    if lse is None:
        lse = torch.empty((Hq, S), dtype=torch.float32, pin_memory=q.is_pinned())
    _check(lib().moba_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), S, Hq, Hkv, d, block_size, topk,
                               out.data_ptr(), lse.data_ptr(), _stream(stream)))
    return out, lse


def pool(k: torch.Tensor, block_size: int, stream=None) -> torch.Tensor:
    """Key mean-pool stage alone: fp32 [Hkv, nblocks-1, 128]."""
    _dev_bf16(k, "k")
    S, Hkv, d = k.shape
    nbp = max(nblocks(S, block_size) - 1, 0)
    if stream is not None:
        stream = _lend(stream, k)
    kmean = _empty(k, stream, (Hkv, max(nbp, 1), d), torch.float32)
    _check(lib().moba_pool(k.data_ptr(), S, Hkv, d, block_size, kmean.data_ptr(), _stream(stream)))
    return kmean[:, :nbp]


def gate(q: torch.Tensor, kmean: torch.Tensor, heads_kv: int, block_size: int, topk: int, stream=None):
    """Gate + top-k stage alone: int32 sel [Hq, S, min(topk, nblocks)]."""
    _dev_bf16(q, "q")
    S, Hq, d = q.shape
    k_eff = min(topk, nblocks(S, block_size))
    if stream is not None:
        stream = _lend(stream, q, kmean)
    sel = _empty(q, stream, (Hq, S, k_eff), torch.int32)
    kp = kmean.data_ptr() if kmean is not None and kmean.numel() else None
    _check(lib().moba_gate(q.data_ptr(), kp, S, Hq, heads_kv, d, block_size, topk, sel.data_ptr(),
                           _stream(stream)))
    return sel


def kv4_cache(batch: int, heads_kv: int, capacity: int, device="cuda") -> torch.Tensor:
    """An empty 4-bit key/value cache: uint8 [batch, heads_kv, tiles, 9216],
    with room for ``capacity`` tokens a sequence (rounded up to whole tiles of
    64 tokens). The caller keeps the sequences' lengths.
    """
    tiles = (capacity + KV4_TILE - 1) // KV4_TILE
    return torch.zeros((batch, heads_kv, tiles, KV4_TILE_BYTES), dtype=torch.uint8, device=device)


def _kv4(x: torch.Tensor, name: str = "kv4"):
    """(batch, heads_kv, capacity, device index) of a cache."""
    if x.dim() != 4 or x.dtype != torch.uint8 or x.shape[3] != KV4_TILE_BYTES or not (x.is_cuda and x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor [batch, heads_kv, tiles, {KV4_TILE_BYTES}]")
    return x.shape[0], x.shape[1], x.shape[2] * KV4_TILE, x.get_device()


def _on(x, name: str, dtype, shape, device: int):
    """Address of a contiguous tensor of this type, shape and device (None stays None)."""
    if x is None:
        return None
    if x.dtype != dtype or x.shape != shape or x.get_device() != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{device}")
    return x.data_ptr()


def _call(device: int, stream, fn, *args) -> None:
    """fn(*args, stream) with `device` current (a switch only when another one is)."""
    # the current stream's handle as such: the object around it would cost a microsecond, a tenth of a small call
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == device:
        _check(fn(*args, raw))
        return
    with torch.cuda.device(device):
        _check(fn(*args, raw))


def kv4_append(k: torch.Tensor, v: torch.Tensor, kv4: torch.Tensor, start: torch.Tensor, cu=None, acc=None,
               stream=None) -> None:
    """Store new tokens in a 4-bit cache.

    k, v [T, Hkv, 128] bf16 hold the new tokens of the sequences one after
    another; ``cu`` (int32 [batch + 1], on the GPU) gives their offsets, None
    the same number for each. Sequence b's first one goes to place
    ``start[b]`` (int32 [batch], on the GPU). ``acc`` (fp32 [batch, Hkv,
    capacity]) is set to zero there.
    """
    batch, hkv, cap, dev = _kv4(kv4)
    T = k.shape[0]
    kp = _on(k, "k", torch.bfloat16, (T, hkv, HEAD_DIM), dev)
    vp = _on(v, "v", torch.bfloat16, (T, hkv, HEAD_DIM), dev)
    cp = _on(cu, "cu", torch.int32, (batch + 1,), dev)
    sp = _on(start, "start", torch.int32, (batch,), dev)
    ap = _on(acc, "acc", torch.float32, (batch, hkv, cap), dev)
    if T == 0:
        return
    if stream is not None:
        stream = _lend(stream, k, v, kv4, start, cu, acc)
    _call(dev, stream, lib().moba_kv4_append, kp, vp, T, cp, sp, batch, hkv, HEAD_DIM, cap, kv4.data_ptr(), ap)


def kv4_load(kv4: torch.Tensor, lengths: torch.Tensor, n: int, first=None, stream=None):
    """Tokens first[b] .. first[b] + n - 1 of a 4-bit cache (``first`` int32
    [batch] on the GPU; None: from token 0) as bf16: (k, v), each
    [batch, n, Hkv, 128], exact, zero from ``lengths[b]`` on.
    """
    batch, hkv, cap, dev = _kv4(kv4)
    lp = _on(lengths, "lengths", torch.int32, (batch,), dev)
    fp = _on(first, "first", torch.int32, (batch,), dev)
    if not 0 <= n <= cap:
        raise ValueError("n must be in [0, capacity]")
    shape = (batch, n, hkv, HEAD_DIM)
    if stream is None:
        k = kv4.new_empty(shape, dtype=torch.bfloat16)
        v = torch.empty_like(k)
    else:
        stream = _lend(stream, kv4, lengths, first)
        k, v = (_empty(kv4, stream, shape, torch.bfloat16) for _ in "kv")
    if n:
        _call(dev, stream, lib().moba_kv4_load, kv4.data_ptr(), lp, fp, batch, hkv, HEAD_DIM, cap, n, k.data_ptr(),
              v.data_ptr())
    return k, v


def kv4_pool(kv4: torch.Tensor, lengths: torch.Tensor, block_size: int, kmean=None, stream=None) -> torch.Tensor:
    """Mean keys of a 4-bit cache's complete blocks: fp32
    [batch, Hkv, capacity // block_size, 128], zero for the other blocks.
    """
    batch, hkv, cap, dev = _kv4(kv4)
    lp = _on(lengths, "lengths", torch.int32, (batch,), dev)
    if block_size < 1:
        raise ValueError("block_size must be positive")
    shape = (batch, hkv, cap // block_size, HEAD_DIM)
    mp = _on(kmean, "kmean", torch.float32, shape, dev)
    if stream is not None:
        stream = _lend(stream, kv4, lengths, kmean)
    if kmean is None:
        kmean = kv4.new_empty(shape, dtype=torch.float32) if stream is None else \
            _empty(kv4, stream, shape, torch.float32)
        mp = kmean.data_ptr()
    if shape[2]:
        _call(dev, stream, lib().moba_kv4_pool, kv4.data_ptr(), lp, batch, hkv, HEAD_DIM, cap, block_size, mp)
    return kmean


def kv4_attend(q: torch.Tensor, kv4: torch.Tensor, lengths: torch.Tensor, cu=None, kmean=None, block_size: int = 0,
               topk: int = 0, acc=None, out=None, lse=None, stream=None):
    """Attention of each sequence's last tokens over its 4-bit cache.

    q [T, Hq, 128] bf16 holds the queries of the sequences one after another
    (``cu`` as in ``kv4_append``): those of the last tokens of each, which
    ``lengths`` (int32 [batch], on the GPU) already counts. Every key at or
    before a query is attended, or with ``kmean`` (``kv4_pool``'s) its own
    block and the ``topk - 1`` best past blocks, as in ``fwd_chunk``.
    ``acc`` (fp32 [batch, Hkv, capacity]) grows by the tokens' attention
    weights. ``out`` may be ``q`` where no weights are asked for. Returns
    (out [T, Hq, 128] bf16, lse [Hq, T] fp32).
    """
    batch, hkv, cap, dev = _kv4(kv4)
    if q.dim() != 3:
        raise ValueError("q must be [T, heads_q, head_dim]")
    T, hq, _ = q.shape
    qp = _on(q, "q", torch.bfloat16, (T, hq, HEAD_DIM), dev)
    cp = _on(cu, "cu", torch.int32, (batch + 1,), dev)
    lp = _on(lengths, "lengths", torch.int32, (batch,), dev)
    ap = _on(acc, "acc", torch.float32, (batch, hkv, cap), dev)
    mp = None
    if kmean is not None:
        if block_size < 1 or topk < 1:
            raise ValueError("kmean needs block_size and topk")
        mp = _on(kmean, "kmean", torch.float32, (batch, hkv, cap // block_size, HEAD_DIM), dev)
        mp = mp if kmean.numel() else None  # less than a block of room: every key is in the own block
    elif block_size or topk:
        raise ValueError("block_size and topk need kmean")
    op = _on(out, "out", torch.bfloat16, (T, hq, HEAD_DIM), dev)
    ep = _on(lse, "lse", torch.float32, (hq, T), dev)
    if op is not None and abs(op - qp) < q.nbytes and (op != qp or acc is not None):
        raise ValueError("out must not overlap q (without acc it may be q): rows are read after others are written")
    if stream is not None:
        stream = _lend(stream, q, kv4, lengths, cu, kmean, acc, out, lse)
    if out is None:
        out = torch.empty_like(q) if stream is None else _empty(q, stream, q.shape, torch.bfloat16)
        op = out.data_ptr()
    if lse is None:
        lse = kv4.new_empty((hq, T), dtype=torch.float32) if stream is None else \
            _empty(kv4, stream, (hq, T), torch.float32)
        ep = lse.data_ptr()
    if T:
        _call(dev, stream, lib().moba_kv4_attend, qp, T, cp, kv4.data_ptr(), lp, mp, batch, hq, hkv, HEAD_DIM, cap,
              block_size, topk, ap, op, ep)
    return out, lse


def kv4_evict(kv4: torch.Tensor, acc: torch.Tensor, lengths: torch.Tensor, budget: int, recent: int,
              dst: torch.Tensor, dst_acc: torch.Tensor, stream=None):
    """Bring a 4-bit cache down to ``budget`` tokens a sequence by accumulated
    weight: the last ``recent`` tokens and the heaviest others of each kv head
    go, in their order, into ``dst`` and ``dst_acc`` (another cache and its
    weights, with room for the budget).

    Returns (lengths int32 [batch] of the new cache, kept int32
    [batch, Hkv, budget]: the old index of every kept token, padded with -1).
    """
    batch, hkv, cap, dev = _kv4(kv4)
    db, dh, dcap, ddev = _kv4(dst, "dst")
    if (db, dh, ddev) != (batch, hkv, dev):
        raise ValueError("dst must be a cache of the same sequences and heads on the same device")
    if acc is None or dst_acc is None:
        raise ValueError("acc and dst_acc are required")
    ap = _on(acc, "acc", torch.float32, (batch, hkv, cap), dev)
    dp = _on(dst_acc, "dst_acc", torch.float32, (batch, hkv, dcap), dev)
    lp = _on(lengths, "lengths", torch.int32, (batch,), dev)
    if not 1 <= budget <= dcap or not 0 <= recent <= budget:
        raise ValueError("budget must be in [1, dst's capacity] and recent in [0, budget]")
    if stream is not None:
        stream = _lend(stream, kv4, acc, lengths, dst, dst_acc)
    new = _empty(lengths, stream, (batch,), torch.int32)
    kept = _empty(lengths, stream, (batch, hkv, budget), torch.int32)
    _call(dev, stream, lib().moba_kv4_evict, kv4.data_ptr(), ap, lp, batch, hkv, HEAD_DIM, cap, budget, recent,
          dst.data_ptr(), dp, dcap, kept.data_ptr(), new.data_ptr())
    return new, kept


def device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the kernels' status word."""
    return lib().moba_device_status(_stream(stream))


def selftest_bounded_wait(timeout_us: int = 20000, stream=None) -> int:
    return lib().moba_selftest_bounded_wait(timeout_us, _stream(stream))


def effective_flops(seqlen: int, heads_q: int, block_size: int, topk: int, head_dim: int = HEAD_DIM) -> float:
    """Selected-block FLOPs: 4*d*Hq per unmasked (query, key) pair.

    A query t attends min(topk-1, t//B) full past blocks plus the keys of its
    own block up to itself.
    """
    nb = nblocks(seqlen, block_size)
    k_eff = min(topk, nb)
    pairs = 0
    for b in range(nb):
        t0, t1 = b * block_size, min(seqlen, (b + 1) * block_size)
        n = t1 - t0
        pairs += n * min(k_eff - 1, b) * block_size + n * (n + 1) // 2
    return 4.0 * head_dim * heads_q * pairs
