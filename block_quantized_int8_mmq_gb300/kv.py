"""The 8-bit key/value cache: position rotation, appending, attention and reading back
(include/mmq.h, "8-bit key/value cache").

    cache = KVCache.empty(pages, heads, dim, page=64)       # records in device memory
    rope = Rope(cos, sin)                                   # f32 [positions, rotary / 2]
    batch = KVBatch(starts, lens, table, tokens, max_new)   # which rows belong to which sequence
    q = mmq_kv_append(cache, batch, k, v, q=q, rope=rope)   # k and v into the cache, q rotated
    out = mmq_kv_attend(cache, batch, q)                    # [tokens, q heads, dim]

The handles only keep tensors alive and their addresses together; a program makes them once
(a batch once per set of tensors: its tensors' contents may change between calls) and every
computation runs in the library's kernels.  The cache's device has to be the current one.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import MMQError, _lib, _stream

BLOCK_TOKENS = 32
F32, BF16, F16 = 0, 1, 2
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class _Batch(ctypes.Structure):
    _fields_ = [("starts", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("seqs", ctypes.c_int32), ("tokens", ctypes.c_int32),
                ("max_new", ctypes.c_int32), ("table_pages", ctypes.c_int32)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("rotary", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


def _bind():
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    _lib.mmq_kv_block_bytes.argtypes = [I64]
    _lib.mmq_kv_block_bytes.restype = ctypes.c_size_t
    _lib.mmq_kv_workspace_bytes.argtypes = [I64]
    _lib.mmq_kv_workspace_bytes.restype = ctypes.c_size_t
    _lib.mmq_kv_append.argtypes = [P, P, I, P, P, P, I64, P, P, P]
    _lib.mmq_kv_read.argtypes = [P, P, I, P, P, P]
    _lib.mmq_kv_attend.argtypes = [P, P, I, P, I64, F, I64, P, P, P, ctypes.c_size_t, P]


_bind()


def _device_tensor(t, dtype, what):
    if t.dtype != dtype or not t.is_cuda:
        raise ValueError(f"{what} must be a {dtype} CUDA tensor, got {t.dtype} on {t.device}")
    return t


def mmq_kv_block_bytes(dim: int) -> int:
    """Bytes of the record of one block: 32 tokens of one head."""
    return int(_lib.mmq_kv_block_bytes(int(dim)))


def mmq_kv_workspace_bytes(dim: int) -> int:
    return int(_lib.mmq_kv_workspace_bytes(int(dim)))


class KVCache:
    """data: uint8 [pages, heads, page / 32, 64 * dim + 16] records, contiguous, on the GPU.  What
    it holds for tokens that were never appended does not matter."""

    def __init__(self, data):
        _device_tensor(data, torch.uint8, "the cache")
        if data.dim() != 4 or not data.is_contiguous():
            raise ValueError("the cache is a contiguous [pages, heads, page / 32, record bytes] tensor")
        self.data = data
        self.pages, self.heads, blocks, rec = data.shape
        self.page, self.dim = blocks * BLOCK_TOKENS, (rec - 16) // 64
        if mmq_kv_block_bytes(self.dim) != rec:
            raise ValueError(f"records of {rec} bytes: 64 * dim + 16 with dim 64, 128 or 256 are taken")
        self.device = data.device
        self._c = _Cache(data.data_ptr(), self.pages, self.page, self.heads, self.dim)
        self._p = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, pages: int, heads: int, dim: int, page: int = 64, device="cuda"):
        rec = mmq_kv_block_bytes(dim)
        if rec == 0 or page < BLOCK_TOKENS or page % BLOCK_TOKENS:
            raise ValueError("dim must be 64, 128 or 256 and page a multiple of 32")
        return cls(torch.empty((pages, heads, page // BLOCK_TOKENS, rec), dtype=torch.uint8, device=device))


class KVBatch:
    """Sequences and their new tokens (see include/mmq.h): int32 CUDA tensors starts [seqs + 1],
    lens [seqs] (the lengths WITH the new tokens) and table [seqs, pages]; tokens: rows of the
    packed row arrays; max_new: no sequence has more new tokens."""

    def __init__(self, starts, lens, table, tokens: int, max_new: int):
        for t, what in ((starts, "starts"), (lens, "lens"), (table, "table")):
            _device_tensor(t, torch.int32, what)
        seqs = lens.shape[0]
        if lens.dim() != 1 or starts.shape != (seqs + 1,) or table.dim() != 2 or table.shape[0] != seqs:
            raise ValueError("starts is [seqs + 1], lens [seqs] and table [seqs, pages]")
        if not starts.is_contiguous() or not lens.is_contiguous() or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("starts, lens and the rows of table must be contiguous")
        if lens.device != starts.device or table.device != starts.device:
            raise ValueError("starts, lens and table must be on one device")
        self.device = starts.device
        self.starts, self.lens, self.table, self.tokens, self.max_new = starts, lens, table, int(tokens), int(max_new)
        stride = table.stride(0) if seqs > 1 else table.shape[1]
        self._c = _Batch(starts.data_ptr(), lens.data_ptr(), table.data_ptr(), stride, seqs, self.tokens,
                         self.max_new, table.shape[1])
        self._p = ctypes.addressof(self._c)


class Rope:
    """Rotation tables cos, sin: f32 [positions, rotary / 2].  Pairs (i, i + rotary / 2), or
    (2i, 2i + 1) where interleaved."""

    def __init__(self, cos, sin, interleaved: bool = False):
        for t in (cos, sin):
            _device_tensor(t, torch.float32, "a rotation table")
        if cos.dim() != 2 or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin are contiguous [positions, rotary / 2] tensors")
        if cos.device != sin.device:
            raise ValueError("cos and sin must be on one device")
        self.device = cos.device
        self.cos, self.sin, self.interleaved = cos, sin, bool(interleaved)
        self._c = _Rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1], int(self.interleaved))
        self._p = ctypes.addressof(self._c)


def _refuse(t, what, shape, dtype, device):
    """Why a row array is refused (the calls' own checks are one comparison each)."""
    if t.dim() != 3 or t.shape[0] != shape[0] or t.shape[2] != shape[2] or (shape[1] and t.shape[1] != shape[1]):
        raise ValueError(f"{what} has shape {tuple(t.shape)}: [{shape[0]}, {shape[1] or 'heads'}, {shape[2]}] is wanted")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{what} is {t.dtype}: float32, bfloat16 and float16 are taken")
    if t.dtype != dtype or t.device != device:
        raise ValueError(f"{what} is {t.dtype} on {t.device}: {dtype} on {device} is wanted")
    raise ValueError(f"{what}: the last axis must be contiguous")


def _elsewhere(what, t, device):
    raise ValueError(f"{what} is on {t.device}, the cache on {device}")


def _here(device):
    """The library launches on the current device, whatever stream and addresses it gets."""
    current = torch.cuda.current_device()
    if current != device.index:
        raise ValueError(f"the cache is on {device}, the current device is cuda:{current}: call it under "
                         f"torch.cuda.device({device.index})")


def _stream_of(device, stream):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _stream(stream)


def _empty(shape, dtype, device, stream):
    """A tensor for what a call returns.  On a stream other than the current one it is that stream's memory,
    which nothing pending elsewhere uses, and given back once the current stream is done with it too."""
    if stream is None or int(_stream(stream).value or 0) == torch._C._cuda_getCurrentRawStream(device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    torch.cuda.set_stream(stream if isinstance(stream, torch.cuda.Stream)
                          else torch.cuda.ExternalStream(int(stream), device=device))
    try:
        t = torch.empty(shape, dtype=dtype, device=device)
    finally:
        torch.cuda.set_stream(current)
    t.record_stream(current)
    return t


def _out(t, shape, dtype, cache, what):
    if t.shape != shape or t.dtype != dtype or t.device != cache.device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} {tuple(shape)} tensor on {cache.device}")
    return t


_ROW_BYTES = ctypes.sizeof(_Rows)


class _Rows3(ctypes.Structure):
    _fields_ = [(f"{n}{i}", t) for i in range(3) for n, t in _Rows._fields_]


def mmq_kv_append(cache, batch, k, v, q=None, rope=None, q_out=None, stream=None):
    """Keys and values [tokens, cache.heads, dim] into the cache, rotated by `rope` on the way (the
    values are not rotated); returns the rotated queries [tokens, q heads, dim] where q is given."""
    dt, dev, shape = k.dtype, cache.device, (batch.tokens, cache.heads, cache.dim)
    _here(dev)
    d = _DTYPES.get(dt)
    ks, vs = k.stride(), v.stride()
    if d is None or k.shape != shape or k.device != dev or ks[-1] != 1:
        _refuse(k, "k", shape, dt, dev)
    if v.dtype != dt or v.shape != shape or v.device != dev or vs[-1] != 1:
        _refuse(v, "v", shape, dt, dev)
    if batch.device != dev:
        _elsewhere("the batch", batch, dev)
    turn = None
    if rope is not None:
        if rope.device != dev:
            _elsewhere("the rotation tables", rope, dev)
        turn = rope._p
    if q is None:
        rows = _Rows3(k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1])
        p = ctypes.addressof(rows)
        st = _lib.mmq_kv_append(cache._p, batch._p, d, p, p + _ROW_BYTES, None, 0, turn, None, _stream_of(dev, stream))
    else:
        qs, qshape = q.stride(), q.shape
        if q.dtype != dt or len(qshape) != 3 or qshape[0] != shape[0] or qshape[2] != shape[2] or q.device != dev or qs[-1] != 1:
            _refuse(q, "q", (shape[0], 0, shape[2]), dt, dev)
        if q_out is None:
            q_out = _empty(qshape, dt, dev, stream)
        else:
            _out(q_out, qshape, dt, cache, "q_out")
        rows = _Rows3(k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], q.data_ptr(), qs[0], qs[1])
        p = ctypes.addressof(rows)
        st = _lib.mmq_kv_append(cache._p, batch._p, d, p, p + _ROW_BYTES, p + 2 * _ROW_BYTES, qshape[1], turn,
                                q_out.data_ptr(), _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_kv_append", st)
    return q_out if q is not None else None


def mmq_kv_read(cache, batch, dtype=torch.float32, k_out=None, v_out=None, stream=None):
    """The cached keys and values of the batch's tokens, [tokens, cache.heads, dim] of `dtype`."""
    d, dev, shape = _DTYPES.get(dtype), cache.device, (batch.tokens, cache.heads, cache.dim)
    _here(dev)
    if d is None:
        raise ValueError(f"{dtype}: float32, bfloat16 and float16 are taken")
    if batch.device != dev:
        _elsewhere("the batch", batch, dev)
    if k_out is None:
        k_out = _empty(shape, dtype, dev, stream)
    else:
        _out(k_out, shape, dtype, cache, "k_out")
    if v_out is None:
        v_out = _empty(shape, dtype, dev, stream)
    else:
        _out(v_out, shape, dtype, cache, "v_out")
    st = _lib.mmq_kv_read(cache._p, batch._p, d, k_out.data_ptr(), v_out.data_ptr(), _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_kv_read", st)
    return k_out, v_out


_WS_ZERO = 16384  # bytes at a workspace's beginning that start at zero
_workspaces: dict = {}


_is_capturing = None


def _captured(raw):
    """Whether a raw stream is being captured (torch asks this of the current stream only, and making
    another one current for the question takes ten times as long)."""
    global _is_capturing
    if _is_capturing is None:
        _is_capturing = ctypes.CDLL("libcuda.so.1").cuStreamIsCapturing
        _is_capturing.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    status = ctypes.c_int(0)
    return _is_capturing(raw, ctypes.addressof(status)) == 0 and status.value != 0


def _workspace(cache, stream):
    """The package's own workspace of a stream: calls on one stream run one after another.  A captured call
    gets one of the graph's memory, zeroed in the graph: its replays may run beside anything."""
    s = torch._C._cuda_getCurrentRawStream(cache.device.index) if stream is None else int(_stream(stream).value or 0)
    captured = _captured(s)
    key = (cache.device.index, s, cache.dim)
    ws = None if captured else _workspaces.get(key)
    if ws is None:
        with torch.cuda.stream(stream if stream is None or isinstance(stream, torch.cuda.Stream)
                               else torch.cuda.ExternalStream(s, device=cache.device)):
            ws = torch.empty(mmq_kv_workspace_bytes(cache.dim), dtype=torch.uint8, device=cache.device)
            ws[:_WS_ZERO].zero_()
            if not captured:
                _workspaces[key] = ws
    return ws


def _clean_workspaces():
    """A call that gave up may have left counts in its workspace."""
    for ws in _workspaces.values():
        torch.cuda.synchronize(ws.device)
        ws[:_WS_ZERO].zero_()
        torch.cuda.synchronize(ws.device)


def mmq_kv_attend(cache, batch, q, scale=None, window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of the rotated queries [tokens, q heads, dim] over the cache: [tokens, q
    heads, dim].  scale: 1 / sqrt(dim) by default.  window: how many of the latest tokens a row
    sees (0: all).  lse: an f32 [tokens, q heads] tensor for the logarithm of the softmax's sum.
    workspace: a uint8 tensor of mmq_kv_workspace_bytes(dim) bytes, its first 16384 zero, that no call
    that may overlap this one uses.  By default the package keeps one for each stream, and a captured call
    has one of the graph's own, zeroed by a node of the graph (1 us) that a workspace given here saves."""
    dt, dev, qs, qshape = q.dtype, cache.device, q.stride(), q.shape
    _here(dev)
    d = _DTYPES.get(dt)
    if d is None or len(qshape) != 3 or qshape[0] != batch.tokens or qshape[2] != cache.dim or q.device != dev or qs[-1] != 1:
        _refuse(q, "q", (batch.tokens, 0, cache.dim), dt, dev)
    if batch.device != dev:
        _elsewhere("the batch", batch, dev)
    if out is None:
        out = _empty(qshape, dt, dev, stream)
    else:
        _out(out, qshape, dt, cache, "out")
    if lse is not None:
        _out(lse, qshape[:2], torch.float32, cache, "lse")
    if workspace is None:
        workspace = _workspace(cache, stream)
    elif workspace.dtype != torch.uint8 or workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {cache.device}")
    if scale is None:
        scale = 1.0 / math.sqrt(cache.dim)
    rows = _Rows(q.data_ptr(), qs[0], qs[1])
    st = _lib.mmq_kv_attend(cache._p, batch._p, d, ctypes.addressof(rows), qshape[1], scale, window, out.data_ptr(),
                            None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                            _stream_of(dev, stream))
    if st != 0:
        raise MMQError("mmq_kv_attend", st)
    return out
