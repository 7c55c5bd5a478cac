"""ctypes binding of the 8-bit K/V cache (bsa_cache_* in include/bsa.h).
Argument marshalling only: every step runs in the library's CUDA kernels."""
from __future__ import annotations

import ctypes
import threading
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import Plan, _check, library

CACHE_E4M3 = 0
CACHE_INT8 = 1
CACHE_CAUSAL = 0x1
_KINDS = {"e4m3": CACHE_E4M3, "int8": CACHE_INT8}
_CODES = {torch.float8_e4m3fn: CACHE_E4M3, torch.int8: CACHE_INT8}
_ELEMENTS = {torch.bfloat16: 0, torch.float16: 1}


class CacheC(ctypes.Structure):
    """Mirror of bsa_cache (include/bsa.h)."""
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k", "v", "k_scale", "v_scale", "block_table", "seq_lens", "page_refs", "control")] + [
        (n, ctypes.c_int32) for n in (
            "kind", "num_pages", "Hkv", "page_size", "d", "scale_block", "max_seqs", "max_pages")]


class RowsC(ctypes.Structure):
    """Mirror of bsa_rows."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_h", ctypes.c_int64),
                ("stride_t", ctypes.c_int64)]


_bound = None
_calls = {}  # entry points by name, without the prefix


def _library() -> ctypes.CDLL:
    global _bound
    if _bound is not None:
        return _bound
    lib = library()
    P, I, F, VP, N = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    C, R = ctypes.POINTER(CacheC), ctypes.POINTER(RowsC)
    lib.bsa_cache_control_bytes.restype = N
    lib.bsa_cache_control_bytes.argtypes = [I]
    lib.bsa_cache_attention_workspace_bytes.restype = N
    lib.bsa_cache_attention_workspace_bytes.argtypes = [C, I, I, I, I, I]
    lib.bsa_cache_forward_workspace_bytes.restype = N
    lib.bsa_cache_forward_workspace_bytes.argtypes = [P, C]
    for name, args in {
            "init": [C, VP], "status": [C, VP, ctypes.POINTER(ctypes.c_int32)], "resize": [C, VP, VP, I, VP],
            "fork": [C, VP, VP, I, VP], "compact": [C, VP], "copy_pages": [C, C, VP, VP, I, VP],
            "append": [C, R, R, I, VP, VP, VP, I, I, VP],
            "attention": [C, R, R, VP, I, VP, VP, I, I, I, I, I, I, F, VP, N, VP],
            "forward": [P, C, VP, VP, I, VP, VP, F, VP, N, VP]}.items():
        f = getattr(lib, "bsa_cache_" + name)
        f.restype = I
        f.argtypes = args
        _calls[name] = f
    _bound = lib
    return lib


class Cache:
    """A paged K/V cache in 8 bits over caller-owned tensors (see bsa_cache):

    k, v            codes [num_pages, Hkv, page_size, d], float8_e4m3fn or int8
    k_scale, v_scale  float32 [num_pages, Hkv, page_size / scale_block]
    block_table     int32 [max_seqs, max_pages], -1 = no page
    lens            int32 [max_seqs]
    refs            int32 [num_pages], sequences that hold each page
    control         int32 scratch and status words (made here when None)

    All contiguous CUDA tensors of one device.  The object keeps them and
    holds no other state; ``cache_create`` makes an empty cache."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 block_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                 control: Optional[torch.Tensor] = None):
        if k.dtype not in _CODES or k.dim() != 4 or not k.is_cuda:
            raise ValueError("k must be a CUDA float8_e4m3fn or int8 tensor [num_pages, Hkv, page_size, d]")
        if v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v differ in shape or type")
        pages, hkv, page, d = k.shape
        if k_scale.dim() != 3 or tuple(k_scale.shape[:2]) != (pages, hkv) or k_scale.shape != v_scale.shape:
            raise ValueError("k_scale and v_scale must be [num_pages, Hkv, page_size / scale_block]")
        per = k_scale.shape[2]
        if per < 1 or page % per:
            raise ValueError("k_scale does not divide a page into blocks")
        if block_table.dim() != 2 or tuple(lens.shape) != (block_table.shape[0],) or tuple(refs.shape) != (pages,):
            raise ValueError("block_table must be [max_seqs, max_pages], lens [max_seqs], refs [num_pages]")
        self.device, self._index = k.device, k.device.index
        need = int(_library().bsa_cache_control_bytes(pages)) // 4
        if control is None:
            control = torch.zeros(need, dtype=torch.int32, device=k.device)
        for name, t, dtype in (("k", k, k.dtype), ("v", v, k.dtype), ("k_scale", k_scale, torch.float32),
                               ("v_scale", v_scale, torch.float32), ("block_table", block_table, torch.int32),
                               ("lens", lens, torch.int32), ("refs", refs, torch.int32),
                               ("control", control, torch.int32)):
            if t.dtype != dtype or t.device != k.device or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor on {k.device}")
        if control.numel() < need:
            raise ValueError(f"control must hold {need} elements")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.block_table, self.lens, self.refs, self.control = block_table, lens, refs, control
        self.scale_block = page // per
        self._c = CacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(),
                         lens.data_ptr(), refs.data_ptr(), control.data_ptr(), _CODES[k.dtype], pages, hkv, page, d,
                         self.scale_block, block_table.shape[0], block_table.shape[1])
        self._ref = ctypes.byref(self._c)
        self._workspace_bytes = {}  # by call geometry (a size, nothing of any call's data)

    num_pages = property(lambda self: self._c.num_pages)
    heads = property(lambda self: self._c.Hkv)
    page_size = property(lambda self: self._c.page_size)
    d = property(lambda self: self._c.d)
    max_seqs = property(lambda self: self._c.max_seqs)
    max_pages = property(lambda self: self._c.max_pages)


def cache_create(num_pages: int, heads: int, page_size: int, d: int, max_seqs: int, max_pages: int,
                 kind: str = "e4m3", scale_block: Optional[int] = None, device="cuda") -> Cache:
    """An empty cache (bsa_cache_init): ``kind`` "e4m3" or "int8", a scale for every ``scale_block`` tokens
    (default: min(page_size, 64))."""
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}")
    sb = min(page_size, 64) if scale_block is None else scale_block
    if sb < 1 or page_size % sb:
        raise ValueError("scale_block must divide page_size")
    codes = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    z = lambda *s, dtype: torch.zeros(s, dtype=dtype, device=device)
    pool = lambda: z(num_pages, heads, page_size, d, dtype=torch.uint8).view(codes)
    scale = lambda: z(num_pages, heads, page_size // sb, dtype=torch.float32)
    c = Cache(pool(), pool(), scale(), scale(), z(max_seqs, max_pages, dtype=torch.int32),
              z(max_seqs, dtype=torch.int32), z(num_pages, dtype=torch.int32))
    _call(c, "init", c._ref, _stream(c, None))
    return c


# The raw handle of a device's current stream (the object that
# torch.cuda.current_stream builds around it costs 2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(c: Cache, stream) -> int:
    return _raw_stream(c._index) if stream is None else stream.cuda_stream


_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(c: Cache, name: str, *args) -> None:
    """One entry point, on the cache's device."""
    f = _calls[name]
    if _device() == c._index:
        status = f(*args)
    else:
        with torch.cuda.device(c._index):
            status = f(*args)
    if status:
        _check(status, "bsa_cache_" + name)


def _list(c: Cache, t: Optional[torch.Tensor], name: str, n: Optional[int] = None) -> Optional[int]:
    """Pointer of an int32 list on the cache's device (None stays None)."""
    if t is None:
        return None
    if (t.dtype != torch.int32 or t.get_device() != c._index or t.dim() != 1 or not t.is_contiguous()
            or (n is not None and t.shape[0] != n)):
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor" + (f" [{n}]" if n is not None else ""))
    return t.data_ptr()


def _rows(c: Cache, t: torch.Tensor, name: str):
    """bsa_rows of a tensor [batch, heads, tokens, d], by reference."""
    if t.dtype not in _ELEMENTS or t.get_device() != c._index or t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be a 4-dimensional CUDA bfloat16 or float16 tensor with contiguous rows")
    b, h, r, _ = t.stride()
    if (b | h | r) & 7:  # a dimension of one element has no stride of its own
        b, h, r = (x if n > 1 else 0 for x, n in zip((b, h, r), t.shape))
    return ctypes.byref(RowsC(t.data_ptr(), b, h, r))


def cache_append(c: Cache, k: torch.Tensor, v: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                 counts: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantise and store tokens (bsa_cache_append): k, v [n, Hkv, T, d], bfloat16
    or float16 (any strides between rows), of which the first ``counts[i]`` of row i become the
    tokens ``start[i]``.. of sequence ``seqs[i]``; by default all T, as the
    sequence's last ones, sequences 0 .. n-1."""
    n, h, T, d = k.shape
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("k and v differ in shape or type")
    if h != c.heads or d != c.d:
        raise ValueError("k and v must be [n, Hkv, T, d] of the cache's Hkv and d")
    _call(c, "append", c._ref, _rows(c, k, "k"), _rows(c, v, "v"), _ELEMENTS[k.dtype],
          seqs if seqs is None else _list(c, seqs, "seqs", n), counts if counts is None else _list(c, counts, "counts", n),
          start if start is None else _list(c, start, "start", n), n, T, _stream(c, stream))


def cache_attention(c: Cache, q: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                    mask: Optional[torch.Tensor] = None, bk: int = 0, causal: bool = False,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of q [B, Hq, nq, d], bfloat16 or float16, over the cached tokens
    of sequences ``seqs`` (default 0 .. B-1) (bsa_cache_attention).  ``mask`` u8 [B, Hq, NKB]
    selects blocks of ``bk`` keys per query head; ``causal``: the queries are
    the sequence's last nq tokens.  Returns (O, LSE)."""
    B, Hq, nq, d = q.shape
    if d != c.d:
        raise ValueError("q must be [B, Hq, nq, d] of the cache's d")
    qr = _rows(c, q, "q")
    NKB, mptr = 0, None
    if mask is not None:
        if (mask.dtype != torch.uint8 or mask.device != c.device or mask.dim() != 3
                or mask.shape[:2] != q.shape[:2] or not mask.is_contiguous()):
            raise ValueError("mask must be a contiguous CUDA uint8 tensor [B, Hq, NKB]")
        NKB, mptr = mask.shape[2], mask.data_ptr()
        if NKB == 0:
            raise ValueError("mask has no key blocks")
    if stream is not None and (out is None or lse is None):
        with torch.cuda.stream(stream):  # memory that this stream may write
            out = torch.empty_like(q) if out is None else out
            lse = torch.empty((B, Hq, nq), dtype=torch.float32, device=c.device) if lse is None else lse
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and type")
    if lse is None:
        lse = torch.empty((B, Hq, nq), dtype=torch.float32, device=c.device)
    elif (lse.dtype != torch.float32 or lse.device != c.device or lse.shape != q.shape[:3]
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous CUDA float32 tensor [B, Hq, nq]")
    key = (B, Hq, nq, NKB, bk)
    need = c._workspace_bytes.get(key)
    if need is None:
        need = int(_bound.bsa_cache_attention_workspace_bytes(c._ref, *key))
        if len(c._workspace_bytes) > 256:
            c._workspace_bytes.clear()
        c._workspace_bytes[key] = need
    handle = _stream(c, stream)
    args = (c._ref, qr, _rows(c, out, "out"), lse.data_ptr(), _ELEMENTS[q.dtype],
            seqs if seqs is None else _list(c, seqs, "seqs", B), mptr, NKB, bk, B, Hq, nq,
            CACHE_CAUSAL if causal else 0, 0.0 if scale is None else scale)
    if handle == 0 and need <= _KEPT_BYTES:
        with _kept_lock:  # the call's kernels are enqueued one after another
            ws = _kept.get(c._index)
            if ws is None:
                with torch.cuda.stream(torch.cuda.default_stream(c.device)):  # (not a given stream's caller's)
                    ws = _kept[c._index] = torch.empty(_KEPT_BYTES, dtype=torch.uint8, device=c.device)
            _call(c, "attention", *args, ws.data_ptr(), need, handle)
    else:
        ws = _scratch(c, need, stream)
        _call(c, "attention", *args, ws.data_ptr(), need, handle)
    return out, lse


# Scratch of calls on a device's default stream: they are in order with each
# other, and never captured into a graph, so one piece serves them all (an
# allocation per call costs a third of a small call's time).  Other streams'
# calls, and larger ones, take theirs from the allocator.
_KEPT_BYTES = 16 << 20
_kept = {}
_kept_lock = threading.Lock()


def _scratch(c: Cache, need: int, stream) -> torch.Tensor:
    """Memory for one call, of the stream's own: what it held before, and what
    will hold it next, are in order with the call."""
    if stream is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=c.device)
    with torch.cuda.stream(stream):
        return torch.empty(max(need, 16), dtype=torch.uint8, device=c.device)


def cache_forward(p: Plan, c: Cache, q: torch.Tensor, seqs: Optional[torch.Tensor] = None, causal: bool = False,
                  split: bool = False, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``forward`` of plan ``p`` with keys and values from the cache's
    sequences ``seqs`` (default 0 .. B-1) (bsa_cache_forward): key lengths are
    the sequences', and with ``causal`` the queries are their last Nq tokens.
    Queries and O are bfloat16, as everywhere in the forward; float16 is for
    ``cache_append`` and ``cache_attention`` alone.  Returns (O, LSE)."""
    L = p.layout
    if (q.dtype != torch.bfloat16 or q.device != c.device or not q.is_contiguous()
            or tuple(q.shape) != (L.B, L.H, L.NQB * L.bq, c.d)):
        raise ValueError("q must be a contiguous CUDA bfloat16 tensor [B, Hq, Nq, d] of the plan's shape")
    for name, t, dtype, shape in (("out", out, torch.bfloat16, q.shape), ("lse", lse, torch.float32, q.shape[:3])):
        if t is not None and (t.dtype != dtype or t.device != c.device or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor {list(shape)}")
    if stream is not None and (out is None or lse is None):
        with torch.cuda.stream(stream):  # memory that this stream may write
            out = torch.empty_like(q) if out is None else out
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if lse is None else lse
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    need = int(_bound.bsa_cache_forward_workspace_bytes(p.handle, c._ref))
    ws = workspace
    if ws is None:
        ws = _scratch(c, need, stream)
    elif ws.dtype != torch.uint8 or ws.device != c.device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    _call(c, "forward", p.handle, c._ref, _list(c, seqs, "seqs", L.B), q.data_ptr(),
          (_lib.FWD_CAUSAL if causal else 0) | (_lib.FWD_SPLIT_P if split else 0), out.data_ptr(), lse.data_ptr(),
          0.0 if scale is None else scale, ws.data_ptr(), ws.numel(), _stream(c, stream))
    return out, lse


def cache_resize(c: Cache, new_lens: torch.Tensor, seqs: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> None:
    """Set sequences' lengths, taking and giving back pages (bsa_cache_resize);
    blocks that a sequence enters hold nothing until ``cache_append`` stores it.
    A token that a growth by one takes is to be stored before the sequence grows
    further."""
    n = new_lens.shape[0]
    _call(c, "resize", c._ref, _list(c, seqs, "seqs", n), _list(c, new_lens, "new_lens"), n, _stream(c, stream))


def cache_free(c: Cache, seqs: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Free sequences, all of them by default (bsa_cache_resize to length 0)."""
    n = c.max_seqs if seqs is None else seqs.shape[0]
    _call(c, "resize", c._ref, _list(c, seqs, "seqs"), None, n, _stream(c, stream))


def cache_fork(c: Cache, src: torch.Tensor, dst: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Let empty sequences dst[i] share the tokens of src[i] (bsa_cache_fork)."""
    n = src.shape[0]
    _call(c, "fork", c._ref, _list(c, src, "src"), _list(c, dst, "dst", n), n, _stream(c, stream))


def cache_compact(c: Cache, stream: Optional[torch.cuda.Stream] = None) -> None:
    """Move the held pages to the front of the pools (bsa_cache_compact)."""
    _call(c, "compact", c._ref, _stream(c, stream))


def cache_copy_pages(dst: Cache, src: Cache, dst_pages: torch.Tensor, src_pages: torch.Tensor,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """Copy pages src_pages[i] of ``src`` to pages dst_pages[i] of ``dst``
    (bsa_cache_copy_pages)."""
    if dst.device != src.device:
        raise ValueError("dst and src must be on one device")
    n = dst_pages.shape[0]
    _call(dst, "copy_pages", dst._ref, src._ref, _list(dst, dst_pages, "dst_pages"),
          _list(dst, src_pages, "src_pages", n), n, _stream(dst, stream))


def cache_status(c: Cache, stream: Optional[torch.cuda.Stream] = None) -> Tuple[int, int]:
    """(status, detail) the cache's kernels recorded since the last report;
    synchronises, and clears it (bsa_cache_status)."""
    det = ctypes.c_int32(0)
    with torch.cuda.device(c._index):
        st = _bound.bsa_cache_status(c._ref, _stream(c, stream), ctypes.byref(det))
    return st, det.value
