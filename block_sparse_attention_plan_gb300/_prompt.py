"""ctypes binding of the operators on prompts' rows (bsa_rope_*, bsa_prompt_* in
include/bsa.h).  Argument marshalling only: every step runs in the library's
CUDA kernels."""
from __future__ import annotations

import ctypes
import threading
from typing import Optional, Tuple

import torch

from ._cache import _KEPT_BYTES, RowsC, _device, _kept_lock, _kept_scratch, _raw_stream
from ._lib import _check, library

_ELEMENTS = {torch.bfloat16: 0, torch.float16: 1}
_PAIRS = {"half": 0, "neighbours": 1}
_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}
ROPE_INVERSE = 0x1
PROMPT_CAUSAL = 0x1


class RopeC(ctypes.Structure):
    """Mirror of bsa_rope (include/bsa.h)."""
    _fields_ = [("steps", ctypes.c_void_p), ("amplitude", ctypes.c_float), ("rot", ctypes.c_int32),
                ("pairs", ctypes.c_int32)]


_bound = None


def _library() -> ctypes.CDLL:
    global _bound
    if _bound is not None:
        return _bound
    lib = library()
    I, D, F, VP, N = ctypes.c_int, ctypes.c_double, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    R = ctypes.POINTER(RowsC)
    lib.bsa_prompt_workspace_bytes.restype = N
    lib.bsa_prompt_workspace_bytes.argtypes = [I, I, I, I]
    for name, args in {
            "bsa_rope_steps": [I, D, I, D, D, VP, ctypes.POINTER(ctypes.c_float)],
            "bsa_prompt_attention": [R, R, R, R, VP, I, VP, I, I, I, I, I, I, F, VP, N, VP],
            "bsa_prompt_status": [VP, VP, ctypes.POINTER(ctypes.c_int32)],
            "bsa_rope_apply": [ctypes.POINTER(RopeC), R, R, I, R, R, I, I, VP, I, I, I, I, VP]}.items():
        f = getattr(lib, name)
        f.restype = I
        f.argtypes = args
    _bound = lib
    return lib


def _call(index: int, name: str, *args) -> None:
    """One entry point, on device `index`."""
    f = getattr(_bound, name)
    if _device() == index:
        status = f(*args)
    else:
        with torch.cuda.device(index):
            status = f(*args)
    if status:
        _check(status, name)


def _new(t: torch.Tensor, stream) -> torch.Tensor:
    """Memory like ``t`` that ``stream`` may write."""
    if stream is None:
        o = torch.empty_like(t)
        return o if o.stride(-1) == 1 else torch.empty(t.shape, dtype=t.dtype, device=t.device)
    with torch.cuda.stream(stream):
        return _new(t, None)


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """Memory that ``stream`` may write."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class _Rows(threading.local):
    """The bsa_rows of a call: the library reads them while it is called, so a host thread has four that it fills
    anew (building one costs a microsecond)."""

    def __init__(self):
        self.rows = [RowsC() for _ in range(4)]
        self.refs = [ctypes.byref(r) for r in self.rows]


_call_rows = _Rows()


def _rows(t: torch.Tensor, index: int, name: str, slot: int):
    """bsa_rows ``slot`` of the call: a tensor [batch, heads, tokens, d] or packed [tokens, heads, d] on device
    `index`, by reference."""
    st = t.stride()
    if t.dtype not in _ELEMENTS or t.get_device() != index or len(st) not in (3, 4) or st[-1] != 1:
        raise ValueError(f"{name} must be a CUDA bfloat16 or float16 tensor [B, H, T, d] or [T, H, d] with contiguous rows")
    if len(st) == 4:
        b, h, r, _ = st
    else:
        r, h, _ = st
        b = 0
    if (b | h | r) & 7:  # a dimension of one element has no stride of its own
        n = t.shape
        nb, nh, nr = n[:3] if len(st) == 4 else (1, n[1], n[0])
        b, h, r = (x if k > 1 else 0 for x, k in ((b, nb), (h, nh), (r, nr)))
    c = _call_rows
    o = c.rows[slot]
    o.data, o.stride_b, o.stride_h, o.stride_t = t.data_ptr(), b, h, r
    return c.refs[slot]


class Rope:
    """Rotary positions over a tensor of steps (see bsa_rope): ``steps`` int64 [rot / 2] on the device (the bits
    of the unsigned words f_i / (2 pi) 2^64), ``amplitude``, ``pairs`` "half" or "neighbours".  ``rope_create`` makes
    one from a base and a scaling; frequencies of another rule come in as steps."""

    def __init__(self, steps: torch.Tensor, amplitude: float = 1.0, pairs: str = "half"):
        if steps.dtype != torch.int64 or not steps.is_cuda or steps.dim() != 1 or not steps.is_contiguous():
            raise ValueError("steps must be a contiguous CUDA int64 tensor [rot / 2]")
        if pairs not in _PAIRS:
            raise ValueError(f"pairs must be one of {sorted(_PAIRS)}")
        _library()
        self.steps, self.amplitude, self.pairs = steps, float(amplitude), pairs
        self.device, self._index = steps.device, steps.device.index
        self._c = RopeC(steps.data_ptr(), self.amplitude, 2 * steps.shape[0], _PAIRS[pairs])
        self._ref = ctypes.byref(self._c)

    rot = property(lambda self: self._c.rot)


def rope_create(rot: int, base: float = 10000.0, pairs: str = "half", scaling: str = "none", factor: float = 1.0,
                original: int = 0, device="cuda") -> Rope:
    """Rotary positions of the first ``rot`` elements of a row, frequencies base^(-2 i / rot) (bsa_rope_steps).
    ``pairs``: "half" (i, i + rot / 2) or "neighbours" (2 i, 2 i + 1).  ``scaling`` for contexts ``factor`` times
    as long as the trained one: "none", "linear", "base", or "parts" (``original``: the trained length)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    lib = _library()
    words = (ctypes.c_int64 * 64)()
    amp = ctypes.c_float(1.0)
    _check(lib.bsa_rope_steps(int(rot), float(base), _SCALINGS[scaling], float(factor), float(original), words,
                              ctypes.byref(amp)), "bsa_rope_steps")
    return Rope(torch.tensor(list(words)[:rot // 2], dtype=torch.int64).to(device), amp.value, pairs)


def rope(r: Rope, q: torch.Tensor, k: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
         inverse: bool = False, out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions of q and (not None) k, bfloat16 or float16: [B, H, T, d], any strides between rows, with
    ``positions`` int32 [B, T]; or packed [T, H, d] with ``positions`` [T] (bsa_rope_apply).  Without positions
    they are 0 .. T-1.  ``inverse`` turns back, which also takes gradients of the outputs to those of the inputs.
    ``out_q``, ``out_k``: where the results go, q and k themselves for a call in place.  Returns (q, k) turned;
    where gradients are recorded and q or k requires them, results that belong to the graph (and given outputs are
    refused)."""
    if (q.requires_grad or (k is not None and k.requires_grad)) and torch.is_grad_enabled():
        if out_q is not None or out_k is not None:
            raise ValueError("out_q and out_k are for calls that record no gradients")
        return _Turn.apply(r, q, k, positions, inverse, stream)
    index = r._index
    qr = _rows(q, index, "q", 0)
    shape = q.shape
    if len(shape) == 3:
        B = 1
        T, Hq, d = shape
        where = (T,)
    else:
        B, Hq, T, d = shape
        where = (B, T)
    kr = ko = pptr = None
    Hk = 0
    if k is None and out_k is not None:
        raise ValueError("out_k without k")
    if k is not None:
        kr = _rows(k, index, "k", 1)
        ks = k.shape
        if len(ks) != len(shape) or k.dtype != q.dtype or ks[0] != shape[0] or ks[2:] != shape[2:]:
            raise ValueError("q and k differ in more than their heads")
        Hk = ks[1]
        if out_k is None:
            out_k = _new(k, stream)
        elif out_k.shape != ks or out_k.dtype != k.dtype:
            raise ValueError("out_k must have k's shape and type")
        ko = _rows(out_k, index, "out_k", 2)
    if positions is not None:
        if (positions.dtype != torch.int32 or positions.get_device() != index or not positions.is_contiguous()
                or positions.shape != where):
            raise ValueError("positions must be a contiguous CUDA int32 tensor " + ("[T]" if len(where) == 1 else "[B, T]"))
        pptr = positions.data_ptr()
    if out_q is None:
        out_q = _new(q, stream)
    elif out_q.shape != shape or out_q.dtype != q.dtype:
        raise ValueError("out_q must have q's shape and type")
    if B * T * d * (Hq + Hk) == 0:
        return out_q, out_k
    _call(index, "bsa_rope_apply", r._ref, qr, _rows(out_q, index, "out_q", 3), Hq, kr, ko, Hk, _ELEMENTS[q.dtype],
          pptr, B, T, d, ROPE_INVERSE if inverse else 0, _raw_stream(index) if stream is None else stream.cuda_stream)
    return out_q, out_k


class _Turn(torch.autograd.Function):
    """``rope`` as a node of the graph: the gradients are turned the other way."""

    @staticmethod
    def forward(ctx, r, q, k, positions, inverse, stream):
        ctx.rope, ctx.inverse = r, inverse
        ctx.save_for_backward(positions)
        return rope(r, q, k, positions, inverse, stream=stream)

    @staticmethod
    def backward(ctx, gq, gk):
        positions, = ctx.saved_tensors
        gq, gk = (g if g is None or _takes(g) else g.contiguous() for g in (gq, gk))
        gq, gk = rope(ctx.rope, gq, gk, positions, not ctx.inverse)
        return None, gq, gk, None, None, None


def _takes(t: torch.Tensor) -> bool:
    """Rows that the library reads as they lie."""
    return t.stride(-1) == 1 and not t.data_ptr() & 15 and not any(s & 7 for n, s in zip(t.shape, t.stride()[:-1]) if n > 1)


def prompt_workspace_bytes(n: int, T: int, Hq: int, Hkv: int) -> int:
    """Workspace bytes of a call on n prompts of T tokens together (bsa_prompt_workspace_bytes; 0 for bad
    arguments)."""
    return int(_library().bsa_prompt_workspace_bytes(n, T, Hq, Hkv))


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor, causal: bool = True,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of whole prompts packed behind one another (bsa_prompt_attention): q [T, Hq, d], k, v
    [T, Hkv, d], bfloat16 or float16 with any strides between rows; ``offsets`` int32 [n + 1]: prompt i has rows
    offsets[i] .. offsets[i + 1] - 1.  ``workspace`` (uint8, prompt_workspace_bytes) is taken from the allocator when
    None; one that is given can be asked what the kernels recorded (``prompt_status``).  Returns (O [T, Hq, d],
    LSE [T, Hq]); rows of no prompt are not written.  The results belong to no graph of gradients."""
    index = q.get_device()
    rows = [_rows(q, index, "q", 0), _rows(k, index, "k", 1), _rows(v, index, "v", 2)]
    shape, ks = q.shape, k.shape
    if len(shape) != 3 or index < 0:
        raise ValueError("q must be a CUDA tensor [T, Hq, d]")
    T, Hq, d = shape
    if len(ks) != 3 or ks != v.shape or ks[0] != T or ks[2] != d or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must be [T, Hkv, d] of q's T, d and type")
    if (offsets.dtype != torch.int32 or offsets.get_device() != index or offsets.dim() != 1 or offsets.shape[0] < 2
            or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous CUDA int32 tensor [n + 1]")
    n, Hkv = offsets.shape[0] - 1, ks[1]
    if out is None:
        out = _new(q, stream)
    elif out.shape != shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and type")
    rows.append(_rows(out, index, "out", 3))
    if lse is None:
        lse = _empty((T, Hq), torch.float32, q.device, stream)
    elif (lse.dtype != torch.float32 or lse.get_device() != index or lse.shape != (T, Hq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous CUDA float32 tensor [T, Hq]")
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    lib = _library()
    if T * Hq * d == 0:
        return out, lse
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    args = (*rows, lse.data_ptr(), _ELEMENTS[q.dtype], offsets.data_ptr(), n, T, Hq, Hkv, d, PROMPT_CAUSAL if causal else 0,
            0.0 if scale is None else scale)
    if workspace is not None:
        _call(index, "bsa_prompt_attention", *args, workspace.data_ptr(), workspace.numel(), handle)
        return out, lse
    need = lib.bsa_prompt_workspace_bytes(n, T, Hq, Hkv)
    if handle == 0 and need <= _KEPT_BYTES:
        with _kept_lock:  # the call's kernels are enqueued one after another
            _call(index, "bsa_prompt_attention", *args, _kept_scratch(index, q.device).data_ptr(), need, handle)
    else:
        ws = _empty((max(need, 16),), torch.uint8, q.device, stream)
        _call(index, "bsa_prompt_attention", *args, ws.data_ptr(), need, handle)
    return out, lse


def prompt_status(workspace: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> Tuple[int, int]:
    """(status, detail) that the kernels of the last ``prompt_attention`` with this workspace recorded;
    synchronises (bsa_prompt_status)."""
    det = ctypes.c_int32(0)
    index = workspace.get_device()
    with torch.cuda.device(index):
        st = _library().bsa_prompt_status(workspace.data_ptr(), _raw_stream(index) if stream is None else stream.cuda_stream,
                                          ctypes.byref(det))
    return st, det.value
