"""ctypes binding of the operators on prompts' rows (bsa_rope_*, bsa_prompt_* in
include/bsa.h).  Argument marshalling only: every step runs in the library's
CUDA kernels."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._cache import RowsC, _device, _raw_stream
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


def _rows(t: torch.Tensor):
    """bsa_rows of a tensor [batch, heads, tokens, d] or packed [tokens, heads, d], by reference."""
    if t.dim() == 4:
        b, h, r, _ = t.stride()
        nb, nh, nr, _ = t.shape
    else:
        r, h, _ = t.stride()
        nr, nh, _ = t.shape
        b, nb = 0, 1
    if (b | h | r) & 7:  # a dimension of one element has no stride of its own
        b, h, r = (x if n > 1 else 0 for x, n in ((b, nb), (h, nh), (r, nr)))
    return ctypes.byref(RowsC(t.data_ptr(), b, h, r))


class Rope:
    """Rotary positions over a tensor of steps (see bsa_rope): ``steps`` int64 [rot / 2] on the device (the bits
    of the unsigned words), ``amplitude``, ``pairs`` "half" or "neighbours".  ``rope_create`` makes one from
    frequencies."""

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
    ``out_q``, ``out_k``: where the results go, q and k themselves for a call in place.  Returns (q, k) turned."""
    dims = q.dim()
    for name, t, o in (("q", q, out_q), ("k", k, out_k)):
        if t is None:
            continue
        if t.dtype not in _ELEMENTS or t.get_device() != r._index or t.dim() not in (3, 4) or t.stride(-1) != 1:
            raise ValueError(f"{name} must be a CUDA bfloat16 or float16 tensor [B, H, T, d] or [T, H, d] with contiguous rows")
        if o is not None and (o.shape != t.shape or o.dtype != t.dtype or o.get_device() != r._index or o.stride(-1) != 1):
            raise ValueError(f"out_{name} must have {name}'s shape, type and device, and contiguous rows")
    B, T, at = (1, q.shape[0], 1) if dims == 3 else (q.shape[0], q.shape[2], 1)
    if k is not None and (k.dim() != dims or k.dtype != q.dtype
                          or k.shape[:at] + k.shape[at + 1:] != q.shape[:at] + q.shape[at + 1:]):
        raise ValueError("q and k differ in more than their heads")
    pptr = None
    if positions is not None:
        if (positions.dtype != torch.int32 or positions.get_device() != r._index or not positions.is_contiguous()
                or tuple(positions.shape) != ((T,) if dims == 3 else (B, T))):
            raise ValueError("positions must be a contiguous CUDA int32 tensor " + ("[T]" if dims == 3 else "[B, T]"))
        pptr = positions.data_ptr()
    if out_q is None:
        out_q = _new(q, stream)
    if k is not None and out_k is None:
        out_k = _new(k, stream)
    if q.numel() == 0 and (k is None or k.numel() == 0):
        return out_q, out_k
    if k is None:
        kr = ko = None
        Hk = 0
    else:
        kr, ko, Hk = _rows(k), _rows(out_k), k.shape[at]
    _call(r._index, "bsa_rope_apply", r._ref, _rows(q), _rows(out_q), q.shape[at], kr, ko, Hk, _ELEMENTS[q.dtype],
          pptr, B, T, q.shape[-1], ROPE_INVERSE if inverse else 0,
          _raw_stream(r._index) if stream is None else stream.cuda_stream)
    return out_q, out_k


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
    LSE [T, Hq]); rows of no prompt are not written."""
    index = q.get_device()
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype not in _ELEMENTS or not t.is_cuda or t.get_device() != index or t.dim() != 3 or t.stride(2) != 1:
            raise ValueError(f"{name} must be a CUDA bfloat16 or float16 tensor [T, H, d] with contiguous rows")
    T, Hq, d = q.shape
    if k.shape != v.shape or k.shape[0] != T or k.shape[2] != d or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("k and v must be [T, Hkv, d] of q's T, d and type")
    if (offsets.dtype != torch.int32 or offsets.get_device() != index or offsets.dim() != 1 or offsets.shape[0] < 2
            or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous CUDA int32 tensor [n + 1]")
    n, Hkv = offsets.shape[0] - 1, k.shape[1]
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or out.get_device() != index or out.stride(2) != 1):
        raise ValueError("out must have q's shape, type and device, and contiguous rows")
    if lse is not None and (lse.dtype != torch.float32 or lse.get_device() != index or tuple(lse.shape) != (T, Hq)
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous CUDA float32 tensor [T, Hq]")
    if workspace is not None and (workspace.dtype != torch.uint8 or workspace.get_device() != index or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA uint8 tensor")
    lib = _library()
    if out is None:
        out = _new(q, stream)
    if lse is None or workspace is None:
        need = int(lib.bsa_prompt_workspace_bytes(n, T, Hq, Hkv)) if workspace is None else 0
        with torch.cuda.stream(stream):  # (None: the current one)
            if lse is None:
                lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
            if workspace is None:
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if q.numel() == 0:
        return out, lse
    _call(index, "bsa_prompt_attention", _rows(q), _rows(k), _rows(v), _rows(out), lse.data_ptr(), _ELEMENTS[q.dtype],
          offsets.data_ptr(), n, T, Hq, Hkv, d, PROMPT_CAUSAL if causal else 0, 0.0 if scale is None else scale,
          workspace.data_ptr(), workspace.numel(), _raw_stream(index) if stream is None else stream.cuda_stream)
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
