"""Python binding of the flamia C ABI (include/flamia.h).

Argument marshalling only: torch tensors supply device pointers and the
current CUDA stream; every step of the attention path runs in the library's
own CUDA kernels.  There is no fallback: if the library is missing or a call
returns an error status, a RuntimeError is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libflamia.so")

FLAMIA_OK = 0
FORMAT_MXFP8 = 0
FORMAT_MXFP8_NVFP4 = 1
FORMAT_HADAMARD = 0x10
FORMAT_TOKEN_SCALES = 0x20
FLAG_NVFP4_QK = 0x1
FLAG_HADAMARD = 0x2
FLAG_NONCAUSAL = 0x4
FLAG_DETERMINISTIC_DQ = 0x8
FLAG_DQ_FP16 = 0x10
FLAG_DQ_CAUSAL_SCALE = 0x20
FLAG_SCHEDULE_STATIC = 0x40
FLAG_SCHEDULE_RULE = 0x80
FLAG_DS_ROW_EXPONENTS = 0x100
FLAG_TOKEN_SCALES = 0x200
FLAG_DS_ZERO_COUNT = 0x400
FLAG_BWD_CTA_PAIR = 0x800
FLAG_BWD_ONE_CTA = 0x1000
FLAG_ROPE_INTERLEAVED = 0x2000
FLAG_ROPE_INVERSE = 0x4000
FLAG_PREFIX_ALWAYS = 0x8000
DEV_BAD_SEQLENS = 0x1
DEV_CAPACITY = 0x2
DEV_TIMEOUT = 0x4
DEV_RANGE = 0x8
DEV_BAD_PAGE = 0x10

_LIB = None


class QTensorStruct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("nvfp4_codes", ctypes.c_void_p), ("nvfp4_scales", ctypes.c_void_p)]


class KVCacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32)]


_i64 = ctypes.c_int64
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_QP = ctypes.POINTER(QTensorStruct)
_CP = ctypes.POINTER(KVCacheStruct)
SIGNATURES = {
    "flamia_quantize_tokenblock": (_i, [_vp, _i, _i, _i, _vp, _i, _i, _vp, _vp, _QP, _vp, _vp]),
    "flamia_quantize_qkv": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _i, _i, _QP, _QP, _QP, _vp,
                                 _vp]),
    "flamia_worklist_bytes": (_sz, [_i, _i]),
    "flamia_build_worklist": (_i, [_vp, _i, _i, _vp, _sz, _vp, _vp]),
    "flamia_attn_fwd": (_i, [_QP, _QP, _QP, _vp, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _vp, _vp]),
    "flamia_attn_fwd_gqa": (_i, [_QP, _QP, _QP, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp,
                                 _vp, _vp]),
    "flamia_fwd_workspace_bytes": (_sz, [_i, _i, _i]),
    "flamia_bwd_ds_counts_offset": (_sz, [_i, _i, _i]),
    "flamia_bwd_workspace_bytes": (_sz, [_i, _i, _i]),
    "flamia_attn_bwd": (_i, [_QP, _QP, _QP, _QP, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp,
                             _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "flamia_attn_bwd_gqa": (_i, [_QP, _QP, _QP, _QP, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i,
                                 _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "flamia_build_worklist_static": (_i, [_vp, _i, _i, _vp, _sz, _vp, _vp]),
    "flamia_rope": (_i, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i, _i, _i, _i, _vp, _i, _f,
                         _i, _vp, _i, _vp, _vp, _vp]),
    "flamia_rope_axes": (_i, [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i, _i, _i, _i, _vp, _vp,
                              _i, _f, _i, _vp, _i64, _i, _vp, _i, _vp, _vp]),
    "flamia_pages_copy": (_i, [_CP, _CP, _vp, _vp, _i, _vp, _vp]),
    "flamia_pages_fork_workspace_bytes": (_sz, [_i, _i]),
    "flamia_pages_fork": (_i, [_vp, _i, _vp, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _sz, _vp, _vp]),
    "flamia_pages_reserve_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "flamia_pages_reserve": (_i, [_CP, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "flamia_pages_compact_workspace_bytes": (_sz, [_i]),
    "flamia_pages_compact": (_i, [_CP, _vp, _vp, _i, _i, _vp, _vp, _sz, _vp, _vp]),
    "flamia_cache_write": (_i, [_CP, _vp, _i64, _vp, _i64, _i, _vp, _i, _vp, _vp, _i, _i, _vp,
                                _vp]),
    "flamia_cache_read": (_i, [_CP, _vp, _i64, _vp, _i64, _i, _vp, _i, _vp, _vp, _i, _vp, _vp]),
    "flamia_attn_cache_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "flamia_attn_cache": (_i, [_CP, _vp, _i64, _i, _i, _vp, _i, _vp, _vp, _i, _f, _i, _i, _vp,
                               _vp, _vp, _sz, _vp, _vp]),
    "flamia_attn_cache_prefix_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i, _i]),
    "flamia_attn_cache_prefix": (_i, [_CP, _vp, _i64, _i, _i, _vp, _i, _vp, _vp, _i, _i, _f, _i,
                                      _vp, _vp, _vp, _sz, _vp, _vp]),
    "flamia_status_str": (ctypes.c_char_p, [_i]),
    "flamia_debug_mma_tile": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "flamia_debug_bounded_waits": (_i, [_vp, _vp, _vp]),
    "flamia_debug_launch_count": (ctypes.c_ulonglong, []),
    "flamia_debug_tmem_ldred": (_i, [_vp, _vp, _vp, _vp]),
    "flamia_debug_pair_mma": (_i, [_i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
}


def load(path: str = LIB_PATH):
    """Loads the built library (raises if it was not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(path):
            raise RuntimeError(f"flamia CUDA library not built ({path}); "
                               "run __graft_entry__.build() first")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


def _check(status: int, what: str):
    if status != FLAMIA_OK:
        msg = load().flamia_status_str(status).decode()
        raise RuntimeError(f"{what} failed: {msg} ({status})")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise RuntimeError("flamia needs CUDA tensors")
    if not t.is_contiguous():
        raise RuntimeError("flamia needs contiguous tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


class QTensor:
    """Caller-owned buffers of one quantised operand (allocated by torch)."""

    def __init__(self, T: int, H: int, d: int, nvfp4: bool = False, device="cuda"):
        self.codes = torch.empty((T, H, d), dtype=torch.uint8, device=device)
        self.scales = torch.empty((H, T), dtype=torch.uint8, device=device)
        self.nvfp4_codes = torch.empty((T, H, d // 2), dtype=torch.uint8, device=device) if nvfp4 else None
        self.nvfp4_scales = torch.empty((T, H, d // 16), dtype=torch.uint8, device=device) if nvfp4 else None

    def struct(self) -> QTensorStruct:
        s = QTensorStruct()
        s.codes = self.codes.data_ptr()
        s.scales = self.scales.data_ptr()
        s.nvfp4_codes = self.nvfp4_codes.data_ptr() if self.nvfp4_codes is not None else None
        s.nvfp4_scales = self.nvfp4_scales.data_ptr() if self.nvfp4_scales is not None else None
        return s


def flamia_quantize_tokenblock(x, cu_seqlens, out: QTensor, fmt: int = FORMAT_MXFP8, o=None,
                               D=None, dev_status=None):
    T, H, d = x.shape
    st = out.struct()
    _check(load().flamia_quantize_tokenblock(
        _ptr(x), T, H, d, _ptr(cu_seqlens), cu_seqlens.numel() - 1, fmt, _ptr(o), _ptr(D),
        ctypes.byref(st), _ptr(dev_status), _stream()), "flamia_quantize_tokenblock")


def flamia_quantize_qkv(xq, xk, xv, cu_seqlens, q: QTensor, k: QTensor, v: QTensor,
                        fmt_qk: int = FORMAT_MXFP8, dev_status=None):
    T, H, d = xq.shape
    sq, sk, sv = q.struct(), k.struct(), v.struct()
    _check(load().flamia_quantize_qkv(
        _ptr(xq), _ptr(xk), _ptr(xv), T, H, xk.shape[1], d, _ptr(cu_seqlens),
        cu_seqlens.numel() - 1, fmt_qk, ctypes.byref(sq), ctypes.byref(sk), ctypes.byref(sv),
        _ptr(dev_status), _stream()), "flamia_quantize_qkv")


def flamia_worklist_bytes(T: int, ndocs: int) -> int:
    return int(load().flamia_worklist_bytes(T, ndocs))


def flamia_build_worklist(cu_seqlens, T: int, wl, dev_status=None):
    _check(load().flamia_build_worklist(_ptr(cu_seqlens), cu_seqlens.numel() - 1, T, _ptr(wl),
                                        wl.numel() * wl.element_size(), _ptr(dev_status),
                                        _stream()), "flamia_build_worklist")


def flamia_build_worklist_static(cu_seqlens, T: int, wl, dev_status=None):
    """Work list with the builder's scratch in the library's static device
    array (no allocation); same output as flamia_build_worklist."""
    _check(load().flamia_build_worklist_static(_ptr(cu_seqlens), cu_seqlens.numel() - 1, T,
                                               _ptr(wl), wl.numel() * wl.element_size(),
                                               _ptr(dev_status), _stream()),
           "flamia_build_worklist_static")


def flamia_attn_fwd(q: QTensor, k: QTensor, v: QTensor, cu_seqlens, T, H, d, softmax_scale,
                    wl, o, lse, flags: int = 0, dev_status=None):
    sq, sk, sv = q.struct(), k.struct(), v.struct()
    _check(load().flamia_attn_fwd(ctypes.byref(sq), ctypes.byref(sk), ctypes.byref(sv),
                                  _ptr(cu_seqlens), cu_seqlens.numel() - 1, T, H, d,
                                  float(softmax_scale), flags, _ptr(wl), _ptr(o), _ptr(lse),
                                  _ptr(dev_status), _stream()), "flamia_attn_fwd")


def flamia_attn_fwd_gqa(q: QTensor, k: QTensor, v: QTensor, cu_seqlens, T, H, H_kv, d,
                        softmax_scale, wl, o, lse, flags: int = 0, dev_status=None):
    sq, sk, sv = q.struct(), k.struct(), v.struct()
    _check(load().flamia_attn_fwd_gqa(ctypes.byref(sq), ctypes.byref(sk), ctypes.byref(sv),
                                      _ptr(cu_seqlens), cu_seqlens.numel() - 1, T, H, H_kv, d,
                                      float(softmax_scale), flags, _ptr(wl), _ptr(o), _ptr(lse),
                                      _ptr(dev_status), _stream()), "flamia_attn_fwd_gqa")


def flamia_bwd_ds_counts_offset(T: int, H: int, d: int) -> int:
    return int(load().flamia_bwd_ds_counts_offset(T, H, d))


def flamia_fwd_workspace_bytes(T: int, H: int, d: int) -> int:
    return int(load().flamia_fwd_workspace_bytes(T, H, d))


def flamia_bwd_workspace_bytes(T: int, H: int, d: int) -> int:
    return int(load().flamia_bwd_workspace_bytes(T, H, d))


def flamia_attn_bwd(q: QTensor, k: QTensor, v: QTensor, dout: QTensor, D, lse, cu_seqlens, T, H,
                    d, softmax_scale, wl, dq, dk, dv, ws, flags: int = 0, dev_status=None):
    sq, sk, sv, sd = q.struct(), k.struct(), v.struct(), dout.struct()
    _check(load().flamia_attn_bwd(ctypes.byref(sq), ctypes.byref(sk), ctypes.byref(sv),
                                  ctypes.byref(sd), _ptr(D), _ptr(lse), _ptr(cu_seqlens),
                                  cu_seqlens.numel() - 1, T, H, d, float(softmax_scale), flags,
                                  _ptr(wl), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                  ws.numel() * ws.element_size(), _ptr(dev_status), _stream()),
           "flamia_attn_bwd")


def flamia_attn_bwd_gqa(q: QTensor, k: QTensor, v: QTensor, dout: QTensor, D, lse, cu_seqlens,
                        T, H, H_kv, d, softmax_scale, wl, dq, dk, dv, ws, flags: int = 0,
                        dev_status=None):
    sq, sk, sv, sd = q.struct(), k.struct(), v.struct(), dout.struct()
    _check(load().flamia_attn_bwd_gqa(ctypes.byref(sq), ctypes.byref(sk), ctypes.byref(sv),
                                      ctypes.byref(sd), _ptr(D), _ptr(lse), _ptr(cu_seqlens),
                                      cu_seqlens.numel() - 1, T, H, H_kv, d, float(softmax_scale),
                                      flags, _ptr(wl), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                      ws.numel() * ws.element_size(), _ptr(dev_status),
                                      _stream()), "flamia_attn_bwd_gqa")


_BF16, _I32 = torch.bfloat16, torch.int32
_INT_MAX = (1 << 31) - 1


def _current():
    """(device index, raw stream) that a call's tensors have to be on and its work goes to."""
    if not torch.cuda.is_initialized():
        return -2, 0  # no tensor is there (CPU tensors answer -1)
    d = torch._C._cuda_getDevice()
    return d, torch._C._cuda_getCurrentRawStream(d)


def _elsewhere(name):
    raise RuntimeError(f"{name}: flamia needs tensors on the current CUDA device")


def _rows(x, name, T, heads, d, dev, out=False):
    """(pointer, token stride in elements) of BF16 rows [T, heads, d]: any
    token stride, the heads of a token side by side."""
    if x.dtype is not _BF16 or x.dim() != 3:
        raise RuntimeError(f"{name}: flamia needs BF16 rows [T, heads, d]")
    t, h, n = x.shape
    if t != T or h != heads or n != d:
        raise RuntimeError(f"{name}: shape {tuple(x.shape)}, expected {(T, heads, d)}")
    stride = h * n
    if t > 1 and not x.is_contiguous():
        stride, sh, sd = x.stride()
        if sd != 1 or (h > 1 and sh != n):
            raise RuntimeError(f"{name}: the heads of a token must be contiguous")
        if out and stride < h * n:
            raise RuntimeError(f"{name}: an output's rows must not overlap")
    elif t <= 1 and not x.is_contiguous():  # (whatever the stride of a single token)
        raise RuntimeError(f"{name}: the heads of a token must be contiguous")
    if x.get_device() != dev:
        _elsewhere(name)
    return x.data_ptr(), stride


def _ints(t, name, numel, dev):
    """Pointer of a contiguous int32 tensor (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not _I32 or not t.is_contiguous() or (numel and t.numel() != numel):
        raise RuntimeError(f"{name}: expected a contiguous int32 tensor"
                           + (f" of {numel} entries" if numel else ""))
    if t.get_device() != dev:
        _elsewhere(name)
    return t.data_ptr()


def _page_table(t, nseq, dev):
    if t.dim() != 2 or t.shape[0] != nseq:
        raise RuntimeError(f"page_table: shape {tuple(t.shape)}, expected [{nseq}, pages]")
    return _ints(t, "page_table", 0, dev)


def rope_frequencies(rot_dim: int, base: float = 10000.0, factor: float = 1.0,
                     method: str = "linear", original_len: int = 8192, low: float = 1.0,
                     high: float = 4.0):
    """Angles per position w_i (float64, [rot_dim / 2]) for Rotary, scaled for
    contexts ``factor`` times longer than a model was trained on:

    ``linear``  w_i / factor (positions squeezed);
    ``base``    the base grows to base * factor^(r / (r - 2)), so the slowest
                pair turns ``factor`` times slower and the fastest keeps its pace;
    ``bands``   pairs that turn more than ``high`` times over ``original_len``
                positions keep w_i, those that turn less than ``low`` times take
                w_i / factor, a linear blend between."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    if method not in ("linear", "base", "bands"):
        raise ValueError(f"unknown scaling method {method!r}")
    if method == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    w = base ** (-i / rot_dim)
    if method == "linear":
        w = w / factor
    elif method == "bands":
        turns = original_len * w / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        w = keep * w + (1 - keep) * (w / factor)
    return w


def rope_axes(sections, cyclic: bool = False):
    """The axis of every pair, for Rotary: the first sections[0] pairs turn with axis 0,
    the next sections[1] with axis 1, and so on; cyclic: axes by turns (0, 1, 2, 0, 1, 2,
    ..), each until it has its pairs."""
    left = [int(n) for n in sections]
    if not left or min(left) < 0:
        raise ValueError("sections must be counts of pairs")
    if not cyclic:
        return [a for a, n in enumerate(left) for _ in range(n)]
    return [a for turn in range(max(left)) for a, n in enumerate(left) if turn < n]


class Rotary:
    """Rotary positions with the angles p * frequencies[i] (see
    rope_frequencies); holds the device table of turns per position.

    axes (see rope_axes): the axis of each pair.  Calls then take ``positions``, int32
    [axes, T], instead of starts: those of every packed token (time, height and width
    of a patch; the same number on all axes for text)."""

    def __init__(self, frequencies, interleaved: bool = False, mscale: float = 1.0,
                 device="cuda", axes=None):
        w = [float(f) for f in frequencies]
        self.rot_dim, self.interleaved, self.mscale = 2 * len(w), bool(interleaved), float(mscale)
        if not all(math.isfinite(f) for f in w):
            raise ValueError("frequencies must be finite")
        steps = [round(f / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for f in w]
        self.turns = torch.tensor([s - (1 << 64) if s >> 63 else s for s in steps],
                                  dtype=torch.int64, device=device)
        self.flags = FLAG_ROPE_INTERLEAVED if interleaved else 0
        self.axes, self.naxes = None, 0
        if axes is not None:
            a = [int(x) for x in axes]
            if len(a) != len(w) or not a or min(a) < 0 or max(a) >= len(w):
                raise ValueError("axes: expected an axis for each pair, fewer axes than pairs or as many")
            self.naxes = max(a) + 1
            self.axes = torch.tensor(a, dtype=torch.uint8, device=device)

    def __call__(self, q, k, cu_seqlens, starts=None, q_out=None, k_out=None,
                 inverse: bool = False, dev_status=None, positions=None):
        """Rotated q and k (k may be None); inverse: gradients of the rotated
        rows -> gradients of the rows.  q_out / k_out may be q / k.  positions: with
        axes, and then instead of starts (it may have more rows than axes are used)."""
        if (positions is None) != (self.axes is None) or not (positions is None or starts is None):
            raise RuntimeError("positions: needed with axes, without starts, and only then")
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format) if q_out is None else q_out
        if k is not None and k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        if positions is None:
            flamia_rope(q, q_out, k, k_out, self, cu_seqlens, starts, inverse, dev_status)
        else:
            flamia_rope_axes(q, q_out, k, k_out, self, positions, cu_seqlens, inverse, dev_status)
        return q_out, k_out


def _positions_fit(rope, positions):
    """Positions belong to a rope with axes (Rotary checks its own calls)."""
    if (positions is None) != (rope is None or rope.axes is None):
        raise RuntimeError("positions: needed for a rope with axes, and only then")


def _rope_rows(q_in, q_out, k_in, k_out, rotary, dev):
    if q_in.dim() != 3:
        raise RuntimeError("q_in: flamia needs BF16 rows [T, heads, d]")
    T, H, d = q_in.shape
    qi, qis = _rows(q_in, "q_in", T, H, d, dev)
    qo, qos = _rows(q_out, "q_out", T, H, d, dev, True)
    H_kv, ki, kis, ko, kos = 0, None, 0, None, 0
    if k_in is not None:
        H_kv = k_in.shape[1]
        ki, kis = _rows(k_in, "k_in", T, H_kv, d, dev)
        ko, kos = _rows(k_out, "k_out", T, H_kv, d, dev, True)
    if rotary.turns.get_device() != dev:
        _elsewhere("turns")
    return qi, qo, qis, qos, ki, ko, kis, kos, T, H, H_kv, d, rotary.turns.data_ptr()


def flamia_rope(q_in, q_out, k_in, k_out, rotary: Rotary, cu_seqlens, starts=None,
                inverse: bool = False, dev_status=None):
    dev, stream = _current()
    rows = _rope_rows(q_in, q_out, k_in, k_out, rotary, dev)
    n = cu_seqlens.numel() - 1
    st = (_LIB or load()).flamia_rope(
        *rows, rotary.rot_dim, rotary.mscale,
        rotary.flags | (FLAG_ROPE_INVERSE if inverse else 0),
        _ints(cu_seqlens, "cu_seqlens", 0, dev), n, _ints(starts, "starts", n, dev),
        _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_rope")


def flamia_rope_axes(q_in, q_out, k_in, k_out, rotary: Rotary, positions, cu_seqlens,
                     inverse: bool = False, dev_status=None):
    dev, stream = _current()
    rows = _rope_rows(q_in, q_out, k_in, k_out, rotary, dev)
    T = q_in.shape[0]
    if (positions.dtype is not _I32 or positions.dim() != 2 or positions.shape[0] < rotary.naxes
            or positions.shape[1] != T or (T > 1 and positions.stride(1) != 1)):
        raise RuntimeError(f"positions: expected int32 [{rotary.naxes}, {T}], tokens side by side")
    if positions.get_device() != dev:
        _elsewhere("positions")
    st = (_LIB or load()).flamia_rope_axes(
        *rows, rotary.axes.data_ptr(), rotary.rot_dim, rotary.mscale,
        rotary.flags | (FLAG_ROPE_INVERSE if inverse else 0), positions.data_ptr(),
        positions.stride(0), rotary.naxes, _ints(cu_seqlens, "cu_seqlens", 0, dev),
        cu_seqlens.numel() - 1, _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_rope_axes")


class KVCache:
    """Paged key-value cache in E4M3 codes with one E8M0 exponent per 32-token
    block and head (token_scales: per token and head).  Position p of sequence
    b is row p % page_size of page page_table[b, p // page_size]; the caller
    hands out the pages."""

    def __init__(self, num_pages: int, page_size: int, H_kv: int, d: int,
                 token_scales: bool = False, device="cuda"):
        shape = (num_pages, H_kv, page_size)
        codes = [torch.zeros(*shape, d, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2)]
        self._set(codes[0], scales[0], codes[1], scales[1], token_scales)

    @classmethod
    def from_buffers(cls, k_codes, k_scales, v_codes, v_scales, token_scales: bool = False):
        """A cache over the caller's uint8 buffers: codes [pages, H_kv,
        page_size, d], scales [pages, H_kv, page_size]."""
        self = cls.__new__(cls)
        self._set(k_codes, k_scales, v_codes, v_scales, token_scales)
        return self

    def _set(self, k_codes, k_scales, v_codes, v_scales, token_scales):
        if k_codes.dim() != 4:
            raise RuntimeError("k_codes: expected [pages, H_kv, page_size, d]")
        for t, name, shape in ((k_codes, "k_codes", k_codes.shape),
                               (v_codes, "v_codes", k_codes.shape),
                               (k_scales, "k_scales", k_codes.shape[:3]),
                               (v_scales, "v_scales", k_codes.shape[:3])):
            if t.dtype is not torch.uint8 or not t.is_contiguous() or t.shape != shape:
                raise RuntimeError(f"{name}: expected contiguous uint8 {tuple(shape)}")
            if not t.is_cuda or t.device != k_codes.device:
                raise RuntimeError(f"{name}: flamia needs CUDA tensors on one device")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = (k_codes, k_scales, v_codes,
                                                                    v_scales)
        self.num_pages, self.H_kv, self.page_size, self.d = k_codes.shape
        self.token_scales = bool(token_scales)
        self._struct = KVCacheStruct(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                     v_scales.data_ptr(), self.num_pages, self.page_size,
                                     self.H_kv, self.d)
        self._ref = ctypes.byref(self._struct)
        self.device_index = k_codes.get_device()

    @property
    def _ws(self):  # (of eager calls)
        return _eager_workspace(*_current())[0]

    def write(self, k, v, cu_seqlens, starts, page_table, dev_status=None):
        """Quantises rows k, v [T, H_kv, d] into positions starts[b] .. of each
        sequence (starts None: 0)."""
        flamia_cache_write(self, k, v, cu_seqlens, starts, page_table, dev_status)

    def read(self, cu_seqlens, starts, page_table, T: int, k_out=None, v_out=None,
             dev_status=None):
        """BF16 rows of positions starts[b] .. of each sequence, packed [T, H_kv, d]."""
        if k_out is None:
            k_out = torch.empty(T, self.H_kv, self.d, dtype=torch.bfloat16,
                                device=self.k_codes.device)
        if v_out is None:
            v_out = torch.empty_like(k_out)
        flamia_cache_read(self, k_out, v_out, cu_seqlens, starts, page_table, dev_status)
        return k_out, v_out

    def copy_pages(self, src, dst, source: "KVCache" = None, dev_status=None):
        """Page dst[i] becomes page src[i] of `source` (None: of this cache); int32
        tensors, pairs with a negative entry are left out.  No page may be a target
        twice, or source and target."""
        flamia_pages_copy(self if source is None else source, self, src, dst, dev_status)

    def attend(self, q, cu_seqlens, starts, page_table, softmax_scale: float, window: int = 0,
               sinks: int = 0, o=None, lse=None, ws=None, dev_status=None, prefix: int = 0,
               always_share: bool = False):
        """(o, lse) of queries q [T, H, d] at positions starts[b] .. over the
        cache.  prefix: the sequences begin with the same so many tokens (those of which
        all new tokens stand at prefix - 1 or behind), which are read once for all of
        them where that is faster (always_share: in any case); with a window each reads
        its own.  Nothing checks that they are the same: every sequence as long as that is
        given the first one's keys and values there, so one that begins with something else
        has to go into another call.  With a prefix read once and more than 8 query rows of
        a K / V head in the batch, softmax weights are rounded to 2^-11 of themselves (plain
        calls: with more than 8 rows a sequence).  ws None: the workspace of the current
        stream and thread (42 MB, made by their first call, shared by all caches; beside it
        one for calls with a prefix, as large as their largest needed), or, while a graph is
        captured, one that belongs to the graph: calls that overlap never share one."""
        T, H = q.shape[0], q.shape[1]
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
        if prefix and not window and not sinks:
            flamia_attn_cache_prefix(self, q, cu_seqlens, starts, page_table, prefix, softmax_scale,
                                     o, lse, ws, dev_status,
                                     FLAG_PREFIX_ALWAYS if always_share else 0)
        else:
            if prefix < 0:
                raise RuntimeError("prefix: expected 0 or more tokens")
            flamia_attn_cache(self, q, cu_seqlens, starts, page_table, softmax_scale, window, sinks,
                              o, lse, ws, dev_status)
        return o, lse


class _Held(threading.local):
    """Workspaces of a thread's eager attend calls, (tensor, pointer, bytes) by (device,
    stream).  Nothing is kept in one, so calls that follow one another share it; two
    threads on one stream do not, as one's kernels may come between the other's."""

    def __init__(self):
        self.ws = {}
        self.prefix = {}  # of calls with a shared prefix: as large as they were


_HELD = _Held()


@functools.lru_cache(maxsize=1024)
def _prefix_bytes(*sizes):
    return int(load().flamia_attn_cache_prefix_workspace_bytes(*sizes))


def _prefix_workspace(dev, stream, size):
    held = _HELD.prefix.get((dev, stream))
    if held is None or held[2] < size:
        # (the one before is the stream's again, behind the calls that use it)
        t = torch.empty(max(1, size), dtype=torch.uint8, device=torch.device("cuda", dev))
        held = _HELD.prefix[dev, stream] = t, t.data_ptr(), t.nbytes
    return held


def _eager_workspace(dev, stream):
    held = _HELD.ws.get((dev, stream))
    if held is None:
        size = flamia_attn_cache_workspace_bytes(1 << 10, 1, 1, 1, 128)  # enough for all calls
        t = torch.empty(size, dtype=torch.uint8, device=torch.device("cuda", dev))
        held = _HELD.ws[dev, stream] = t, t.data_ptr(), size
    return held


def flamia_cache_write(cache: KVCache, k, v, cu_seqlens, starts, page_table, dev_status=None):
    dev, stream = _current()
    T, n = k.shape[0], cu_seqlens.numel() - 1
    kp, ks = _rows(k, "k", T, cache.H_kv, cache.d, dev)
    vp, vs = _rows(v, "v", T, cache.H_kv, cache.d, dev)
    if cache.device_index != dev:
        _elsewhere("cache")
    st = (_LIB or load()).flamia_cache_write(
        cache._ref, kp, ks, vp, vs, T, _ints(cu_seqlens, "cu_seqlens", 0, dev), n,
        _ints(starts, "starts", n, dev), _page_table(page_table, n, dev), page_table.shape[1],
        FORMAT_TOKEN_SCALES if cache.token_scales else FORMAT_MXFP8,
        _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_cache_write")


def flamia_cache_read(cache: KVCache, k_out, v_out, cu_seqlens, starts, page_table,
                      dev_status=None):
    dev, stream = _current()
    T, n = k_out.shape[0], cu_seqlens.numel() - 1
    kp, ks = _rows(k_out, "k_out", T, cache.H_kv, cache.d, dev, True)
    vp, vs = _rows(v_out, "v_out", T, cache.H_kv, cache.d, dev, True)
    if cache.device_index != dev:
        _elsewhere("cache")
    st = (_LIB or load()).flamia_cache_read(
        cache._ref, kp, ks, vp, vs, T, _ints(cu_seqlens, "cu_seqlens", 0, dev), n,
        _ints(starts, "starts", n, dev), _page_table(page_table, n, dev), page_table.shape[1],
        _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_cache_read")


def flamia_attn_cache_workspace_bytes(T: int, ndocs: int, H: int, H_kv: int, d: int) -> int:
    return int(load().flamia_attn_cache_workspace_bytes(T, ndocs, H, H_kv, d))


def _attend_rows(cache, q, o, lse, dev):
    """(pointer, stride, T, H) of the queries, pointer of lse."""
    if q.dim() != 3:
        raise RuntimeError("q: flamia needs BF16 rows [T, heads, d]")
    T, H, d = q.shape
    qp, qs = _rows(q, "q", T, H, cache.d, dev)
    if o.dtype is not _BF16 or o.shape != q.shape or not o.is_contiguous():
        raise RuntimeError("o: expected contiguous BF16 of q's shape")
    lp = None
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (H, T) or not lse.is_contiguous():
            raise RuntimeError("lse: expected contiguous float32 [H, T]")
        lp = lse.data_ptr()
        if lse.get_device() != dev:
            _elsewhere("lse")
    if cache.device_index != dev or o.get_device() != dev:
        _elsewhere("cache and o")
    return qp, qs, T, H, lp


def _given_workspace(ws, dev):
    if not ws.is_contiguous():
        raise RuntimeError("ws: expected a contiguous tensor")
    if ws.get_device() != dev:
        _elsewhere("ws")
    return ws.data_ptr(), ws.nbytes


def flamia_attn_cache(cache: KVCache, q, cu_seqlens, starts, page_table, softmax_scale, window,
                      sinks, o, lse, ws=None, dev_status=None):
    dev, stream = _current()
    qp, qs, T, H, lp = _attend_rows(cache, q, o, lse, dev)
    n = cu_seqlens.numel() - 1
    if ws is None:
        if torch._C._cuda_isCurrentStreamCapturing():
            # from the graph's pool: replays of two graphs may overlap
            ws = torch.empty(flamia_attn_cache_workspace_bytes(T, n, H, cache.H_kv, cache.d),
                             dtype=torch.uint8, device=q.device)
            wp, wn = ws.data_ptr(), ws.nbytes
        else:
            _, wp, wn = _eager_workspace(dev, stream)
    else:
        wp, wn = _given_workspace(ws, dev)
    if not (0 <= window <= _INT_MAX and 0 <= sinks <= _INT_MAX):
        # (ctypes would keep the low 32 bits; positions end before, negative ones are refused)
        window, sinks = (max(-1, min(x, _INT_MAX)) for x in (window, sinks))
    st = (_LIB or load()).flamia_attn_cache(
        cache._ref, qp, qs, T, H, _ints(cu_seqlens, "cu_seqlens", 0, dev), n,
        _ints(starts, "starts", n, dev), _page_table(page_table, n, dev), page_table.shape[1],
        float(softmax_scale), window, sinks, o.data_ptr(), lp, wp, wn,
        _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_attn_cache")


def flamia_attn_cache_prefix_workspace_bytes(T: int, ndocs: int, H: int, H_kv: int, d: int,
                                             prefix: int, flags: int = 0) -> int:
    return int(load().flamia_attn_cache_prefix_workspace_bytes(
        T, ndocs, H, H_kv, d, max(-1, min(prefix, _INT_MAX)), flags))


def flamia_attn_cache_prefix(cache: KVCache, q, cu_seqlens, starts, page_table, prefix,
                             softmax_scale, o, lse, ws=None, dev_status=None, flags: int = 0):
    dev, stream = _current()
    qp, qs, T, H, lp = _attend_rows(cache, q, o, lse, dev)
    n = cu_seqlens.numel() - 1
    prefix = max(-1, min(prefix, _INT_MAX))  # (as windows: positions end before)
    lib = _LIB or load()
    if ws is None:
        size = _prefix_bytes(T, n, H, cache.H_kv, cache.d, prefix, flags)  # (0: to be refused)
        if torch._C._cuda_isCurrentStreamCapturing():  # (as in flamia_attn_cache)
            ws = torch.empty(max(1, size), dtype=torch.uint8, device=q.device)
            wp, wn = ws.data_ptr(), ws.nbytes
        else:
            _, wp, wn = _prefix_workspace(dev, stream, size)
    else:
        wp, wn = _given_workspace(ws, dev)
    st = lib.flamia_attn_cache_prefix(
        cache._ref, qp, qs, T, H, _ints(cu_seqlens, "cu_seqlens", 0, dev), n,
        _ints(starts, "starts", n, dev), _page_table(page_table, n, dev), page_table.shape[1],
        prefix, float(softmax_scale), flags, o.data_ptr(), lp, wp, wn,
        _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_attn_cache_prefix")


def flamia_pages_copy(source: KVCache, target: KVCache, src, dst, dev_status=None):
    dev, stream = _current()
    n = src.numel()
    sp, dp = _ints(src, "src", 0, dev), _ints(dst, "dst", n, dev)
    if dst.numel() != n:
        raise RuntimeError(f"dst: expected {n} entries")
    if source.device_index != dev or target.device_index != dev:
        _elsewhere("cache")
    st = (_LIB or load()).flamia_pages_copy(source._ref, target._ref, sp, dp, n,
                                            _ints(dev_status, "dev_status", 0, dev), stream)
    if st:
        _check(st, "flamia_pages_copy")


def flamia_pages_fork_workspace_bytes(n: int, table_stride: int) -> int:
    return int(load().flamia_pages_fork_workspace_bytes(n, table_stride))


def flamia_pages_reserve_workspace_bytes(T: int, nseq: int, table_stride: int,
                                         page_size: int) -> int:
    return int(load().flamia_pages_reserve_workspace_bytes(T, nseq, table_stride, page_size))


def flamia_pages_compact_workspace_bytes(num_pages: int) -> int:
    return int(load().flamia_pages_compact_workspace_bytes(num_pages))


class PagePool:
    """Who uses which page of a cache: page_table int32 [nseq, width] (-1: no page) and
    refs int32 [pages] (slots of the table that hold a page; 0: free), on the device and
    the caller's to read.  Calls on one pool follow one another on one stream (or are
    ordered by the caller); they can be captured.  Errors found on the device (no free
    page, positions outside the table) show in check_status until the caller sets `status`
    to zero."""

    def __init__(self, cache: KVCache, nseq: int, width: int):
        dev = cache.k_codes.device
        self._set(cache, torch.full((nseq, width), -1, dtype=torch.int32, device=dev),
                  torch.zeros(cache.num_pages, dtype=torch.int32, device=dev))

    @classmethod
    def from_buffers(cls, cache: KVCache, page_table, refs):
        """A pool over the caller's tensors, which have to agree."""
        self = cls.__new__(cls)
        self._set(cache, page_table, refs)
        return self

    def _set(self, cache, page_table, refs):
        if page_table.dtype is not _I32 or page_table.dim() != 2 or not page_table.is_contiguous():
            raise RuntimeError("page_table: expected contiguous int32 [sequences, pages]")
        if refs.dtype is not _I32 or refs.shape != (cache.num_pages,) or not refs.is_contiguous():
            raise RuntimeError(f"refs: expected contiguous int32 [{cache.num_pages}]")
        if not page_table.device == refs.device == cache.k_codes.device:
            raise RuntimeError("page_table, refs: expected on the cache's device")
        self.cache, self.page_table, self.refs = cache, page_table, refs
        self.nseq, self.width = page_table.shape
        self.status = torch.zeros(1, dtype=torch.int32, device=refs.device)
        self.live = torch.zeros(1, dtype=torch.int32, device=refs.device)
        self._at = refs.data_ptr(), page_table.data_ptr(), self.status.data_ptr()
        self._sizes = {}    # workspace bytes by call
        self._held = []     # workspaces of eager calls, the last one in use
        self._ws = 0, 0     # its pointer and size

    def _begin(self):
        dev, stream = _current()
        if self.cache.device_index != dev:
            _elsewhere("pool")
        return dev, stream

    def _workspace(self, name, *sizes):
        """(tensor to keep until the call is made, pointer, bytes).  Eager calls follow one
        another and share one, which is never given back while the pool lives (another
        stream may be in it); a captured call has one from its graph's pool."""
        size = self._sizes.get((name, sizes))
        if size is None:
            size = self._sizes[name, sizes] = int(getattr(load(), name)(*sizes))
        if torch._C._cuda_isCurrentStreamCapturing():
            t = torch.empty(max(1, size), dtype=torch.uint8, device=self.refs.device)
            return t, t.data_ptr(), size
        if size > self._ws[1]:
            t = torch.empty(2 * size, dtype=torch.uint8, device=self.refs.device)
            self._held.append(t)
            self._ws = t.data_ptr(), t.nbytes
        return (None,) + self._ws

    def fork(self, parents, children, lens):
        """Sequences children[i] go on from parents[i] (int32 tensors): they give their
        pages back, share those of the parent's first lens[parent] tokens, and
        lens[child] becomes lens[parent] (lens int32 [nseq]).  Negative parents, or None:
        the pages are given back and the length is 0.  Children may be parents of
        others; negative children are left out, and of a child's entries the last counts."""
        dev, stream = self._begin()
        n = children.numel()
        cp = _ints(children, "children", 0, dev)
        pp = _ints(parents, "parents", n, dev)
        if parents is not None and parents.numel() != n:
            raise RuntimeError(f"parents: expected {n} entries")
        lp = _ints(lens, "lens", self.nseq, dev)
        if n == 0:
            return
        refs, table, status = self._at
        keep, wp, wn = self._workspace("flamia_pages_fork_workspace_bytes", n, self.width)
        st = (_LIB or load()).flamia_pages_fork(refs, self.cache.num_pages, table, self.width,
                                                self.nseq, self.cache.page_size, pp, cp, n, lp, wp,
                                                wn, status, stream)
        if st:
            _check(st, "flamia_pages_fork")

    def release(self, sequences, lens):
        """The sequences' pages are given back and their lengths become 0."""
        self.fork(None, sequences, lens)

    def reserve(self, cu_seqlens, starts, T: int = None, granted=None):
        """Pages for the tokens cu_seqlens[b] .. cu_seqlens[b + 1] - 1 at positions
        starts[b] .. of every sequence: what is missing is taken from the free pages, and
        a page with other users is replaced by a copy.  T: an upper bound of the number
        of tokens (None: one that every table row could hold).  granted: int32 [nseq + 1]
        that becomes cu_seqlens, or zeros if pages ran out, positions lie outside the
        table or cu_seqlens is malformed, for the calls that write to the pages."""
        dev, stream = self._begin()
        cp = _ints(cu_seqlens, "cu_seqlens", self.nseq + 1, dev)
        sp = _ints(starts, "starts", self.nseq, dev)
        gp = _ints(granted, "granted", self.nseq + 1, dev)
        if T is None:
            T = min(1 << 20, self.nseq * self.width * self.cache.page_size)
        refs, table, status = self._at
        keep, wp, wn = self._workspace("flamia_pages_reserve_workspace_bytes", T, self.nseq,
                                       self.width, self.cache.page_size)
        st = (_LIB or load()).flamia_pages_reserve(self.cache._ref, refs, table, self.width,
                                                   self.nseq, T, cp, sp, gp, wp, wn, status,
                                                   stream)
        if st:
            _check(st, "flamia_pages_reserve")

    def compact(self, live=None):
        """Moves the used pages to the front of the pool (page table and refs follow) and
        returns their number, int32 [1] on the device (live None: the pool's own tensor,
        the same in every call)."""
        dev, stream = self._begin()
        if live is None:
            live = self.live
        lp = _ints(live, "live", 1, dev)
        refs, table, status = self._at
        keep, wp, wn = self._workspace("flamia_pages_compact_workspace_bytes", self.cache.num_pages)
        st = (_LIB or load()).flamia_pages_compact(self.cache._ref, refs, table, self.width,
                                                   self.nseq, lp, wp, wn, status, stream)
        if st:
            _check(st, "flamia_pages_compact")
        return live

    def check_status(self):
        st = int(self.status.item())
        if st != 0:
            raise RuntimeError(f"flamia device status 0x{st:x}")


def flamia_debug_tmem_ldred(x, vals, mx):
    _check(load().flamia_debug_tmem_ldred(_ptr(x), _ptr(vals), _ptr(mx), _stream()),
           "flamia_debug_tmem_ldred")


def flamia_debug_pair_mma(shape, variant, a, b, sfa, sfb, d_out, tmem_cols, dev_status):
    _check(load().flamia_debug_pair_mma(shape, variant, _ptr(a), _ptr(b), _ptr(sfa), _ptr(sfb),
                                        _ptr(d_out), _ptr(tmem_cols), _ptr(dev_status),
                                        _stream()),
           "flamia_debug_pair_mma")


def flamia_debug_launch_count() -> int:
    """Kernel launches the library has enqueued since it was loaded."""
    return int(load().flamia_debug_launch_count())


def flamia_debug_bounded_waits(turn, dev_status):
    _check(load().flamia_debug_bounded_waits(_ptr(turn), _ptr(dev_status), _stream()),
           "flamia_debug_bounded_waits")


def flamia_debug_mma_tile(mode, N, a_mn, b_mn, variant, a, b, sfa, sfb, d_out, dev_status=None):
    _check(load().flamia_debug_mma_tile(mode, N, a_mn, b_mn, variant, _ptr(a), _ptr(b), _ptr(sfa),
                                        _ptr(sfb), _ptr(d_out), _ptr(dev_status), _stream()),
           "flamia_debug_mma_tile")


class TrainingCall:
    """Buffers and the sequence of C-ABI calls of one attention training call
    (quantise Q, K, V -> work list -> forward -> quantise dO with D -> backward)
    for fixed shapes.  All buffers are torch allocations owned by this object."""

    def __init__(self, T, H, d, cu_seqlens, softmax_scale, nvfp4_qk: bool = False,
                 hadamard: bool = False, causal: bool = True, H_kv=None,
                 deterministic_dq: bool = False, dq_accum: str = "fp32", schedule: str = "dynamic",
                 ds_rows: bool = False, token_scales: bool = False,
                 ds_zero_count: bool = False, bwd_ctas: str = "rule", device="cuda",
                 rope: Rotary = None):
        self.T, self.H, self.d = T, H, d
        self.H_kv = H if H_kv is None else H_kv
        self.scale = softmax_scale
        self.cu = cu_seqlens
        self.flags = ((FLAG_NVFP4_QK if nvfp4_qk else 0) | (FLAG_HADAMARD if hadamard else 0) |
                      (0 if causal else FLAG_NONCAUSAL) |
                      (FLAG_DETERMINISTIC_DQ if deterministic_dq else 0) |
                      {"fp32": 0, "fp16_sequence": FLAG_DQ_FP16,
                       "fp16_causal": FLAG_DQ_FP16 | FLAG_DQ_CAUSAL_SCALE}[dq_accum] |
                      {"dynamic": 0, "rule": FLAG_SCHEDULE_RULE,
                       "static": FLAG_SCHEDULE_STATIC}[schedule] |
                      (FLAG_DS_ROW_EXPONENTS if ds_rows else 0) |
                      (FLAG_TOKEN_SCALES if token_scales else 0) |
                      (FLAG_DS_ZERO_COUNT if ds_zero_count else 0))
        # backward only: one- or two-CTA items (head dim 128), or the library's rule
        self.bwd_flags = self.flags | {"rule": 0, "one": FLAG_BWD_ONE_CTA,
                                       "pair": FLAG_BWD_CTA_PAIR}[bwd_ctas]
        self.fmt_qk = ((FORMAT_MXFP8_NVFP4 if nvfp4_qk else FORMAT_MXFP8) |
                       (FORMAT_HADAMARD if hadamard else 0) |
                       (FORMAT_TOKEN_SCALES if token_scales else 0))
        # dO takes the same scale blocks as Q, K and V
        self.fmt_do = FORMAT_MXFP8 | (FORMAT_TOKEN_SCALES if token_scales else 0)
        self.q = QTensor(T, H, d, nvfp4_qk, device)
        self.k = QTensor(T, self.H_kv, d, nvfp4_qk, device)
        self.v = QTensor(T, self.H_kv, d, False, device)
        self.dout = QTensor(T, H, d, False, device)
        ndocs = cu_seqlens.numel() - 1
        self.wl = torch.empty(flamia_worklist_bytes(T, ndocs), dtype=torch.uint8, device=device)
        self.ws = torch.empty(flamia_bwd_workspace_bytes(T, H, d), dtype=torch.uint8, device=device)
        self.o = torch.empty((T, H, d), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((H, T), dtype=torch.float32, device=device)
        self.D = torch.empty((H, T), dtype=torch.float32, device=device)
        self.dq = torch.empty((T, H, d), dtype=torch.bfloat16, device=device)
        self.dk = torch.empty((T, self.H_kv, d), dtype=torch.bfloat16, device=device)
        self.dv = torch.empty_like(self.dk)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        # the work list is built on a side stream while Q, K, V are quantised;
        # high priority, so its small launches take SMs ahead of the waiting
        # CTAs of the quantiser's one large launch
        self.side = torch.cuda.Stream(device, priority=-1)
        self.wl_ready = torch.cuda.Event()
        # rotary positions (document-local): rotated Q and K before the
        # quantiser, dQ and dK turned back in place after the backward
        self.rope = rope
        self.positions = None
        if rope is not None:
            self.xq = torch.empty((T, H, d), dtype=torch.bfloat16, device=device)
            self.xk = torch.empty((T, self.H_kv, d), dtype=torch.bfloat16, device=device)

    def forward(self, xq, xk, xv, positions=None):
        """positions: for a rope with axes (kept for the backward)."""
        _positions_fit(self.rope, positions)
        main = torch.cuda.current_stream()
        if self.rope is not None:
            self.positions = positions
            xq, xk = self.rope(xq, xk, self.cu, q_out=self.xq, k_out=self.xk,
                               dev_status=self.status, positions=positions)
        # cu_seqlens is ready and the previous call has finished with the list
        self.side.wait_stream(main)
        with torch.cuda.stream(self.side):
            flamia_build_worklist(self.cu, self.T, self.wl, dev_status=self.status)
            self.wl_ready.record(self.side)
        flamia_quantize_qkv(xq, xk, xv, self.cu, self.q, self.k, self.v, self.fmt_qk,
                            dev_status=self.status)
        main.wait_event(self.wl_ready)
        flamia_attn_fwd_gqa(self.q, self.k, self.v, self.cu, self.T, self.H, self.H_kv, self.d,
                            self.scale, self.wl, self.o, self.lse, self.flags,
                            dev_status=self.status)
        return self.o, self.lse

    def backward(self, xdo):
        flamia_quantize_tokenblock(xdo, self.cu, self.dout, self.fmt_do, o=self.o, D=self.D,
                                   dev_status=self.status)
        flamia_attn_bwd_gqa(self.q, self.k, self.v, self.dout, self.D, self.lse, self.cu, self.T,
                            self.H, self.H_kv, self.d, self.scale, self.wl, self.dq, self.dk,
                            self.dv, self.ws, self.bwd_flags, dev_status=self.status)
        if self.rope is not None:
            self.rope(self.dq, self.dk, self.cu, q_out=self.dq, k_out=self.dk, inverse=True,
                      dev_status=self.status, positions=self.positions)
        return self.dq, self.dk, self.dv

    def __call__(self, xq, xk, xv, xdo, positions=None):
        self.forward(xq, xk, xv, positions)
        return self.backward(xdo)

    def ds_zero_counts(self):
        """(nonzero dS entries, those rounded to zero) of the last backward
        with ds_zero_count (reads device memory: call after it completed)."""
        off = flamia_bwd_ds_counts_offset(self.T, self.H, self.d)
        c = self.ws[off:off + 16].view(torch.int64).cpu()
        return int(c[0]), int(c[1])

    def check_status(self):
        st = int(self.status.item())
        if st != 0:
            raise RuntimeError(f"flamia device status 0x{st:x}")


class DecodeCall:
    """Buffers and the sequence of C-ABI calls of one serving step over a
    KVCache (rotary positions -> cache write -> attention) for T rows of new
    tokens of nseq sequences (cu_seqlens may end before T: the rows behind are
    padding, and sequences may be empty).  The calls read cu_seqlens, starts and page_table
    on the device, so a captured step can be replayed while the caller updates
    them in place.

    pool: the step begins with pages for its tokens (PagePool.reserve) and takes the
    pool's page table; where it cannot have them it does nothing more (check_status), as
    other sequences may hold the pages that it would write to.  `granted` holds the step's
    offsets then: cu_seqlens, or zeros, so lengths are to grow by granted.diff().  prefix,
    always_share: the sequences begin with the same so many tokens, read once for all of
    them (KVCache.attend, which says what is not checked)."""

    def __init__(self, cache: KVCache, T: int, nseq: int, H: int, softmax_scale: float,
                 rope: Rotary = None, window: int = 0, sinks: int = 0, pool: PagePool = None,
                 prefix: int = 0, always_share: bool = False):
        if pool is not None and (pool.cache is not cache or pool.nseq != nseq):
            raise RuntimeError("pool: expected one over this cache with a row a sequence")
        dev = cache.k_codes.device
        self.cache, self.T, self.H, self.scale = cache, T, H, float(softmax_scale)
        self.rope, self.window, self.sinks = rope, int(window), int(sinks)
        self.pool, self.prefix, self.always_share = pool, int(prefix), bool(always_share)
        self.o = torch.empty((T, H, cache.d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((H, T), dtype=torch.float32, device=dev)
        size = (flamia_attn_cache_workspace_bytes(T, nseq, H, cache.H_kv, cache.d)
                if self.window or not self.prefix else
                flamia_attn_cache_prefix_workspace_bytes(T, nseq, H, cache.H_kv, cache.d, self.prefix,
                                                         FLAG_PREFIX_ALWAYS if always_share else 0))
        self.ws = torch.empty(size, dtype=torch.uint8, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.granted = None if pool is None else torch.zeros(nseq + 1, dtype=torch.int32, device=dev)
        if rope is not None:
            self.q = torch.empty((T, H, cache.d), dtype=torch.bfloat16, device=dev)
            self.k = torch.empty((T, cache.H_kv, cache.d), dtype=torch.bfloat16, device=dev)

    def __call__(self, q, k, v, cu_seqlens, starts, page_table=None, positions=None):
        """o [T, H, d] of the new tokens at positions starts[b] .. of each
        sequence; rows behind the last sequence are left as they were.  page_table:
        without a pool; positions: for a rope with axes."""
        if (page_table is None) != (self.pool is not None):
            raise RuntimeError("page_table: needed without a pool, and only then")
        _positions_fit(self.rope, positions)
        if self.pool is not None:
            self.pool.reserve(cu_seqlens, starts, self.T, self.granted)
            cu_seqlens = self.granted
            page_table = self.pool.page_table
        if self.rope is not None:
            q, k = self.rope(q, k, cu_seqlens, starts if self.rope.axes is None else None,
                             q_out=self.q, k_out=self.k, dev_status=self.status,
                             positions=positions)
        self.cache.write(k, v, cu_seqlens, starts, page_table, dev_status=self.status)
        self.cache.attend(q, cu_seqlens, starts, page_table, self.scale, self.window, self.sinks,
                          o=self.o, lse=self.lse, ws=self.ws, dev_status=self.status,
                          prefix=self.prefix, always_share=self.always_share)
        return self.o

    def check_status(self):
        st = int(self.status.item()) | (0 if self.pool is None else int(self.pool.status.item()))
        if st != 0:
            raise RuntimeError(f"flamia device status 0x{st:x}")
