"""Binding of libmi_decode: the operators beside the projections of a decode step.

* ``Decode.w4_linear``  -- linear layer with 4-bit weights and group scales, for few tokens;
* ``Decode.kv_append``  -- keys and values of new tokens, rotated by their positions, into a
  paged 8-bit cache with a scale for each page and head;
* ``Decode.kv_read``    -- the values of cached tokens;
* ``Decode.kv_attend``  -- attention over that cache (grouped heads, causal, a window with
  first tokens that stay visible), one query a sequence or ragged many.

Operations, layouts and rules are those of ``include/mi_decode.h``; torch supplies device
memory and the stream.  The four calls check and marshal their arguments in an extension
module (``bind/decode_calls.cpp``), because a decode step's kernels take microseconds; the
rest of the library is reached with ctypes.  A call returns
without synchronising, and every call may be captured into a graph.  Work goes to the
current stream, or to ``stream`` (a torch stream, or a handle as an integer), whose memory
the results are then, as if it were the current one.  ``kv_attend`` uses the
handle's workspace: calls that may overlap on different streams need handles of their own.

    from dense_fp16_gemm_hgemm_amd import decode
    d = decode.Decode()
    w = decode.w4_quantize(weight)                       # [N, K] -> W4 (qweight, scales, zeros, n, group)
    y = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=w.n, group=w.group)
    cache = decode.KvCache.empty(pages, kv_heads, head_dim, page_size=64)
    q = d.kv_append(cache, k, v, table, past, q=q, rope=decode.rope_table(max_len, head_dim))
    o = d.kv_attend(q, cache, table, past + 1, max_len=max_len)

``python -m dense_fp16_gemm_hgemm_amd.decode_step`` runs them together.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch  # imported first so that both use one HIP runtime

__all__ = ["Decode", "DecodeError", "KvCache", "W4", "w4_pack", "w4_unpack", "w4_quantize",
           "rope_table", "LIB_PATH"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmi_decode.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built: run `python dense_fp16_gemm_hgemm_amd/build.py`")
_lib = ctypes.CDLL(LIB_PATH)
try:
    from . import _decode_calls as _calls  # needs torch and the library above
except ImportError as e:
    raise ImportError("_decode_calls.so is not built for this Python and torch: run "
                      "`python dense_fp16_gemm_hgemm_amd/build.py`") from e

MI_DECODE_OK = 0
MI_DECODE_ERR_INVALID_ARG = 1
MI_DECODE_ERR_UNSUPPORTED = 2
MI_DECODE_ERR_NO_DEVICE = 3
MI_DECODE_ERR_HIP = 4
MI_DECODE_CREATE_NO_DEVICE = 1

_p, _i32, _i64, _u32, _f32 = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                              ctypes.c_float)


class _Cache(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("pages", _i64),
                ("kv_heads", _i32), ("page_size", _i32), ("head_dim", _i32), ("code", _i32)]


class _Batch(ctypes.Structure):
    _fields_ = [("table", _p), ("lens", _p), ("cu", _p), ("table_stride", _i64),
                ("table_cols", _i32), ("batch", _i32), ("tokens", _i32), ("max_tokens", _i32)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", _p), ("token_stride", _i64), ("head_stride", _i64)]


def _sig(name, restype, *argtypes):
    f = getattr(_lib, name)
    f.restype = restype
    f.argtypes = list(argtypes)
    return f


_create = _sig("mi_decode_create", ctypes.c_int, ctypes.POINTER(_p), _u32)
_destroy = _sig("mi_decode_destroy", ctypes.c_int, _p)
_device = _sig("mi_decode_device", ctypes.c_int, _p)
_status_string = _sig("mi_decode_status_string", ctypes.c_char_p, ctypes.c_int)
_last_hip_error = _sig("mi_decode_last_hip_error", ctypes.c_int, _p)
_w4_linear = _sig("mi_decode_w4_linear", ctypes.c_int, _p, ctypes.c_int, _i64, _i64, _i64, _i64, _p,
                  _i64, _p, _p, _p, _p, _p, _i64, _p)
# structs are passed by address (ctypes.byref)
_kv_append = _sig("mi_decode_kv_append", ctypes.c_int, _p, _p, ctypes.c_int, _p, _p, _p, _p, _i64,
                  _i32, _i32, _i32, _p, _p, _p)
_kv_read = _sig("mi_decode_kv_read", ctypes.c_int, _p, _p, ctypes.c_int, _p, _p, _p, _p)
_kv_attend = _sig("mi_decode_kv_attend", ctypes.c_int, _p, _p, ctypes.c_int, _p, _i64, _i32, _p, _p,
                  _f32, _i32, _i32, _p)

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}
_byref = ctypes.byref


class DecodeError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        name = _status_string(status).decode()
        super().__init__(f"{what}: {name}" if what else name)


def _check(st, what):
    if st:
        raise DecodeError(st, what)


def _dtype(x, name):
    d = _DTYPES.get(x.dtype)
    if d is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {x.dtype}")
    return d


def _on(device, **tensors):
    for name, x in tensors.items():
        if x is not None and x.device != device:
            raise ValueError(f"{name} must be on {device}, got {x.device}")


def _raw(stream, device):
    """A stream's handle: of a torch stream on `device`, or an integer as it is."""
    if not isinstance(stream, torch.cuda.Stream):
        return stream
    if stream.device != device:
        raise ValueError(f"stream must be on {device}, got {stream.device}")
    return stream.cuda_stream


def _done(result, what):
    """A call's result, or DecodeError for the status that the library returned."""
    if type(result) is int:
        raise DecodeError(result, what)
    return result


# ------------------------------------------------------- 4-bit weights --

class W4(NamedTuple):
    """4-bit weights laid out for ``Decode.w4_linear``."""
    qweight: torch.Tensor            # int32 [ceil(N / 16), ceil(K / 128), 64, 4]
    scales: torch.Tensor             # [ceil(K / group), 16 ceil(N / 16)] fp16 or bf16
    zeros: Optional[torch.Tensor]    # uint8, the scales' shape; None: 8 everywhere
    n: int
    k: int
    group: int


def _by_group(x, rows, fill):
    """[N, groups] -> [groups, 16 ceil(N / 16)]."""
    out = torch.full((x.shape[1], rows), fill, dtype=x.dtype, device=x.device)
    out[:, :x.shape[0]] = x.t()
    return out


def w4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None,
            group: int = 128) -> W4:
    """Codes [N, K] (0..15), scales and zeros [N, ceil(K / group)] in the kernels' layout
    (``include/mi_decode.h``).  A weight is (code - zero) * scale; zeros None means 8."""
    if codes.dim() != 2:
        raise ValueError("codes must be [N, K]")
    if group < 32 or group % 32:
        raise ValueError(f"group must be a positive multiple of 32, got {group}")
    N, K = codes.shape
    groups = -(-K // group)
    if tuple(scales.shape) != (N, groups) or (zeros is not None and tuple(zeros.shape) != (N, groups)):
        raise ValueError(f"scales and zeros must have shape {(N, groups)}")
    _dtype(scales, "scales")
    for name, x in (("codes", codes), ("zeros", zeros)):
        if x is not None and x.numel() and not bool(((x >= 0) & (x <= 15)).all()):
            raise ValueError(f"{name} must be 0..15")
    nb, kb = -(-N // 16), -(-K // 128)
    full = torch.zeros((nb * 16, kb * 128), dtype=torch.int64, device=codes.device)
    full[:N, :K] = codes.to(torch.int64)
    e = torch.arange(8, device=codes.device)
    tiles = full.view(nb, 16, kb, 4, 4, 8) << (4 * (e // 2) + 16 * (e % 2))  # n-tile, r, k-tile, j, c, e
    words = tiles.sum(-1).permute(0, 2, 4, 1, 3).reshape(nb, kb, 64, 4)      # entry l = 16 c + r, word j
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32).contiguous()
    z = None if zeros is None else _by_group(zeros.to(torch.uint8), nb * 16, 8)
    return W4(words, _by_group(scales, nb * 16, 0), z, N, K, group)


def w4_unpack(w: W4) -> torch.Tensor:
    """The weights [N, K] that ``w`` stands for, in float32."""
    nb, kb = w.qweight.shape[:2]
    e = torch.arange(8, device=w.qweight.device, dtype=torch.int32)
    c = (w.qweight[..., None] >> (4 * (e // 2) + 16 * (e % 2))) & 15
    c = c.view(nb, kb, 4, 16, 4, 8).permute(0, 3, 1, 4, 2, 5).reshape(nb * 16, kb * 128)[:w.n, :w.k]
    g = torch.arange(w.k, device=c.device) // w.group
    z = 8 if w.zeros is None else w.zeros.int().t()[:w.n, g]
    return (c - z).float() * w.scales.float().t()[:w.n, g]


def w4_quantize(weight: torch.Tensor, group: int = 128, symmetric: bool = True) -> W4:
    """[N, K] fp16 or bf16 weights to 4 bits: for each row and `group` columns the scale
    that takes the largest magnitude to 7 (symmetric), or the range to 0..15."""
    _dtype(weight, "weight")
    N, K = weight.shape
    groups = -(-K // group)
    w = torch.zeros((N, groups * group), device=weight.device)
    w[:, :K] = weight.float()
    w = w.view(N, groups, group)
    if symmetric:
        s = (w.abs().amax(-1) / 7).to(weight.dtype)
        zeros = None
        z = torch.full_like(s, 8, dtype=torch.float32)
    else:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        s = ((hi - lo) / 15).to(weight.dtype)
        z = torch.where(s > 0, (-lo / s.float()).round().clamp(0, 15), torch.zeros_like(lo))
        zeros = z.to(torch.uint8)
    sf = s.float()[..., None]
    codes = torch.where(sf > 0, w / sf, torch.zeros_like(w)).round() + z[..., None]
    codes = codes.clamp(0, 15).to(torch.uint8).view(N, -1)[:, :K]
    return w4_pack(codes, s, zeros, group)


def rope_table(positions: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float32 [positions, rot_dim]: cosines, then sines, of position * base^(-2 i / rot_dim),
    with the angles in float64."""
    f = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([angle.cos(), angle.sin()], 1).float()


# --------------------------------------------------------------- cache --

class KvCache:
    """A paged cache: k and v [pages, kv_heads, page_size, head_dim] of int8 or float8_e4m3fn
    codes, k_scale and v_scale float32 [pages, kv_heads].  A value is its code times its
    page's and head's scale.  Calls go by the tensors' addresses, so a cache keeps the tensors
    that it was made of: their elements may change, the attributes may not."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "pages", "kv_heads", "page_size", "head_dim",
                 "device", "_struct", "_at", "_dev")

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("k and v must be alike: [pages, kv_heads, page_size, head_dim]")
        if k.dtype not in _CODES:
            raise TypeError(f"k and v must be torch.int8 or torch.float8_e4m3fn, got {k.dtype}")
        if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2]:
            raise ValueError("k_scale and v_scale must have shape [pages, kv_heads]")
        if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
            raise TypeError("k_scale and v_scale must be torch.float32")
        for name, x in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if not x.is_cuda:
                raise ValueError(f"{name} must be on the GPU")
            if not x.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        _on(k.device, v=v, k_scale=k_scale, v_scale=v_scale)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self.device = k.device
        self._struct = _Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                              self.pages, self.kv_heads, self.page_size, self.head_dim, _CODES[k.dtype])
        self._at, self._dev = ctypes.addressof(self._struct), k.device.index

    def __setattr__(self, name, value):
        if hasattr(self, "_dev"):
            raise AttributeError(f"a KvCache keeps the tensors that it was made of: {name} cannot be set")
        object.__setattr__(self, name, value)

    @classmethod
    def empty(cls, pages, kv_heads, head_dim, page_size=64, dtype=torch.int8, device="cuda"):
        """A cache with no tokens (scales zero, codes zero)."""
        codes = lambda: torch.zeros((pages, kv_heads, page_size, head_dim), dtype=torch.uint8,  # noqa: E731
                                    device=device).view(dtype)
        scale = lambda: torch.zeros((pages, kv_heads), dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(), codes(), scale(), scale())


# -------------------------------------------------------------- handle --

class Decode:
    """A library handle on the current device; its calls take tensors of that device."""

    def __init__(self, inspect_only: bool = False):
        h = _p()
        _check(_create(_byref(h), MI_DECODE_CREATE_NO_DEVICE if inspect_only else 0), "mi_decode_create")
        self.handle = h.value
        self.device = _device(h)  # -1: inspect_only

    def close(self):
        if getattr(self, "handle", None):
            _destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def last_hip_error(self):
        return _last_hip_error(self.handle)

    def w4_linear(self, x, qweight, scales, zeros=None, *, n, group=128, bias=None, out=None, stream=None):
        """x [M, K] times the 4-bit weights [n, K]: [M, n] in x's type, sums in float32."""
        return _done(_calls.w4_linear(self.handle, self.device, x, qweight, scales, zeros, n, group, bias, out,
                                      stream if stream is None else _raw(stream, x.device)),
                     "mi_decode_w4_linear")

    def kv_append(self, cache, k, v, table, past, cu_new=None, max_new=None, *, q=None, rope=None,
                  interleaved=False, q_out=None, stream=None):
        """Append k and v [tokens, kv_heads, head_dim] after the `past` tokens of each sequence;
        returns q [tokens, q_heads, head_dim] turned by its positions (None without q).
        Without cu_new one token a sequence; max_new: the most that a sequence has of them,
        which saves work where it is far below all tokens (the default with cu_new)."""
        return _done(_calls.kv_append(self.handle, self.device, cache._at, cache._dev, k, v, table, past, cu_new, max_new, q, rope,
                                      interleaved, q_out, stream if stream is None else _raw(stream, cache.device)), "mi_decode_kv_append")

    def kv_read(self, cache, table, start, cu=None, *, tokens=None, max_tokens=None, dtype=torch.float16,
                stream=None):
        """The values of the cached tokens at positions start[b] + i, i < cu[b + 1] - cu[b]:
        k and v [tokens, kv_heads, head_dim].  Without cu one token a sequence; with it
        `tokens` is needed, how many there are in all (cu lies on the device)."""
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be torch.float16 or torch.bfloat16, got {dtype}")
        if tokens is None:
            if cu is not None:
                raise ValueError("kv_read needs tokens, the number of tokens in all, where cu is given")
            tokens = start.shape[0]
        return _done(_calls.kv_read(self.handle, self.device, cache._at, cache._dev, table, start, cu, tokens, max_tokens,
                                    dtype == torch.bfloat16,
                                    stream if stream is None else _raw(stream, cache.device)), "mi_decode_kv_read")

    def kv_attend(self, q, cache, table, lens, cu_q=None, max_q=None, *, max_len=None, window=0, sinks=0,
                  scale=None, out=None, stream=None):
        """softmax(scale q k^T) v over the cache for q [tokens, q_heads, head_dim]: each
        sequence's queries are the last of its lens[b] tokens.  Without cu_q one query a
        sequence; max_q: the most that a sequence has, which saves work where it is far
        below all queries (the default with cu_q).  scale: head_dim ** -0.5.
        Sequences with one query each are faster in a call of their own than in one with
        prompt pieces of many, which is planned for the longest."""
        return _done(_calls.kv_attend(self.handle, self.device, cache._at, cache._dev, q, table, lens, cu_q, max_q, max_len,
                                      window, sinks, scale, out,
                                      stream if stream is None else _raw(stream, cache.device)), "mi_decode_kv_attend")
