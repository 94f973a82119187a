"""The 8-bit prefix operators on CUDA tensors: argument marshalling over the
pae_quantize_rows, pae_linear_i8 and pae_kv8_* calls of include/pae.h.

Every call runs on its tensors' device and on that device's current stream, as
PyTorch's own operators do, so allocation and use stay in order.
"""
from __future__ import annotations

import struct
from typing import Optional, Tuple

import torch

import flow_matching_action_pi0_b200 as _fm

_CODES = {torch.float32: 0, torch.bfloat16: 1}  # PAE_FP32, PAE_BF16

# A small call costs its launch on the device and this module on the host, so
# arguments go to the library as packed bytes (pae_kv8_query, stride pairs) and
# messages are put together only when a check fails.
_QUERY = struct.Struct("5P12q5if")  # pae_kv8_query
_PAIR = struct.Struct("2q").pack
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_int8, _int32, _float32, _bfloat16 = torch.int8, torch.int32, torch.float32, torch.bfloat16


class _Library:
    """libpae's functions with c_void_p (p), c_int (i), c_longlong (q),
    c_size_t (z) or c_float (f) arguments (bytes pass as pointers), looked up
    on first use."""

    _types = {"pae_quantize_rows": "pqiiifppp", "pae_linear_i8": "ppppiiipqip", "pae_kv8_write": "pppppppiiip",
              "pae_kv8_read": "pppppppiiip", "pae_kv8_attention": "pppzp"}

    def __getattr__(self, name):
        import ctypes
        kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int, "q": ctypes.c_longlong, "z": ctypes.c_size_t, "f": ctypes.c_float}
        f = _fm.lib()[name]  # an object of its own: the package's prototype stays
        f.restype = ctypes.c_int
        f.argtypes = [kinds[c] for c in self._types[name]]
        setattr(self, name, f)
        return f


_lib = _Library()


def _call(device: int, f, *args) -> None:
    """f(*args, stream) on the device's current stream, with the device current."""
    if device == _current_device():
        status = f(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _raw_stream(device))
    if status:
        _fm._check(status)


def _check_device(first: torch.Tensor, *others) -> int:
    """Ordinal of the CUDA device that all tensors (None: absent) are on."""
    device = first.get_device()
    if device < 0:
        raise ValueError("tensors must be on a CUDA device")
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"tensors are on {first.device} and {t.device}: one device is needed")
    return device


def _dtype_code(dtype: torch.dtype, what: str) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"{what} must be torch.float32 or torch.bfloat16, not {dtype}")
    return code


_MOST = 1 << 30  # of a size: the library takes 32-bit integers


def _check_vector(t: torch.Tensor, n: int, dtype: torch.dtype, what: str) -> None:
    if t.dtype != dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n}")


def quantize_rows(x: torch.Tensor, rms_eps: Optional[float] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [rows, width] (float32 or bfloat16, unit stride along width) ->
    (codes int8 [rows, width], scale float32 [rows]).  rms_eps: quantise the
    RMSNorm x / sqrt(mean(x^2) + rms_eps) of each row instead of x."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, width]")
    rows, width = x.shape
    if width < 1:
        raise ValueError("x must have width >= 1")
    if rows > _MOST or width > _MOST:
        raise ValueError("x must have at most 2^30 rows and columns")
    ldx, unit = x.stride()
    if unit != 1 and width > 1:
        raise ValueError("x must be contiguous along width")
    code = _dtype_code(x.dtype, "x")
    if rms_eps is not None and not rms_eps > 1e-45:  # (the library takes a float, 0 stands for no norm)
        raise ValueError("rms_eps must be positive")
    device = _check_device(x)
    codes = x.new_empty((rows, width), dtype=_int8)
    scale = x.new_empty((rows,), dtype=_float32)
    _call(device, _lib.pae_quantize_rows, x.data_ptr(), ldx if rows > 1 else width, rows, width,
          code, rms_eps or 0.0, codes.data_ptr(), scale.data_ptr())
    return codes, scale


def linear_i8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(x [tokens, k] int8 times w [n, k] int8 transposed) * x_scale[token] *
    w_scale[channel] -> [tokens, n] in out_dtype (or into `out`)."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [tokens, k] and w [n, k]")
    tokens, k = x.shape
    n, kw = w.shape
    if k != kw:
        raise ValueError("x [tokens, k] and w [n, k] must share k")
    if tokens > _MOST or n > _MOST or k > _MOST:
        raise ValueError("tokens, n and k must be at most 2^30")
    if x.dtype != _int8 or w.dtype != _int8:
        raise ValueError("x and w must be int8 codes")
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    _check_vector(x_scale, tokens, _float32, "x_scale")
    _check_vector(w_scale, n, _float32, "w_scale")
    device = _check_device(x, x_scale, w, w_scale, out)
    if out is None:
        out = x.new_empty((tokens, n), dtype=out_dtype)
    elif out.shape != (tokens, n) or (out.stride(1) != 1 and n > 1):
        raise ValueError("out must be [tokens, n], contiguous along n")
    code = _dtype_code(out.dtype, "out")
    _call(device, _lib.pae_linear_i8, x.data_ptr(), x_scale.data_ptr(), w.data_ptr(),
          w_scale.data_ptr(), tokens, n, k, out.data_ptr(), out.stride(0) if tokens > 1 else n, code)
    return out


class Kv8Plan:
    """Sizes and workspace of KvCacheInt8.attend for one call shape.  Calls
    that may overlap (different streams, graphs replayed side by side) need a
    plan each."""

    def __init__(self, key, workspace: Optional[torch.Tensor], device: int):
        self.key = key
        self.workspace = workspace
        self.bytes = 0 if workspace is None else workspace.numel()
        self.device = device


class KvCacheInt8:
    """An int8 K/V cache: codes k, v [n_slots, n_kv_heads, capacity, head_dim]
    and scales k_scale, v_scale [n_slots, n_kv_heads, capacity]."""

    def __init__(self, n_slots: int, n_kv_heads: int, capacity: int, head_dim: int, device="cuda"):
        shape = (n_slots, n_kv_heads, capacity, head_dim)
        self.k = torch.zeros(shape, dtype=torch.int8, device=device)
        self.v = torch.zeros(shape, dtype=torch.int8, device=device)
        self.k_scale = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self.v_scale = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self.shape = shape
        self.device = self.k.device
        self._c = _fm.pae_kv8(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                              n_slots, n_kv_heads, capacity, head_dim)
        self._p = bytes(self._c)

    # ------------------------------------------------------------ write, read
    def _seqs(self, cu_rows, start) -> Tuple[int, Optional[int], Optional[int]]:
        n_seq = 1
        cu = at = None
        if cu_rows is not None:
            n_seq = cu_rows.shape[0] - 1
            if n_seq > self.shape[0]:
                raise ValueError(f"cu_rows names {n_seq} sequences, the cache has {self.shape[0]} slots")
            _check_vector(cu_rows, n_seq + 1, _int32, "cu_rows")
            cu = cu_rows.data_ptr()
        if start is not None:
            _check_vector(start, n_seq, _int32, "start")
            at = start.data_ptr()
        return n_seq, cu, at

    def _strides(self, t: torch.Tensor, what: str) -> bytes:
        rows, heads, d = t.shape if t.dim() == 3 else (0, -1, 0)
        if heads != self.shape[1] or d != self.shape[3] or t.stride(2) != 1:
            raise ValueError(f"{what} must be [rows, {self.shape[1]}, {self.shape[3]}], contiguous along the last dimension")
        return _PAIR(t.stride(0) if rows > 1 else 0, t.stride(1) if heads > 1 else 0)

    def write(self, k: torch.Tensor, v: torch.Tensor, cu_rows: Optional[torch.Tensor] = None,
              start: Optional[torch.Tensor] = None) -> None:
        """Quantise rows k, v [n_rows, n_kv_heads, head_dim] into the cache:
        sequence b (slot b) is rows [cu_rows[b], cu_rows[b + 1]), placed from
        position start[b] on (int32 tensors; None: one sequence, position 0).
        Rows outside every sequence or past the capacity are dropped."""
        if k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must have the same shape and type")
        if k.dim() != 3 or k.shape[0] > _MOST:
            raise ValueError("k and v must be [rows, n_kv_heads, head_dim] with at most 2^30 rows")
        code = _dtype_code(k.dtype, "k and v")
        ks, vs = self._strides(k, "k"), self._strides(v, "v")
        n_seq, cu, at = self._seqs(cu_rows, start)
        device = _check_device(self.k, k, v, cu_rows, start)
        _call(device, _lib.pae_kv8_write, self._p, k.data_ptr(), v.data_ptr(), ks, vs, cu, at,
              n_seq, k.shape[0], code)

    def read(self, cu_rows: Optional[torch.Tensor], start: Optional[torch.Tensor], n_rows: int,
             dtype: torch.dtype = torch.bfloat16) -> Tuple[torch.Tensor, torch.Tensor]:
        """The rows that write places for the same arguments, as the values
        their codes stand for; rows without a place are zeros."""
        if not 0 <= n_rows <= _MOST:
            raise ValueError("n_rows must be in [0, 2^30]")
        code = _dtype_code(dtype, "dtype")
        n_seq, cu, at = self._seqs(cu_rows, start)
        device = _check_device(self.k, cu_rows, start)
        shape = (n_rows, self.shape[1], self.shape[3])
        k, v = self.k.new_empty(shape, dtype=dtype), self.k.new_empty(shape, dtype=dtype)
        _call(device, _lib.pae_kv8_read, self._p, k.data_ptr(), v.data_ptr(), None, None, cu, at,
              n_seq, n_rows, code)
        return k, v

    # -------------------------------------------------------------- attention
    def plan(self, n_seq: int, n_q: int, n_q_heads: int, fresh: int = 0) -> Kv8Plan:
        """Allocate the workspace of attend calls of this shape."""
        need = _fm.pae_kv8_workspace(self._c, n_seq, n_q, n_q_heads, fresh)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        return Kv8Plan((n_seq, n_q, n_q_heads, fresh), ws, self.k.get_device())

    def _rows(self, t: torch.Tensor, heads: int, what: str) -> Tuple[int, int, int]:
        if t.dim() != 4 or t.dtype != _bfloat16 or t.shape[2] != heads or t.shape[3] != self.shape[3] or t.stride(3) != 1:
            raise ValueError(f"{what} must be bfloat16 [n_seq, n, {heads}, {self.shape[3]}], contiguous along the last dimension")
        n0, n1, n2, _ = t.shape
        s0, s1, s2, _ = t.stride()
        return s0 if n0 > 1 else 0, s1 if n1 > 1 else 0, s2 if n2 > 1 else 0

    def attend(self, q: torch.Tensor, lens: torch.Tensor, causal: bool = False, k_new: Optional[torch.Tensor] = None,
               v_new: Optional[torch.Tensor] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               plan: Optional[Kv8Plan] = None) -> torch.Tensor:
        """q [n_seq, n_q, n_q_heads, head_dim] bfloat16 over cached positions
        [0, lens[b]) of slot b (lens int32), and fresh k_new, v_new [n_seq,
        n_new, n_kv_heads, head_dim] that every query sees; causal: query i
        sees positions [0, lens[b] - n_q + i].  Queries that see no key give
        zeros.  Returns [n_seq, n_q, n_q_heads, head_dim] bfloat16."""
        if q.dim() != 4:
            raise ValueError("q must be [n_seq, n_q, n_q_heads, head_dim]")
        n_seq, n_q, hq, _ = q.shape
        if scale is not None and scale == 0.0:
            raise ValueError("scale must not be 0")
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new go together")
        device = _check_device(self.k, q, lens, k_new, v_new, out)
        _check_vector(lens, n_seq, _int32, "lens")
        qs = self._rows(q, hq, "q")
        n_new, kp, vp, ks, vs = 0, 0, 0, (0, 0, 0), (0, 0, 0)
        if k_new is not None:
            hk = self.shape[1]
            if k_new.shape != v_new.shape or k_new.shape[0] != n_seq:
                raise ValueError("k_new and v_new must be [n_seq, n_new, n_kv_heads, head_dim]")
            n_new, kp, vp = k_new.shape[1], k_new.data_ptr(), v_new.data_ptr()
            if n_new > _MOST:
                raise ValueError("k_new and v_new must have at most 2^30 rows")
            ks, vs = self._rows(k_new, hk, "k_new"), self._rows(v_new, hk, "v_new")
        if out is None:
            out = q.new_empty(q.shape)
        elif out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        os = self._rows(out, hq, "out")
        key = (n_seq, n_q, hq, n_new)
        if plan is None:
            plan = self.plan(*key)
        elif plan.key != key or plan.device != device:
            raise ValueError(f"the plan is for {plan.key} on device {plan.device}, the call is {key} on {device}")
        query = _QUERY.pack(lens.data_ptr(), q.data_ptr(), out.data_ptr(), kp, vp, *qs, *os, *ks, *vs, n_seq, n_q, hq,
                            n_new, 1 if causal else 0, scale or 0.0)
        ws = plan.workspace
        _call(device, _lib.pae_kv8_attention, self._p, query, None if ws is None else ws.data_ptr(),
              plan.bytes)
        return out


__all__ = ["quantize_rows", "linear_i8", "KvCacheInt8", "Kv8Plan"]
