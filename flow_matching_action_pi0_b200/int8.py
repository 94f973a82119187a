"""The 8-bit prefix operators on CUDA tensors: argument marshalling over the
pae_quantize_rows, pae_linear_i8 and pae_kv8_* calls of include/pae.h.

Every call runs on its tensors' device and on that device's current stream, as
PyTorch's own operators do, so allocation and use stay in order.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

import flow_matching_action_pi0_b200 as _fm

_CODES = {torch.float32: 0, torch.bfloat16: 1}  # PAE_FP32, PAE_BF16


def _need(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def _same_device(first: torch.Tensor, **tensors) -> None:
    _need(first.is_cuda, "tensors must be on a CUDA device")
    for name, t in tensors.items():
        if t is not None:
            _need(t.device == first.device, f"{name} is on {t.device}, not on {first.device}")


def _dtype_code(dtype: torch.dtype, what: str) -> int:
    _need(dtype in _CODES, f"{what} must be torch.float32 or torch.bfloat16, not {dtype}")
    return _CODES[dtype]


def _vector(t: torch.Tensor, n: int, dtype: torch.dtype, what: str) -> None:
    _need(t.dtype == dtype and t.shape == (n,) and t.is_contiguous(), f"{what} must be a contiguous {dtype} vector of {n}")


def quantize_rows(x: torch.Tensor, rms_eps: Optional[float] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [rows, width] (float32 or bfloat16, unit stride along width) ->
    (codes int8 [rows, width], scale float32 [rows]).  rms_eps: quantise the
    RMSNorm x / sqrt(mean(x^2) + rms_eps) of each row instead of x."""
    _need(x.dim() == 2 and x.shape[1] >= 1, "x must be [rows, width] with width >= 1")
    _need(x.stride(1) == 1 or x.shape[1] == 1, "x must be contiguous along width")
    code = _dtype_code(x.dtype, "x")
    _need(rms_eps is None or rms_eps > 0, "rms_eps must be positive")
    _same_device(x)
    rows, width = x.shape
    ldx = x.stride(0) if rows > 1 else width
    with torch.cuda.device(x.device):
        codes = torch.empty((rows, width), dtype=torch.int8, device=x.device)
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        _fm.pae_quantize_rows(x.data_ptr(), ldx, rows, width, code, rms_eps or 0.0, codes.data_ptr(), scale.data_ptr())
    return codes, scale


def linear_i8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(x [tokens, k] int8 times w [n, k] int8 transposed) * x_scale[token] *
    w_scale[channel] -> [tokens, n] in out_dtype (or into `out`)."""
    _need(x.dim() == 2 and w.dim() == 2 and x.shape[1] == w.shape[1], "x [tokens, k] and w [n, k] must share k")
    _need(x.dtype == torch.int8 and w.dtype == torch.int8, "x and w must be int8 codes")
    _need(x.is_contiguous() and w.is_contiguous(), "x and w must be contiguous")
    (tokens, k), n = x.shape, w.shape[0]
    _vector(x_scale, tokens, torch.float32, "x_scale")
    _vector(w_scale, n, torch.float32, "w_scale")
    _same_device(x, x_scale=x_scale, w=w, w_scale=w_scale, out=out)
    with torch.cuda.device(x.device):
        if out is None:
            out = torch.empty((tokens, n), dtype=out_dtype, device=x.device)
        _need(out.shape == (tokens, n) and (out.stride(1) == 1 or n == 1), "out must be [tokens, n], contiguous along n")
        code = _dtype_code(out.dtype, "out")
        _fm.pae_linear_i8(x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), tokens, n, k,
                          out.data_ptr(), out.stride(0) if tokens > 1 else n, code)
    return out


class Kv8Plan:
    """Sizes and workspace of KvCacheInt8.attend for one call shape.  Calls
    that may overlap (different streams, graphs replayed side by side) need a
    plan each."""

    def __init__(self, key, workspace: Optional[torch.Tensor]):
        self.key = key
        self.workspace = workspace


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

    # ------------------------------------------------------------ write, read
    def _seqs(self, cu_rows, start) -> Tuple[int, Optional[int], Optional[int]]:
        n_seq = 1 if cu_rows is None else int(cu_rows.shape[0]) - 1
        _same_device(self.k, cu_rows=cu_rows, start=start)
        if cu_rows is not None:
            _vector(cu_rows, n_seq + 1, torch.int32, "cu_rows")
        if start is not None:
            _vector(start, n_seq, torch.int32, "start")
        return n_seq, None if cu_rows is None else cu_rows.data_ptr(), None if start is None else start.data_ptr()

    def _rows(self, t: torch.Tensor, what: str):
        _need(t.dim() == 3 and t.shape[1:] == (self.shape[1], self.shape[3]) and t.stride(2) == 1,
              f"{what} must be [rows, {self.shape[1]}, {self.shape[3]}], contiguous along the last dimension")
        return [t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0]

    def write(self, k: torch.Tensor, v: torch.Tensor, cu_rows: Optional[torch.Tensor] = None,
              start: Optional[torch.Tensor] = None) -> None:
        """Quantise rows k, v [n_rows, n_kv_heads, head_dim] into the cache:
        sequence b (slot b) is rows [cu_rows[b], cu_rows[b + 1]), placed from
        position start[b] on (int32 tensors; None: one sequence, position 0).
        Rows outside every sequence or past the capacity are dropped."""
        _need(k.shape == v.shape and k.dtype == v.dtype, "k and v must have the same shape and type")
        code = _dtype_code(k.dtype, "k and v")
        ks, vs = self._rows(k, "k"), self._rows(v, "v")
        n_seq, cu, at = self._seqs(cu_rows, start)
        _same_device(self.k, k=k, v=v)
        with torch.cuda.device(self.device):
            _fm.pae_kv8_write(self._c, k.data_ptr(), v.data_ptr(), ks, vs, cu, at, n_seq, k.shape[0], code)

    def read(self, cu_rows: Optional[torch.Tensor], start: Optional[torch.Tensor], n_rows: int,
             dtype: torch.dtype = torch.bfloat16) -> Tuple[torch.Tensor, torch.Tensor]:
        """The rows that write places for the same arguments, as the values
        their codes stand for; rows without a place are zeros."""
        code = _dtype_code(dtype, "dtype")
        n_seq, cu, at = self._seqs(cu_rows, start)
        with torch.cuda.device(self.device):
            k = torch.empty((n_rows, self.shape[1], self.shape[3]), dtype=dtype, device=self.device)
            v = torch.empty_like(k)
            _fm.pae_kv8_read(self._c, k.data_ptr(), v.data_ptr(), None, None, cu, at, n_seq, n_rows, code)
        return k, v

    # -------------------------------------------------------------- attention
    def plan(self, n_seq: int, n_q: int, n_q_heads: int, fresh: int = 0) -> Kv8Plan:
        """Allocate the workspace of attend calls of this shape."""
        need = _fm.pae_kv8_workspace(self._c, n_seq, n_q, n_q_heads, fresh)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        return Kv8Plan((n_seq, n_q, n_q_heads, fresh), ws)

    def attend(self, q: torch.Tensor, lens: torch.Tensor, causal: bool = False, k_new: Optional[torch.Tensor] = None,
               v_new: Optional[torch.Tensor] = None, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               plan: Optional[Kv8Plan] = None) -> torch.Tensor:
        """q [n_seq, n_q, n_q_heads, head_dim] bfloat16 over cached positions
        [0, lens[b]) of slot b (lens int32), and fresh k_new, v_new [n_seq,
        n_new, n_kv_heads, head_dim] that every query sees; causal: query i
        sees positions [0, lens[b] - n_q + i].  Queries that see no key give
        zeros.  Returns [n_seq, n_q, n_q_heads, head_dim] bfloat16."""
        d, hk = self.shape[3], self.shape[1]

        def rows(t, heads, what):
            _need(t.dtype == torch.bfloat16 and t.dim() == 4 and t.shape[2:] == (heads, d) and t.stride(3) == 1,
                  f"{what} must be bfloat16 [n_seq, n, {heads}, {d}], contiguous along the last dimension")
            return tuple(s if n > 1 else 0 for s, n in zip(t.stride()[:3], t.shape[:3]))

        _need(q.dim() == 4, "q must be [n_seq, n_q, n_q_heads, head_dim]")
        n_seq, n_q, hq = q.shape[:3]
        _need((k_new is None) == (v_new is None), "k_new and v_new go together")
        _same_device(self.k, q=q, lens=lens, k_new=k_new, v_new=v_new, out=out)
        _vector(lens, n_seq, torch.int32, "lens")
        qs = _fm.pae_kv8_query(lens=lens.data_ptr(), q=q.data_ptr(), n_seq=n_seq, n_q=n_q, n_q_heads=hq,
                               causal=int(causal), scale=0.0 if scale is None else scale)
        _need(scale is None or scale != 0.0, "scale must not be 0")
        qs.q_strides = rows(q, hq, "q")
        if k_new is not None:
            _need(k_new.shape == v_new.shape and k_new.shape[0] == n_seq, "k_new and v_new must be [n_seq, n_new, ...]")
            qs.n_new, qs.k_new, qs.v_new = k_new.shape[1], k_new.data_ptr(), v_new.data_ptr()
            qs.k_new_strides, qs.v_new_strides = rows(k_new, hk, "k_new"), rows(v_new, hk, "v_new")
        with torch.cuda.device(self.device):
            if out is None:
                out = torch.empty((n_seq, n_q, hq, d), dtype=torch.bfloat16, device=self.device)
            _need(out.shape == q.shape, "out must have the shape of q")
            qs.out, qs.out_strides = out.data_ptr(), rows(out, hq, "out")
            if plan is None:
                plan = self.plan(n_seq, n_q, hq, qs.n_new)
            _need(plan.key == (n_seq, n_q, hq, qs.n_new), f"the plan is for {plan.key}")
            ws = plan.workspace
            _need(ws is None or ws.device == self.device, "the plan's workspace is on another device")
            _fm.pae_kv8_attention(self._c, qs, ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0)
        return out


__all__ = ["quantize_rows", "linear_i8", "KvCacheInt8", "Kv8Plan"]
