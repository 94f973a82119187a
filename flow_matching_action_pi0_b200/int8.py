"""The 8-bit prefix operators on CUDA tensors: the pae_quantize_rows,
pae_linear_i8 and pae_kv8_* calls of include/pae.h.

Every call runs on its tensors' device and on that device's current stream, as
PyTorch's own operators do, so allocation and use stay in order.  Arguments are
checked and results allocated in csrc/int8_tensors.cpp: on small inputs a call
costs its host side, and in Python that was more than the kernels' time.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

import flow_matching_action_pi0_b200 as _fm
from flow_matching_action_pi0_b200 import build as _build


def _bind():
    try:
        from flow_matching_action_pi0_b200 import _int8_tensors as ops
    except ImportError as e:
        raise RuntimeError(f"{_build.TENSORS} is not built, or not against this PyTorch ({e}); "
                           "run `python -m flow_matching_action_pi0_b200.build`") from e
    lib = _fm.lib()
    names = ("pae_quantize_rows", "pae_linear_i8", "pae_kv8_write", "pae_kv8_read", "pae_kv8_attention")
    ops.bind(tuple(ctypes.cast(lib[name], ctypes.c_void_p).value for name in names), _fm._check)
    return ops


_ops = _bind()


def quantize_rows(x: torch.Tensor, rms_eps: Optional[float] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x [rows, width] (float32 or bfloat16, unit stride along width) ->
    (codes int8 [rows, width], scale float32 [rows]).  rms_eps: quantise the
    RMSNorm x / sqrt(mean(x^2) + rms_eps) of each row instead of x."""
    return _ops.quantize_rows(x, rms_eps)


def linear_i8(x: torch.Tensor, x_scale: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
              out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(x [tokens, k] int8 times w [n, k] int8 transposed) * x_scale[token] *
    w_scale[channel] -> [tokens, n] in out_dtype (or into `out`)."""
    return _ops.linear_i8(x, x_scale, w, w_scale, out_dtype, out)


class Kv8Plan:
    """Sizes and workspace of KvCacheInt8.attend for one call shape.  Calls
    that may overlap (different streams, graphs replayed side by side) need a
    plan each."""

    def __init__(self, key: Tuple[int, int, int, int], workspace: Optional[torch.Tensor]):
        self.key = key  # n_seq, n_q, n_q_heads, fresh
        self.workspace = workspace
        self._args = (*key, workspace)


class KvCacheInt8:
    """An int8 K/V cache: codes k, v [n_slots, n_kv_heads, capacity, head_dim]
    and scales k_scale, v_scale [n_slots, n_kv_heads, capacity].  The tensors may
    be filled in place; they stay the cache's own."""

    # the calls take the addresses that were found once: another tensor in the
    # place of one of these would leave them in freed memory
    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    k_scale = property(lambda self: self._k_scale)
    v_scale = property(lambda self: self._v_scale)

    def __init__(self, n_slots: int, n_kv_heads: int, capacity: int, head_dim: int, device="cuda"):
        shape = (n_slots, n_kv_heads, capacity, head_dim)
        self._k = torch.zeros(shape, dtype=torch.int8, device=device)
        self._v = torch.zeros(shape, dtype=torch.int8, device=device)
        self._k_scale = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self._v_scale = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self.shape = shape
        self.device = self.k.device
        self._c = _fm.pae_kv8(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                              n_slots, n_kv_heads, capacity, head_dim)
        self._p, self._device = bytes(self._c), self.k.get_device()

    def write(self, k: torch.Tensor, v: torch.Tensor, cu_rows: Optional[torch.Tensor] = None,
              start: Optional[torch.Tensor] = None) -> None:
        """Quantise rows k, v [n_rows, n_kv_heads, head_dim] into the cache:
        sequence b (slot b) is rows [cu_rows[b], cu_rows[b + 1]), placed from
        position start[b] on (int32 tensors; None: one sequence, position 0).
        Rows outside every sequence or past the capacity are dropped."""
        _ops.kv8_write(self._p, self._device, k, v, cu_rows, start)

    def read(self, cu_rows: Optional[torch.Tensor], start: Optional[torch.Tensor], n_rows: int,
             dtype: torch.dtype = torch.bfloat16) -> Tuple[torch.Tensor, torch.Tensor]:
        """The rows that write places for the same arguments, as the values
        their codes stand for; rows without a place are zeros."""
        return _ops.kv8_read(self._p, self._device, cu_rows, start, n_rows, dtype)

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
        if plan is None:
            if q.dim() != 4:
                raise ValueError("q must be [n_seq, n_q, n_q_heads, head_dim]")
            plan = self.plan(*q.shape[:3], 0 if k_new is None else k_new.shape[1])
        return _ops.kv8_attend(self._p, self._device, q, lens, causal, k_new, v_new, scale, out, plan._args)


__all__ = ["quantize_rows", "linear_i8", "KvCacheInt8", "Kv8Plan"]
