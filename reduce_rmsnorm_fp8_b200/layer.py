"""The calls of a layer around its attention, on torch tensors: the FP8
products with their epilogue, the per-head norm and rotation, and the paged
FP8 cache of keys and values.  The checks and the marshalling are in C++
(csrc/rrf_torch.cpp, built in-tree as _rrf_torch.so): these calls are short,
and a call's own time counts.

The calls have no gradient.  Where autograd records (outside torch.no_grad()),
a tensor that requires grad is refused.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import RRF_ACT_GELU, RRF_ACT_GELU_TANH, RRF_ACT_NONE, RRF_ACT_RELU, RRF_ACT_SILU

try:
    from . import _rrf_torch as _call
except ImportError as e:
    raise ImportError(f"_rrf_torch.so is missing or was built for another torch ({e}): build it "
                      "with `python -m reduce_rmsnorm_fp8_b200.build`") from e

_inf = float("inf")


def _bind(lib):
    """Let the binding call the functions of ``lib`` (the loaded librrf.so)."""
    _call.bind(_lib._raise_on, *[ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.rrf_scaled_mm_fp8_act, lib.rrf_scaled_mm_mxfp8_act, lib.rrf_qk_norm_rope,
        lib.rrf_kv_cache_write_fp8, lib.rrf_qk_norm_rope_kv_cache_fp8,
        lib.rrf_kv_cache_read_fp8)])


_bind(_lib.lib)


# ------------------------------------------- products with their epilogue ---

_ACTIVATIONS = {None: RRF_ACT_NONE, "none": RRF_ACT_NONE, "relu": RRF_ACT_RELU,
                "gelu": RRF_ACT_GELU, "gelu_tanh": RRF_ACT_GELU_TANH, "silu": RRF_ACT_SILU}


def _activation(name):
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(filter(None, _ACTIVATIONS))}")
    return _ACTIVATIONS[name]


def rrf_scaled_mm_fp8_act(a, a_scale, b, b_scale, bias=None, activation="none", residual=None,
                          out=None):
    """out = RN_bf16(act((a @ b^T) * a_scale * b_scale + bias) + residual):
    rrf_scaled_mm_fp8 with the rest of a projection in its epilogue, rounded
    once.  activation: "none", "relu", "gelu" (erf), "gelu_tanh" or "silu";
    residual: bf16 [M, N] or None; pass it as out too for an update in place.
    Returns out, bf16 [M, N]."""
    return _call.scaled_mm_fp8_act(a, a_scale, b, b_scale, bias, _activation(activation),
                                   residual, out)


def rrf_scaled_mm_mxfp8_act(a, sa, b, sb, bias=None, activation="none", residual=None, out=None):
    """rrf_scaled_mm_mxfp8 with the epilogue of rrf_scaled_mm_fp8_act: sa and
    sb are E8M0 scale codes in the blocked order.  Returns out, bf16 [M, N]."""
    return _call.scaled_mm_mxfp8_act(a, sa, b, sb, bias, _activation(activation), residual, out)


# ---------------------------------------- heads, rotation and the FP8 cache ---

class RrfKvCache(ctypes.Structure):
    """The C struct rrf_kv_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64),
                ("code_strides", ctypes.c_int64 * 3), ("scale_strides", ctypes.c_int64 * 3)]


def rope_table(max_positions: int, rot_dim: int, theta: float = 10000.0, device="cuda"):
    """The cos_sin table of the plain rotation: angle p * theta^(-2i / rot_dim)
    for position p and pair i, taken in float64 and rounded to float32 once;
    [max_positions, rot_dim], cosines first.  Prepared once, not a step of a
    call."""
    if rot_dim <= 0 or rot_dim % 16:
        raise ValueError("rot_dim must be a positive multiple of 16")
    i = torch.arange(rot_dim // 2, device=device, dtype=torch.float64)
    p = torch.arange(max_positions, device=device, dtype=torch.float64)
    angle = p[:, None] * torch.pow(float(theta), -2.0 * i / rot_dim)
    return torch.cat((angle.cos(), angle.sin()), dim=1).float()


def rrf_qk_norm_rope(q, k, q_gamma, k_gamma, eps, weight_offset, cos_sin, positions,
                     interleaved=False, q_out=None, k_out=None):
    """RMS norm of every head with gamma + weight_offset, then the rotation of
    its first cos_sin.shape[1] values (cos_sin None: the norm alone).  q, k:
    bf16 [tokens, heads, head_dim] with any token and head strides (parts of a
    projection's output); cos_sin: float32 [max_positions, rot_dim]
    (rope_table); positions: int64 [tokens].  q_out, k_out: new contiguous
    tensors if None; pass q and k for an update in place.  Returns (q_out,
    k_out)."""
    return _call.qk_norm_rope(q, k, q_gamma, k_gamma, eps, weight_offset, cos_sin, positions,
                              interleaved, q_out, k_out)


def rrf_kv_cache_write_fp8(k, v, slots, k_cache, k_scales, v_cache, v_scales, scale_ub=_inf):
    """Quantise keys and values, bf16 [tokens, kv_heads, head_dim], into slots
    of a paged cache: one scale per token and head.  slots: int64 [tokens]
    (page * page_size + place; negative: a padding token, not stored; the
    others must differ).  k_cache, v_cache: float8_e4m3fn [pages, page_size,
    kv_heads, head_dim]; k_scales, v_scales: float32 [pages, page_size,
    kv_heads]; any strides that keep a head's codes contiguous, the same for
    keys and values.  Updates the cache."""
    _call.kv_cache_write_fp8(k, v, slots, k_cache, k_scales, v_cache, v_scales, scale_ub)


def rrf_qk_norm_rope_kv_cache_fp8(q, k, v, q_gamma, k_gamma, eps, weight_offset, cos_sin,
                                  positions, slots, k_cache, k_scales, v_cache, v_scales,
                                  scale_ub=_inf, interleaved=False, q_out=None):
    """rrf_qk_norm_rope and rrf_kv_cache_write_fp8 in one pass: q normalised,
    rotated and written to q_out (new if None; q for an update in place), k
    normalised, rotated and quantised into its slots, v quantised into its
    slots.  Returns q_out."""
    return _call.qk_norm_rope_kv_cache_fp8(q, k, v, q_gamma, k_gamma, eps, weight_offset, cos_sin,
                                           positions, interleaved, slots, k_cache, k_scales,
                                           v_cache, v_scales, scale_ub, q_out)


def rrf_kv_cache_read_fp8(k_cache, k_scales, v_cache, v_scales, block_table, seq_starts, k_out,
                          v_out):
    """Read a batch's keys and values back as bf16: row seq_starts[s] + t of
    k_out and v_out (contiguous bf16 [rows, kv_heads, head_dim]) gets place
    t % page_size of page block_table[s][t // page_size].  block_table: int32
    [sequences, pages per sequence]; seq_starts: int32 [sequences + 1].  Rows
    of no sequence stay as they are.  Returns (k_out, v_out)."""
    return _call.kv_cache_read_fp8(k_cache, k_scales, v_cache, v_scales, block_table, seq_starts,
                                   k_out, v_out)
