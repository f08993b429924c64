"""Python face of lix_rotary: rotary positions of queries and keys, forward and gradient.

As in ops.py, the functions check and marshal arguments and call the C ABI
(include/lix_rotary.h); the arithmetic runs in the HIP kernel.
"""

import math
from typing import NamedTuple, Optional

import torch

from . import _lib
from .ops import _need, _stream

_DTYPES = {torch.bfloat16: _lib.LIX_BF16, torch.float16: _lib.LIX_FP16, torch.float32: _lib.LIX_FP32}
_LAYOUTS = {"half": _lib.LIX_ROTARY_HALF, "interleaved": _lib.LIX_ROTARY_INTERLEAVED}


class Rotary(NamedTuple):
    """How positions enter a head: dimensions [start, start + 2 * len(inv_freq)) are rotated in pairs
    (i, i + rot/2) ("half") or (2i, 2i+1) ("interleaved"), and multiplied by scale."""
    inv_freq: torch.Tensor
    layout: str = "half"
    start: int = 0
    scale: float = 1.0


def rotary_frequencies(rot, theta=10000.0, scaling=None, factor=1.0, original_max_position=None, beta_fast=32.0,
                       beta_slow=1.0, low_freq_factor=1.0, high_freq_factor=4.0, device=None):
    """Inverse frequencies (fp64 [rot/2], radians per position) and the scale of the rotated part.

    theta^(-2i/rot), changed for contexts `factor` times the original by `scaling`:
      None      as they are, scale 1
      "linear"  all divided by factor, scale 1
      "ntk"     theta multiplied by factor^(rot/(rot-2)), scale 1
      "yarn"    divided by factor where a pair turns fewer than beta_slow times over
                original_max_position, kept where it turns more than beta_fast times, a linear blend
                over the pairs between; scale 0.1 ln(factor) + 1
      "llama3"  divided by factor below low_freq_factor turns over original_max_position, kept above
                high_freq_factor turns, blended linearly in the turns between; scale 1
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and at least 2, got {rot}")
    if factor < 1.0:
        raise ValueError(f"factor must be at least 1, got {factor}")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("ntk scaling needs rot > 2")
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2.0 * i / rot)
    scale = 1.0
    if scaling in ("yarn", "llama3") and not original_max_position:
        raise ValueError(f"{scaling} scaling needs original_max_position")
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair_of(turns):          # the pair that turns so many times over the original context
            return rot * math.log(original_max_position / (turns * 2 * math.pi)) / (2 * math.log(theta))
        low, high = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rot - 1)
        keep = 1.0 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f / factor * (1.0 - keep) + f * keep
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling == "llama3":
        turns = original_max_position * f / (2 * math.pi)
        keep = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0, 1)
        f = f / factor * (1.0 - keep) + f * keep
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device) if device is not None else f, scale


def _rotate(x, positions, inv_freq, layout, start, scale, inverse, out=None):
    shape, strides = x.shape, x.stride()
    N0, N1, H, sh = (*shape[:3], strides[2]) if len(shape) == 4 else (*shape[:2], 1, 0)
    p0, p1 = positions.stride()
    ps = positions.shape
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    so = out.stride()
    st = _lib.load().lix_rotary(x.data_ptr(), strides[0], strides[1], sh, positions.data_ptr(),
                                p0 if ps[0] == N0 else 0, p1 if ps[1] == N1 else 0, inv_freq.data_ptr(), N0, N1, H,
                                shape[-1], 2 * inv_freq.shape[0], start, _LAYOUTS[layout], scale, inverse,
                                _DTYPES[x.dtype], out.data_ptr(), so[0], so[1], so[2] if len(shape) == 4 else 0,
                                _stream(x.device))
    _lib.check(st, "lix_rotary")
    return out


class RotaryFunction(torch.autograd.Function):
    """rotary's gradient: the inverse rotation of the upstream gradient (again differentiable)."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, layout, start, scale, inverse):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = (layout, start, scale, inverse)
        return _rotate(x, positions, inv_freq, layout, start, scale, inverse)

    @staticmethod
    def backward(ctx, dy):
        positions, inv_freq = ctx.saved_tensors
        layout, start, scale, inverse = ctx.how
        dy = dy if dy.stride(-1) == 1 else dy.contiguous()
        return RotaryFunction.apply(dy, positions, inv_freq, layout, start, scale, not inverse), *(None,) * 6


def rotary(x, positions, inv_freq, layout="half", start=0, scale=1.0, out=None):
    """lix_rotary: x [N0, N1, H, D] or [N0, N1, D] (bf16, fp16 or fp32; SBHD or BSHD, any strides with
    the last dimension contiguous), its dimensions [start, start + 2 * len(inv_freq)) rotated by
    positions * inv_freq and multiplied by scale.

    positions: int32, [N0, N1], [N0, 1], [1, N1] or [N0].  inv_freq: fp64 on x's device
    (rotary_frequencies).  out: a tensor like x to write to, x itself included; only where no gradient
    is recorded.  The result carries gradients to x.
    """
    if not isinstance(x, torch.Tensor) or x.dtype not in _DTYPES:
        raise TypeError("x must be a bfloat16, float16 or float32 tensor")
    if x.dim() not in (3, 4):
        raise ValueError(f"x must be [N0, N1, H, D] or [N0, N1, D], got shape {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if x.stride(-1) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    if not isinstance(positions, torch.Tensor) or positions.dtype != torch.int32:
        raise TypeError("positions must be an int32 tensor")
    if positions.dim() == 1:
        positions = positions[:, None]
    N0, N1 = x.shape[0], x.shape[1]
    if positions.dim() != 2 or positions.shape[0] not in (1, N0) or positions.shape[1] not in (1, N1):
        raise ValueError(f"positions must broadcast to [{N0}, {N1}], got shape {tuple(positions.shape)}")
    _need(inv_freq, "inv_freq", torch.float64, 1)
    if positions.get_device() != x.get_device() or inv_freq.get_device() != x.get_device():
        raise ValueError("x, positions and inv_freq must be on the same device")
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    if out is not None:
        if torch.is_grad_enabled() and x.requires_grad:
            raise ValueError("out cannot be given where a gradient is recorded")
        if out.dtype != x.dtype or out.shape != x.shape or out.device != x.device or out.stride(-1) != 1:
            raise ValueError("out must have x's shape, dtype and device and a contiguous last dimension")
        return _rotate(x, positions, inv_freq, layout, int(start), float(scale), False, out)
    if torch.is_grad_enabled() and x.requires_grad:
        return RotaryFunction.apply(x, positions, inv_freq, layout, int(start), float(scale), False)
    return _rotate(x, positions, inv_freq, layout, int(start), float(scale), False)


def rotate_indexer_inputs(index_q, index_k, compress_ratio, how: Rotary, q_positions: Optional[torch.Tensor] = None,
                          k_positions: Optional[torch.Tensor] = None):
    """index_q [S,B,H,D] and index_k [Skv,B,D] with their positions: query t at t and compressed key s at
    s * compress_ratio, the first token of its group, unless positions are given (as for rotary)."""
    if q_positions is None:
        q_positions = torch.arange(index_q.shape[0], dtype=torch.int32, device=index_q.device)
    if k_positions is None:
        k_positions = torch.arange(index_k.shape[0], dtype=torch.int32, device=index_k.device) * int(compress_ratio)
    return (rotary(index_q, q_positions, how.inv_freq, how.layout, how.start, how.scale),
            rotary(index_k, k_positions, how.inv_freq, how.layout, how.start, how.scale))
