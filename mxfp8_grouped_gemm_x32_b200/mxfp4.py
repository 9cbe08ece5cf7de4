"""MXFP4 quantisation of tensors (moe_mlp_quantize_mxfp4 and back): E2M1 codes,
two per byte, with one E8M0 scale per 32 values along the last axis, the
scales in the library's blocked layout.  The layer's own weights go through
GroupedMLP.quantize_weights_mxfp4; these calls are for any other tensor and for
reading MXFP4 tensors back."""
from __future__ import annotations

import torch

from . import lib
from .layer import _DTYPES, _raw_stream, check_tensor, on_device


def _scale_bytes(groups: int, rows: int, K: int) -> int:
    """lib.moe_mx_scale_bytes without the call into the library."""
    return groups * -(-rows // 128) * -(-K // 128) * 512


def _extent(shape):
    """(groups, rows, K) of a tensor's shape: all leading axes but the last
    two are groups."""
    if len(shape) < 1:
        raise ValueError("expected at least one axis")
    groups = 1
    for d in shape[:-2]:
        groups *= d
    return groups, shape[-2] if len(shape) > 1 else 1, shape[-1]


def quantize(x: torch.Tensor):
    """x fp32 or bf16 [..., rows, K], K a multiple of 32 -> (codes uint8
    [..., rows, K/2], the even element in the low half of a byte; scales uint8,
    blocked, of lib.moe_mx_scale_bytes(groups, rows, K) bytes, groups the
    product of the axes before the last two).  Every group's scales fill whole
    tiles of 128 rows, so [N, 1, K] takes 128 rows of scales per row, eight
    times its codes' bytes: flatten such a tensor to [N, K] first."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"x: expected a torch.Tensor, got {type(x).__name__}")
    dt = _DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x: expected float32 or bfloat16, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"x: expected a tensor on a CUDA device, got {x.device}")
    groups, rows, K = _extent(x.shape)
    if K % 32:
        raise ValueError(f"x: the last axis must be a multiple of 32, got {K}")
    if not x.is_contiguous():
        raise ValueError("x: must be contiguous")
    with on_device(x.device):
        codes = torch.empty(*x.shape[:-1], K // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(_scale_bytes(groups, rows, K), dtype=torch.uint8, device=x.device)
        lib.moe_mlp_quantize_mxfp4(x.data_ptr(), dt, groups, rows, K, codes.data_ptr(), K // 2,
                                   scales.data_ptr(), _raw_stream(x.device.index))
    return codes, scales


def dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The values that quantize()'s codes [..., rows, K/2] and blocked scales
    stand for, fp32 or bf16 [..., rows, K]."""
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"dtype: expected torch.float32 or torch.bfloat16, got {dtype}")
    if not isinstance(codes, torch.Tensor):
        raise TypeError(f"codes: expected a torch.Tensor, got {type(codes).__name__}")
    if not codes.is_cuda:
        raise ValueError(f"codes: expected a tensor on a CUDA device, got {codes.device}")
    groups, rows, half = _extent(codes.shape)
    if half % 16:
        raise ValueError(f"codes: the last axis must be a multiple of 16, got {half}")
    if codes.dtype != torch.uint8:
        raise TypeError(f"codes: expected torch.uint8, got {codes.dtype}")
    if not codes.is_contiguous():
        raise ValueError("codes: must be contiguous")
    check_tensor(scales, "scales", torch.uint8, (_scale_bytes(groups, rows, 2 * half),), codes.device)
    with on_device(codes.device):
        out = torch.empty(*codes.shape[:-1], 2 * half, dtype=dtype, device=codes.device)
        lib.moe_mlp_dequantize_mxfp4(codes.data_ptr(), half, scales.data_ptr(), groups, rows, 2 * half, dt,
                                     out.data_ptr(), _raw_stream(codes.device.index))
    return out
