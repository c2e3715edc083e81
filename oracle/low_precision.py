"""The 8-bit linear layer and the 4-bit cache rows, plain numpy in 64 bits (TEST INFRASTRUCTURE ONLY).

The formats are the library's own (the pages describe none) and are stated here as their definition.  A scale is a
stored number, so its rounding (fp32 for 8-bit rows, bf16 for 4-bit rows) is part of the format; everything else is
exact.  Values are float64 arrays.
"""
from __future__ import annotations

import dataclasses

import numpy as np
import torch

TINY = 2.0 ** -126


def _bf16(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.float32)
    return torch.from_numpy(x.reshape(-1).copy()).bfloat16().double().numpy().reshape(x.shape)


def quant_rows_i8(x):
    """x [T, K] -> (codes [T, K], scale [T]); numpy's rint rounds ties to even."""
    x = np.asarray(x, np.float64)
    amax = np.abs(x).max(axis=1, initial=0.0)
    with np.errstate(over="ignore", invalid="ignore"):
        scale = (amax.astype(np.float32) / np.float32(127.0)).astype(np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    dead = (scale < TINY) & ~bad
    use = np.where(bad | dead, 1.0, scale)
    codes = np.rint(np.where((bad | dead)[:, None], 0.0, x) / use[:, None])
    return codes, np.where(bad, np.nan, np.where(dead, 0.0, scale))


def quant_weight_i8(w):
    """w [K, N] -> (codes [N, K], scale [N])."""
    return quant_rows_i8(np.asarray(w, np.float64).T)


def linear_i8(x, w_codes, w_scale, bias=None, silu=False):
    codes, scale = quant_rows_i8(x)
    y = codes @ np.asarray(w_codes, np.float64).T * scale[:, None] * np.asarray(w_scale, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return y / (1 + np.exp(-y)) if silu else y


def quant4(x):
    """x [..., d] -> (codes 0..15, scale, zero): every row by itself."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    lo, hi = np.minimum(x.min(-1), 0.0), np.maximum(x.max(-1), 0.0)
    with np.errstate(over="ignore"):
        scale = _bf16((hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15.0))
    bad |= ~np.isfinite(scale)
    dead = (scale < TINY) & ~bad
    use = np.where(bad | dead, 1.0, scale)
    zero = np.where(bad | dead, 0.0, np.clip(np.rint(-lo / use), 0, 15))
    codes = np.clip(np.rint(x / use[..., None]) + zero[..., None], 0, 15)
    codes = np.where((bad | dead)[..., None], 0.0, codes)
    return codes.astype(np.uint8), np.where(bad, np.nan, np.where(dead, 0.0, scale)), zero


def dequant4(codes, scale, zero):
    return np.asarray(scale)[..., None] * (np.asarray(codes, np.float64) - np.asarray(zero)[..., None])


def pack4(codes):
    """Codes [..., d] -> bytes [..., d / 2], one 32-bit word at a time."""
    codes = np.asarray(codes, np.uint32)
    d = codes.shape[-1]
    words = np.zeros(codes.shape[:-1] + (d // 8,), np.uint32)
    for e in range(8):
        words |= codes[..., e::8] << np.uint32(4 * (e // 2 + 4 * (e % 2)))
    return words.astype("<u4").view(np.uint8).reshape(codes.shape[:-1] + (d // 2,))


def unpack4(byte):
    words = np.ascontiguousarray(byte).view("<u4")
    out = np.zeros(words.shape[:-1] + (words.shape[-1] * 8,), np.uint8)
    for e in range(8):
        out[..., e::8] = (words >> np.uint32(4 * (e // 2 + 4 * (e % 2)))) & 15
    return out


@dataclasses.dataclass
class Pools4:
    """A 4-bit cache: torch tensors as the library takes them."""
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor


def quant_pool(pool):
    """[num_pages, H, P, d] rows -> (bytes, scales) torch tensors; slots of NaN become rows with scale NaN."""
    codes, scale, zero = quant4(pool.double().numpy())
    meta = torch.from_numpy(np.stack([scale, zero], -1)).bfloat16()
    return torch.from_numpy(pack4(codes)), meta


def dequant_pool(byte, meta):
    m = meta.double().numpy()
    return torch.from_numpy(dequant4(unpack4(byte.numpy()), m[..., 0], m[..., 1]))


def quantised(pb):
    """(Pools4, the same synth.PagedBatch with the pools holding the values the codes stand for)."""
    kp, ks = quant_pool(pb.k_pool)
    vp, vs = quant_pool(pb.v_pool)
    return Pools4(kp, vp, ks, vs), dataclasses.replace(pb, k_pool=dequant_pool(kp, ks), v_pool=dequant_pool(vp, vs))
