"""Plain references of the linear layers and norms, in 64 bits on the CPU (the
quantiser's four fp32 roundings are part of its definition and kept)."""
from __future__ import annotations

import numpy as np
import torch

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
UE4M3 = np.array([m / 512.0 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8.0) for e in range(16) for m in range(8)][:127])


def _nearest_even(a: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the table value nearest to a >= 0, ties to the even index, saturating."""
    a = np.minimum(a, table[-1])
    lo = np.searchsorted(table, a, side="right") - 1
    hi = np.minimum(lo + 1, len(table) - 1)
    dlo, dhi = a - table[lo], table[hi] - a
    return np.where((dhi < dlo) | ((dhi == dlo) & (lo % 2 == 1)), hi, lo)


def quantize(x: torch.Tensor, g: float = 1.0):
    """(codes [rows, K] one per element, scale bytes [rows, K/16]) of fp32-valued rows."""
    v = x.float().numpy().reshape(x.shape[0], -1, 16)
    f = np.float32
    a = np.abs(v).max(-1)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        s = _nearest_even(((a / f(6.0)) / f(g)).astype(np.float64), UE4M3)
        gs = (f(g) * UE4M3[s].astype(f)).astype(f)
        inv = np.where(s > 0, f(1.0) / gs, f(0.0)).astype(f)
    r = (v * inv[..., None]).astype(f)
    c = _nearest_even(np.abs(r).astype(np.float64), MAGS) | (np.signbit(r).astype(np.int64) << 3)
    return c.reshape(x.shape[0], -1).astype(np.uint8), s.astype(np.uint8)


def computed_g(x: torch.Tensor) -> float:
    a = np.float32(x.float().abs().max().item()) / np.float32(2688.0)
    return float(max(a, np.float32(2.0 ** -64)))


def values(codes: np.ndarray, scales: np.ndarray, g: float) -> torch.Tensor:
    """The values in 64 bits of codes [rows, K] and scale bytes [rows, K/16]."""
    v = MAGS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    v = v.reshape(codes.shape[0], -1, 16) * (float(g) * UE4M3[scales])[..., None]
    return torch.from_numpy(v.reshape(codes.shape[0], -1))


def pack_codes(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def tile(scales: np.ndarray) -> np.ndarray:
    """The documented byte order, entry by entry."""
    rows, nb = scales.shape
    chunks = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * chunks * 512, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * chunks + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = scales
    return out


def make_packed(rows: int, K: int, seed: int, std: float = 1.0, outliers: int = 2):
    """(bf16 source [rows, K], codes, scale bytes, g) with outlier channels and a computed g."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=gen) * std
    if outliers:
        x[:, torch.randperm(K, generator=gen)[:outliers]] *= 20.0
    x = x.bfloat16()
    g = computed_g(x) if rows else 1.0
    c, s = quantize(x, g)
    return x, c, s, g


def packed_to(dev, codes, scales, g):
    return (torch.from_numpy(pack_codes(codes)).to(dev), torch.from_numpy(tile(scales)).to(dev),
            torch.tensor([g], dtype=torch.float32, device=dev))
