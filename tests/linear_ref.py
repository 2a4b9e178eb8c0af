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
    v = x.float().numpy().reshape(x.shape[0], x.shape[1] // 16, 16)
    f = np.float32
    a = np.abs(v).max(-1)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        s = _nearest_even(((a / f(6.0)) / f(g)).astype(np.float64), UE4M3)
        gs = (f(g) * UE4M3[s].astype(f)).astype(f)
        inv = np.where(s > 0, f(1.0) / gs, f(0.0)).astype(f)
    r = (v * inv[..., None]).astype(f)
    c = _nearest_even(np.abs(r).astype(np.float64), MAGS) | (np.signbit(r).astype(np.int64) << 3)
    return c.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def computed_g(x: torch.Tensor) -> float:
    a = np.float32(x.float().abs().max().item()) / np.float32(2688.0)
    return float(max(a, np.float32(2.0 ** -64)))


def values(codes: np.ndarray, scales: np.ndarray, g: float) -> torch.Tensor:
    """The values in 64 bits of codes [rows, K] and scale bytes [rows, K/16]."""
    v = MAGS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    v = v.reshape(codes.shape[0], codes.shape[1] // 16, 16) * (float(g) * UE4M3[scales])[..., None]
    return torch.from_numpy(v.reshape(codes.shape))


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


# ------------------------------------------------ norms around a branch --
#
# The formulas in 64 bits with a bound on how far fp32 arithmetic may be off,
# first order in u = 2^-24.  A row's sums run over at most 64 terms a thread, 5
# exchanges and 16 warps: DEPTH roundings.  The root's relative error is half of
# its sum's, plus 2 units in the last place (4u) of the reciprocal root.

U = 2.0 ** -24
DEPTH = 90
ROOT = DEPTH / 2 + 8


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2 if t != torch.float64 else 0.0


def norm64(v, layer, eps, dv=None):
    """(norm(v), 1/root, bound on the computed norm) for v off by at most dv."""
    dv = torch.zeros_like(v) if dv is None else dv
    dm = torch.zeros_like(v[..., :1])
    c = v
    if layer:
        dm = dv.mean(-1, keepdim=True) + DEPTH * U * v.abs().mean(-1, keepdim=True)
        c = v - v.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    n = c * r
    dc = dv + dm + U * v.abs()
    # the root sees its values' errors through mean(n dc); a shift common to all of a row cancels there
    own = dv + U * v.abs()
    rel = ROOT * U + r * (n.abs() * own).mean(-1, keepdim=True) + (r * dm) ** 2
    return n, r, r * dc + n.abs() * (rel + 2 * U)


def _f64(t, default=None):
    return t.double() if t is not None else default


def norm_gate64(x, h, post, gate, pre, scale, shift, groups, layer, eps):
    """dict(y, z) in 64 bits and dict of bounds before the outputs' rounding."""
    M, C = x.shape
    G = groups
    v = lambda t: t.double().view(-1, 1, C) if t is not None else None
    x3 = x.double().view(G, -1, C)
    one = torch.ones(1, 1, C, dtype=torch.float64, device=x.device)
    post, gate, pre = (one if t is None else v(t) for t in (post, gate, pre))
    scale, shift = (0 * one if t is None else v(t) for t in (scale, shift))
    y, dy = x3, torch.zeros_like(x3)
    if h is not None:
        m, _, dm = norm64(h.double().view(G, -1, C), layer, eps)
        y = x3 + gate * post * m
        dy = (gate * post).abs() * (dm + 2 * U * m.abs()) + U * y.abs()
    n, _, dn = norm64(y, layer, eps, dy)
    w = pre * (1 + scale)
    z = n * w + shift
    dz = w.abs() * (dn + 3 * U * n.abs()) + U * z.abs()
    return {"y": y.reshape(M, C), "z": z.reshape(M, C)}, {"y": dy.reshape(M, C), "z": dz.reshape(M, C)}


def _norm_grad64(v, g, dg, layer, eps):
    """Gradient of norm at v for the gradient g of its result (known within dg), and its bound."""
    n, r, dn = norm64(v, layer, eps)
    c = (g * n).mean(-1, keepdim=True)
    dc = (g.abs() * dn + dg * n.abs() + DEPTH * U * (g * n).abs()).mean(-1, keepdim=True)
    mg, dmg = 0.0, 0.0
    if layer:
        mg = g.mean(-1, keepdim=True)
        dmg = (dg + DEPTH * U * g.abs()).mean(-1, keepdim=True)
    out = r * (g - mg - n * c)
    rel = dn / n.abs().clamp(min=1e-300)  # the root's part of it; the mean's shift stands in dn itself
    root = torch.minimum(rel, torch.full_like(rel, 1.0)).amin(-1, keepdim=True) + ROOT * U
    bound = r * (dg + dmg + n.abs() * dc + dn * c.abs() + 4 * U * (g.abs() + (n * c).abs()) + 4 * U * (abs(mg)))
    return out, bound + out.abs() * root, n, dn


def norm_gate_backward64(dz, dy, y, h, post, gate, pre, scale, groups, layer, eps):
    M, C = y.shape
    G = groups
    r3 = lambda t: t.double().view(G, -1, C)
    v = lambda t: t.double().view(-1, 1, C)
    one = torch.ones(1, 1, C, dtype=torch.float64, device=y.device)
    post, gate, pre = (one if t is None else v(t) for t in (post, gate, pre))
    scale = 0 * one if scale is None else v(scale)
    gate, scale = gate.expand(G, 1, C), scale.expand(G, 1, C)
    dz3 = r3(dz)
    g = dz3 * pre * (1 + scale)
    dv, ddv, n, dn = _norm_grad64(r3(y), g, 3 * U * g.abs(), layer, eps)
    dyv = r3(dy) if dy is not None else torch.zeros_like(dv)
    dx = dyv + dv
    ddx = ddv + U * dx.abs()
    rows = M // G

    def colsum(term, err):
        return term.sum(1), (err + (rows + 16) * U * term.abs()).sum(1)

    out, bound = {}, {}
    out["dx"], bound["dx"] = dx.reshape(M, C), ddx.reshape(M, C)
    out["dshift"], bound["dshift"] = colsum(dz3, 0 * dz3)
    s, e = colsum(dz3 * n, dz3.abs() * dn + U * (dz3 * n).abs())
    out["dscale"], bound["dscale"] = s * pre[:, 0], e * pre[:, 0].abs() + 2 * U * (s * pre[:, 0]).abs()
    w = 1 + scale[:, 0]
    out["dpre_weight"] = (s * w).sum(0)
    bound["dpre_weight"] = (e * w.abs() + (G + 12) * U * (s * w).abs()).sum(0)
    if h is not None:
        g = dx * gate * post
        dh, ddh, m, dm = _norm_grad64(r3(h), g, (gate * post).abs() * ddx + 3 * U * g.abs(), layer, eps)
        out["dh"], bound["dh"] = dh.reshape(M, C), ddh.reshape(M, C)
        s, e = colsum(dx * m, ddx * m.abs() + dx.abs() * dm + U * (dx * m).abs())
        out["dgate"], bound["dgate"] = s * post[:, 0], e * post[:, 0].abs() + 2 * U * (s * post[:, 0]).abs()
        out["dpost_weight"] = (s * gate[:, 0]).sum(0)
        bound["dpost_weight"] = (e * gate[:, 0].abs() + (G + 12) * U * (s * gate[:, 0]).abs()).sum(0)
    return out, bound


def worst(got, want, bound) -> float:
    """Largest error in units of the bound, which grows by half a step of got's type."""
    b = bound * (1 + 2.0 ** -10) + want.abs() * half_step(got.dtype) + 1e-37
    d = (got.double() - want).abs() / b
    return float(d.max()) if d.numel() else 0.0
