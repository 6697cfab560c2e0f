"""Plain definitions of the 4-bit matrix operators and the table lookup with its gradient, for the tests.

Codes, scales and zero points follow the fp32 steps of the definition in numpy (whose fp32 quotients are correctly
rounded), so they are compared bit for bit; products and sums are taken in 64 bits.
"""
from __future__ import annotations

import numpy as np
import torch

F32 = np.float32


def to_bf16(v: np.ndarray) -> np.ndarray:
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32."""
    return torch.from_numpy(np.ascontiguousarray(v, dtype=F32)).to(torch.bfloat16).float().numpy()


def quantize_int4(x: torch.Tensor, group: int, scale_bf16: bool, asym: bool):
    """(codes [N, K] 0..15, scale fp32 [N, G], zero [N, G]) of x, one group at a time."""
    v = x.float().numpy()
    N, K = v.shape
    G = -(-K // group)
    codes = np.zeros((N, K), np.int64)
    scale, zero = np.zeros((N, G), F32), np.full((N, G), 8, np.int64)
    for g in range(G):
        b = v[:, g * group:(g + 1) * group]
        if asym:
            lo, hi = np.minimum(b.min(1), F32(0)), np.maximum(b.max(1), F32(0))
            s = hi / F32(15) - lo / F32(15)
        else:
            s = np.abs(b).max(1) / F32(7)
        s = s.astype(F32)
        if scale_bf16:
            s = to_bf16(s)
        s[s == 0] = 1
        c = np.rint(b / s[:, None])
        assert c.dtype == F32
        if asym:
            z = np.clip(np.rint(-lo / s), 0, 15)
            zero[:, g] = z.astype(np.int64)
            c = np.clip(c + z[:, None], 0, 15)
        else:
            c = np.clip(c, -8, 7) + 8
        codes[:, g * group:(g + 1) * group] = c.astype(np.int64)
        scale[:, g] = s
    return codes, scale, zero


def pack(codes: np.ndarray, zero: np.ndarray, group: int) -> np.ndarray:
    """uint8 [N, ceil(K/2)]; the unused nibble of an odd row holds the zero point of its group."""
    N, K = codes.shape
    if K % 2:
        codes = np.concatenate([codes, zero[:, -1:]], 1)
        if K % group == 0:  # pragma: no cover - groups are even
            raise AssertionError
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q: np.ndarray, K: int) -> np.ndarray:
    c = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    return c[:, :K].astype(np.int64)


def spread(per_group: np.ndarray, group: int, K: int) -> np.ndarray:
    return np.repeat(per_group, group, 1)[:, :K]


def values(codes, scale, zero, group: int) -> np.ndarray:
    """fp32(scale * (code - zero)) [N, K]."""
    K = codes.shape[1]
    return (codes - spread(zero, group, K)).astype(F32) * spread(scale.astype(F32), group, K)


def product(x: np.ndarray, codes, scale, zero, group: int, bias=None):
    """(y, S) in 64 bits: x W^T + bias, and the sum of the magnitudes of its terms."""
    w = (codes - spread(zero, group, codes.shape[1])).astype(np.float64) * spread(scale.astype(np.float64), group, codes.shape[1])
    y, S = x.astype(np.float64) @ w.T, np.abs(x).astype(np.float64) @ np.abs(w).T
    if bias is not None:
        y, S = y + bias.astype(np.float64), S + np.abs(bias)
    return y, S


def lookup(tokens: np.ndarray, table: np.ndarray, alpha: float) -> np.ndarray:
    """fp32(alpha * table[token]), zero rows outside the table."""
    ok = (tokens >= 0) & (tokens < len(table))
    rows = table[np.where(ok, tokens, 0)] * F32(alpha)
    return np.where(ok[:, None], rows, F32(0)).astype(F32)


def lookup_grad(tokens: np.ndarray, grad: np.ndarray, V: int, alpha: float, padding_idx=None):
    """(d, S, n) in 64 bits: the gradient, the sum of the magnitudes of its terms, and the terms per row."""
    d, S, n = np.zeros((V, grad.shape[1])), np.zeros((V, grad.shape[1])), np.zeros(V, np.int64)
    keep = (tokens >= 0) & (tokens < V)
    if padding_idx is not None:
        keep &= tokens != padding_idx
    g = grad.astype(np.float64)
    a = float(F32(alpha))
    np.add.at(d, tokens[keep], a * g[keep])
    np.add.at(S, tokens[keep], abs(a) * np.abs(g[keep]))
    np.add.at(n, tokens[keep], 1)
    return d, S, n
