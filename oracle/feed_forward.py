"""float64 reference of the gated feed-forward block and its compressed forms, in NumPy.

    h = act(x W_gᵀ) ⊙ (x W_uᵀ),  act = GeLU g·Φ(g) or SiLU g·σ(g)
("Griffin：将门控线性循环与局部注意力混合以实现高效的语言模型", §MLP块, Fig. 2(b), before the
down projection), its reverse-mode derivative, the 8-bit activation checkpoint (int8 codes and
one power of two for each 32 channels) and matrices of 4-bit codes with group scales.
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc


def act(g, name):
    g = np.asarray(g, dtype=np.float64)
    if name == "gelu":
        return g * 0.5 * erfc(-g / math.sqrt(2.0))
    return g / (1.0 + np.exp(-g))


def act_slope(g, name):
    g = np.asarray(g, dtype=np.float64)
    if name == "gelu":
        return 0.5 * erfc(-g / math.sqrt(2.0)) + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    r = 1.0 / (1.0 + np.exp(-g))
    return r * (1.0 + g * (1.0 - r))


def glu_forward(x, W_gate, W_up, name):
    return act(x @ W_gate.T, name) * (x @ W_up.T)


def glu_backward(x, W_gate, W_up, dh, name):
    g, u = x @ W_gate.T, x @ W_up.T
    dg = dh * u * act_slope(g, name)
    du = dh * act(g, name)
    return {"dx": dg @ W_gate + du @ W_up, "dW_gate": dg.T @ x, "dW_up": du.T @ x, "h": act(g, name) * u}


def act8_pack(x):
    """(codes [N][C], scales [N][⌈C/32⌉], both int64): for each group the smallest −127 ≤ e ≤ 121 with
    |rint(x / 2^e)| ≤ 127, by trying every exponent in turn, or 121 where none does, with the codes
    held within ±127 (127 · 2^121 is the largest multiple that is a finite number of either type); the
    scale is e + 127, or 255 where the group is not finite."""
    x = np.asarray(x, dtype=np.float64)
    N, C = x.shape
    groups = -(-C // 32)
    codes = np.zeros((N, C), dtype=np.int64)
    scales = np.zeros((N, groups), dtype=np.int64)
    for n in range(N):
        for j in range(groups):
            v = x[n, 32 * j:32 * j + 32]
            if not np.all(np.isfinite(v)):
                scales[n, j] = 255
                continue
            e = -127
            while e < 121 and np.max(np.abs(np.rint(np.ldexp(v, -e)))) > 127:
                e += 1
            codes[n, 32 * j:32 * j + 32] = np.clip(np.rint(np.ldexp(v, -e)), -127, 127).astype(np.int64)
            scales[n, j] = e + 127
    return codes, scales


def act8_unpack(codes, scales):
    N, C = codes.shape
    e = np.repeat(scales, 32, axis=1)[:, :C]
    return np.where(e == 255, np.nan, np.ldexp(codes.astype(np.float64), (e - 127).astype(np.int32)))


def w4_dequantize(codes, scales, group):
    """codes [N][K/2] bytes (even k in the low four bits), scales [N][K/group] → Ŵ [N][K]."""
    codes = np.asarray(codes).astype(np.int64)
    N, half = codes.shape
    q = np.empty((N, 2 * half))
    q[:, 0::2] = codes % 16
    q[:, 1::2] = codes // 16
    return (q - 8.0) * np.repeat(np.asarray(scales, dtype=np.float64), group, axis=1)
