"""How far the gated feed-forward block's kernels may be from the float64 oracle, element by element.

A product of two bf16 numbers is exact in float32; a sum of n of them in float32, in any order and
with partial sums cut off instead of rounded (tensor cores), is off by at most n·2^-23 of the sum of
magnitudes (SUM). The activation s(g)·g in float32: Abramowitz & Stegun's 7.1.26 is off by
0.75e-7 in Φ, the hardware's exponential and reciprocal by 2^-22 each, and about ten float32
operations follow: ACT = 2e-6 relative to |g| (and to 1 for the slope, whose largest value is 1.13).
|act'| ≤ 1.13 and |act''| ≤ 0.8 for both activations (GeLU: √2·φ-type extrema at 1.1289 and 0.798;
SiLU: 1.0998 and 0.5). A rounding to bf16 is off by half a step, 2^-8 of the value, or by half of
the smallest step there is, 2^-134."""
import numpy as np

SUM = 2.0 ** -23
ACT = 2e-6
HALF = 2.0 ** -8
TINY = 2.0 ** -133


def _products(x, Wg, Wu):
    D = x.shape[1]
    g, u = x @ Wg.T, x @ Wu.T
    eg = D * SUM * (np.abs(x) @ np.abs(Wg).T)
    eu = D * SUM * (np.abs(x) @ np.abs(Wu).T)
    return g, u, eg, eu


def forward_bound(x, Wg, Wu, act, h):
    """|kernel's h − h|, at most."""
    g, u, eg, eu = _products(x, Wg, Wu)
    a = np.abs(act(g))
    ea = 1.13 * eg + ACT * (np.abs(g) + eg)
    e = ea * np.abs(u) + (a + ea) * eu
    return (e + HALF * (np.abs(h) + e)) * (1 + 1e-6) + TINY


def backward_bounds(x, Wg, Wu, dh, act, slope):
    """The same for dx, dW_gate and dW_up: dg and du are rounded to bf16 before their products."""
    g, u, eg, eu = _products(x, Wg, Wu)
    N, H = dh.shape
    a, s = np.abs(act(g)), np.abs(slope(g))
    ea = 1.13 * eg + ACT * (np.abs(g) + eg)
    es = 0.8 * eg + ACT * (1.13 + np.abs(g) * 0.4)
    dg, du = np.abs(dh) * np.abs(u) * s, np.abs(dh) * a
    edg = np.abs(dh) * (es * np.abs(u) + (s + es) * eu)
    edu = np.abs(dh) * ea
    edg = edg + HALF * (dg + edg) + TINY
    edu = edu + HALF * (du + edu) + TINY
    dgm, dum = dg + edg, du + edu

    def out(err, size, terms, ref_size):
        e = err + terms * SUM * size
        return (e + HALF * (ref_size + e)) * (1 + 1e-6) + TINY

    dx_ref = np.abs(dh * u * slope(g) @ Wg + dh * act(g) @ Wu)
    return {
        "dx": out(edg @ np.abs(Wg) + edu @ np.abs(Wu), dgm @ np.abs(Wg) + dum @ np.abs(Wu), 2 * H, dx_ref),
        "dW_gate": out(edg.T @ np.abs(x), dgm.T @ np.abs(x), N, np.abs((dh * u * slope(g)).T @ x)),
        "dW_up": out(edu.T @ np.abs(x), dum.T @ np.abs(x), N, np.abs((dh * act(g)).T @ x)),
    }


def w4_bound(x, W, y):
    """|kernel's y − x Ŵᵀ|: q − 8 is exact, a group's sum is a float32 sum, its scale multiplies it and
    the scaled sums add in float32, eight warps' after one another."""
    K = x.shape[1]
    e = (K + 16) * SUM * (np.abs(x) @ np.abs(W).T)
    return e, (e + HALF * (np.abs(y) + e)) * (1 + 1e-6) + TINY
