"""References in 64 bits of the dense operators (gated feed-forward block, projection with adapters) and
element-wise error bounds that follow from the arithmetic of the kernels.

Products of bf16 values are exact in fp32; a sum of K of them in the tensor cores loses at most one unit in the
last place (2^-23 of the running sum of magnitudes) per addition, so its error is at most K 2^-23 sum|a||b|: that is
gamma(K) below.  A rounding to bf16 is off by at most half a step, 2^-8 of the value (plus half the smallest
subnormal, far below everything here).  The activations use the fast exponential and division (relative error
below 2^-20 each)."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8          # half a step of bf16, relative
FAST = 2.0 ** -18      # the activation and its slope, in units of the values they are made of
GELU_C = math.sqrt(2.0 / math.pi)


def gamma(K: int) -> float:
    return (K + 8) * 2.0 ** -23


def f64(t: torch.Tensor) -> torch.Tensor:
    return t.to(torch.float64)


def activation(z: torch.Tensor, act: str):
    """act(z), act'(z) in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    w = GELU_C * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(2 * w)
    return z * s, s + z * s * (1 - s) * 2 * GELU_C * (1 + 3 * 0.044715 * z ** 2)


def slope_size(z: torch.Tensor, act: str) -> torch.Tensor:
    """The size of the terms of act'(z), which its error scales with (the GELU argument is clamped at 12)."""
    if act == "silu":
        return 1 + z.abs()
    c = z.abs().clamp(max=12.0)
    return 1 + 2 * GELU_C * c * (1 + 3 * 0.044715 * c * c)


def split_bank(bank: torch.Tensor, d: int, I: int):
    """Wg, Wu [I][d], Wd [d][I] of a bf16 bank, in 64 bits."""
    n = I * d
    return (f64(bank[:n]).view(I, d), f64(bank[n:2 * n]).view(I, d), f64(bank[2 * n:3 * n]).view(d, I))


def block_forward(x, bank, d, I, act):
    """(g, u, y) in 64 bits and the bounds of the kernels' g, u (kept, in bf16) and y."""
    wg, wu, wd = split_bank(bank, d, I)
    X = f64(x)
    g, u = X @ wg.T, X @ wu.T
    dg, du = gamma(d) * (X.abs() @ wg.abs().T), gamma(d) * (X.abs() @ wu.abs().T)
    a, slope = activation(g, act)
    h = a * u
    # first order in the errors of g and u, and the product of both
    dh = slope.abs() * u.abs() * dg + a.abs() * du + 1.2 * dg * du + 0.6 * u.abs() * dg * dg + FAST * h.abs()
    dh = dh + U * (h.abs() + dh)
    y = h @ wd.T
    dy = dh @ wd.abs().T + gamma(I) * ((h.abs() + dh) @ wd.abs().T)
    return (g, u, y), (dg + U * (g.abs() + dg), du + U * (u.abs() + du), dy + U * (y.abs() + dy))


def block_backward(x, bank, pre, dy, d, I, act):
    """(dx, dWgu, dWd) in 64 bits from the kept g and u, and their bounds."""
    wg, wu, wd = split_bank(bank, d, I)
    X, DY = f64(x), f64(dy)
    g, u = f64(pre[:, :I]), f64(pre[:, I:])
    T = x.shape[0]
    a, slope = activation(g, act)
    dh = DY @ wd
    e_dh = gamma(d) * (DY.abs() @ wd.abs())
    h, dg, du = a * u, dh * u * slope, dh * a

    def rounded(v, e):
        return e + U * (v.abs() + e)

    e_h = rounded(h, FAST * h.abs())
    e_dg = rounded(dg, e_dh * (u * slope).abs() + FAST * (dh * u).abs() * slope_size(g, act))
    e_du = rounded(du, e_dh * a.abs() + FAST * du.abs())
    w = torch.cat([wg, wu])
    dgu, e_dgu = torch.cat([dg, du], 1), torch.cat([e_dg, e_du], 1)
    dx, dw, dwd = dgu @ w, dgu.T @ X, DY.T @ h
    e_dx = rounded(dx, e_dgu @ w.abs() + gamma(2 * I) * ((dgu.abs() + e_dgu) @ w.abs()))
    e_dw = rounded(dw, e_dgu.T @ X.abs() + gamma(T) * ((dgu.abs() + e_dgu).T @ X.abs()))
    e_dwd = rounded(dwd, DY.abs().T @ e_h + gamma(T) * (DY.abs().T @ (h.abs() + e_h)))
    return (dx, dw, dwd), (e_dx, e_dw, e_dwd)


def lora(x, w, a, b, scale, ids):
    """y in 64 bits and its bound; ids outside [0, n) take no adapter."""
    X, W = f64(x), f64(w)
    y, e = X @ W.T, gamma(x.shape[1]) * (X.abs() @ W.abs().T)
    n, r, K = a.shape
    for k in torch.unique(ids).tolist():
        if not 0 <= k < n:
            continue
        rows = (ids == k).nonzero().flatten()
        s = 1.0 if scale is None else float(scale[k])
        A, B, R = f64(a[k]), f64(b[k]), X[rows]
        v = s * (R @ A.T)
        ev = (gamma(K) + 2.0 ** -23) * abs(s) * (R.abs() @ A.abs().T)
        ev = ev + U * (v.abs() + ev)
        y[rows] += v @ B.T
        e[rows] += ev @ B.abs().T + gamma(K + r) * ((v.abs() + ev) @ B.abs().T)
        e[rows] += gamma(r) * (R.abs() @ W.abs().T)      # the longer accumulation
    return y, e + U * (y.abs() + e)


def assert_within(got, want, bound, what=""):
    err = (f64(got) - want).abs()
    ok = torch.isfinite(f64(got)) & (err <= bound + 1e-30)
    if not bool(ok.all()):
        i = (~ok).nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} values off; first at {i}: got "
                             f"{float(got[tuple(i)])}, want {float(want[tuple(i)])}, bound {float(bound[tuple(i)]):.3g}")


# The relative Frobenius norm of a gradient's error.  A weight gradient's operand (dg, du or h) is rounded once and so
# is the gradient, each by at most U of a value.  The operand's errors meet the other operand's independent rows, so
# that over the gradient they add up as the terms themselves do: at most U again, together 2 U.  A fifth more for the
# fp32 sums (below 2^-23 of the terms' running sum for each 16 of T tokens: 1e-3 at 10^5).
NORM = 2.4 * U


def norm_error(got, want) -> float:
    return float((f64(got) - want).norm() / want.norm())
