"""64-bit references of the operators around the recurrent step (test
infrastructure), each with the magnitude its rounding errors scale with: the
same sums over absolute values.  Written from the definitions, token by token.
"""

from __future__ import annotations

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}


def silu(x):
    return x / (1 + torch.exp(-x))


def conv(x, starts, w, bias, h0, act):
    """-> (y, |y| magnitude, states): x [T, C], h0 [n, W-1, C] or None."""
    n, (C, W) = len(starts) - 1, w.shape
    x, w = x.double(), w.double()
    b = bias.double() if bias is not None else x.new_zeros(C)
    h = h0.double() if h0 is not None else x.new_zeros(n, W - 1, C)
    y, mag, h1 = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(h)
    for s in range(n):
        rows = torch.cat([h[s], x[starts[s]:starts[s + 1]]], 0)
        for t in range(starts[s + 1] - starts[s]):
            win = rows[t:t + W] * w.t()
            y[starts[s] + t] = b + win.sum(0)
            mag[starts[s] + t] = b.abs() + win.abs().sum(0)
        h1[s] = rows[rows.shape[0] - (W - 1):]
    # |d silu / dx| < 1.1, and the function's own rounding is relative to |y|
    return (silu(y), 1.1 * mag + silu(y).abs(), h1) if act else (y, mag, h1)


def conv_tol(mag, W, dtype):
    """W + 1 roundings of the sum, at most 8 more units for the activation (the
    fast exponential and division are within a few ulp), one of the output."""
    return mag * ((W + 1 + 8) * U[torch.float32]) + mag * (U[dtype] if dtype != torch.float32 else 0)


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def ssm(starts, q, k, v, dt, a, d, bias, S0, use_softplus=True):
    """q, k [T, G, dk], v [T, H, dv], dt [T, H], S0 [n, H, dv, dk] or None.
    -> (o [T, H, dv], S1, magnitude of o, magnitude of S1, largest |dt a|)."""
    n, (T, H, dv), (G, dk) = len(starts) - 1, v.shape, q.shape[1:]
    q, k = (z.double().repeat_interleave(H // G, 1) for z in (q, k))
    v = v.double()
    x = dt.double() + (bias.double() if bias is not None else 0)
    x = softplus(x) if use_softplus else x
    lam = x * a.double()
    S = S0.double().clone() if S0 is not None else v.new_zeros(n, H, dv, dk)
    A = S.abs()
    dd = d.double()[:, None] if d is not None else v.new_zeros(H, 1)
    o, mo = torch.zeros_like(v), torch.zeros_like(v)
    for s in range(n):
        for t in range(starts[s], starts[s + 1]):
            e = torch.exp(lam[t])[:, None, None]
            S[s] = e * S[s] + (x[t][:, None] * v[t])[..., None] * k[t][:, None]
            A[s] = e * A[s] + (x[t][:, None] * v[t]).abs()[..., None] * k[t].abs()[:, None]
            o[t] = (S[s] * q[t][:, None]).sum(-1) + dd * v[t]
            mo[t] = (A[s] * q[t].abs()[:, None]).sum(-1) + (dd * v[t]).abs()
    top = float(lam.abs().max()) if T else 0.0
    return o, S, mo, A, top


def ssm_tol(mo, ms, top, longest, dk, dtype):
    """Tolerances of o and S1.  fp32 part: a term of the state passes at most
    `longest` decays, each exponential right to 4 units and its argument dt * a
    to 8 (softplus, product), so to 4 + 8 * top relative, plus 2 roundings a
    step; the sum over d_k adds d_k roundings.  For bf16, o may also carry one
    rounding of each term's weight or state (2^-8), and its own (2^-8)."""
    f = U[torch.float32]
    ts = ms * (longest * (6 + 8 * min(top, 88.0)) + 8) * f
    to = mo * (longest * (6 + 8 * min(top, 88.0)) + dk + 8) * f
    if dtype == torch.bfloat16:
        to = to + mo * (2 * U[dtype] + U[dtype] ** 2)
    return to + 1e-30, ts + 1e-30


def norm(x, res, w, eps):
    h = x.double() + (res.double() if res is not None else 0)
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return h, h * r * w.double()
