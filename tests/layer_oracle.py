"""Plain 64-bit implementations of the sequence-layer operators, step by step from their definitions (CPU, torch)."""
import decimal
import functools
import math
from decimal import Decimal

import torch


decimal.getcontext().prec = 60
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@functools.lru_cache(maxsize=None)
def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=4096, fast=32.0, slow=1.0):
    """Angles per position, in 60 digits so that far positions keep theirs, and the factor m."""
    f, base, factor = [], Decimal(base), Decimal(factor)
    if scaling == "ntk":
        base = base * factor ** (Decimal(rot) / (rot - 2))
    for i in range(rot // 2):
        w = base ** (Decimal(-2 * i) / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "yarn":
            g = min(Decimal(1), max(Decimal(0), (original * w / TWO_PI - Decimal(slow)) / (Decimal(fast) - Decimal(slow))))
            w *= g + (1 - g) / factor
        f.append(w)
    m = 0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0
    return f, m


def rotate(x, positions, rot, layout="half", inverse=False, **how):
    """x [..., heads, d] in 64 bits, positions [...]."""
    f, m = frequencies(rot, **how)
    y = x.double().clone()
    flat, pos = y.reshape(-1, *y.shape[-2:]), [int(p) for p in positions.reshape(-1)]
    for r, p in enumerate(pos):
        for i, w in enumerate(f):
            a0, b0 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            t = float((p * w) % TWO_PI)
            c, s = m * math.cos(t), m * math.sin(t)
            if inverse:
                s = -s
            a, b = flat[r, :, a0].clone(), flat[r, :, b0].clone()
            flat[r, :, a0], flat[r, :, b0] = a * c - b * s, b * c + a * s
    return flat.reshape(y.shape)


def norm(x, w, eps):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def norm_gradient(t, x, w, eps):
    """(dx, dw) of sum(t * norm(x, w))."""
    x, t, w = x.double(), t.double(), w.double()
    rms = torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, u = x / rms, t * w
    return (u - n * (u * n).mean(-1, keepdim=True)) / rms, (t * n).reshape(-1, x.shape[-1]).sum(0)


def linear(q, k, v, g, scale, s0=None):
    """(o [T, H, dv], S [H, dk, dv]) of one sequence; q [T, H, dk], k and v with fewer heads; g [H]."""
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    S = torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64) if s0 is None else s0.double().clone()
    lam = torch.exp(g.double())[:, None, None]
    o = torch.zeros(q.shape[0], H, v.shape[2], dtype=torch.float64)
    for t in range(q.shape[0]):
        S = lam * S + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * torch.einsum("hd,hde->he", q[t], S)
    return o, S


def linear_gradient(do, q, k, v, g, scale, s0=None, ds=None):
    """(dq, dk, dv, ds0) of one sequence."""
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    q, do = q.double(), do.double()
    kw, vw = k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    T, dk_, dv_ = q.shape[0], q.shape[2], v.shape[2]
    lam = torch.exp(g.double())[:, None, None]
    S = torch.zeros(H, dk_, dv_, dtype=torch.float64) if s0 is None else s0.double().clone()
    R = torch.zeros(H, dk_, dv_, dtype=torch.float64) if ds is None else ds.double().clone()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(kw), torch.zeros_like(vw)
    for t in range(T):
        S = lam * S + kw[t][:, :, None] * vw[t][:, None, :]
        dq[t] = scale * torch.einsum("hde,he->hd", S, do[t])
    for t in reversed(range(T)):
        R = R + scale * q[t][:, :, None] * do[t][:, None, :]
        dk[t] = torch.einsum("hde,he->hd", R, vw[t])
        dv[t] = torch.einsum("hde,hd->he", R, kw[t])
        R = lam * R
    return dq, dk.unflatten(1, (H // G, G)).sum(2), dv.unflatten(1, (H // G, G)).sum(2), R
