"""Plain 64-bit forms of the operators of a prompt's chunk (chunk attention, head norms,
projections), on the CPU, with the error each fp32 kernel may have; built as those of
_decoder_ref are, and with its constants."""
from __future__ import annotations

import math

import numpy as np
import torch

from _decoder_ref import U32, UP, f64, gather


def attend_chunk(q, k_pages, v_pages, table, starts, lens, scale, softcap=0.0, window=0, k_scale=None, v_scale=None):
    """(out, bound, lse, bound) of rows starts[0]..starts[-1] - 1, the other rows NaN: see
    moe_kv_attend_chunk. table, starts and lens on the host. Every token uses the rows it
    attends to and no others."""
    T, Hq, D = q.shape
    Hk, G = k_pages.shape[1], q.shape[1] // k_pages.shape[1]
    q = f64(q)
    out, eo = (torch.full((T, Hq, D), x, dtype=torch.float64) for x in (torch.nan, 0.0))
    lse, el = (torch.full((T, Hq), x, dtype=torch.float64) for x in (torch.nan, 0.0))
    for b in range(len(lens)):
        n, total = starts[b + 1] - starts[b], max(int(lens[b]), 0)
        rows = slice(starts[b], starts[b + 1])
        if n == 0 or total == 0:
            out[rows], lse[rows] = 0.0, -torch.inf
            continue
        pos = total - n + torch.arange(n)
        lo = max(0, total - n + 1 - window) if window else 0
        j = torch.arange(lo, total)
        seen = j <= pos[:, None]
        if window:
            seen &= j > pos[:, None] - window
        for h in range(Hk):
            k = gather(k_pages, table, b, lo, total, h) * (1.0 if k_scale is None else float(k_scale[h]))
            v = gather(v_pages, table, b, lo, total, h) * (1.0 if v_scale is None else float(v_scale[h]))
            # what no token of the chunk sees is left out; what only some see stays, and is
            # looked at by those alone where it is not finite
            k, v = (torch.where(seen.any(0)[:, None], x, 0.0) for x in (k, v))
            odd = ~torch.isfinite(v).all(1)
            vf = torch.where(torch.isfinite(v), v, 0.0)
            heads = slice(h * G, (h + 1) * G)
            qs = q[rows, heads]
            s = torch.einsum("ngd,jd->ngj", qs, k) * scale
            # a dot product of D terms, the scale and the conversion to base two
            es = (D + 6) * U32 * torch.einsum("ngd,jd->ngj", qs.abs(), k.abs()) * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                es = es + softcap * 2.0 ** -20
            es = es + 4 * U32 * s.abs()
            s = torch.where(seen[:, None], s, -torch.inf)
            es = torch.where(seen[:, None] & torch.isfinite(es), es, 0.0).amax(2, keepdim=True)
            m = s.amax(2, keepdim=True)
            p = torch.exp(s - torch.where(torch.isfinite(m), m, 0.0))
            L = p.sum(2, keepdim=True)
            p = p / torch.where(L == 0, 1.0, L)
            # weights: twice the scores' error, the exponential (2^-21), their rounding in the
            # product; the sum over the positions
            rel = 2 * es + 2.0 ** -21 + UP + 2 * len(j) * U32
            o = torch.einsum("ngj,jd->ngd", p, vf)
            for i in torch.nonzero(odd).flatten().tolist():
                o = torch.where(seen[:, i, None, None], o + (v[i] - vf[i]), o)
            out[rows, heads] = o
            eo[rows, heads] = rel * torch.einsum("ngj,jd->ngd", p, vf.abs())
            lse[rows, heads] = (m + torch.log(L))[..., 0]
            el[rows, heads] = (es[..., 0] + 2.0 ** -21 + len(j) * U32
                               + 4 * U32 * torch.nan_to_num(lse[rows, heads], neginf=0.0).abs())
    return out, eo, lse, el


def head_norm(x, w, eps, offset):
    """(value, relative bound): x [T, heads, d] normed per head."""
    x = f64(x)
    if w is None:
        return x, 0.0
    d = x.shape[-1]
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * (f64(w) + offset)
    # a mean of d squares (halved by the root), the root, the quotient, the weight's sum and two products
    return y, ((d + 2) / 2 + 8) * U32


def rotate64(x, positions, inv_freq, adjacent):
    """Rotation of values that are held in 64 bits already."""
    half = len(inv_freq)
    y = x.clone()
    if half == 0:
        return y
    ang = np.outer(np.asarray(positions, np.float64), np.asarray(inv_freq, np.float64))
    c, s = torch.from_numpy(np.cos(ang))[:, None], torch.from_numpy(np.sin(ang))[:, None]
    i = slice(0, 2 * half, 2) if adjacent else slice(0, half)
    j = slice(1, 2 * half, 2) if adjacent else slice(half, 2 * half)
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def linear(x, w, bias, activation, residual):
    """(value, bound): see moe_linear."""
    x, w = f64(x), f64(w)
    z = x @ w.T
    # products of bf16 numbers are exact in fp32; a sum of K terms in any order
    e = (x.shape[1] + 2) * U32 * (x.abs() @ w.abs().T)
    if bias is not None:
        z = z + f64(bias)
        e = e + U32 * z.abs()
    if activation == "silu":
        # |silu'| <= 1.1; exponential, sum, quotient
        y, e = z * torch.sigmoid(z), 1.1 * e + 2.0 ** -20 * (z * torch.sigmoid(z)).abs()
    elif activation == "gelu_tanh":
        # |gelu'| <= 1.13; the hyperbolic tangent to 2^-21 of itself or of one, times z / 2
        y = 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        e = 1.13 * e + 2.0 ** -20 * z.abs()
    elif activation == "sigmoid":
        y, e = torch.sigmoid(z), 0.25 * e + 2.0 ** -20
    else:
        y = z
    if residual is not None:
        y = y + f64(residual)
        e = e + U32 * y.abs()
    return y, e
