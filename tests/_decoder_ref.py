"""Plain 64-bit forms of the decoder-layer operators (block norm, cache append,
paged attention), on the CPU, with the error each fp32 kernel may have.

Every function returns the value and a bound on the kernel's distance from it,
element by element, before the output type's own rounding:
  * fp32 arithmetic is off by U32 = 2^-24 relative per operation;
  * a sum of n terms in any order is off by at most n * U32 * sum |terms|;
  * softmax weights that go through a product in the cache's 16-bit operand type
    are rounded once: UP relative (half a bf16 step).
`rounded` adds the output's rounding: half a step of its type.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float8_e4m3fn": 2.0 ** -4}
TINY = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float8_e4m3fn": 2.0 ** -10}  # half the smallest step
UP = 2.0 ** -8


def f64(t):
    return None if t is None else t.detach().float().cpu().double() if "float8" in str(t.dtype) else \
        t.detach().cpu().double()


def rounded(value, bound, dtype):
    name = str(dtype).rsplit(".", 1)[-1]
    return bound + HALF[name] * (value.abs() + bound) + TINY[name]


def assert_close(got, value, bound, what=""):
    """got (any float type) against value within bound; infinities and NaN in the same places."""
    g = f64(got)
    assert g.shape == value.shape, (what, g.shape, value.shape)
    fine = torch.isfinite(value)
    assert torch.equal(torch.isfinite(g), fine), f"{what}: finite in other places"
    assert torch.equal(torch.isnan(g), torch.isnan(value)), f"{what}: NaN in other places"
    assert torch.equal(g[~fine & ~torch.isnan(value)], value[~fine & ~torch.isnan(value)]), f"{what}: infinities"
    over = ((g - value).abs() - bound)[fine]
    if over.numel() and float(over.max()) > 0:
        d = (g - value).abs()
        d[~fine] = 0
        at = int((d - torch.where(fine, bound, torch.inf)).argmax())
        raise AssertionError(f"{what}: off by {float(d.reshape(-1)[at]):.3g}, allowed "
                             f"{float(bound.expand_as(value).reshape(-1)[at]):.3g} at flat index {at}")


# ---- block norm -------------------------------------------------------------------

def block_norm(x, o, gate, w_post, w_pre, eps, scale, offset):
    """(r, bound on r, h, bound on h): see moe_block_norm."""
    x, o, gate, w_post, w_pre = map(f64, (x, o, gate, w_post, w_pre))
    H = x.shape[1]
    # a mean of H squares (relative (H + 2) U32, halved by the root), the root, the quotient and
    # at most five products per term
    rel = ((H + 2) / 2 + 8) * U32
    a = torch.zeros_like(x) if o is None else o
    if w_post is not None:
        a = a / torch.sqrt((a * a).mean(1, keepdim=True) + eps) * (w_post + offset)
    if gate is not None:
        a = a * (gate if gate.dim() == 2 else gate[None])
    r = x + scale * a
    er = rel * (scale * a).abs() + 2 * U32 * (x.abs() + (scale * a).abs())
    if w_pre is None:
        return r, er, None, None
    inv = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    h = r * inv * (w_pre + offset)
    # er moves h directly and through the mean of the squares
    stat = ((r.abs() * er).sum(1, keepdim=True) / (r * r).sum(1, keepdim=True).clamp(min=1e-300))
    eh = er * inv * (w_pre + offset).abs() + h.abs() * (rel + stat)
    return r, er, h, eh


# ---- append -----------------------------------------------------------------------

def rotate(x, positions, inv_freq, adjacent):
    """(value, bound): x [T, heads, d] with its leading 2 * len(inv_freq) channels turned."""
    x = f64(x)
    half = len(inv_freq)
    y, e = x.clone(), torch.zeros_like(x)
    if half == 0:
        return y, e
    ang = np.outer(np.asarray(positions, np.float64), np.asarray(inv_freq, np.float64))
    c, s = torch.from_numpy(np.cos(ang))[:, None], torch.from_numpy(np.sin(ang))[:, None]
    i = slice(0, 2 * half, 2) if adjacent else slice(0, half)
    j = slice(1, 2 * half, 2) if adjacent else slice(half, 2 * half)
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    # the half turn in fp32 (2^-25 of [-1, 1], times pi), 2^-32 of a turn cut off, sine and cosine
    # to 2 ulp, two products and a sum: below 2^-21 of |a| + |b|; the 64-bit angles themselves
    # carry 2^-52 of their size
    m = (2.0 ** -21 + torch.from_numpy(np.abs(ang))[:, None] * 2.0 ** -52) * (a.abs() + b.abs())
    e[..., i], e[..., j] = m, m
    return y, e


# ---- attention --------------------------------------------------------------------

def gather(pool, table, seq, lo, n, head):
    """Rows lo..n-1 of one sequence and head, 64-bit, [n - lo, d]; pool is indexed as
    [page, head, slot, d]."""
    page = pool.shape[2]
    j = torch.arange(lo, n)
    t = table[seq, j // page].long().to(pool.device)
    sl = (j % page).to(pool.device)
    if "float8" in str(pool.dtype):
        return pool.view(torch.uint8)[t, head, sl].view(pool.dtype).float().cpu().double()
    return pool[t, head, sl].cpu().double()


def attend(q, k_pages, v_pages, table, lens, scale, softcap=0.0, window=0, k_scale=None, v_scale=None):
    """(out, bound, lse, bound): see moe_kv_attend. table and lens on the host."""
    B, Hq, D = q.shape
    Hk, G = k_pages.shape[1], q.shape[1] // k_pages.shape[1]
    q = f64(q)
    out, eo = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    lse, el = torch.full((B, Hq), -torch.inf, dtype=torch.float64), torch.zeros(B, Hq, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        lo = max(0, n - window) if window else 0
        if n <= 0:
            continue
        for h in range(Hk):
            k = gather(k_pages, table, b, lo, n, h) * (1.0 if k_scale is None else float(k_scale[h]))
            v = gather(v_pages, table, b, lo, n, h) * (1.0 if v_scale is None else float(v_scale[h]))
            qs = q[b, h * G:(h + 1) * G]
            s = qs @ k.T * scale
            # a dot product of D terms, the scale and the conversion to base two
            es = (D + 6) * U32 * (qs.abs() @ k.abs().T * abs(scale))
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                es = es + softcap * 2.0 ** -20
            es = es + 4 * U32 * s.abs()
            es = torch.nan_to_num(es).amax(1, keepdim=True)
            p = torch.softmax(s, 1)
            # weights: twice the scores' error, the exponential (2^-21), their rounding in the
            # product; the sum over n - lo terms
            rel = 2 * es + 2.0 ** -21 + UP + 2 * (n - lo) * U32
            out[b, h * G:(h + 1) * G] = p @ v
            eo[b, h * G:(h + 1) * G] = rel * (p @ v.abs())
            L = torch.logsumexp(s, 1)
            lse[b, h * G:(h + 1) * G] = L
            el[b, h * G:(h + 1) * G] = es[:, 0] + 2.0 ** -21 + (n - lo) * U32 + 4 * U32 * L.abs()
    return out, eo, lse, el
