"""Attention under a window and over pages, and norms with rotation: the
definitions in 64 bits (CPU), with error bounds of the kernels' arithmetic.

Attention's bounds are attn_ref's: half a step of the type for every
probability and for the result, float32 sums, scores off by D 2^-24 of their
terms' sizes.  Partial results are float32, joined by weights 2^x with x off by
2^-23 of itself: within the same terms.

Norms and rotation: float32 throughout, rounded once.  The sum of D squares is
off by D 2^-24, its root by half of that and 2^-23 (v_rsq_f32), three products and the
sum of two by 2^-24 each; cosine and sine are off by 4 2^-24 (of 1), the angle
by 2^-24 of a turn; so an element of a pair (a, b) is off by (D / 2 + 8) 2^-24
(|a| + |b|) and 2^-22 pi (|a| + |b|), and by half a step of the type of itself
(subnormal float16: of 2^-14).
"""
import math

import torch

from attn_ref import E32, U, check, starts      # noqa: F401


def attend(q, k, v, lq, lk, window=None, sinks=0, scale=None):
    """Packed sequences of lq rows and lk keys, causal: O, LSE and their bounds."""
    dt = q.dtype
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    H, G, D = q.shape[1], q.shape[1] // k.shape[1], q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, bound = torch.full(q.shape, math.nan, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse, lse_bound = torch.full(q.shape[:2], math.nan, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    u, q0, k0 = U[dt], 0, 0
    for n, m in zip(lq, lk):
        rows = slice(q0, q0 + n)
        q0, at, k0 = q0 + n, k0, k0 + m
        if n == 0:
            continue
        if m == 0:
            out[rows], lse[rows] = 0.0, -math.inf
            continue
        Q = q[rows].transpose(0, 1)
        K, V = (x[at:at + m].transpose(0, 1).repeat_interleave(G, 0) for x in (k, v))
        p, j = torch.arange(m - n, m)[:, None], torch.arange(m)
        see = j <= p
        if window is not None:
            see = see & ((j > p - window) | (j < sinks))
        x = (Q @ torch.where(see.any(0)[:, None], K, 0.0).transpose(1, 2) * scale).masked_fill(~see, -math.inf)
        top = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        l = e.sum(-1, keepdim=True)
        w = e / torch.where(l == 0, 1.0, l)
        fin = torch.where(torch.isfinite(V), V, 0.0)
        o = w @ fin
        # infinities and NaN reach the rows that see them
        for bad in (math.inf, -math.inf, math.nan):
            is_bad = torch.isnan(V) if math.isnan(bad) else V == bad
            if bool(is_bad.any()):
                hit = (see.double().expand(H, n, m) @ is_bad.double()) > 0
                o = o + torch.where(hit, bad, 0.0)
        size = w @ fin.abs()
        ds = (D + 4) * E32 * scale * (Q.abs() @ torch.where(see.any(0)[:, None], K, 0.0).abs().transpose(1, 2))
        ds = torch.where(see, ds, 0.0).amax(-1, keepdim=True)
        rel = 2 * ds + (m + 16) * E32 + 2 * torch.where(top == -math.inf, 0.0, top).abs() * 2.0 ** -23
        tiny = 2.0 ** -25 * (see.double() @ fin.abs()) if dt == torch.float16 else 0.0
        of = torch.where(torch.isfinite(o), o, 0.0).abs()
        b = (u + rel) * size + tiny + u * (1 + u) * of + 2 * u * u * size + 2.0 ** -24
        out[rows], bound[rows] = o.transpose(0, 1), b.transpose(0, 1)
        ls = torch.where(l > 0, torch.log(l) + top, -math.inf)[..., 0]
        lse[rows] = ls.T
        lse_bound[rows] = (rel[..., 0] + 4 * 2.0 ** -23 * (1 + torch.where(ls == -math.inf, 0.0, ls).abs())).T
    return out, lse, bound, lse_bound


def gather(cache, table, lens):
    """The keys of all sequences, side by side, from the pages of a cache."""
    cache, table, size = cache.detach().cpu(), table.cpu().tolist(), cache.shape[1]
    rows = [cache[table[s][j // size], j % size] for s, n in enumerate(lens) for j in range(n)]
    return torch.stack(rows) if rows else cache.new_zeros((0,) + tuple(cache.shape[2:]))


def norm_rotary(x, weight, positions, rotary, freqs, axes_of=None, interleaved=False, eps=1e-6):
    """x [rows, heads, dim]; positions [axes, rows]: the result and its bound."""
    dt, D = x.dtype, x.shape[-1]
    y = x.detach().cpu().double()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.detach().cpu().double()
    pairs = rotary // 2
    axes_of = [0] * pairs if axes_of is None else axes_of
    out, size = y.clone(), y.abs().clone()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        t = positions[axes_of[i]].cpu().double() * freqs[i]
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    u = U[dt]
    bound = ((D / 2 + 12) * E32 + math.pi * 2.0 ** -22) * size * (1 + u) + u * out.abs()
    if dt == torch.float16:
        bound = torch.maximum(bound, bound - u * out.abs() + 2.0 ** -25)
    return out, bound


def default_freqs(rotary, base=10000.0):
    return [base ** (-2.0 * i / rotary) for i in range(rotary // 2)]
