"""The attention operators' definitions in 64 bits (CPU), with error bounds of
the kernels' arithmetic for the tests.

Bounds.  u is half a step of the type (2^-8 bf16, 2^-11 fp16).  Products of
16-bit values are exact in float32; a score sums D of them and is off by at
most D 2^-24 scale sum_d |q_d k_d|, which changes a probability by that
relative amount twice (numerator and the row's sum).  Every probability is
then rounded to the type once (u relative; fp16 below 2^-14: 2^-25 of the row's
largest, which is 1 or more), the sums over the keys are float32 (2^-24 a term),
and the result is rounded once (u of itself).
"""
import itertools
import math

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E32 = 2.0 ** -24


def starts(lens):
    return [0] + list(itertools.accumulate(lens))


def attention(q, k, v, cu_q, cu_k, causal, scale):
    """O, LSE and O's and LSE's bounds; rows outside every sequence are NaN."""
    dt = q.dtype
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    D = q.shape[2]
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    bound = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], math.nan, dtype=torch.float64)
    lse_bound = torch.zeros(q.shape[:2], dtype=torch.float64)
    u = U[dt]
    for s in range(len(cu_q) - 1):
        n, m = cu_q[s + 1] - cu_q[s], cu_k[s + 1] - cu_k[s]
        rows = slice(cu_q[s], cu_q[s + 1])
        if n <= 0:
            continue
        Q = q[rows].transpose(0, 1)
        K = k[cu_k[s]:cu_k[s + 1]].transpose(0, 1).repeat_interleave(G, 0)
        V = v[cu_k[s]:cu_k[s + 1]].transpose(0, 1).repeat_interleave(G, 0)
        see = torch.ones((n, m), dtype=torch.bool)
        if causal:
            see = see.tril(m - n)
        x = (Q @ K.transpose(1, 2) * scale).masked_fill(~see, -math.inf)
        top = x.amax(-1, keepdim=True) if m else torch.full((H, n, 1), -math.inf, dtype=torch.float64)
        p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        l = p.sum(-1, keepdim=True)
        w = p / torch.where(l == 0, 1.0, l)
        V0 = torch.where(see.any(0)[:, None], V, 0.0) if m else V
        o = w @ V0
        # errors
        ds = (D + 4) * E32 * scale * (Q.abs() @ K.abs().transpose(1, 2)) if m else torch.zeros((H, n, 0))
        ds = torch.where(see, ds, 0.0).amax(-1, keepdim=True) if m else torch.zeros((H, n, 1))
        rel = 2 * ds + (m + 16) * E32 + 2 * torch.where(top == -math.inf, 0.0, top).abs() * 2.0 ** -23
        tiny = 2.0 ** -25 * (see.double() @ V0.abs()) if dt == torch.float16 else 0.0
        e = (u + rel) * (w @ V0.abs()) + tiny + u * (1 + u) * o.abs() + 2 * u * u * (w @ V0.abs()) + 2.0 ** -24
        out[rows], bound[rows] = o.transpose(0, 1), e.transpose(0, 1)
        ls = torch.where(l > 0, torch.log(l) + top, -math.inf)[..., 0]
        lse[rows] = ls.T
        lse_bound[rows] = (rel[..., 0] + 4 * 2.0 ** -23 * (1 + torch.where(ls == -math.inf, 0.0, ls).abs())).T
    return out, lse, bound, lse_bound


def check(got, want, bound, what=""):
    """Every value within its bound, infinities and NaN in the same places."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    odd = ~torch.isfinite(want)
    same = torch.isnan(want) & torch.isnan(got) | (want == got)
    assert bool(same[odd].all()), f"{what}: infinities or NaN differ"
    d = (got - want).abs()
    bad = ~odd & ~(d <= bound)
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, first at {at}: "
                             f"{float(got[at])} for {float(want[at])} +- {float(bound[at]):.3e}")
