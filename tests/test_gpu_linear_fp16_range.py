"""Linear attention in fp16 where something leaves fp16's range, or falls below
it, while the operands and the results do not: states, scores, a chunk's decayed
values.  Against the recurrence in 64 bits.

Bounds (u = 2^-11, A = scale sum_j lambda^(i-j) sum_d |q_id k_jd| |v_j| over all
keys and the first state, y: the same sum without q and scale).  Outputs: a
score is held in two parts (2^-21 of its row's largest in the chunk or better,
and every tested row's values are of one size: 32 keys, 2^-16 A), the state's
copy is rounded once (u A), the result once (u of itself; 2^-25 where it is
subnormal), the rest is float32: D products and 72 sums of 2^-24, 2^-22 a chunk
for the powers of lambda, 2^-20 more.  States: float32 terms, 72 sums of 2^-24, 2^-22
a chunk, 2^-21; values below float32's normal range (2^-126) count as nothing."""
import math

import pytest
import torch

import attn_ref as R
import chip_fusion_amd as cf

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def _flush(msg):
    print(f"\n[case] {msg}", flush=True)


def _randn(seed, shape, std=1.0, dtype=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _cu(lens):
    return torch.tensor(R.starts(lens), dtype=torch.int32, device="cuda")


def recurrence(q, k, v, decay, state, scale):
    """One sequence: O, its bound, the state after it and its bound."""
    n, H, D = q.shape
    q, k, v, g = (x.detach().cpu().double() for x in (q, k, v, decay))
    lam = torch.exp(g)[:, None, None]
    x = torch.zeros((H, D, D), dtype=torch.float64) if state is None else state.detach().cpu().double()[0]
    y = x.abs()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    for t in range(n):
        term = k[t][:, :, None] * v[t][:, None, :]
        x, y = lam * x + term, lam * y + term.abs()
        out[t] = scale * (q[t][:, None] @ x)[:, 0]
        A = scale * (q[t].abs()[:, None] @ y)[:, 0]
        rel = (D + 72) * R.E32 + (t // 32 + 1) * 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -16
        bound[t] = (U * (1 + U) + rel) * A + U * out[t].abs() + 2.0 ** -25
    return out, bound, x[None], ((72 * R.E32 + (n // 32 + 1) * 2.0 ** -22 + 2.0 ** -21) * y + 2.0 ** -126)[None]


def _check(what, q, k, v, decay, state, scale=None):
    n, H, D = q.shape
    plan = cf.LinearAttention("f16", H, H, D, scale=scale)
    got, after = plan.run(q, k, v, decay, _cu([n]), state=state)
    torch.cuda.synchronize()
    want, b, ws, bs = recurrence(q, k, v, decay, state, D ** -0.5 if scale is None else scale)
    assert bool((want.abs() < 65504).all())
    R.check(got, want, b, f"{what}: O")
    R.check(after, ws, bs, f"{what}: state")
    return got, after


@pytest.mark.parametrize("D,n", [(64, 400), (128, 900), (64, 1700)])
@pytest.mark.parametrize("zero", ["k", "v"])
def test_states_that_decay_to_nothing(D, n, zero):
    """Hundreds of masked tokens (zero keys or values) after a state: it decays
    through all of float32's range, whole and cut into segments, and on behind
    them tokens count as before."""
    decay = torch.tensor([-0.7, -0.25, -0.06, 0.0], device="cuda")
    _flush(f"decaying state {D} {n} {zero}")
    q, k, v = _randn(1, (n, 4, D)), _randn(2, (n, 4, D), 0.7), _randn(3, (n, 4, D))
    (k if zero == "k" else v)[:n - 20] = 0
    _check("decayed", q, k, v, decay, _randn(4, (1, 4, D, D), 4.0, torch.float32))


@pytest.mark.parametrize("size", [1e-36, 1e-40, 2.0 ** -120, 2.0 ** -149, 1e30])
@pytest.mark.parametrize("n", [40, 600])
def test_states_of_any_size(size, n):
    _flush(f"state of {size}, {n} tokens")
    q, k, v = _randn(1, (n, 2, 64)), torch.zeros((n, 2, 64), dtype=torch.float16, device="cuda"), _randn(3, (n, 2, 64))
    state = torch.full((1, 2, 64, 64), size, device="cuda")
    state[:, :, ::3] = 0
    # (large states: outputs in range, by the scale)
    _check("tiny", q, k, v, torch.tensor([-0.01, -0.3], device="cuda"), state, None if size < 1 else 1e-30)


def test_scores_past_fp16():
    """Scores past 65504 of operands and results that fit."""
    D, n = 128, 100
    decay = torch.tensor([-0.5, -0.02], device="cuda")
    big = torch.full((n, 2, D), 100.0, dtype=torch.float16, device="cuda")
    _flush("scores past fp16: all alike")
    _check("alike", big, big, torch.full_like(big, 0.001), decay, None)
    _flush("scores past fp16: scale 1")
    q, k = _randn(1, (n, 2, D), 30.0), _randn(2, (n, 2, D), 30.0)
    q, k = (x + 25 * torch.sign(x) for x in (q, k))
    k[::2] = q[::2]                                     # large at the token itself
    v = torch.sign(_randn(3, (n, 2, D))) * 0.01
    state = _randn(4, (1, 2, D, D), 0.1, torch.float32)
    got, after = _check("scale 1", q, k, v, decay, state, 1.0)
    # a prompt's first token is what a step gives
    one, s = cf.LinearAttention("f16", 2, 2, D, scale=1.0).step(q[:1], k[:1], v[:1], decay, state)
    want, b, ws, bs = recurrence(q[:1], k[:1], v[:1], decay, state, 1.0)
    R.check(one, want, b)
    R.check(got[:1], want, b)


def test_scores_past_fp16_beside_infinities():
    """The same where a later value is infinite: rows before it, whose scores
    are large, stay right."""
    D, n = 64, 70
    _flush("scores past fp16 beside an infinity")
    q = torch.full((n, 1, D), 200.0, dtype=torch.float16, device="cuda")
    v = torch.full((n, 1, D), 0.001, dtype=torch.float16, device="cuda")
    decay = torch.tensor([-1.0], device="cuda")
    want, b, _, _ = recurrence(q, q, v, decay, None, 0.125)
    v[50, 0, 7] = math.inf
    got, after = cf.LinearAttention("f16", 1, 1, D).run(q, q, v, decay, _cu([n]))
    torch.cuda.synchronize()
    assert not torch.isfinite(got[50:, 0, 7]).any() and not torch.isfinite(after[0, 0, :, 7]).any()
    keep = torch.ones((n, 1, D), dtype=torch.bool)
    keep[50:, 0, 7] = False
    # (the careful pass takes each score's first part alone: U of A more)
    R.check(got.cpu()[keep], want[keep], (b + U * want.abs())[keep])


def test_zero_queries_on_large_states():
    """Rows of zeros stay zeros, however large the state is."""
    _flush("zero queries")
    q, k, v = (torch.zeros((40, 2, 64), dtype=torch.float16, device="cuda") for _ in range(3))
    k[20:], v[20:] = 1.0, 2.0
    state = _randn(4, (1, 2, 64, 64), 1e38, torch.float32).clamp(-3e38, 3e38)
    for scale in (None, 1e6):
        got, _ = cf.LinearAttention("f16", 2, 2, 64, scale=scale).run(q, k, v, torch.tensor([0.0, -0.1], device="cuda"),
                                                                      _cu([40]), state=state)
        torch.cuda.synchronize()
        assert bool((got == 0).all())


def test_scores_below_fp16():
    """Scores of 2^-20 and below with values of thousands."""
    D, n = 64, 100
    decay = torch.tensor([-0.5, -0.02], device="cuda")
    for std in (1e-3, 1e-4):
        _flush(f"scores below fp16: {std}")
        q, k = _randn(1, (n, 2, D), std), _randn(2, (n, 2, D), std)
        k[::2] = q[::2]
        v = torch.sign(_randn(3, (n, 2, D))) * 30000.0
        _check("small scores", q, k, v, decay, None)


@pytest.mark.parametrize("D,n", [(64, 43), (128, 64 + 11), (64, 1600)])
@pytest.mark.parametrize("rate", [-0.3, -0.7, -2.0])
def test_terms_that_decay_within_a_chunk(D, n, rate):
    """Tokens early in a chunk whose others are masked: their terms are small
    at its end, and the state, which is float32, holds nothing else."""
    _flush(f"decayed terms {D} {n} {rate}")
    q, k, v = _randn(1, (n, 2, D)), _randn(2, (n, 2, D), 0.7), _randn(3, (n, 2, D))
    decay = torch.tensor([rate, rate / 2], device="cuda")
    at = torch.arange(n, device="cuda")
    masked = at % 32 >= 11
    masked[:n // 3] = False
    masked[-10:] = True                               # and none behind them
    v[masked] = 0
    _check("masked", q, k, v, decay, None)


@pytest.mark.parametrize("n", [50, 1100])
def test_small_values(n):
    """Values near fp16's smallest: a decayed one still has float32's bits."""
    _flush(f"small values {n}")
    q, k, v = _randn(1, (n, 2, 64)), _randn(2, (n, 2, 64), 0.7), _randn(3, (n, 2, 64), 1e-5)
    _check("small", q, k, v, torch.tensor([-0.2, -0.03], device="cuda"), None)
