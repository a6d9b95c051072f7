"""Attention whose keys are split over workgroups (partial results joined by a
second kernel) against the definition in 64 bits: what the join may write."""
import ctypes
import math

import pytest
import torch

import attn_ref as R
import chip_fusion_amd as cf

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _flush(msg):
    print(f"\n[case] {msg}", flush=True)


def _randn(seed, shape, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _at(starts):
    return torch.tensor(starts, dtype=torch.int32, device="cuda")


def _is_split(plan, seqs, rows, keys):
    n = ctypes.c_size_t()
    assert cf.lib().b2b_attn_workspace(plan._h, seqs, rows, keys, ctypes.byref(n)) == 0
    return n.value > 0


def _many(n):
    """Starts of n sequences of 0, 1 or 2 rows behind three rows of nobody's."""
    at = [3]
    for i in range(n):
        at.append(at[-1] + (0, 1, 2, 1)[i % 4])
    return at


CASES = [
    # dtype, heads, kv heads, dim, rows, their starts, keys, their starts, causal
    ("bf16", 4, 2, 64, 40, [5, 25], 2300, [0, 2300], True),
    ("f16", 4, 1, 96, 40, [0, 25], 2300, [100, 2100], False),
    ("bf16", 32, 8, 128, 128, [0, 77], 4096, [0, 4096], True),        # a padded batch of one
    ("f16", 3, 3, 72, 50, [25, 35, 5, 15], 3000, [0, 900, 900, 3000], False),    # starts out of order, rows between
    ("f16", 2, 1, 64, 30, [30, 30], 2000, [0, 2000], True),           # all rows are nobody's
    ("bf16", 1, 1, 64, 140, _many(130), 70000, [530 * i for i in range(131)], True),   # more sequences than lanes
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_outside_the_sequences_stay(case):
    """Rows of O and of the log-sum-exp that belong to no sequence keep what
    they hold, and the others are right, where keys are split as where not."""
    dtype, H, Hkv, D, rows, cu_q, keys, cu_k, causal = CASES[case]
    _flush(f"split, rows outside {CASES[case][:5]} causal {causal}")
    q, k, v = _randn(1, (rows, H, D), DT[dtype], 1.5), _randn(2, (keys, Hkv, D), DT[dtype]), _randn(3, (keys, Hkv, D), DT[dtype])
    plan = cf.Attention(dtype, H, Hkv, D, causal=causal)
    assert _is_split(plan, len(cu_q) - 1, rows, keys)
    O, lse = torch.full_like(q, 7.0), torch.full((rows, H), 7.0, device="cuda")
    plan.run(q, k, v, _at(cu_q), _at(cu_k), O=O, lse=lse)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attention(q, k, v, cu_q, cu_k, causal, D ** -0.5)
    live = torch.zeros(rows, dtype=torch.bool)
    for s in range(len(cu_q) - 1):
        live[cu_q[s]:cu_q[s + 1]] = True
    assert bool((O.cpu()[~live] == 7.0).all()) and bool((lse.cpu()[~live] == 7.0).all())
    # joining parts: a few more roundings in 32 bits
    R.check(O.cpu()[live], want[live], b[live] + 2.0 ** -20 * want[live].abs(), "O")
    R.check(lse.cpu()[live], want_lse[live], bl[live] + 2.0 ** -20, "LSE")
    O2 = torch.full_like(q, 7.0)
    plan.run(q, k, v, _at(cu_q), _at(cu_k), O=O2)               # without a log-sum-exp
    assert torch.equal(O2, O)


def test_graph_replays_with_fewer_rows():
    """A captured call whose keys are split, replayed with sequences that fill
    fewer rows than the tensors have: the others stay, replay after replay."""
    H, Hkv, D, rows, keys = 4, 1, 128, 20, 2100
    plan = cf.Attention("bf16", H, Hkv, D)
    assert _is_split(plan, 2, rows, keys)
    q, k, v = _randn(1, (rows, H, D), torch.bfloat16, 1.5), _randn(2, (keys, Hkv, D), torch.bfloat16), \
        _randn(3, (keys, Hkv, D), torch.bfloat16)
    cu_q, cu_k, O = _at([0, 17, 20]), _at([0, 1200, 2100]), torch.full_like(q, 7.0)
    _flush("split graph, fewer rows")
    plan.run(q, k, v, cu_q, cu_k, O=O)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run(q, k, v, cu_q, cu_k, O=O)
    for a, b in [([0, 17, 20], [0, 1200, 2100]), ([0, 5, 12], [0, 900, 2000]), ([2, 2, 3], [0, 0, 2100]), ([4, 4, 4], [0, 5, 9])]:
        cu_q.copy_(_at(a)), cu_k.copy_(_at(b)), O.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want, _, bound, _ = R.attention(q, k, v, a, b, True, D ** -0.5)
        lo, hi = a[0], a[-1]
        R.check(O[lo:hi], want[lo:hi], bound[lo:hi] + 2.0 ** -20 * want[lo:hi].abs())
        assert bool((O[:lo] == 7.0).all()) and bool((O[hi:] == 7.0).all())


@pytest.mark.parametrize("dtype,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_infinities_of_little_weight_stay(dtype, D, causal):
    """An infinite value among keys whose weight is far below float32's range
    beside another part's (their scores differ by 300): its column is infinite
    as the definition has it, whichever part comes first."""
    n, keys, H = 9, 3000, 2
    for at, big in ((10, keys - 40), (keys - 40, 10)):
        _flush(f"infinity of little weight {dtype} {D} {causal} {at}")
        q = torch.ones((n, H, D), dtype=DT[dtype], device="cuda")
        k, v = torch.zeros((keys, H, D), dtype=DT[dtype], device="cuda"), _randn(3, (keys, H, D), DT[dtype])
        k[big] = 300.0 / D
        v[at, 0, 5], v[at, 1, 3], v[at, 1, 4] = math.inf, -math.inf, math.nan
        plan = cf.Attention(dtype, H, H, D, causal=causal, scale=1.0)
        assert _is_split(plan, 1, n, keys)
        got = plan.run(q, k, v, _at([0, n]), _at([0, keys]))
        torch.cuda.synchronize()
        want, _, b, _ = R.attention(q, k, torch.where(torch.isfinite(v), v, 0.0), [0, n], [0, keys], causal, 1.0)
        want[:, 0, 5], want[:, 1, 3], want[:, 1, 4] = math.inf, -math.inf, math.nan
        R.check(got, want, b + 2.0 ** -20)


def test_infinities_of_little_weight_in_a_prefix_stay():
    H, D, P, S, T = 2, 64, 1000, 40, torch.bfloat16
    _flush("infinity of little weight, prefix")
    q, k = torch.ones((3, H, D), dtype=T, device="cuda"), torch.zeros((3, S, H, D), dtype=T, device="cuda")
    k[:, 7] = 300.0 / D
    kp, vp, v = torch.zeros((P, H, D), dtype=T, device="cuda"), _randn(2, (P, H, D), T), _randn(3, (3, S, H, D), T)
    vp[500, 0, 5], vp[20, 1, 7] = math.inf, -math.inf
    lens = _at([S, 0, 8])
    got = cf.PrefixAttention("bf16", H, H, D, scale=1.0).run(q, kp, vp, k, v, lens)
    torch.cuda.synchronize()
    odd = ~torch.isfinite(got)
    assert bool(odd[:, 0, 5].all()) and bool(odd[:, 1, 7].all()) and int(odd.sum()) == 6
