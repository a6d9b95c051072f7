"""Attention over packed sequences and behind a shared prefix against the
definition in 64 bits, at the sizes, masks and layouts where it can go wrong."""
import itertools
import math
import sys

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


def _cu(lens):
    return torch.tensor(R.starts(lens), dtype=torch.int32, device="cuda")


def _case(dtype, heads, kv, dim, lq, lk, seed=1, std=1.5):
    T = DT[dtype]
    q = _randn(seed, (sum(lq), heads, dim), T, std)
    k = _randn(seed + 1, (sum(lk), kv, dim), T)
    v = _randn(seed + 2, (sum(lk), kv, dim), T)
    return q, k, v


CASES = [
    # dtype, heads, kv heads, dim, query lengths, key lengths, causal
    ("f16", 1, 1, 64, [1], [1], True),
    ("bf16", 2, 1, 8, [3, 1], [3, 1], True),
    ("f16", 4, 4, 40, [63, 64, 65], [63, 64, 65], True),
    ("bf16", 4, 2, 64, [127, 0, 1, 129, 2], [127, 0, 1, 129, 2], True),
    ("f16", 6, 2, 72, [31, 33], [95, 97], True),              # pieces behind earlier keys
    ("bf16", 8, 1, 80, [5, 70], [64, 71], False),
    ("f16", 3, 1, 96, [100], [300], True),
    ("bf16", 5, 5, 128, [257], [257], True),
    ("f16", 8, 2, 128, [300, 20], [300, 20], False),
    ("bf16", 8, 2, 128, [40, 9], [12, 0], True),              # more rows than keys: the first see none
    ("f16", 2, 2, 64, [50, 3], [0, 7], False),                # a sequence without keys
    ("f16", 24, 2, 112, [17], [1500], True),                  # few rows, many keys: split
    ("bf16", 2, 2, 128, [260], [2100], False),
    ("f16", 4, 1, 64, [600], [600], True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case):
    dtype, H, Hkv, D, lq, lk, causal = CASES[case]
    _flush(f"attention {CASES[case]}")
    q, k, v = _case(dtype, H, Hkv, D, lq, lk)
    O = torch.full_like(q, math.nan)
    plan = cf.Attention(dtype, H, Hkv, D, causal=causal)
    got, lse = plan.run(q, k, v, _cu(lq), _cu(lk), O=O, lse=True)
    assert got is O
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attention(q, k, v, R.starts(lq), R.starts(lk), causal, D ** -0.5)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")
    again = plan.run(q, k, v, _cu(lq), _cu(lk))
    assert torch.equal(again, got)          # the same values on every run


@pytest.mark.parametrize("seqs", [1, 65, 200])
def test_many_sequences(seqs):
    """More sequences than a wave scans at once, empty ones among them."""
    lens = [(7 * i) % 23 for i in range(seqs)]
    _flush(f"attention {seqs} sequences")
    q, k, v = _case("bf16", 4, 2, 64, lens, lens, seed=11)
    got = cf.Attention("bf16", 4, 2, 64).run(q, k, v, _cu(lens))
    torch.cuda.synchronize()
    want, _, b, _ = R.attention(q, k, v, R.starts(lens), R.starts(lens), True, 0.125)
    R.check(got, want, b)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("seqs", [40, 64])
def test_sequences_of_all_sizes(causal, seqs):
    """Every tile of every sequence is taken, in whatever order they start: rows
    and keys of very different numbers, more rows than keys among them."""
    lq = [(37 * i * i) % 241 if i % 5 else 0 for i in range(seqs)]
    lk = [(53 * i) % 401 if i % 7 else 0 for i in range(seqs)]
    _flush(f"attention {seqs} sequences of all sizes, causal {causal}")
    q, k, v = _case("f16", 6, 2, 40, lq, lk, seed=13)
    O = torch.full_like(q, math.nan)
    got, lse = cf.Attention("f16", 6, 2, 40, causal=causal).run(q, k, v, _cu(lq), _cu(lk), O=O, lse=True)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attention(q, k, v, R.starts(lq), R.starts(lk), causal, 40 ** -0.5)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")


@pytest.mark.parametrize("scale", [None, 0.02, 3.0])
def test_scale_and_large_scores(scale):
    """Scores from nearly equal to one key taking all of the weight."""
    _flush(f"attention scale {scale}")
    q, k, v = _case("bf16", 2, 2, 64, [150], [150], seed=21, std=8.0)
    got, lse = cf.Attention("bf16", 2, 2, 64, scale=scale).run(q, k, v, _cu([150]), lse=True)
    torch.cuda.synchronize()
    want, wl, b, bl = R.attention(q, k, v, [0, 150], [0, 150], True, 0.125 if scale is None else scale)
    R.check(got, want, b)
    R.check(lse, wl, bl)


def test_rising_scores_move_the_maximum():
    """Keys in rising order of their scores: the running maximum moves in every
    tile, by less and by more than the lag that is allowed."""
    for step in (0.2, 3.0):
        _flush(f"attention rising by {step}")
        n = 400
        q = torch.ones((n, 1, 64), dtype=torch.float16, device="cuda")
        k = (torch.arange(n, device="cuda").float()[:, None, None] * (step / 64)).expand(n, 1, 64).half().contiguous()
        v = _randn(5, (n, 1, 64), torch.float16)
        got, lse = cf.Attention("f16", 1, 1, 64, causal=False, scale=1.0).run(q, k, v, _cu([n]), lse=True)
        torch.cuda.synchronize()
        want, wl, b, bl = R.attention(q, k, v, [0, n], [0, n], False, 1.0)
        R.check(got, want, b)
        R.check(lse, wl, bl)


def test_layouts():
    """Slices of a fused projection, head-major storage, padded rows."""
    H, Hkv, D, n = 6, 2, 64, 140
    cu = _cu([100, 40])
    fused = _randn(31, (n, (H + 2 * Hkv) * D + 24), torch.float16)
    q, k, v = (fused[:, a * D:b * D].view(n, b - a, D) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    plan = cf.Attention("f16", H, Hkv, D)
    want = plan.run(q.contiguous(), k.contiguous(), v.contiguous(), cu)
    _flush("attention layouts: fused projection")
    assert torch.equal(plan.run(q, k, v, cu), want)
    _flush("attention layouts: head-major")
    hm = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    O = torch.full((H, n, D), math.nan, dtype=torch.float16, device="cuda").transpose(0, 1)
    assert plan.run(hm(q), hm(k), hm(v), cu, O=O) is O
    assert torch.equal(O, want)
    ref, _, b, _ = R.attention(q, k, v, [0, 100, 140], [0, 100, 140], True, 0.125)
    R.check(want, ref, b)


def test_offsets_past_32_bits():
    """Keys and values whose rows, and whose requests, lie gigabytes apart."""
    H, D, n, far = 2, 64, 2200, 1 << 20
    T = torch.bfloat16
    q, k, v = _case("bf16", H, 1, D, [5], [n], seed=17)
    room = torch.zeros((n * far,), dtype=T, device="cuda")           # 4.6 GB; K and V in turn along its rows
    K, V = room.as_strided((n, 1, D), (far, D, 1)), room.as_strided((n, 1, D), (far, D, 1), far // 2)
    K.copy_(k), V.copy_(v)
    _flush("attention far rows")
    got = cf.Attention("bf16", H, 1, D).run(q, K, V, _cu([5]), _cu([n]))
    torch.cuda.synchronize()
    want, _, b, _ = R.attention(q, k, v, [0, 5], [0, n], True, D ** -0.5)
    R.check(got, want, b)
    _flush("prefix far requests")
    B, S = 11, 200                                                    # request i from row 200 i on
    K4, V4 = K[:B * S].as_strided((B, S, 1, D), (S * far, far, D, 1)), V.as_strided((B, S, 1, D), (S * far, far, D, 1))
    q = _randn(3, (B, H, D), T, 1.5)
    lens = torch.full((B,), S, dtype=torch.int32, device="cuda")
    got = cf.PrefixAttention("bf16", H, 1, D).run(q, k[:3], v[:3], K4, V4, lens)
    torch.cuda.synchronize()
    ks = torch.cat([torch.cat([k[:3], k[i * S:(i + 1) * S]]) for i in range(B)])
    vs = torch.cat([torch.cat([v[:3], v[i * S:(i + 1) * S]]) for i in range(B)])
    want, _, b, _ = R.attention(q, ks, vs, list(range(B + 1)), R.starts([S + 3] * B), False, D ** -0.5)
    R.check(got, want, b + 2.0 ** -20 * want.abs())


def test_rows_outside_the_sequences_stay():
    """Rows behind the last sequence are neither read as keys nor written,
    whatever they hold; starts past the tensors are clamped."""
    q, k, v = _case("bf16", 4, 2, 64, [90], [90], seed=41)
    for x in (q, k, v):
        x[60:] = math.nan
    O = torch.full_like(q, 7.0)
    _flush("attention rows outside")
    plan = cf.Attention("bf16", 4, 2, 64, causal=False)
    plan.run(q, k, v, _cu([20, 40]), O=O)
    torch.cuda.synchronize()
    want, _, b, _ = R.attention(q[:60], k[:60], v[:60], [0, 20, 60], [0, 20, 60], False, 0.125)
    R.check(O[:60], want, b)
    assert bool((O[60:] == 7.0).all())
    got = plan.run(q[:60], k[:60], v[:60], torch.tensor([0, 20, 1 << 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, O[:60])


def test_starts_and_lengths_are_clamped():
    """Starts below 0 and past the rows, lengths below 0 and past the own keys:
    as if they were the nearest that fit, and nothing outside is touched."""
    H, Hkv, D, n = 4, 2, 64, 300
    T = torch.float16
    q, k, v = _case("f16", H, Hkv, D, [n], [n], seed=91)
    O = torch.full((n + 40, H, D), 7.0, dtype=T, device="cuda")
    at = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    _flush("starts clamped")
    plan = cf.Attention("f16", H, Hkv, D)
    plan.run(q, k, v, at([-9, 100, 90, 2 * n]), at([-1, 120, 2 * n, 1 << 30]), O=O[:n])
    # 0..100 on keys 0..120; none on the rest; 90.. has no keys left
    want = plan.run(q, k, v, at([0, 100, 100, 100]), at([0, 120, 120, 120]))
    torch.cuda.synchronize()
    assert torch.equal(O[:90], want[:90]) and bool((O[100:n] == 0).all()) and bool((O[n:] == 7).all())
    B, S = 3, 20
    q, k, v = _randn(1, (B, H, D), T), _randn(2, (B, S, Hkv, D), T), _randn(3, (B, S, Hkv, D), T)
    e = k[0, :0]
    plan = cf.PrefixAttention("f16", H, Hkv, D)
    _flush("lengths clamped")
    got = plan.run(q, e, e, k, v, at([-5, S + 100, 7]))
    want = plan.run(q, e, e, k, v, at([0, S, 7]))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool((got[0] == 0).all())


def test_nan_and_infinities_where_they_are_seen():
    """A NaN among a row's keys makes that row NaN and no other; a query's NaN
    its own row; an infinite score ends in NaN as the definition does."""
    q, k, v = _case("f16", 2, 2, 64, [100], [100], seed=51)
    q[70, 0, 3] = math.nan
    k[40, 1] = math.nan
    _flush("attention NaN")
    got = cf.Attention("f16", 2, 2, 64).run(q, k, v, _cu([100]))
    torch.cuda.synchronize()
    nan = torch.isnan(got).any(-1)
    assert nan[70, 0] and int(nan[:, 0].sum()) == 1
    assert not nan[:40, 1].any() and bool(nan[40:, 1].all())


@pytest.mark.parametrize("dtype,D,n,keys", [("f16", 72, 150, 150), ("bf16", 128, 150, 150), ("bf16", 64, 40, 3000)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(dtype, D, n, keys):
    """Infinities and NaN among the values: rows before them in the same tile
    stay finite, rows that see them get them (both signs: NaN)."""
    q, k, v = _case(dtype, 4, 2, D, [n], [keys], seed=55)
    old = keys - n                  # keys before the first row's own
    v[old + 33, 0, 5], v[old + 37, 0, 5] = math.inf, -math.inf
    v[old + 20, 1, 56], v[keys - 1, 1, 0], v[old, 1, 7] = -math.inf, math.nan, math.inf
    _flush(f"attention odd values {dtype} {n} {keys}")
    got = cf.Attention(dtype, 4, 2, D).run(q, k, v, _cu([n]), _cu([keys]))
    torch.cuda.synchronize()
    odd = ~torch.isfinite(v)
    want, _, b, _ = R.attention(q, k, torch.where(odd, 0.0, v), [0, n], [0, keys], True, D ** -0.5)
    for h in range(4):
        for j, d in odd[:, h // 2].nonzero().tolist():
            want[max(j - old, 0):, h, d] += v[j, h // 2, d].double().cpu()
    R.check(got, want, b)


def test_calls_in_python_and_compiled_agree():
    """The same checks and results whether the compiled binding takes a call or
    the one in Python does (here: because a stream is named); no references are
    kept or lost."""
    H, Hkv, D, n = 4, 2, 64, 70
    T = torch.bfloat16
    q, k, v = _case("bf16", H, Hkv, D, [n], [n], seed=23)
    cu, lens = _cu([n]), torch.tensor([5, 0, 9], dtype=torch.int32, device="cuda")
    k4, v4 = _randn(4, (3, 9, Hkv, D), T), _randn(5, (3, 9, Hkv, D), T)
    g = torch.full((H,), -0.1, device="cuda")
    s1, s3 = _randn(6, (1, H, D, D), torch.float32), _randn(7, (3, H, D, D), torch.float32)
    pa, pp, pl = cf.Attention("bf16", H, Hkv, D), cf.PrefixAttention("bf16", H, Hkv, D), cf.LinearAttention("bf16", H, Hkv, D)
    calls = [lambda **x: pa.run(q, k, v, cu, **x), lambda **x: pa.run(q, k, v, cu, cu, lse=True, **x),
             lambda **x: pa.run(q[:3], k, v, _cu([3]), cu, O=torch.empty_like(q[:3]), **x),
             lambda **x: pp.run(q[:3], k, v, k4, v4, lens, **x),
             lambda **x: pl.run(q, k, v, g, cu, **x), lambda **x: pl.run(q, k, v, g, cu, state=s1, **x),
             lambda **x: pl.step(q[:3], k[:3], v[:3], g, s3, **x)]
    _flush("both bindings")
    here = torch.cuda.current_stream()
    for call in calls:
        a, b = call(), call(stream=here)
        a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
        assert len(a) == len(b) and all(torch.equal(x, y) and x.stride() == y.stride() for x, y in zip(a, b))
    assert pa._usual.attention(q, k, v, cu, None, None, False) is not None
    assert pp._usual.prefix(q[:3], k, v, k4, v4, lens, None) is not None
    assert pl._usual.linear(q, k, v, g, cu, s1, None, None) is not None
    assert pl._usual.linear_step(q[:3], k[:3], v[:3], g, s3, None, None) is not None
    held = [q, k, v, cu, k4, v4, lens, g, s1, s3, torch.float32, pa, pp, pl]
    before = [sys.getrefcount(x) for x in held]
    for _ in range(50):
        for call in calls:
            call()
    assert [sys.getrefcount(x) for x in held] == before
    for bad, match in [(dict(Q=q.half()), "Q: dtype"), (dict(K=k[:, :1]), "K: shape"), (dict(V=v[1:]), "V: shape"),
                       (dict(cu_q=cu.long()), "cu_q"), (dict(O=q[:, :, :32]), "O: shape"), (dict(cu_k=_cu([1, 2])), "cu_k"),
                       (dict(V=v.cpu()), "V: a device")]:
        with pytest.raises(ValueError, match=match):
            pa.run(**{**dict(Q=q, K=k, V=v, cu_q=cu), **bad})
    with pytest.raises(cf.B2BError):
        pa.run(q, k, v, cu, O=q)                  # O at Q's address
    pa.close()
    with pytest.raises(cf.B2BError):
        pa.run(q, k, v, cu)
    torch.cuda.synchronize()


def test_empty_calls():
    plan = cf.Attention("f16", 2, 2, 64)
    e = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    assert plan.run(e, e, e, _cu([])).shape == (0, 2, 64)
    q = _randn(1, (5, 2, 64), torch.float16)
    out, lse = plan.run(q, e, e, _cu([5]), _cu([0]), lse=True)       # rows without any key
    torch.cuda.synchronize()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_graph_replays_and_streams():
    """Captured twice (each graph with its own workspace) and replayed with new
    values and new lengths in turn; then two streams at once."""
    H, Hkv, D = 4, 1, 128
    plan = cf.Attention("bf16", H, Hkv, D)
    lq, lk = [17, 3], [1200, 900]             # split over keys: uses a workspace
    q, k, v = _case("bf16", H, Hkv, D, lq, lk, seed=61)
    cu_q, cu_k = _cu(lq), _cu(lk)
    _flush("attention graph")
    plan.run(q, k, v, cu_q, cu_k)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(plan.run(q, k, v, cu_q, cu_k))
        graphs.append(g)
    for rep, (a, b) in enumerate([(lq, lk), ([10, 10], [800, 1300]), ([0, 20], [1, 2099])]):
        q2, k2, v2 = _case("bf16", H, Hkv, D, a, b, seed=70 + rep)
        q.copy_(q2), k.copy_(k2), v.copy_(v2), cu_q.copy_(_cu(a)), cu_k.copy_(_cu(b))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = plan.run(q2, k2, v2, _cu(a), _cu(b))
        for o in outs:
            assert torch.equal(o, want), rep
    _flush("attention two streams")
    sets = [_case("bf16", H, Hkv, D, lq, lk, seed=80 + i) for i in range(2)]
    want = [plan.run(*x, _cu(lq), _cu(lk)) for x in sets]
    cq, ck = _cu(lq), _cu(lk)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [plan.run(*x, cq, ck, stream=s) for _ in range(3) for x, s in zip(sets, streams)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


PREFIX = [
    # dtype, heads, kv heads, dim, batch, prefix, own keys
    ("f16", 1, 1, 64, 1, 1, 1),
    ("bf16", 4, 2, 128, 3, 100, 20),
    ("f16", 32, 8, 96, 9, 700, 300),
    ("bf16", 40, 1, 80, 5, 33, 1),           # more heads a key head than a row tile holds
    ("f16", 8, 8, 64, 130, 2000, 65),
    ("bf16", 6, 3, 128, 2, 0, 50),           # no prefix
    ("f16", 6, 3, 120, 4, 65, 0),            # nothing but the prefix
    ("bf16", 16, 4, 128, 7, 5000, 1030),
]


@pytest.mark.parametrize("case", range(len(PREFIX)))
def test_prefix_attention(case):
    dtype, H, Hkv, D, B, P, S = PREFIX[case]
    _flush(f"prefix {PREFIX[case]}")
    T = DT[dtype]
    q, kp, vp = _randn(1, (B, H, D), T, 1.5), _randn(2, (P, Hkv, D), T), _randn(3, (P, Hkv, D), T)
    k, v = _randn(4, (B, S, Hkv, D), T), _randn(5, (B, S, Hkv, D), T)
    lens = [(i * 37) % (S + 1) for i in range(B)]
    lens[-1] = S
    for b, n in enumerate(lens):              # past a request's keys: anything
        k[b, n:], v[b, n:] = math.nan, math.inf
    O = torch.full_like(q, math.nan)
    got = cf.PrefixAttention(dtype, H, Hkv, D).run(q, kp, vp, k, v,
                                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), O=O)
    torch.cuda.synchronize()
    K = torch.cat([torch.cat([kp, k[b, :n]]) for b, n in enumerate(lens)])
    V = torch.cat([torch.cat([vp, v[b, :n]]) for b, n in enumerate(lens)])
    want, _, b, _ = R.attention(q, K, V, list(range(B + 1)), R.starts([P + n for n in lens]), False, D ** -0.5)
    # joining parts: a few more roundings in 32 bits
    R.check(got, want, b + 2.0 ** -20 * want.abs(), "O")


def test_prefix_graph_replays():
    """Captured twice and replayed with new keys and lengths in turn, eager calls
    in between."""
    H, Hkv, D, B, P, S = 8, 2, 128, 6, 1500, 300
    T = torch.bfloat16
    plan = cf.PrefixAttention("bf16", H, Hkv, D)
    mk = lambda i: (_randn(i, (B, H, D), T, 1.5), _randn(i + 1, (P, Hkv, D), T), _randn(i + 2, (P, Hkv, D), T),
                    _randn(i + 3, (B, S, Hkv, D), T), _randn(i + 4, (B, S, Hkv, D), T),
                    (torch.arange(B, device="cuda", dtype=torch.int32) * 61 + 7 * i) % (S + 1))
    args = mk(1)
    _flush("prefix graph")
    plan.run(*args)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(plan.run(*args))
        graphs.append(g)
    for rep in range(3):
        new = mk(20 + 10 * rep)
        for a, b in zip(args, new):
            a.copy_(b)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = plan.run(*new)
        for o in outs:
            assert torch.equal(o, want), rep


def test_prompt_then_tokens():
    """As they are used together: a prompt's last row by Attention is what
    PrefixAttention gives for that token behind the rest of the prompt."""
    H, Hkv, D, P, S = 8, 2, 128, 500, 37
    T = torch.bfloat16
    k, v = _randn(7, (P + S, Hkv, D), T), _randn(8, (P + S, Hkv, D), T)
    q = _randn(9, (P + S, H, D), T)
    _flush("prompt then tokens")
    whole = cf.Attention("bf16", H, Hkv, D).run(q, k, v, _cu([P + S]))
    B = S                                      # request b holds the first b + 1 keys behind the prefix
    own_k, own_v = k[None, P:].expand(B, S, Hkv, D), v[None, P:].expand(B, S, Hkv, D)
    lens = torch.arange(1, S + 1, dtype=torch.int32, device="cuda")
    tok = cf.PrefixAttention("bf16", H, Hkv, D).run(q[P:], k[:P], v[:P], own_k, own_v, lens)
    torch.cuda.synchronize()
    want, _, b, _ = R.attention(q, k, v, [0, P + S], [0, P + S], True, D ** -0.5)
    R.check(whole, want, b)
    R.check(tok, want[P:], b[P:] + 2.0 ** -20)
