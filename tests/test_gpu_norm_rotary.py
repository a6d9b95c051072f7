"""Norms of queries and keys with their rotation, alone and into a paged cache,
against the definition in 64 bits."""
import math

import pytest
import torch

import chip_fusion_amd as cf
import paged_ref as R

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _flush(msg):
    print(f"\n[case] {msg}", flush=True)


def _randn(seed, shape, dtype, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# dtype, heads, kv heads, dim, rotary, rows, interleaved, norm
CASES = [
    ("f16", 1, 1, 8, 8, 1, False, True),
    ("bf16", 2, 1, 64, 64, 3, False, True),
    ("f16", 5, 5, 72, 72, 7, False, True),           # partners in the other half of a lane's piece
    ("bf16", 6, 2, 80, 40, 33, False, True),
    ("f16", 24, 4, 96, 96, 130, True, True),
    ("bf16", 32, 8, 128, 128, 600, False, True),
    ("f16", 16, 2, 128, 64, 2049, False, False),
    ("bf16", 8, 8, 64, 32, 4101, True, False),
    ("f16", 3, 1, 40, 24, 513, False, True),
    ("bf16", 40, 40, 128, 120, 5, False, True),
    ("f16", 4, 4, 56, 0, 11, False, True),           # the norm alone
    ("bf16", 64, 1, 16, 8, 511, True, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_run(case):
    dtype, H, Hkv, D, rot, T, inter, norm = CASES[case]
    _flush(f"rotary {CASES[case]}")
    dt = DT[dtype]
    q, k = _randn(1, (T, H, D), dt, 1.5), _randn(2, (T, Hkv, D), dt, 0.7, 0.2)
    qw, kw = (_randn(3 + i, (D,), dt, 0.2, 1.0) if norm else None for i in range(2))
    pos = torch.randint(0, 300000, (T,), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    plan = cf.NormRotary(dtype, H, Hkv, D, rotary_dim=rot, interleaved=inter, eps=1e-6 if norm else None)
    got = plan.run(q, k, pos, qw, kw)
    kept = q.clone(), k.clone()
    torch.cuda.synchronize()
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        want, bound = R.norm_rotary(x, w, pos[None], rot, R.default_freqs(rot), None, inter, 1e-6 if norm else None)
        R.check(y, want, bound)
    # in place, the same values
    assert plan.run(q, k, pos, qw, kw, Q_out=q, K_out=k) == (q, k)
    torch.cuda.synchronize()
    assert torch.equal(q, got[0]) and torch.equal(k, got[1]) and not torch.equal(kept[0], q)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("order", ["sections", "alternating"])
def test_several_axes(order, inter):
    H, Hkv, D, T = 4, 2, 96, 700
    _flush(f"axes {order} {inter}")
    q, k = _randn(11, (T, H, D), torch.float16), _randn(12, (T, Hkv, D), torch.float16)
    pos = torch.randint(-50, 100000, (3, T), generator=torch.Generator().manual_seed(6), dtype=torch.int32).cuda()
    axes = [0] * 16 + [1] * 12 + [2] * 20 if order == "sections" else [i % 3 for i in range(48)]
    kw = dict(sections=(16, 12, 20)) if order == "sections" else dict(axes_of=axes)
    freqs = [0.9 ** i for i in range(48)]
    got = cf.NormRotary("f16", H, Hkv, D, freqs=freqs, interleaved=inter, eps=None, **kw).run(q, k, pos)
    wide = torch.zeros((3, T + 5), dtype=torch.int32, device="cuda")       # axes further apart than rows
    wide[:, :T] = pos
    again = cf.NormRotary("f16", H, Hkv, D, freqs=freqs, interleaved=inter, eps=None, **kw).run(q, k, wide[:, :T])
    one = pos[:1].expand(3, T)                     # text: the same place on every axis
    alike = cf.NormRotary("f16", H, Hkv, D, freqs=freqs, interleaved=inter, eps=None, **kw).run(q, k, one)
    plain = cf.NormRotary("f16", H, Hkv, D, freqs=freqs, interleaved=inter, eps=None).run(q, k, pos[0])
    torch.cuda.synchronize()
    assert torch.equal(alike[0], plain[0]) and torch.equal(alike[1], plain[1])
    for x, y, z in ((q, got[0], again[0]), (k, got[1], again[1])):
        want, bound = R.norm_rotary(x, None, pos, D, freqs, axes, inter, None)
        R.check(y, want, bound)
        assert torch.equal(y, z)


def test_far_positions_and_wide_strides():
    """Positions up to 2^31 and below 0; slices of a fused projection, heads first."""
    H, Hkv, D, T = 4, 2, 64, 9
    _flush("far positions, strides")
    dt = torch.bfloat16
    fused = _randn(21, (T, (H + 2 * Hkv) * D), dt)
    q, k = fused[:, :H * D].view(T, H, D), fused[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
    pos = _int([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9, 123456789, 2 ** 24 + 1, 7])
    out = torch.full((H, T + 1, D), math.nan, dtype=dt, device="cuda")
    q_out = out[:, :T].transpose(0, 1)
    plan = cf.NormRotary("bf16", H, Hkv, D)
    got = plan.run(q, k, pos, Q_out=q_out)
    torch.cuda.synchronize()
    for x, y in ((q, got[0]), (k, got[1])):
        want, bound = R.norm_rotary(x, None, pos[None], D, R.default_freqs(D))
        R.check(y, want, bound)
    assert bool(torch.isnan(out[:, T]).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-20])
def test_norms_of_odd_heads(dtype, eps):
    """Heads of zeros, of the largest and the smallest values, one element alone;
    a NaN or an infinity stays in its head."""
    D, dt = 128, DT[dtype]
    _flush(f"odd heads {dtype} {eps}")
    top = torch.finfo(dt).max
    rows = [[0.0] * D, [top] * D, [-top, top] * (D // 2), [1e-5] * D, [torch.finfo(dt).tiny] * D, [0.0] * (D - 1) + [3.0],
            [1.0] * D]
    x = torch.tensor(rows, dtype=torch.float64).to(dt).view(-1, 1, D).cuda()
    pos = _int(range(len(rows)))
    plan = cf.NormRotary(dtype, 1, 1, D, eps=eps)
    got, _ = plan.run(x, x.clone(), pos)
    odd = _randn(31, (4, 3, D), dt)
    odd[1, 1, 5], odd[2, 0, 100], odd[3, 2, 64] = math.nan, math.inf, -math.inf
    got2, _ = cf.NormRotary(dtype, 3, 3, D, eps=eps).run(odd, odd.clone(), _int([3, 4, 5, 6]))
    torch.cuda.synchronize()
    # (eps reaches the kernel in float32)
    e32 = float(torch.tensor(eps, dtype=torch.float32))
    want, bound = R.norm_rotary(x, None, pos[None], D, R.default_freqs(D), eps=e32)
    R.check(got, want, bound)
    fine = torch.ones((4, 3), dtype=torch.bool)
    fine[1, 1] = fine[2, 0] = fine[3, 2] = False
    want, bound = R.norm_rotary(odd, None, _int([3, 4, 5, 6])[None], D, R.default_freqs(D), eps=e32)
    R.check(got2[fine.cuda()], want[fine], bound[fine])
    assert bool(torch.isnan(got2[1, 1]).all()) and bool(torch.isnan(got2[2, 0]).any())


def _pool(seed, lens, size, Hkv, D, dt, layout="rows", width=None):
    """Caches and a table of pages in no order; places of no page hold -1."""
    need = [-(-n // size) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), max(need + [1]) if width is None else width), -1, dtype=torch.int32)
    for s, n in enumerate(need):
        for i in range(n):
            table[s, i] = order.pop()
    caches = []
    for i in range(2):
        if layout == "rows":
            caches.append(torch.full((pages, size, Hkv, D), 7.0, dtype=dt, device="cuda"))
        elif layout == "heads":
            caches.append(torch.full((pages, Hkv, size, D), 7.0, dtype=dt, device="cuda").transpose(1, 2))
        else:               # keys and values of a page side by side, rows padded
            if i == 0:
                both = torch.full((pages, 2, size, Hkv, D + 8), 7.0, dtype=dt, device="cuda")
            caches.append(both[:, i, :, :, :D])
    return caches[0], caches[1], table.cuda()


# dtype, heads, kv heads, dim, rotary, page, new tokens, keys before, layout
APPENDS = [
    ("f16", 4, 2, 64, 64, 16, [1, 1, 1], [0, 15, 16], "rows"),
    ("bf16", 8, 2, 128, 128, 7, [5, 0, 40, 1], [3, 4, 0, 13], "heads"),
    ("f16", 6, 1, 80, 48, 1, [3, 9], [0, 2], "both"),
    ("bf16", 2, 2, 96, 96, 64, [300], [77], "rows"),
    ("f16", 8, 8, 40, 0, 32, [2] * 70, [31] * 70, "heads"),        # more sequences than a wave scans at once
    ("bf16", 32, 8, 128, 128, 16, [2100, 2000], [5, 0], "rows"),
]


@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(case):
    dtype, H, Hkv, D, rot, size, lq, before, layout = APPENDS[case]
    _flush(f"append {APPENDS[case][:6]} {layout}")
    dt, T = DT[dtype], sum(lq)
    lens = [a + b for a, b in zip(lq, before)]
    kc, vc, table = _pool(3, lens, size, Hkv, D, dt, layout)
    q, k, v = _randn(1, (T, H, D), dt), _randn(2, (T, Hkv, D), dt), _randn(3, (T, Hkv, D), dt)
    qw, kw = (_randn(4 + i, (D,), dt, 0.2, 1.0) for i in range(2))
    cu = None if all(n == 1 for n in lq) else _int(R.starts(lq))
    plan = cf.NormRotary(dtype, H, Hkv, D, rotary_dim=rot)
    want_k, want_v = kc.cpu().double(), vc.cpu().double()
    got = plan.append(q, k, v, kc, vc, table, _int(lens), cu, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    pos = torch.tensor([b + i for n, b in zip(lq, before) for i in range(n)])[None]
    want, bound = R.norm_rotary(q, qw, pos, rot, R.default_freqs(rot))
    R.check(got, want, bound, "Q")
    want, bound = R.norm_rotary(k, kw, pos, rot, R.default_freqs(rot))
    bound_k, tab, t = torch.zeros_like(want_k), table.cpu(), 0
    for s, (n, b) in enumerate(zip(lq, before)):
        for i in range(n):
            at = int(tab[s, (b + i) // size]), (b + i) % size
            want_k[at], bound_k[at], want_v[at] = want[t], bound[t], v[t].cpu().double()
            t += 1
    R.check(kc, want_k, bound_k, "keys")            # the new rows, and nothing else
    assert torch.equal(vc.cpu().double(), want_v)


def test_append_writes_nothing_elsewhere():
    """Rows of no sequence, places before 0 and past the table, entries of no page."""
    H, Hkv, D, size, dt = 2, 1, 64, 4, torch.float16
    _flush("append, rows and pages that are not there")
    q, k, v = (_randn(41 + i, (12, h, D), dt) for i, h in enumerate((H, Hkv, Hkv)))
    kc, vc = (torch.full((3, size, Hkv, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    table = _int([[0, -1], [5, 1], [2, 2 ** 31 - 1], [-2 ** 31, 2]])
    # sequence 0: 3 rows, 2 keys: the first lies before 0; 1: places 3, 4 of pages 5 (none) and 1;
    # 2: places 7 and 8, the last past the table; 3: none; rows 10, 11 in no sequence
    cu, lens = _int([0, 3, 5, 7, 10]), _int([2, 5, 9, 1 << 30])
    q_out = torch.full_like(q, math.nan)
    plan = cf.NormRotary("f16", H, Hkv, D, eps=None)
    plan.append(q, k, v, kc, vc, table, lens, cu, Q_out=q_out)
    torch.cuda.synchronize()
    want = torch.full((3, size, Hkv, D), 7.0, dtype=dt)
    want[0, 0], want[0, 1], want[1, 0] = v[1].cpu(), v[2].cpu(), v[4].cpu()
    assert torch.equal(vc.cpu(), want)
    assert bool((kc[want.cuda() == 7.0] == 7.0).all())
    assert bool(torch.isfinite(q_out[:10]).all()) and bool(torch.isnan(q_out[10:]).all())
    # starts and lengths that are no sequences at all
    plan.append(q, k, v, kc, vc, table, _int([-5, -2 ** 31, 2 ** 31 - 1, 0]), _int([9, -3, 2 ** 31 - 1, 2, -7]), Q_out=q_out)
    torch.cuda.synchronize()


def test_positions_beside_the_places():
    """An image's tokens have positions of several axes, their keys the places."""
    H, Hkv, D, size, dt = 4, 2, 64, 8, torch.bfloat16
    _flush("append, positions of their own")
    lq, before = [11, 6], [4, 0]
    lens = [15, 6]
    kc, vc, table = _pool(9, lens, size, Hkv, D, dt)
    q, k, v = (_randn(51 + i, (17, h, D), dt) for i, h in enumerate((H, Hkv, Hkv)))
    pos = torch.randint(0, 5000, (2, 17), generator=torch.Generator().manual_seed(8), dtype=torch.int32).cuda()
    plan = cf.NormRotary("bf16", H, Hkv, D, sections=(10, 22))
    got = plan.append(q, k, v, kc, vc, table, _int(lens), _int(R.starts(lq)), positions=pos)
    alone = plan.run(q, k, pos)
    torch.cuda.synchronize()
    assert torch.equal(got, alone[0])
    new = torch.cat([R.gather(kc, table, lens)[4:15], R.gather(kc, table, lens)[15:]])
    assert torch.equal(new, alone[1].cpu())


def test_another_stream_and_a_graph():
    H, Hkv, D, size, dt = 8, 2, 128, 16, torch.bfloat16
    _flush("append on another stream and in a graph")
    lens = [33, 20, 1]
    kc, vc, table = _pool(5, [64, 64, 64], size, Hkv, D, dt)
    q, k, v = (_randn(61 + i, (3, h, D), dt) for i, h in enumerate((H, Hkv, Hkv)))
    n = _int(lens)
    plan = cf.NormRotary("bf16", H, Hkv, D)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.append(q, k, v, kc, vc, table, n, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        plan.append(q, k, v, kc, vc, table, n, Q_out=out)
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        kc2, vc2 = torch.full_like(kc, 7.0), torch.full_like(vc, 7.0)
        want = plan.append(q, k, v, kc2, vc2, table, n)
        torch.cuda.synchronize()
        if step == 0:
            assert torch.equal(out, got)
        assert torch.equal(out, want)
        for s in range(3):
            at = int(table[s, (int(n[s]) - 1) // size]), (int(n[s]) - 1) % size
            assert torch.equal(kc[at], kc2[at]) and torch.equal(vc[at], v[s])
        n += 1
        q.copy_(_randn(70 + step, q.shape, dt))


def test_no_rows():
    plan = cf.NormRotary("f16", 2, 1, 64)
    q, k = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda"), torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    got = plan.run(q, k, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert got[0].shape == q.shape and got[1].shape == k.shape
    cache = torch.zeros((2, 4, 1, 64), dtype=torch.float16, device="cuda")
    assert plan.append(q, k, k, cache, cache.clone(), _int([[0]]), _int([0]), _int([0, 0])).shape == q.shape
