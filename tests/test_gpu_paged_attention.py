"""Attention under a window and over pages against the definition in 64 bits, at
the sizes, masks and layouts where it can go wrong."""
import math

import pytest
import torch

import chip_fusion_amd as cf
import paged_ref as R
from test_gpu_norm_rotary import DT, _flush, _int, _pool, _randn

pytestmark = pytest.mark.gpu


def _fill(cache, table, lens, seed, std=1.0, behind=math.nan):
    """Values for the sequences' keys; `behind` in every other place."""
    size, tab = cache.shape[1], table.cpu()
    cache.fill_(behind)
    x = _randn(seed, (sum(lens),) + tuple(cache.shape[2:]), cache.dtype, std)
    page = torch.tensor([int(tab[s, j // size]) for s, n in enumerate(lens) for j in range(n)], dtype=torch.long, device="cuda")
    slot = torch.tensor([j % size for n in lens for j in range(n)], dtype=torch.long, device="cuda")
    if len(page):
        cache[page, slot] = x
    return x


# dtype, heads, kv heads, dim, query lengths, key lengths, window, sinks
WINDOWS = [
    ("f16", 1, 1, 64, [1], [1], 1, 0),
    ("bf16", 2, 1, 8, [3, 1], [3, 1], 2, 1),
    ("f16", 4, 4, 40, [63, 64, 65], [63, 64, 65], 16, 0),
    ("bf16", 4, 2, 64, [127, 0, 1, 129, 2], [127, 0, 1, 129, 2], 33, 4),
    ("f16", 6, 2, 72, [31, 33], [95, 97], 32, 32),              # pieces behind earlier keys
    ("bf16", 8, 1, 80, [5, 70], [400, 71], 64, 1),
    ("f16", 3, 1, 96, [100], [300], 100, 40),
    ("bf16", 5, 5, 128, [257], [257], 1, 0),                     # a row sees itself alone
    ("f16", 8, 2, 128, [300, 20], [300, 20], 1 << 30, 0),        # every earlier key
    ("bf16", 8, 2, 128, [40, 9], [12, 0], 5, 3),                 # more rows than keys: the first see none
    ("f16", 2, 2, 64, [50, 3], [0, 7], 4, 2),                    # a sequence without keys
    ("f16", 24, 2, 112, [17], [1500], 1100, 70),                 # few rows, many keys: cut
    ("bf16", 2, 2, 128, [260], [2100], 700, 500),
    ("f16", 4, 1, 64, [600], [600], 200, 1 << 30),               # sinks without end
    ("bf16", 4, 1, 128, [700, 3], [2000, 900], 129, 31),
    ("f16", 8, 8, 64, [77], [77], 16, 4),
]


@pytest.mark.parametrize("case", range(len(WINDOWS)))
def test_window(case):
    dtype, H, Hkv, D, lq, lk, window, sinks = WINDOWS[case]
    _flush(f"window {WINDOWS[case]}")
    dt = DT[dtype]
    q, k, v = _randn(1, (sum(lq), H, D), dt, 1.5), _randn(2, (sum(lk), Hkv, D), dt), _randn(3, (sum(lk), Hkv, D), dt)
    O = torch.full_like(q, math.nan)
    plan = cf.Attention(dtype, H, Hkv, D, window=window, sinks=sinks)
    got, lse = plan.run(q, k, v, _int(R.starts(lq)), _int(R.starts(lk)), O=O, lse=True)
    again = plan.run(q, k, v, _int(R.starts(lq)), _int(R.starts(lk)))
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk, window, sinks)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")
    assert got is O and torch.equal(again, got)          # the same values on every run


@pytest.mark.parametrize("seqs", [1, 64, 65, 200])
@pytest.mark.parametrize("window", [None, 20])
def test_many_sequences(seqs, window):
    """More sequences than a wave scans at once, empty ones among them, over pages
    and side by side."""
    lq = [(7 * i) % 23 for i in range(seqs)]
    lk = [n + (31 * i) % 190 for i, n in enumerate(lq)]
    _flush(f"{seqs} sequences, window {window}")
    H, Hkv, D = 4, 2, 64
    kc, vc, table = _pool(1, lk, 16, Hkv, D, torch.bfloat16)
    k, v = _fill(kc, table, lk, 2), _fill(vc, table, lk, 3)
    q = _randn(1, (sum(lq) + 2, H, D), torch.bfloat16, 1.5)             # two rows of no sequence
    O = torch.full_like(q, 7.0)
    got, lse = cf.PagedAttention("bf16", H, Hkv, D, 16, window=window, sinks=3 if window else 0).run(
        q, kc, vc, table, _int(lk), _int(R.starts(lq)), O=O, lse=True)
    torch.cuda.synchronize()
    n = sum(lq)
    want, want_lse, b, bl = R.attend(q[:n], k, v, lq, lk, window, 3)
    R.check(got[:n], want, b, "O")
    R.check(lse[:n], want_lse, bl, "LSE")
    assert bool((got[n:] == 7.0).all())
    if window:
        O2 = torch.full_like(q, 7.0)
        cf.Attention("bf16", H, Hkv, D, window=window, sinks=3).run(q, k, v, _int(R.starts(lq)), _int(R.starts(lk)), O=O2)
        torch.cuda.synchronize()
        R.check(O2[:n], want, b, "side by side")
        assert bool((O2[n:] == 7.0).all())


# dtype, heads, kv heads, dim, page, query lengths, key lengths, window, sinks, layout
PAGED = [
    ("f16", 1, 1, 64, 16, [1], [1], None, 0, "rows"),
    ("bf16", 8, 8, 64, 16, [1, 1, 1], [300, 17, 16], None, 0, "heads"),
    ("f16", 8, 2, 128, 1, [1, 1], [33, 70], None, 0, "rows"),              # a page a key
    ("bf16", 4, 2, 40, 7, [3, 0, 20, 1], [50, 9, 20, 0], None, 0, "both"),  # pages that end inside tiles
    ("f16", 6, 1, 80, 24, [40, 2], [100, 64], 30, 5, "heads"),
    ("bf16", 16, 2, 96, 32, [4, 4, 4], [900, 31, 4], None, 0, "rows"),     # 32 rows a key head: the waves take keys
    ("f16", 24, 4, 72, 64, [5, 6], [700, 650], 300, 33, "rows"),
    ("bf16", 32, 8, 128, 16, [1] * 9, [1, 31, 32, 33, 257, 1000, 2000, 3001, 5000], None, 0, "rows"),   # cut
    ("f16", 32, 8, 128, 128, [1] * 5, [4000, 1, 0, 2500, 129], 1000, 100, "heads"),
    ("bf16", 8, 2, 128, 64, [300, 1], [2500, 3500], None, 0, "rows"),
    ("f16", 2, 2, 64, 256, [200], [200], None, 0, "rows"),
    ("bf16", 64, 1, 64, 16, [3], [200], None, 0, "rows"),                  # more heads a key head than a wave's rows
    ("f16", 4, 2, 64, 5, [9, 3], [4, 0], None, 0, "rows"),                 # more rows than keys: the first see none
    ("bf16", 130, 1, 16, 16, [1, 1], [600, 3], 64, 64, "rows"),            # more than a tile's rows a token
]


def _paged(case, behind=math.nan):
    dtype, H, Hkv, D, size, lq, lk, window, sinks, layout = case
    kc, vc, table = _pool(7, lk, size, Hkv, D, DT[dtype], layout)
    k, v = _fill(kc, table, lk, 2, behind=behind), _fill(vc, table, lk, 3, behind=behind)
    q = _randn(1, (sum(lq), H, D), DT[dtype], 1.5)
    cu = None if all(n == 1 for n in lq) else _int(R.starts(lq))
    return cf.PagedAttention(dtype, H, Hkv, D, size, window=window, sinks=sinks), q, kc, vc, table, cu, k, v


@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged(case):
    """Places behind the sequences' keys, and pages of none, hold NaN."""
    _flush(f"paged {PAGED[case]}")
    lq, lk, window, sinks = PAGED[case][5:9]
    plan, q, kc, vc, table, cu, k, v = _paged(PAGED[case])
    O = torch.full_like(q, math.nan)
    got, lse = plan.run(q, kc, vc, table, _int(lk), cu, O=O, lse=True)
    again = plan.run(q, kc, vc, table, _int(lk), cu)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk, window, sinks)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")
    assert got is O and torch.equal(again, got)


@pytest.mark.parametrize("group", [1, 4, 6])
@pytest.mark.parametrize("before", [0, 1, 31, 500])
def test_chunks_of_all_sizes(group, before):
    """Chunks on both sides of the rows that a wave and a tile hold."""
    lq = [1, 5, 8, 9, 32, 33, 127, 128, 129, 200]
    lk = [n + before for n in lq]
    _flush(f"chunks, group {group}, {before} keys before")
    case = ("bf16", 2 * group, 2, 64, 16, lq, lk, None, 0, "rows")
    plan, q, kc, vc, table, cu, k, v = _paged(case)
    got, lse = plan.run(q, kc, vc, table, _int(lk), cu, lse=True)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")


@pytest.mark.parametrize("dtype,H,Hkv,D,size", [("bf16", 8, 2, 128, 16), ("f16", 12, 2, 96, 24), ("f16", 8, 8, 64, 1)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (700, 40)])
def test_single_tokens_and_chunks_together(dtype, H, Hkv, D, size, window, sinks):
    """Mostly single tokens, few and many keys, whole and cut; a chunk among them
    whose rows fill tiles; requests that pad the batch; pages that sequences share."""
    lq = [1] * 30 + [40] + [0, 1, 1]
    lk = [(37 * i * i) % 300 + 1 for i in range(28)] + [6000, 2500, 1900, 0, 0, 5]
    _flush(f"single tokens and a chunk {dtype} {D} window {window}")
    case = (dtype, H, Hkv, D, size, lq, lk, window, sinks, "rows")
    plan, q, kc, vc, table, cu, k, v = _paged(case)
    got, lse = plan.run(q, kc, vc, table, _int(lk), cu, lse=True)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk, window, sinks)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")
    # a second request behind the longest one's pages
    share, n = table[28:29].expand(3, -1).contiguous(), _int([6000, 6000, 5999])
    q3 = torch.cat([q[28:29], q[28:29], q[:1]])
    both = plan.run(q3, kc, vc, share, n)
    torch.cuda.synchronize()
    at = sum(lk[:28])
    want, _, b, _ = R.attend(q3, *(torch.cat([x[at:at + 6000], x[at:at + 6000], x[at:at + 5999]]) for x in (k, v)), [1] * 3,
                             n.tolist(), window, sinks)
    R.check(both, want, b, "shared pages")


@pytest.mark.parametrize("window,sinks", [(None, 0), (45, 0), (45, 10)])
@pytest.mark.parametrize("rows", [1, 4, 150])
def test_infinities_and_nan_reach_the_rows_that_see_them(window, sinks, rows):
    H, Hkv, D, size, n = 2, 1, 64, 16, 260
    _flush(f"infinities, window {window} {sinks}, {rows} rows")
    case = ("f16", H, Hkv, D, size, [rows], [n], window, sinks, "rows")
    plan, q, kc, vc, table, cu, k, v = _paged(case)
    tab = table.cpu()
    for key, col, x in ((3, 1, math.inf), (60, 2, -math.inf), (200, 3, math.nan), (255, 5, math.inf), (259, 6, math.nan),
                        (220, 7, math.inf), (251, 7, -math.inf), (258, 63, -math.inf)):
        v[key, 0, col] = x
        vc[int(tab[0, key // size]), key % size, 0, col] = x
    got = plan.run(q, kc, vc, table, _int([n]), cu)
    torch.cuda.synchronize()
    want, _, b, _ = R.attend(q, k, v, [rows], [n], window, sinks)
    R.check(got, want, b)
    if window:
        got = cf.Attention("f16", H, Hkv, D, window=window, sinks=sinks).run(q, k, v, _int([0, rows]), _int([0, n]))
        torch.cuda.synchronize()
        R.check(got, want, b, "side by side")


@pytest.mark.parametrize("rows", [1, 2, 40])
@pytest.mark.parametrize("window,sinks", [(None, 0), (4000, 50)])
def test_infinities_in_parts(rows, window, sinks):
    """Cut keys: infinities and NaN in parts of any weight, and in keys that nobody sees."""
    H, Hkv, D, size, n = 8, 2, 64, 16, 6500
    _flush(f"infinities in parts, {rows} rows, window {window}")
    case = ("bf16", H, Hkv, D, size, [rows], [n], window, sinks, "rows")
    plan, q, kc, vc, table, cu, k, v = _paged(case)
    tab = table.cpu()
    for key, col, x in ((3, 1, math.inf), (60, 2, -math.inf), (1200, 3, math.nan), (3000, 4, math.inf), (5000, 5, -math.inf),
                        (6000, 5, math.inf), (6470, 6, math.nan), (6499, 7, math.inf)):
        v[key, 0, col] = x
        vc[int(tab[0, key // size]), key % size, 0, col] = x
    got, lse = plan.run(q, kc, vc, table, _int([n]), cu, lse=True)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, [rows], [n], window, sinks)
    R.check(got, want, b)
    R.check(lse, want_lse, bl)
    # one part holds all the weight: the others' infinities stay
    q2 = q.clone()
    q2[:] = k[6400].repeat_interleave(H // Hkv, 0) * 40
    got = plan.run(q2, kc, vc, table, _int([n]), cu)
    torch.cuda.synchronize()
    want, _, _, _ = R.attend(q2, k, v, [rows], [n], window, sinks)
    odd = ~torch.isfinite(want)
    assert not bool(torch.isfinite(got.cpu()[odd]).any()) and bool(torch.isfinite(got.cpu()[~odd]).all())


def test_keys_of_nan_that_a_row_does_not_see():
    """NaN among keys: rows that see them are NaN, others as they would be."""
    H, Hkv, D, n = 2, 2, 64, 200
    _flush("keys of NaN")
    q, k, v = (_randn(i, (n, h, D), torch.bfloat16) for i, h in ((1, H), (2, Hkv), (3, Hkv)))
    k[90, 0, 7] = math.nan
    got = cf.Attention("bf16", H, Hkv, D, window=30, sinks=2).run(q, k, v, _int([0, n]))
    torch.cuda.synchronize()
    hit = torch.zeros((n, H), dtype=torch.bool)
    hit[90:120, 0] = True
    assert torch.equal(torch.isnan(got).all(-1).cpu(), hit) and torch.equal(torch.isnan(got).any(-1).cpu(), hit)
    k2 = k.clone()
    k2[90, 0, 7] = 0.0
    want, _, b, _ = R.attend(q, k2, v, [n], [n], 30, 2)
    R.check(got[~hit.cuda()], want[~hit], b[~hit])


def test_lengths_and_pages_that_are_not_there():
    """Lengths past the table, entries of no page, starts out of order: clamped,
    nothing outside is read or written."""
    H, Hkv, D, size = 4, 2, 64, 8
    _flush("bad lengths and entries")
    kc, vc = _randn(1, (5, size, Hkv, D), torch.float16), _randn(2, (5, size, Hkv, D), torch.float16)
    table = _int([[0, 1, 2, 3], [-7, 99, 2 ** 31 - 1, -2 ** 31], [4, 3, 2, 1]])
    lens = [2 ** 31 - 1, 30, -5]
    q = _randn(3, (9, H, D), torch.float16)
    plan = cf.PagedAttention("f16", H, Hkv, D, size)
    got = plan.run(q, kc, vc, table, _int(lens), _int([0, 3, 6, 9]))
    torch.cuda.synchronize()
    fixed = _int([[0, 1, 2, 3], [0, 4, 4, 0], [4, 3, 2, 1]])
    k, v = (R.gather(c, fixed, [32, 30, 0]) for c in (kc, vc))
    want, _, b, _ = R.attend(q, k, v, [3, 3, 3], [32, 30, 0])
    R.check(got, want, b)
    for cu in ([-5, -2 ** 31, 2 ** 31 - 1, 0], [9, 0, 9, 0], [0, 9, 0, 9]):
        for window in (None, 3):
            out = cf.PagedAttention("f16", H, Hkv, D, size, window=window).run(q, kc, vc, table, _int(lens), _int(cu))
            assert out.shape == q.shape
            torch.cuda.synchronize()
    # a cache without pages, a table without places
    none = torch.empty((0, size, Hkv, D), dtype=torch.float16, device="cuda")
    got, lse = plan.run(q, none, none, table, _int([5, 5, 5]), _int([0, 3, 6, 9]), lse=True)
    got2 = plan.run(q, kc, vc, _int([[], [], []]).view(3, 0), _int([5, 5, 5]), _int([0, 3, 6, 9]))
    torch.cuda.synchronize()
    assert not bool(got.any()) and not bool(got2.any()) and bool((lse == -math.inf).all())


def test_a_cache_past_32_bits():
    """Pages whose offsets pass 2^32 bytes."""
    H, Hkv, D, size, dt = 2, 1, 128, 256, torch.float16
    _flush("a cache of more than 4 GB")
    pages = 36000                       # 2.4 GB of keys and of values, side by side
    both = torch.zeros((pages, 2, size, Hkv, D), dtype=dt, device="cuda")
    lens, at = [600, 256], [[35999, 3, 20000], [34000, 5, 6]]
    table = _int(at)
    kc, vc = both[:, 0], both[:, 1]
    for i, c in enumerate((kc, vc)):
        for s in range(2):
            for p in range(3):
                c[at[s][p]] = _randn(10 * i + 3 * s + p, (size, Hkv, D), dt)
    q = _randn(50, (2, H, D), dt, 1.5)
    got = cf.PagedAttention("f16", H, Hkv, D, size).run(q, kc, vc, table, _int(lens))
    torch.cuda.synchronize()
    k, v = (R.gather(c[torch.tensor(sum(at, []), device="cuda")], torch.arange(6).view(2, 3), lens) for c in (kc, vc))
    want, _, b, _ = R.attend(q, k, v, [1, 1], lens)
    R.check(got, want, b)


def test_a_table_with_wider_rows_and_a_fused_projection():
    H, Hkv, D, size = 4, 2, 64, 16
    _flush("strides")
    lq, lk = [2, 7], [40, 23]
    case = ("bf16", H, Hkv, D, size, lq, lk, None, 0, "rows")
    plan, q, kc, vc, table, cu, k, v = _paged(case)
    wide = torch.full((2, 50), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    fused = torch.zeros((9, H + 2, D), dtype=torch.bfloat16, device="cuda")
    fused[:, 1:H + 1] = q
    O = torch.full((H, 9, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    plan.run(fused[:, 1:H + 1], kc, vc, wide[:, :table.shape[1] + 1], _int(lk), cu, O=O[:, :, :D].transpose(0, 1))
    torch.cuda.synchronize()
    want, _, b, _ = R.attend(q, k, v, lq, lk)
    R.check(O[:, :, :D].transpose(0, 1), want, b)
    assert bool((O[:, :, D:] == 7.0).all())


def test_streams_and_graphs():
    """Replays with new lengths, tables, queries and keys; two graphs and an eager
    call, each with its own workspace; the side stream's output is the same."""
    H, Hkv, D, size, dt = 8, 2, 128, 16, torch.bfloat16
    _flush("paged graphs")
    lens = [4000, 1, 777]
    kc, vc, table = _pool(3, [4096] * 3, size, Hkv, D, dt)
    kc.copy_(_randn(1, kc.shape, dt))
    vc.copy_(_randn(2, vc.shape, dt))
    q, n = _randn(4, (3, H, D), dt, 1.5), _int(lens)
    plans = [cf.PagedAttention("bf16", H, Hkv, D, size), cf.PagedAttention("bf16", H, Hkv, D, size, window=1500, sinks=4)]
    outs, graphs = [torch.empty_like(q) for _ in plans], []
    for plan, out in zip(plans, outs):
        plan.run(q, kc, vc, table, n)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.run(q, kc, vc, table, n, O=out)
        graphs.append(g)
    side = torch.cuda.Stream()
    for step in range(4):
        for g in graphs:
            g.replay()
        eager = [plan.run(q, kc, vc, table, n) for plan in plans]
        side.wait_stream(torch.cuda.current_stream())
        other = [plan.run(q, kc, vc, table, n, stream=side) for plan in plans]
        torch.cuda.synchronize()
        L = n.tolist()
        k, v = R.gather(kc, table, L), R.gather(vc, table, L)
        for i, (w, s) in enumerate(((None, 0), (1500, 4))):
            want, _, b, _ = R.attend(q, k, v, [1] * 3, L, w, s)
            R.check(outs[i], want, b, f"graph {i}, step {step}")
            assert torch.equal(eager[i], outs[i]) and torch.equal(other[i], outs[i])
        n.copy_(_int([[10, 4096, 31], [2222, 0, 33], [1, 1, 1], [5, 5, 5]][step]))
        q.copy_(_randn(20 + step, q.shape, dt))
        table.copy_(table.flip(0))


def test_no_rows_and_no_sequences():
    plan = cf.PagedAttention("f16", 2, 1, 64, 16, window=5)
    kc = torch.zeros((3, 16, 1, 64), dtype=torch.float16, device="cuda")
    q = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda")
    assert plan.run(q, kc, kc.clone(), _int([[0]]), _int([0]), _int([0, 0])).shape == q.shape
    assert plan.run(q, kc, kc.clone(), torch.empty((0, 4), dtype=torch.int32, device="cuda"), _int([])).shape == q.shape


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_decoder_step_after_step(dtype):
    """As they are used together: a chunk of each prompt and then single tokens,
    normed, turned and appended, each attending over the pages under a window."""
    H, Hkv, D, size, window, sinks, dt = 8, 2, 64, 16, 70, 3, DT[dtype]
    _flush(f"a decoder {dtype}")
    total = [150, 90, 201]
    kc, vc, table = _pool(4, total, size, Hkv, D, dt)
    rot, att = cf.NormRotary(dtype, H, Hkv, D), cf.PagedAttention(dtype, H, Hkv, D, size, window=window, sinks=sinks)
    whole = cf.Attention(dtype, H, Hkv, D, window=window, sinks=sinks)
    x = [[_randn(10 * s + i, (n, h, D), dt) for i, h in enumerate((H, Hkv, Hkv))] for s, n in enumerate(total)]
    qw, kw = (_randn(90 + i, (D,), dt, 0.2, 1.0) for i in range(2))
    done, out = [0, 0, 0], [[], [], []]
    for chunk in ([100, 90, 64], [49, 0, 64], [1, 0, 72], [0, 0, 1]):
        lens = [a + b for a, b in zip(done, chunk)]
        q, k, v = (torch.cat([x[s][i][done[s]:lens[s]] for s in range(3)]) for i in range(3))
        cu, n = _int(R.starts(chunk)), _int(lens)
        q = rot.append(q, k, v, kc, vc, table, n, cu, q_weight=qw, k_weight=kw, Q_out=q)
        o = att.run(q, kc, vc, table, n, cu)
        torch.cuda.synchronize()
        for s, part in enumerate(torch.split(o, chunk)):
            out[s].append(part)
        done = lens
    assert done == total
    cu = _int(R.starts(total))
    pos = torch.cat([torch.arange(n) for n in total]).int().cuda()
    q, k = rot.run(torch.cat([y[0] for y in x]), torch.cat([y[1] for y in x]), pos, qw, kw)
    v = torch.cat([y[2] for y in x])
    once = whole.run(q, k, v, cu)
    torch.cuda.synchronize()
    want, _, b, _ = R.attend(q, k, v, total, total, window, sinks)
    R.check(torch.cat([torch.cat(y) for y in out]), want, b, "step by step")
    R.check(once, want, b, "at once")
