"""Paged and windowed attention, norms and appends where a call leaves the common
paths: keys cut among more sequences than a wave looks at at once, many rows over
caches past 4 GB, pages further apart than 32 bits, eight rows a workgroup, starts
out of order between guarded rows."""
import math

import pytest
import torch

import chip_fusion_amd as cf
import paged_ref as R
from test_gpu_norm_rotary import DT, _flush, _int, _pool, _randn
from test_gpu_paged_attention import _fill

pytestmark = pytest.mark.gpu


def _lengths(seqs, chunks):
    """Contexts on both sides of every 64th sequence, long ones among short ones;
    chunks: new tokens of some of the sequences, one of the others."""
    chunks = {s: n for s, n in chunks.items() if s < seqs}
    lq = [chunks.get(s, 1) for s in range(seqs)]
    lk = [n + (31 * s) % 90 for s, n in enumerate(lq)]
    for i, s in enumerate((0, 3, 62, 63, 64, 65, 70, 127, 128, 129, seqs - 1)):
        if s < seqs and s not in chunks:
            lk[s] = 2000 + 400 * i
    for i, s in enumerate(chunks):
        if chunks[s] > 1:
            lk[s] += 1500 + 500 * i
    return lq, lk


@pytest.mark.parametrize("seqs", [65, 130, 200])
@pytest.mark.parametrize("dtype,H,Hkv,D,size", [("bf16", 8, 2, 64, 16), ("f16", 4, 1, 128, 24)])
@pytest.mark.parametrize("kind", ["single tokens", "chunks among them"])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1300, 40)])
def test_keys_cut_among_many_sequences(seqs, dtype, H, Hkv, D, size, kind, window, sinks):
    _flush(f"cut keys, {seqs} sequences, {kind}, {dtype} {D}, window {window}")
    chunks = {} if kind == "single tokens" else {1: 40, 2: 0, 5: 8, 61: 70, 66: 150, 68: 0, seqs - 2: 33}
    lq, lk = _lengths(seqs, chunks)
    kc, vc, table = _pool(1, lk, size, Hkv, D, DT[dtype])
    k, v = _fill(kc, table, lk, 2), _fill(vc, table, lk, 3)
    q = _randn(1, (sum(lq), H, D), DT[dtype], 1.5)
    cu = None if kind == "single tokens" else _int(R.starts(lq))
    plan = cf.PagedAttention(dtype, H, Hkv, D, size, window=window, sinks=sinks)
    O = torch.full_like(q, math.nan)
    got, lse = plan.run(q, kc, vc, table, _int(lk), cu, O=O, lse=True)
    again = plan.run(q, kc, vc, table, _int(lk), cu)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk, window, sinks)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")
    assert torch.equal(again, got)


@pytest.mark.parametrize("seqs", [65, 140])
def test_window_cut_among_many_sequences(seqs):
    """Side by side: pieces of prompts behind earlier keys."""
    _flush(f"cut keys under a window, {seqs} sequences side by side")
    H, Hkv, D, window, sinks = 4, 2, 96, 900, 50
    lq, lk = _lengths(seqs, {1: 40, 2: 0, 5: 8, 61: 70, 66: 150, 68: 0, seqs - 2: 33})
    q = _randn(1, (sum(lq), H, D), torch.float16, 1.5)
    k, v = (_randn(2 + i, (sum(lk), Hkv, D), torch.float16) for i in range(2))
    plan = cf.Attention("f16", H, Hkv, D, window=window, sinks=sinks)
    got, lse = plan.run(q, k, v, _int(R.starts(lq)), _int(R.starts(lk)), lse=True)
    torch.cuda.synchronize()
    want, want_lse, b, bl = R.attend(q, k, v, lq, lk, window, sinks)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")


@pytest.mark.parametrize("window", [None, 300])
def test_chunks_over_a_cache_past_32_bits(window):
    """Many rows, pages of whole groups, whose offsets pass 2^32 bytes; the last
    rows appended there."""
    H, Hkv, D, size, dt = 4, 1, 128, 256, torch.float16
    _flush(f"chunks over a cache of more than 4 GB, window {window}")
    pages = 36000                       # 2.4 GB of keys and of values, side by side
    both = torch.zeros((pages, 2, size, Hkv, D), dtype=dt, device="cuda")
    lens, lq, at = [600, 256], [45, 50], [[35999, 3, 20000], [34000, 5, 6]]
    table, cu = _int(at), _int(R.starts(lq))
    kc, vc = both[:, 0], both[:, 1]
    for i, c in enumerate((kc, vc)):
        for s in range(2):
            for p in range(3):
                c[at[s][p]] = _randn(10 * i + 3 * s + p, (size, Hkv, D), dt)
    q, k, v = (_randn(50 + i, (sum(lq), h, D), dt, 1.5) for i, h in enumerate((H, Hkv, Hkv)))
    plain = cf.NormRotary("f16", H, Hkv, D, rotary_dim=0, eps=None)         # the new rows as they are
    q = plain.append(q, k, v, kc, vc, table, _int(lens), cu)
    plan = cf.PagedAttention("f16", H, Hkv, D, size, window=window)
    got, lse = plan.run(q, kc, vc, table, _int(lens), cu, lse=True)
    torch.cuda.synchronize()
    K, V = (R.gather(c[torch.tensor(sum(at, []), device="cuda")], torch.arange(6).view(2, 3), lens) for c in (kc, vc))
    for x, y in ((K, k), (V, v)):
        assert torch.equal(torch.cat([x[555:600], x[806:]]), y.cpu())
    want, want_lse, b, bl = R.attend(q, K, V, lq, lens, window)
    R.check(got, want, b, "O")
    R.check(lse, want_lse, bl, "LSE")


@pytest.mark.parametrize("rows", [1, 60])
def test_pages_further_apart_than_32_bits(rows):
    """Three pages, 2^31 elements and more from one to the next."""
    H, Hkv, D, size, dt = 2, 1, 64, 32, torch.bfloat16
    _flush(f"pages 4 GB apart, {rows} rows")
    far = 2 ** 31 + 64
    one = size * Hkv * D
    buf = torch.empty(2 * far + 2 * one, dtype=dt, device="cuda")
    kc, vc = (buf.as_strided((3, size, Hkv, D), (far, Hkv * D, D, 1), i * one) for i in range(2))
    for i, c in enumerate((kc, vc)):
        for p in range(3):
            c[p] = _randn(5 * i + p, (size, Hkv, D), dt)
    n = 90
    table, lens, cu = _int([[2, 0, 1]]), _int([n]), _int([0, rows])
    q, k, v = (_randn(60 + i, (rows, h, D), dt, 1.5) for i, h in enumerate((H, Hkv, Hkv)))
    plain = cf.NormRotary("bf16", H, Hkv, D, rotary_dim=0, eps=None)
    q = plain.append(q, k, v, kc, vc, table, lens, cu)
    got = cf.PagedAttention("bf16", H, Hkv, D, size).run(q, kc, vc, table, lens, cu)
    torch.cuda.synchronize()
    K, V = (R.gather(torch.stack([c[2], c[0], c[1]]), torch.arange(3)[None], [n]) for c in (kc, vc))
    assert torch.equal(K[n - rows:], k.cpu()) and torch.equal(V[n - rows:], v.cpu())
    want, _, b, _ = R.attend(q, K, V, [rows], [n])
    R.check(got, want, b)


@pytest.mark.parametrize("dtype,H,Hkv,D,rot,norm,given", [
    ("f16", 16, 4, 64, 64, True, False), ("bf16", 12, 4, 128, 64, False, True), ("bf16", 4, 4, 72, 48, True, False)])
def test_append_of_many_rows_of_many_sequences(dtype, H, Hkv, D, rot, norm, given):
    """Eight rows a workgroup, whose sequences are found 64 at a time, empty ones
    and sequences of one row among them, workgroups whose rows belong to several."""
    dt, size, seqs = DT[dtype], 16, 150
    lq = [(37 * s) % 61 if s % 5 else s % 2 for s in range(seqs)]
    lq[80], lq[149] = 700, 300
    before = [(53 * s) % 40 for s in range(seqs)]
    T, lens = sum(lq), [a + b for a, b in zip(lq, before)]
    assert T >= 4096
    _flush(f"append of {T} rows of {seqs} sequences, {dtype} {D}")
    kc, vc, table = _pool(3, lens, size, Hkv, D, dt)
    rows = T + 3                        # three rows of no sequence
    q, k, v = (_randn(1 + i, (rows, h, D), dt) for i, h in enumerate((H, Hkv, Hkv)))
    qw, kw = (_randn(4 + i, (D,), dt, 0.2, 1.0) if norm else None for i in range(2))
    place = torch.tensor([b + i for n, b in zip(lq, before) for i in range(n)])
    pos = (7 * place + 3 if given else place)[None]
    want_k, want_v = kc.cpu().double(), vc.cpu().double()
    out = torch.full_like(q, math.nan)
    plan = cf.NormRotary(dtype, H, Hkv, D, rotary_dim=rot, eps=1e-6 if norm else None)
    handed = torch.cat([pos[0], torch.zeros(3, dtype=torch.long)]).int().cuda() if given else None
    plan.append(q, k, v, kc, vc, table, _int(lens), _int(R.starts(lq)), positions=handed, q_weight=qw, k_weight=kw, Q_out=out)
    torch.cuda.synchronize()
    eps = 1e-6 if norm else None
    want, bound = R.norm_rotary(q[:T], qw, pos, rot, R.default_freqs(rot), eps=eps)
    R.check(out[:T], want, bound, "Q")
    assert bool(torch.isnan(out[T:]).all())
    want, bound = R.norm_rotary(k[:T], kw, pos, rot, R.default_freqs(rot), eps=eps)
    tab = table.cpu()
    page = torch.tensor([int(tab[s, (b + i) // size]) for s, (n, b) in enumerate(zip(lq, before)) for i in range(n)])
    bound_k = torch.zeros_like(want_k)
    want_k[page, place % size], bound_k[page, place % size] = want, bound
    want_v[page, place % size] = v[:T].cpu().double()
    R.check(kc, want_k, bound_k, "keys")            # the new rows, and nothing else
    assert torch.equal(vc.cpu().double(), want_v)


@pytest.mark.parametrize("window", [None, 3])
@pytest.mark.parametrize("cu", [[-5, -2 ** 31, 2 ** 31 - 1, 0], [9, 0, 9, 0], [0, 9, 0, 9], [3, 2, 1, 0], [8, 9, 2 ** 31 - 1, 9]])
def test_starts_out_of_order_write_nothing_outside(cu, window):
    """Starts that are no sequences: the rows around the output, the inputs and the
    pages' other places stay as they were."""
    H, Hkv, D, size, dt = 4, 2, 64, 8, torch.float16
    _flush(f"starts {cu}, window {window}")
    kc, vc = _randn(1, (5, size, Hkv, D), dt), _randn(2, (5, size, Hkv, D), dt)
    table, lens = _int([[0, 1, 2, 3], [-7, 99, 2 ** 31 - 1, -2 ** 31], [4, 3, 2, 1]]), _int([2 ** 31 - 1, 30, -5])
    guarded = [torch.full((9 + 400, H, D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    q = _randn(3, (9, H, D), dt)
    kept = [x.clone() for x in (q, kc, vc)]
    plan = cf.PagedAttention("f16", H, Hkv, D, size, window=window)
    plan.run(q, kc, vc, table, lens, _int(cu), O=guarded[0][200:209])
    if window:
        flat = [x.reshape(-1, Hkv, D) for x in (kc, vc)]
        cf.Attention("f16", H, Hkv, D, window=window).run(q, *flat, _int(cu), _int([0, 50, -3, 2 ** 31 - 1]), O=guarded[1][200:209])
    torch.cuda.synchronize()
    for g in guarded:
        assert bool((g[:200] == 7.0).all()) and bool((g[209:] == 7.0).all())
        assert bool(torch.isfinite(g).all())
    assert all(torch.equal(x, y) for x, y in zip((q, kc, vc), kept))
