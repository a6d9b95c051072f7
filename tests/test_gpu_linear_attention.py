"""Linear attention with a decay for each head: prompts in chunks and single
tokens against the recurrence in 64 bits.

Bounds.  A token's output is a sum over the keys of scale lambda^(i-j) (q_i.k_j)
v_j and a product with the state before its chunk.  The score and the copy of
the state are each rounded to the type once (u relative; a state's copy in
fp16 is scaled by a power of two, its values below 2^-28 of the largest lost;
scores in fp16 below 2^-14 are off by 2^-25), and the result once (u of itself); the rest is float32: with
A = scale sum_j lambda^(i-j) sum_d |q_id k_jd| |v_j| over all keys and the first
state, every term of it is counted with u and 2^-24 for each of its sums (D
products of a score, 64 keys, one multiplication a chunk) and 2^-21 for its
powers of lambda.  States: the same sum without q, every term in float32 with
2^-23 a chunk for its factor."""
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


def _cu(lens):
    return torch.tensor(R.starts(lens), dtype=torch.int32, device="cuda")


def recurrence(q, k, v, log_decay, cu, state, scale):
    """O and states with their bounds (64 bits, on the CPU)."""
    dt, H, D = q.dtype, q.shape[1], q.shape[2]
    q, k, v, g = (x.detach().cpu().double() for x in (q, k, v, log_decay))
    G = H // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    lam = torch.exp(g)[:, None, None]
    n = len(cu) - 1
    S = torch.zeros((n, H, D, D), dtype=torch.float64) if state is None else state.detach().cpu().double()
    out, bound = torch.full(q.shape, math.nan, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    after, after_bound = S.clone(), torch.zeros_like(S)
    u = R.U[dt]
    for s in range(n):
        x, y, c = S[s].clone(), S[s].abs(), 0.0          # state, the sum of its terms' magnitudes
        for t in range(cu[s], cu[s + 1]):
            x = lam * x + k[t][:, :, None] * v[t][:, None, :]
            y = lam * y + (k[t][:, :, None] * v[t][:, None, :]).abs()
            out[t] = scale * (q[t][:, None] @ x)[:, 0]
            A = scale * (q[t].abs()[:, None] @ y)[:, 0]
            i = t - cu[s]
            rel = (D + 64 + 8) * R.E32 + (i // 64 + 1) * 2.0 ** -22 + 2.0 ** -20
            tiny = 2.0 ** -25 * 64 * v[cu[s]:t + 1].abs().amax(0) + 2.0 ** -26 * A if dt == torch.float16 else 0.0
            bound[t] = (u * (1 + u) + rel) * A + u * out[t].abs() + tiny + 1e-30
        length = cu[s + 1] - cu[s]
        after[s], after_bound[s] = x, ((64 + 8) * R.E32 + (length // 64 + 1) * 2.0 ** -22 + 2.0 ** -21) * y
    return out, bound, after, after_bound


def _case(dtype, H, Hkv, D, lens, seed=1, state=True, decay=None):
    T, n = DT[dtype], sum(lens)
    q, k, v = _randn(seed, (n, H, D), T), _randn(seed + 1, (n, Hkv, D), T, 0.7), _randn(seed + 2, (n, Hkv, D), T)
    g = -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda") / H) if decay is None else decay
    s0 = _randn(seed + 3, (len(lens), H, D, D), torch.float32, 4.0) if state else None
    return q, k, v, g.float(), s0


CASES = [
    # dtype, heads, kv heads, dim, lengths, a first state
    ("f16", 1, 1, 64, [1], False),
    ("bf16", 2, 1, 64, [63, 64, 65], True),
    ("f16", 4, 4, 128, [31, 0, 1, 100], True),
    ("bf16", 6, 3, 128, [200, 130], False),
    ("bf16", 2, 2, 64, [0, 5], True),
    ("f16", 2, 2, 64, [1300], True),             # cut into segments
    ("bf16", 3, 1, 128, [1200, 1, 700, 512], True),
    ("f16", 1, 1, 128, [1025], False),
    ("bf16", 1, 1, 64, [3, 0] * 35 + [1300, 9, 700], True),      # more sequences than a wave scans at once, some cut
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_linear_attention(case):
    dtype, H, Hkv, D, lens, state = CASES[case]
    _flush(f"linear {CASES[case]}")
    q, k, v, g, s0 = _case(dtype, H, Hkv, D, lens, state=state)
    O, S = torch.full_like(q, math.nan), torch.full((len(lens), H, D, D), math.nan, device="cuda")
    plan = cf.LinearAttention(dtype, H, Hkv, D)
    got, after = plan.run(q, k, v, g, _cu(lens), state=s0, O=O, state_out=S)
    assert got is O and after is S
    torch.cuda.synchronize()
    want, b, ws, bs = recurrence(q, k, v, g, R.starts(lens), s0, D ** -0.5)
    R.check(got, want, b, "O")
    R.check(after, ws, bs, "state")
    again, after2 = plan.run(q, k, v, g, _cu(lens), state=s0)
    assert torch.equal(again, got) and torch.equal(after2, after)
    if s0 is not None:                            # the states in place
        got2, after3 = plan.run(q, k, v, g, _cu(lens), state=s0, state_out=s0)
        assert after3 is s0 and torch.equal(got2, got) and torch.equal(s0, after)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_steps(dtype, D):
    H, Hkv, B = 4, 2, 5
    _flush(f"linear step {dtype} {D}")
    q, k, v, g, s0 = _case(dtype, H, Hkv, D, [1] * B, seed=11)
    plan = cf.LinearAttention(dtype, H, Hkv, D, scale=0.3)
    got, after = plan.step(q, k, v, g, s0)
    torch.cuda.synchronize()
    want, b, ws, bs = recurrence(q, k, v, g, list(range(B + 1)), s0, 0.3)
    R.check(got, want, b, "O")
    R.check(after, ws, bs, "state")
    before = s0.clone()
    got2, after2 = plan.step(q, k, v, g, s0, state_out=s0)
    assert after2 is s0 and torch.equal(s0, after) and torch.equal(got2, got)
    assert not torch.equal(before, s0)


def test_prompt_then_steps():
    """As they are used together: a prompt, then tokens one at a time, is the
    longer prompt; and a prompt in two pieces is the whole one."""
    H, Hkv, D, P, N = 4, 2, 128, 150, 6
    _flush("linear prompt then steps")
    q, k, v, g, s0 = _case("bf16", H, Hkv, D, [P + N], seed=21)
    plan = cf.LinearAttention("bf16", H, Hkv, D)
    want, b, ws, bs = recurrence(q, k, v, g, [0, P + N], s0, D ** -0.5)
    whole, after = plan.run(q, k, v, g, _cu([P + N]), state=s0)
    R.check(whole, want, b)
    out, state = plan.run(q[:P], k[:P], v[:P], g, _cu([P]), state=s0)
    R.check(out, want[:P], b[:P])
    for t in range(P, P + N):
        o, state = plan.step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g, state, state_out=state)
        R.check(o, want[t:t + 1], b[t:t + 1])
    R.check(state, ws, 2 * bs)
    o2, state2 = plan.run(q[100:], k[100:], v[100:], g, _cu([P + N - 100]),
                          state=plan.run(q[:100], k[:100], v[:100], g, _cu([100]), state=s0)[1])
    R.check(o2, want[100:], b[100:])
    R.check(state2, ws, 2 * bs)


def test_decays_from_none_to_all():
    """lambda 1 (a plain sum), 0 (only the token itself), and one whose powers
    run out of float32's range within a chunk."""
    g = torch.tensor([0.0, -math.inf, -5.0, -1e-4], device="cuda")
    for dtype in DT:
        _flush(f"linear decays {dtype}")
        q, k, v, _, s0 = _case(dtype, 4, 4, 64, [300, 2], seed=31)
        got, after = cf.LinearAttention(dtype, 4, 4, 64).run(q, k, v, g, _cu([300, 2]), state=s0)
        torch.cuda.synchronize()
        want, b, ws, bs = recurrence(q, k, v, g, [0, 300, 302], s0, 0.125)
        R.check(got, want, b)
        R.check(after, ws, bs + 1e-30)


@pytest.mark.parametrize("size", [1e-6, 1e6])
def test_fp16_states_out_of_fp16_range(size):
    """States far below and above what fp16 holds: their copy is scaled."""
    _flush(f"linear fp16 state {size}")
    q, k, v, g, s0 = _case("f16", 2, 2, 64, [90], seed=41)
    k.zero_()
    s0 = s0 * size
    q = (q / max(1.0, size / 1e3)).half()            # keep the outputs in range
    got, after = cf.LinearAttention("f16", 2, 2, 64).run(q, k, v, g, _cu([90]), state=s0)
    torch.cuda.synchronize()
    want, b, ws, bs = recurrence(q, k, v, g, [0, 90], s0, 0.125)
    R.check(got, want, b + 2.0 ** -25)              # the output's own subnormals
    R.check(after, ws, bs)


@pytest.mark.parametrize("dtype,D,n", [("f16", 64, 150), ("bf16", 128, 150), ("f16", 128, 1300), ("bf16", 64, 1300)])
def test_values_that_are_not_finite_reach_only_later_rows(dtype, D, n):
    """A value that is not finite spoils its column from its token on, a key
    all of them; the rows before it in the same chunk, and other columns, stay."""
    H, Hkv = 2, 2
    _flush(f"linear odd values {dtype} {D} {n}")
    q, k, v, g, s0 = _case(dtype, H, Hkv, D, [n], seed=61)
    at = n - 50
    v[at, 0, 5], v[at + 3, 0, 40], v[at + 20, 0, D - 1] = math.inf, math.nan, -math.inf
    k[at + 21, 1, 9] = math.nan
    got, after = cf.LinearAttention(dtype, H, Hkv, D).run(q, k, v, g, _cu([n]), state=s0)
    torch.cuda.synchronize()
    odd = torch.zeros((n, H, D), dtype=torch.bool)
    odd[at:, 0, 5] = odd[at + 3:, 0, 40] = odd[at + 20:, 0, D - 1] = True
    odd[at + 21:, 1] = True
    clean = [torch.where(torch.isfinite(x), x, 0.0) for x in (k, v)]
    want, b, ws, bs = recurrence(q, clean[0], clean[1], g, [0, n], s0, D ** -0.5)
    got, after, gone = got.cpu(), after.cpu(), torch.zeros((1, H, D, D), dtype=torch.bool)
    assert not torch.isfinite(got[odd]).any()
    R.check(torch.where(odd, 0.0, got), torch.where(odd, 0.0, want), b, "O")
    gone[:, 0, :, [5, 40, D - 1]] = gone[:, 1, 9] = True
    assert not torch.isfinite(after[gone]).any()
    R.check(torch.where(gone, 0.0, after), torch.where(gone, 0.0, ws), bs, "state")


def test_layouts_and_rows_outside():
    H, Hkv, D, n = 4, 2, 64, 130
    fused = _randn(51, (n, (H + 2 * Hkv) * D), torch.float16)
    q, k, v = (fused[:, a * D:b * D].view(n, b - a, D) for a, b in ((0, H), (H, H + Hkv), (H + Hkv, H + 2 * Hkv)))
    g = torch.full((H,), -0.05, device="cuda")
    plan = cf.LinearAttention("f16", H, Hkv, D)
    _flush("linear layouts")
    want, ws = plan.run(q.contiguous(), k.contiguous(), v.contiguous(), g, _cu([100]))
    hm = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    O = torch.full((H, n, D), 7.0, dtype=torch.float16, device="cuda").transpose(0, 1)
    fused[100:] = math.nan                          # rows behind the last sequence
    for a in ((q, k, v), tuple(hm(x) for x in (q, k, v))):
        _, s = plan.run(*a, g, _cu([100]), O=O)
        assert torch.equal(O[:100], want[:100]) and torch.equal(s, ws)
        assert bool((O[100:] == 7.0).all())
    s0 = torch.randn((3, H, D, D), device="cuda")
    o1, s1 = plan.step(q[:3], k[:3], v[:3], g, s0)
    o2, s2 = plan.step(*(hm(x[:3]) for x in (q, k, v)), g, s0)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


def test_starts_that_go_back_stay_inside():
    """Starts that are out of order ask for more segments than the workspace
    holds: nothing outside it or the tensors is written."""
    H, D, n = 2, 64, 4000
    _flush("linear starts out of order")
    q, k, v, g, _ = _case("f16", H, H, D, [n], seed=71, state=False)
    cu = torch.tensor([0, n, 0, n, -5, 2 * n, 7], dtype=torch.int32, device="cuda")
    seqs = cu.numel() - 1
    plan, L, need = cf.LinearAttention("f16", H, H, D), cf.lib(), ctypes.c_size_t()
    assert L.b2b_linear_attn_workspace(plan._h, seqs, n, ctypes.byref(need)) == 0 and need.value > 0
    guard = 1 << 20
    ws = torch.full((need.value // 4 + 12 * guard,), 7.0, device="cuda")
    O = torch.full((n + 64, H, D), 7.0, dtype=torch.float16, device="cuda")
    after = torch.empty((seqs, H, D, D), device="cuda")
    rows = lambda t: cf.Rows(t.data_ptr(), t.stride(0), t.stride(1))
    assert L.b2b_linear_attn_run(plan._h, seqs, n, rows(q), rows(k), rows(v), rows(O), g.data_ptr(), cu.data_ptr(), None,
                                 after.data_ptr(), ws.data_ptr(), need.value, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert bool((ws[need.value // 4:] == 7).all()) and bool((O[n:] == 7).all())


def test_offsets_past_32_bits():
    """Rows that lie gigabytes apart, inputs and outputs."""
    H, D, n, far = 1, 64, 1200, 1 << 21
    _flush("linear far rows")
    q, k, v, g, s0 = _case("bf16", H, H, D, [n], seed=81)
    room = torch.zeros((n * far,), dtype=torch.bfloat16, device="cuda")           # 5 GB
    Q, K, V, O = [room.as_strided((n, H, D), (far, D, 1), i * far // 4) for i in range(4)]
    Q.copy_(q), K.copy_(k), V.copy_(v)
    got, after = cf.LinearAttention("bf16", H, H, D).run(Q, K, V, g, _cu([n]), state=s0, O=O)
    torch.cuda.synchronize()
    want, b, ws, bs = recurrence(q, k, v, g, [0, n], s0, D ** -0.5)
    R.check(got, want, b, "O")
    R.check(after, ws, bs, "state")


def test_empty_calls():
    plan = cf.LinearAttention("bf16", 2, 1, 64)
    e = lambda h: torch.empty((0, h, 64), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(2, device="cuda")
    s0 = torch.randn((2, 2, 64, 64), device="cuda")
    o, s = plan.run(e(2), e(1), e(1), g, _cu([0, 0]), state=s0)
    assert o.shape == (0, 2, 64) and torch.equal(s, s0)
    assert torch.equal(plan.run(e(2), e(1), e(1), g, _cu([0, 0]))[1], torch.zeros_like(s0))
    assert plan.run(e(2), e(1), e(1), g, _cu([]))[1].shape == (0, 2, 64, 64)
    assert plan.step(e(2), e(1), e(1), g, s0[:0])[0].shape == (0, 2, 64)


def test_graph_replays():
    H, Hkv, D = 4, 4, 128
    plan = cf.LinearAttention("bf16", H, Hkv, D)
    lens = [1100, 300]
    q, k, v, g, s0 = _case("bf16", H, Hkv, D, lens, seed=61)
    cu = _cu(lens)
    _flush("linear graph")
    plan.run(q, k, v, g, cu, state=s0)
    plan.step(q[:2], k[:2], v[:2], g, s0)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            o, s = plan.run(q, k, v, g, cu, state=s0)
            o1, s1 = plan.step(q[:2], k[:2], v[:2], g, s)
        graphs.append(gr)
        outs.append((o, s, o1, s1))
    for rep, ls in enumerate([lens, [700, 700], [1400, 0]]):
        q2, k2, v2, _, s2 = _case("bf16", H, Hkv, D, ls, seed=70 + rep)
        q.copy_(q2), k.copy_(k2), v.copy_(v2), cu.copy_(_cu(ls)), s0.copy_(s2)
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        wo, wst = plan.run(q2, k2, v2, g, _cu(ls), state=s2)
        w1, ws1 = plan.step(q2[:2], k2[:2], v2[:2], g, wst)
        for got in outs:
            for x, y in zip(got, (wo, wst, w1, ws1)):
                assert torch.equal(x, y), rep
