"""The workloads of serving from a paged cache: what is timed and compared.

What a decoder does between its projections, a step after another:

  rotary   norms of queries and keys for each head and their rotation by the
           position, in one pass; positions of one axis or of several (time,
           height, width)
  append   the same for new tokens whose keys and values go into the pages of
           a cache
  paged    attention of a few new tokens of each request, one or a chunk, over
           the pages
  window   attention over packed prompts where a row sees the last keys and the
           first few of its sequence; `paged` has the same window

`run` computes them in plain torch operations in 32 bits (angles in 64), or,
where `own` is true, through the package's plans.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS, BASE = 1e-6, 10000.0


def listed():
    return [
        # one token each of a few requests of a small model; latency
        {"name": "rotary_few", "op": "rotary", "dtype": "f16", "heads": 8, "kv_heads": 8, "dim": 64, "rotary": 64,
         "rows": 3, "norm": True, "axes": 1, "interleaved": False, "far": 4000},
        # a server's step over packed prompts
        {"name": "rotary_packed", "op": "rotary", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "rows": 8001, "norm": True, "axes": 1, "interleaved": False, "far": 200000},
        # text around images and video: time, height and width
        {"name": "rotary_axes", "op": "rotary", "dtype": "f16", "heads": 24, "kv_heads": 4, "dim": 96, "rotary": 96,
         "rows": 5003, "norm": False, "axes": 3, "interleaved": False, "far": 30000},
        # one token of each request of a large batch, into its page
        {"name": "append_step", "op": "append", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "rotary": 128,
         "seqs": 128, "steps": 128, "total": 128, "context": 4000, "page": 16, "norm": True, "interleaved": False,
         "spread": 1},
        # pieces of prompts, half of each head rotated
        {"name": "append_chunk", "op": "append", "dtype": "f16", "heads": 16, "kv_heads": 4, "dim": 64, "rotary": 32,
         "seqs": 5, "steps": 0, "total": 4097, "context": 4096, "page": 64, "norm": True, "interleaved": True,
         "spread": 2},
        # the smallest prompt: latency
        {"name": "window_short", "op": "window", "dtype": "f16", "heads": 8, "kv_heads": 8, "dim": 64, "seqs": 1,
         "steps": 0, "total": 77, "context": 0, "window": 16, "sinks": 4, "lse": False, "spread": 3},
        # packed prompts, lengths 0 and 1 among them
        {"name": "window_packed", "op": "window", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "seqs": 17,
         "steps": 0, "total": 8001, "context": 0, "window": 512, "sinks": 4, "lse": False, "spread": 4},
        # one long document
        {"name": "window_long", "op": "window", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "seqs": 1,
         "steps": 0, "total": 32768, "context": 0, "window": 4096, "sinks": 4, "lse": False, "spread": 5},
        # one token each of a few requests of a small model; latency
        {"name": "paged_few", "op": "paged", "dtype": "f16", "heads": 8, "kv_heads": 8, "dim": 64, "seqs": 3, "steps": 3,
         "total": 3, "context": 300, "page": 16, "window": 0, "sinks": 0, "lse": False, "spread": 6},
        # one token of each request of a decoding batch, contexts of all lengths
        {"name": "paged_step", "op": "paged", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "seqs": 64,
         "steps": 64, "total": 64, "context": 8192, "page": 16, "window": 0, "sinks": 0, "lse": False, "spread": 7},
        # pieces of long prompts against the keys before them
        {"name": "paged_chunk", "op": "paged", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128, "seqs": 4,
         "steps": 0, "total": 2048, "context": 16384, "page": 64, "window": 0, "sinks": 0, "lse": False, "spread": 8},
        # a step that mixes pieces of prompts and single tokens behind long contexts, under a window
        {"name": "paged_mixed", "op": "paged", "dtype": "f16", "heads": 24, "kv_heads": 4, "dim": 96, "seqs": 40,
         "steps": 36, "total": 1500, "context": 30000, "page": 32, "window": 2048, "sinks": 4, "lse": True, "spread": 9},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "window", "paged", "paged"])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 80, 96, 128])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "heads": kv * rng.choice([1, 2, 4, 6]), "kv_heads": kv, "dim": dim}
    if op == "rotary":
        axes = rng.choice([1, 1, 2, 3])
        case.update(rotary=rng.choice([dim, dim, 32, 48]), rows=_log_int(rng, 1, 8000), norm=rng.random() < 0.7, axes=axes,
                    interleaved=rng.random() < 0.3, far=_log_int(rng, 100, 500000))
        return case
    seqs = _log_int(rng, 1, 64)
    steps = rng.choice([0, seqs, rng.randint(0, seqs)]) if op != "window" else 0
    case.update(seqs=seqs, steps=steps, total=steps + (_log_int(rng, seqs, 2000) if steps < seqs else 0),
                spread=rng.randrange(1 << 30))
    if op == "append":
        case.update(rotary=rng.choice([dim, dim, 32, 48]), context=_log_int(rng, 1, 4096), norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.3)
    elif op == "window":
        case.update(total=_log_int(rng, seqs, 9000), context=rng.choice([0, 0, _log_int(rng, 1, 2048)]))
    else:
        case.update(context=_log_int(rng, 1, 8192))
    if op != "append":
        window = _log_int(rng, 1, 4096) if op == "window" else rng.choice([0, _log_int(rng, 1, 4096)])
        case.update(window=window, sinks=rng.choice([0, 1, 4, 100]) if window else 0, lse=rng.random() < 0.5)
    if op != "window":
        case.update(page=rng.choice([1, 16, 16, 32, 64, 128, 256]))
    return case


def _lengths(case):
    """The sequences' new tokens (they sum to `total`, the last `steps` of them
    have one) and how many keys come before each: set by the case, not by the
    seed."""
    rng, steps = random.Random(case["spread"]), case["steps"]
    n, total = case["seqs"] - steps, case["total"] - steps
    weights = [rng.uniform(0.2, 1.0) for _ in range(n)]
    if n >= 4:                      # an empty sequence and one of a single token
        weights[1], weights[2] = 0.0, 0.0
    lens = [int(total * w / sum(weights)) for w in weights]
    if n >= 4:
        lens[2] = 1
    if n:
        lens[0] += total - sum(lens)
    lens += [1] * steps
    before = [rng.randint(0, case["context"]) for _ in lens]
    before[0] = case["context"]
    return lens, before


def _normal(seed, shape, dtype, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _table(case, lens_k, seed):
    """Pages in no order; the places of a table past a request's pages hold -1."""
    page = case["page"]
    need = [-(-n // page) for n in lens_k]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((len(lens_k), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table.cuda(), pages


def _freqs(case):
    i = torch.arange(case["rotary"] // 2, dtype=torch.float64)
    return BASE ** (-2.0 * i / case["rotary"])


def _sections(case):
    """How many of the rotated pairs follow each axis."""
    pairs, axes = case["rotary"] // 2, case.get("axes", 1)
    first = pairs // axes
    return (first,) * (axes - 1) + (pairs - first * (axes - 1),)


def prepare(case, seed):
    dt, H, Hkv, D = DTYPES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    s, base = {"case": case}, seed * 16
    if case["op"] in ("rotary", "append"):
        # a trained norm's weights lie around 1
        weight = [_normal(base + 8 + i, (D,), dt, 0.2, 1.0) if case["norm"] else None for i in range(2)]
        s.update(q_weight=weight[0], k_weight=weight[1])
    if case["op"] == "rotary":
        T, axes = case["rows"], case["axes"]
        g = torch.Generator(device="cuda").manual_seed(base + 12)
        if axes == 1:           # prompts side by side, each from a place of its own
            at = torch.randint(0, case["far"], (1 + T // 512,), generator=g, device="cuda", dtype=torch.int32)
            row = torch.arange(T, device="cuda", dtype=torch.int32)
            pos = at[(row // 512).long()] + row % 512
        else:                   # frames of 24 x 32 patches from a place of the text on
            row = torch.arange(T, device="cuda", dtype=torch.int32)
            at = torch.randint(0, case["far"], (1,), generator=g, device="cuda", dtype=torch.int32)
            pos = torch.stack([at + row // 768, at + row // 32 % 24, at + row % 32][:axes]).contiguous()
        s.update(q=_normal(base, (T, H, D), dt, 1.5), k=_normal(base + 1, (T, Hkv, D), dt, 0.7, 0.2), positions=pos)
        return s
    lens, before = _lengths(case)
    lens_k = [a + b for a, b in zip(lens, before)]
    T = sum(lens)
    s.update(cu=_starts(lens), rows_of=(lens, before), q=_normal(base, (T, H, D), dt, 1.5))

    def keys(shape, i):
        # keys share a direction, as those of trained models do
        return (_normal(base + i, shape, torch.float32) + _normal(base + 15, shape[-2:], torch.float32, 0.5)).to(dt)

    if case["op"] == "window":
        s.update(cu_k=_starts(lens_k), k=keys((sum(lens_k), Hkv, D), 1), v=_normal(base + 2, (sum(lens_k), Hkv, D), dt, 1.0, 0.25))
        return s
    table, pages = _table(case, lens_k, base + 13)
    shape = (pages, case["page"], Hkv, D)
    s.update(table=table, lens=torch.tensor(lens_k, dtype=torch.int32, device="cuda"), k_cache=keys(shape, 1),
             v_cache=_normal(base + 2, shape, dt, 1.0, 0.25))
    if case["steps"] == case["seqs"]:
        s["cu"] = None              # one token a request
    if case["op"] == "append":
        s.update(k=_normal(base + 3, (T, Hkv, D), dt, 0.7, 0.2), v=_normal(base + 4, (T, Hkv, D), dt, 1.0, 0.25))
    return s


# ---------------------------------------------------------------------------
# The operators in plain form: products, sums, exp and indexing in 32 bits.
# ---------------------------------------------------------------------------
def _places(s):
    """Sequence and place of every new token."""
    if s["cu"] is None:
        seq = torch.arange(s["q"].shape[0], device="cuda")
        return seq, s["lens"].long() - 1
    cu, lens = s["cu"].long(), s["lens"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, lens[seq] - cu[seq + 1] + t


def _plain_turn(c, x, weight, cos, sin):
    y, r = x.float(), c["rotary"]
    if c["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    if c["interleaved"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _plain_rotary(s, positions):
    c = s["case"]
    freqs = _freqs(c).cuda()
    if positions.dim() == 1:
        angle = positions.double()[:, None] * freqs
    else:
        axis = torch.repeat_interleave(torch.arange(len(_sections(c))), torch.tensor(_sections(c))).cuda()
        angle = positions.double()[axis].T * freqs
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return _plain_turn(c, s["q"], s["q_weight"], cos, sin), _plain_turn(c, s["k"], s["k_weight"], cos, sin)


def _plain_append(s):
    c = s["case"]
    seq, at = _places(s)
    q, k = _plain_rotary(s, at)
    page, slot = s["table"][seq, at // c["page"]].long(), at % c["page"]
    s["k_cache"][page, slot] = k
    s["v_cache"][page, slot] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _plain_steps(s):
    """One token a request, all requests at once, their keys padded to the most."""
    c, q = s["case"], s["q"]
    B, H, Hkv, D, page = c["seqs"], c["heads"], c["kv_heads"], c["dim"], c["page"]
    lens = s["lens"].long()
    most = max(s["rows_of"][1]) + 1
    if c["window"] and c["window"] + c["sinks"] < most:
        first = (lens - c["window"]).clamp(min=c["sinks"])
        j = torch.cat([torch.arange(c["sinks"], device="cuda").expand(B, -1),
                       first[:, None] + torch.arange(c["window"], device="cuda")], 1)
    else:
        j = torch.arange(most, device="cuda").expand(B, -1)
    here = j < lens[:, None]
    j = torch.where(here, j, 0)
    at = s["table"].gather(1, j // page).long() * page + j % page
    K = s["k_cache"].view(-1, Hkv, D)[at].float().permute(0, 2, 3, 1).contiguous()
    V = s["v_cache"].view(-1, Hkv, D)[at].float().permute(0, 2, 1, 3).contiguous()
    S = torch.matmul(q.float().view(B, Hkv, H // Hkv, D) * D ** -0.5, K)
    S.masked_fill_(~here[:, None, None], float("-inf"))
    m = S.amax(-1, keepdim=True)
    P = S.sub_(m).exp_()
    l = P.sum(-1, keepdim=True)
    out = (torch.matmul(P, V) / l).view(B, H, D).to(q.dtype)
    return (out, (l.log() + m).view(B, H)) if c["lse"] else out


def _plain_attention(s, block=1024):
    """A sequence after another, `block` rows at a time, against the keys that
    any of them sees."""
    c, q = s["case"], s["q"]
    H, Hkv, D, W = c["heads"], c["kv_heads"], c["dim"], c["window"]
    G = H // Hkv
    out = torch.empty_like(q)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
    q0 = k0 = 0
    for b, (n, before) in enumerate(zip(*s["rows_of"])):
        for r0 in range(0, n, block):
            r1 = min(n, r0 + block)
            at = torch.arange(before + r0, before + r1, device="cuda")
            first = max(0, before + r0 - W + 1) if W else 0
            sinks = min(c["sinks"], first)
            j = torch.arange(first - sinks, before + r1, device="cuda")
            j[:sinks] = torch.arange(sinks, device="cuda")
            if c["op"] == "paged":
                where = s["table"][b, j // c["page"]].long() * c["page"] + j % c["page"]
                K, V = s["k_cache"].view(-1, Hkv, D)[where], s["v_cache"].view(-1, Hkv, D)[where]
            else:
                K, V = s["k"][k0 + j], s["v"][k0 + j]
            K, V = K.float().permute(1, 2, 0).contiguous(), V.float().permute(1, 0, 2).contiguous()
            Q = q[q0 + r0:q0 + r1].float().view(r1 - r0, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * (r1 - r0), D)
            S = torch.matmul(Q, K).mul_(D ** -0.5).view(Hkv, G, r1 - r0, -1)
            hidden = j > at[:, None]
            if W:
                hidden = hidden | ((j <= at[:, None] - W) & (j >= c["sinks"]))
            S.masked_fill_(hidden, float("-inf"))
            m = S.amax(-1, keepdim=True)
            P = S.sub_(m).exp_()
            l = P.sum(-1, keepdim=True)
            O = torch.matmul(P.view(Hkv, G * (r1 - r0), -1), V).view(Hkv, G, r1 - r0, D) / l
            out[q0 + r0:q0 + r1] = O.permute(2, 0, 1, 3).reshape(r1 - r0, H, D).to(q.dtype)
            lse[q0 + r0:q0 + r1] = (l.log() + m).permute(2, 0, 1, 3).reshape(r1 - r0, H)
        q0, k0 = q0 + n, k0 + n + before
    return (out, lse) if c["lse"] else out


# ---------------------------------------------------------------------------
# The package's operators.  A program makes a plan once for a model's heads.
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _plan(kind, dtype, heads, kv_heads, dim, *rest):
    import chip_fusion_amd as cf
    if kind == "rotary":
        rotary, sections, interleaved, norm = rest
        return cf.NormRotary(dtype, heads, kv_heads, dim, rotary_dim=rotary, base=BASE, sections=sections,
                             interleaved=interleaved, eps=EPS if norm else None)
    if kind == "window":
        window, sinks = rest
        return cf.Attention(dtype, heads, kv_heads, dim, window=window, sinks=sinks)
    page, window, sinks = rest
    return cf.PagedAttention(dtype, heads, kv_heads, dim, page, window=window or None, sinks=sinks)


def _own(s):
    c = s["case"]
    shape = (c["dtype"], c["heads"], c["kv_heads"], c["dim"])
    if c["op"] == "window":
        return _plan("window", *shape, c["window"], c["sinks"]).run(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], lse=c["lse"])
    if c["op"] == "paged":
        return _plan("paged", *shape, c["page"], c["window"], c["sinks"]).run(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], lse=c["lse"])
    plan = _plan("rotary", *shape, c["rotary"], _sections(c), c["interleaved"], c["norm"])
    if c["op"] == "rotary":
        return plan.run(s["q"], s["k"], s["positions"], s["q_weight"], s["k_weight"])
    q = plan.append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                    q_weight=s["q_weight"], k_weight=s["k_weight"])
    return q, s["k_cache"], s["v_cache"]


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "rotary":
        return _plain_rotary(state, state["positions"])
    if c["op"] == "append":
        return _plain_append(state)
    if c["op"] == "paged" and c["steps"] == c["seqs"]:
        return _plain_steps(state)
    return _plain_attention(state)


# ---------------------------------------------------------------------------
# Bytes and operations that no form of the operator does without.
# ---------------------------------------------------------------------------
def _seen(at, case):
    """Keys that a row in place `at` sees."""
    W = case["window"]
    return at + 1 if not W else min(at + 1, W) + min(case["sinks"], max(0, at + 1 - W))


def work(case):
    H, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rotary":
        T = case["rows"]
        return {"bytes": 2 * D * T * 2 * (H + Hkv) + 4 * T * case["axes"], "flops": 10 * D * T * (H + Hkv)}
    lens, before = _lengths(case)
    T = sum(lens)
    if case["op"] == "append":
        return {"bytes": 2 * D * T * 2 * (H + 2 * Hkv) + 8 * case["seqs"], "flops": 10 * D * T * (H + Hkv)}
    pairs = keys = 0
    for n, b in zip(lens, before):
        if not n:
            continue
        pairs += sum(_seen(at, case) for at in range(b, b + n))
        first = max(0, b - case["window"] + 1) if case["window"] else 0
        keys += b + n - first + min(first, case["sinks"])
    return {"bytes": 2 * D * (2 * T * H + 2 * keys * Hkv) + (4 * T * H if case["lse"] else 0), "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def _exact_rotary(case, x, weight, positions):
    """x [rows, heads, dim] in 64 bits; positions[a] the rows' places on axis a."""
    if case["norm"]:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dim"] + EPS) * weight.double()
    out, pair = x.clone(), 0
    for axis, n in enumerate(_sections(case)):
        for i in range(pair, pair + n):
            angle = positions[axis].double() * math.pow(BASE, -2.0 * i / case["rotary"])
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rotary"] // 2)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            out[..., a], out[..., b] = z.real, z.imag
        pair += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    H, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rotary":
        pos = s["positions"] if case["axes"] > 1 else s["positions"][None]
        return (_exact_rotary(case, s["q"].double(), s["q_weight"], pos),
                _exact_rotary(case, s["k"].double(), s["k_weight"], pos))
    lens, before = _lengths(case)
    table = s["table"].tolist() if case["op"] != "window" else None
    if case["op"] == "append":
        where, at = [], []
        for b, (n, m) in enumerate(zip(lens, before)):
            for p in range(m, m + n):
                where.append(table[b][p // case["page"]] * case["page"] + p % case["page"])
                at.append(p)
        where, pos = torch.tensor(where, device="cuda"), torch.tensor([at], device="cuda")
        out = [_exact_rotary(case, s["q"].double(), s["q_weight"], pos)]
        new = [_exact_rotary(case, s["k"].double(), s["k_weight"], pos), s["v"].double()]
        for cache, x in zip((s["k_cache"], s["v_cache"]), new):
            whole = cache.double()
            whole.view(-1, Hkv, D)[where] = x
            out.append(whole)
        return tuple(out)
    G, W = H // Hkv, case["window"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(lens, before)):
        if n and table is not None:
            row = torch.tensor([table[b][i // case["page"]] * case["page"] + i % case["page"] for i in range(n + m)], device="cuda")
            K, V = s["k_cache"].view(-1, Hkv, D)[row], s["v_cache"].view(-1, Hkv, D)[row]
        elif n:
            K, V = s["k"][k0:k0 + n + m], s["v"][k0:k0 + n + m]
        for r in range(0, n, 4096):
            e = min(n, r + 4096)
            lo = max(0, m + r - W) if W else 0
            key = torch.cat([torch.arange(min(case["sinks"], lo), device="cuda"), torch.arange(lo, m + e, device="cuda")])
            gap = torch.arange(m + r, m + e, device="cuda")[:, None] - key      # how far behind the row a key lies
            see = gap >= 0
            if W:
                see = see & ((gap < W) | (key < case["sinks"]))
            for h in range(H):
                x = s["q"][q0 + r:q0 + e, h].double() @ K[key, h // G].double().T / math.sqrt(D)
                x = torch.where(see, x, float("-inf"))
                lse[q0 + r:q0 + e, h] = torch.logsumexp(x, -1)
                out[q0 + r:q0 + e, h] = torch.softmax(x, -1) @ V[key, h // G].double()
        q0, k0 = q0 + n, k0 + n + m
    return (out, lse) if case["lse"] else out
