"""The attention operators' workloads: what is timed and compared.

Three operators of a language model whose work is a cascade of two products
with the intermediate kept on chip:

  attention  prompts: packed sequences, grouped heads, causal or not, keys
             that were there before the prompt (a prompt taken in pieces)
  prefix     one new token for each request of a batch, whose requests share
             one long prefix and have a few keys of their own
  linear     attention without a softmax, a decay for each head and a state
             instead of a cache: whole prompts, and one token at a time

`run` computes them in plain torch operations in 32 bits, or, where `own` is
true, through the package's plans.
"""
import functools
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest prompt: one short request of a small model; latency
        {"name": "attention_one_short", "op": "attention", "dtype": "f16", "heads": 8, "kv_heads": 8, "dim": 64,
         "seqs": 1, "total": 77, "context": 0, "causal": True, "lse": False, "spread": 1},
        # an ordinary step of a server that packs waiting prompts, lengths 0 and 1 among them
        {"name": "attention_packed", "op": "attention", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "seqs": 17, "total": 8001, "context": 0, "causal": True, "lse": False, "spread": 2},
        # prompts taken in pieces: a piece of each prompt against the keys before it
        {"name": "attention_pieces", "op": "attention", "dtype": "f16", "heads": 24, "kv_heads": 4, "dim": 96,
         "seqs": 6, "total": 2500, "context": 4096, "causal": True, "lse": True, "spread": 3},
        # an encoder's batch: every row sees its whole sequence
        {"name": "attention_encoder", "op": "attention", "dtype": "f16", "heads": 16, "kv_heads": 16, "dim": 64,
         "seqs": 24, "total": 9000, "context": 0, "causal": False, "lse": False, "spread": 4},
        # one long document
        {"name": "attention_long", "op": "attention", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "seqs": 1, "total": 16384, "context": 0, "causal": True, "lse": False, "spread": 5},
        # a few requests behind a short system prompt; latency
        {"name": "prefix_few", "op": "prefix", "dtype": "f16", "heads": 8, "kv_heads": 8, "dim": 64,
         "batch": 3, "prefix": 300, "own_keys": 33, "spread": 6},
        # an ordinary decoding batch behind a few thousand tokens of instructions
        {"name": "prefix_batch", "op": "prefix", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "batch": 32, "prefix": 4097, "own_keys": 512, "spread": 7},
        # many samples of one long document
        {"name": "prefix_long", "op": "prefix", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "batch": 128, "prefix": 32768, "own_keys": 1000, "spread": 8},
        # packed prompts going on from the states of earlier ones
        {"name": "linear_packed", "op": "linear", "dtype": "bf16", "heads": 32, "kv_heads": 32, "dim": 128,
         "seqs": 9, "total": 8200, "state": True, "spread": 9},
        # one long document
        {"name": "linear_long", "op": "linear", "dtype": "f16", "heads": 16, "kv_heads": 16, "dim": 128,
         "seqs": 1, "total": 32768, "state": False, "spread": 10},
        # one token of a few requests; latency
        {"name": "linear_step_few", "op": "linear_step", "dtype": "f16", "heads": 8, "kv_heads": 8, "dim": 64,
         "batch": 2},
        # one token of each request of a large batch
        {"name": "linear_step_batch", "op": "linear_step", "dtype": "bf16", "heads": 32, "kv_heads": 32, "dim": 128,
         "batch": 128},
    ]


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "prefix", "linear", "linear_step"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4])
    case = {"op": op, "dtype": rng.choice(["f16", "bf16"]), "heads": kv * group, "kv_heads": kv}
    if op == "attention":
        seqs = _log_int(rng, 1, 24)
        case.update(dim=rng.choice([64, 80, 96, 128]), seqs=seqs, total=_log_int(rng, seqs, 9000),
                    context=rng.choice([0, 0, _log_int(rng, 1, 2048)]), causal=rng.random() < 0.75,
                    lse=rng.random() < 0.5, spread=rng.randrange(1 << 30))
    elif op == "prefix":
        case.update(dim=rng.choice([64, 80, 96, 128]), batch=_log_int(rng, 1, 128),
                    prefix=_log_int(rng, 1, 20000), own_keys=_log_int(rng, 1, 1000),
                    spread=rng.randrange(1 << 30))
    elif op == "linear":
        seqs = _log_int(rng, 1, 12)
        case.update(dim=rng.choice([64, 128]), seqs=seqs, total=_log_int(rng, seqs, 20000),
                    state=rng.random() < 0.5, spread=rng.randrange(1 << 30))
    else:
        case.update(dim=rng.choice([64, 128]), batch=_log_int(rng, 1, 128))
    return case


def _lengths(case):
    """The sequences' lengths (they sum to `total`) and how many keys come
    before each: set by the case, not by the seed."""
    rng, n, total = random.Random(case["spread"]), case["seqs"], case["total"]
    weights = [rng.uniform(0.2, 1.0) for _ in range(n)]
    if n >= 4:                      # an empty sequence and one of a single token
        weights[1], weights[2] = 0.0, 0.0
    lens = [int(total * w / sum(weights)) for w in weights]
    if n >= 4:
        lens[2] = 1
    lens[0] += total - sum(lens)
    before = [rng.randint(0, case.get("context", 0)) for _ in range(n)]
    return lens, before


def _own_lengths(case):
    rng = random.Random(case["spread"])
    lens = [rng.randint(1, case["own_keys"]) for _ in range(case["batch"])]
    lens[0] = case["own_keys"]
    if case["batch"] >= 4:          # a request that has no keys of its own
        lens[2] = 0
    return lens


def _normal(seed, shape, dtype, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _log_decay(heads):
    """The usual slopes: from about half a token's memory to a few hundred tokens'."""
    h = torch.arange(1, heads + 1, dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / heads)).float().cuda()


def prepare(case, seed):
    dt, H, Hkv, D = DTYPES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case}
    base = seed * 16

    def keys(shape, i):
        # keys share a direction, as those of trained models do
        return (_normal(base + i, shape, torch.float32) + _normal(base + 15, shape[-2:], torch.float32, 0.5)).to(dt)

    if case["op"] == "attention":
        lens, before = _lengths(case)
        lens_k = [a + b for a, b in zip(lens, before)]
        s.update(cu_q=_starts(lens), cu_k=_starts(lens_k), longest_q=max(lens), longest_k=max(lens_k),
                 q=_normal(base, (sum(lens), H, D), dt, 1.5), k=keys((sum(lens_k), Hkv, D), 1),
                 v=_normal(base + 2, (sum(lens_k), Hkv, D), dt, 1.0, 0.25))
    elif case["op"] == "prefix":
        B, P, S = case["batch"], case["prefix"], case["own_keys"]
        s.update(lens=torch.tensor(_own_lengths(case), dtype=torch.int32, device="cuda"),
                 q=_normal(base, (B, H, D), dt, 1.5), kp=keys((P, Hkv, D), 1),
                 vp=_normal(base + 2, (P, Hkv, D), dt, 1.0, 0.25), k=keys((B, S, Hkv, D), 3),
                 v=_normal(base + 4, (B, S, Hkv, D), dt, 1.0, 0.25))
    else:
        step = case["op"] == "linear_step"
        lens = None if step else _lengths(case)[0]
        T = case["batch"] if step else case["total"]
        s.update(q=_normal(base, (T, H, D), dt), k=_normal(base + 1, (T, Hkv, D), dt, 0.7, 0.2),
                 v=_normal(base + 2, (T, Hkv, D), dt), log_decay=_log_decay(H), state=None)
        if not step:
            s.update(cu=_starts(lens), longest=max(lens))
        if step or case["state"]:
            n = T if step else case["seqs"]
            s["state"] = _normal(base + 3, (n, H, D, D), torch.float32, 4.0)
    return s


# ---------------------------------------------------------------------------
# The operators in plain form: products, sums, exp and indexing in 32 bits.
# ---------------------------------------------------------------------------
def _rows_of(cu, longest, total):
    """For sequences side by side, padded to the longest: the packed row each
    place reads, whether it is a row of the sequence, and the way back."""
    cu = cu.long()
    place = torch.arange(longest, device=cu.device)
    row = (cu[:-1, None] + place).clamp(max=max(total - 1, 0))
    here = place < (cu[1:] - cu[:-1])[:, None]
    t = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return row, here, seq, t - cu[seq]


def _plain_attention(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    H, Hkv, D = c["heads"], c["kv_heads"], c["dim"]
    n, Lq, Lk, G = c["seqs"], s["longest_q"], s["longest_k"], H // Hkv
    rq, _, seq, at = _rows_of(s["cu_q"], Lq, q.shape[0])
    rk, here_k, _, _ = _rows_of(s["cu_k"], Lk, k.shape[0])
    Q = q.float()[rq].view(n, Lq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(n, Hkv, G * Lq, D)
    K = k.float()[rk].permute(0, 2, 3, 1).contiguous()
    V = v.float()[rk].permute(0, 2, 1, 3).contiguous()
    S = torch.matmul(Q, K).mul_(D ** -0.5).view(n, Hkv, G, Lq, Lk)
    hidden = ~here_k[:, None, :]
    if c["causal"]:
        lens_q, lens_k = (s["cu_q"][1:] - s["cu_q"][:-1]).long(), (s["cu_k"][1:] - s["cu_k"][:-1]).long()
        i, j = torch.arange(Lq, device=q.device), torch.arange(Lk, device=q.device)
        hidden = hidden | (j > i[:, None] + (lens_k - lens_q)[:, None, None])
    S.masked_fill_(hidden[:, None, None], float("-inf"))
    m = S.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), 0.0, m)
    P = S.sub_(m0).exp_()
    l = P.sum(-1, keepdim=True)
    O = torch.matmul(P.view(n, Hkv, G * Lq, Lk), V).view(n, Hkv, G, Lq, D)
    O = torch.where(l > 0, O / l, 0.0).permute(0, 3, 1, 2, 4).reshape(n, Lq, H, D)
    out = O[seq, at].to(q.dtype)
    if not c["lse"]:
        return out
    lse = (l.log() + m0).view(n, H, Lq).permute(0, 2, 1)
    return out, lse[seq, at]


def _plain_prefix(s):
    c, q = s["case"], s["q"]
    B, H, Hkv, D = c["batch"], c["heads"], c["kv_heads"], c["dim"]
    G, P, S = H // Hkv, c["prefix"], c["own_keys"]
    Q = q.float().view(B, Hkv, G, D) * D ** -0.5
    Kp, Vp = s["kp"].float().permute(1, 2, 0).contiguous(), s["vp"].float().permute(1, 0, 2).contiguous()
    Ko, Vo = s["k"].float().permute(0, 2, 3, 1).contiguous(), s["v"].float().permute(0, 2, 1, 3).contiguous()
    sp = torch.matmul(Q.permute(1, 0, 2, 3).reshape(Hkv, B * G, D), Kp)          # [Hkv, B G, P]
    so = torch.matmul(Q, Ko)                                                      # [B, Hkv, G, S]
    so.masked_fill_((torch.arange(S, device=q.device) >= s["lens"][:, None])[:, None, None], float("-inf"))
    mp = sp.amax(-1).view(Hkv, B, G).permute(1, 0, 2)
    m = torch.maximum(mp, so.amax(-1))
    sp = sp.sub_(m.permute(1, 0, 2).reshape(Hkv, B * G, 1)).exp_()
    so = so.sub_(m[..., None]).exp_()
    l = sp.sum(-1).view(Hkv, B, G).permute(1, 0, 2) + so.sum(-1)
    O = torch.matmul(sp, Vp).view(Hkv, B, G, D).permute(1, 0, 2, 3) + torch.matmul(so, Vo)
    return (O / l[..., None]).reshape(B, H, D).to(q.dtype)


def _plain_linear(s, chunk=128):
    """Chunks of tokens: inside one, the decayed scores; between them, each
    chunk's contribution to the state, summed over the chunks before with the
    decay that lies between (one product with a matrix of decays)."""
    c, q = s["case"], s["q"]
    H, Hkv, D, n = c["heads"], c["kv_heads"], c["dim"], c["seqs"]
    C = chunk
    N = -(-max(s["longest"], 1) // C)
    row, here, seq, at = _rows_of(s["cu"], N * C, q.shape[0])

    def chunks(x):
        x = torch.where(here[..., None, None], x.float()[row], 0.0).view(n, N, C, -1, D)
        return x.repeat_interleave(H // x.shape[3], 3).permute(0, 3, 1, 2, 4).contiguous()   # [n, H, N, C, D]

    Q, K, V = chunks(q), chunks(s["k"]), chunks(s["v"])
    g = s["log_decay"].float()
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    gap = i[:, None] - i
    decay = torch.where(gap >= 0, torch.exp(gap.clamp(min=0) * g[:, None, None]), 0.0)       # [H, C, C]
    S = torch.matmul(Q, K.transpose(-1, -2)).mul_(decay[:, None])
    O = torch.matmul(S, V)
    lens = (s["cu"][1:] - s["cu"][:-1]).float()
    c0 = torch.arange(N, device=q.device, dtype=torch.float32) * C
    # a chunk's state counts up to its last token (the sequence's, in the last chunk)
    last = torch.minimum(lens[:, None], c0 + C) - c0 - 1                                       # [n, N]
    left = (last[:, :, None] - i).clamp(min=0)                                                # [n, N, C]
    U = torch.matmul((K * torch.exp(left[:, None] * g[None, :, None, None])[..., None]).transpose(-1, -2), V)
    first = torch.zeros((n, H, D, D), device=q.device) if s["state"] is None else s["state"]
    # state before chunk x: the first state after x C tokens, and chunk y < x after (x - 1 - y) C
    x = torch.arange(N, device=q.device, dtype=torch.float32)
    between = x[:, None] - 1 - x
    W = torch.where(between >= 0, torch.exp(between.clamp(min=0) * C * g[:, None, None]), 0.0)
    before = torch.matmul(W, U.view(n, H, N, D * D)).view(n, H, N, D, D)
    before += torch.exp(x * C * g[:, None])[None, :, :, None, None] * first[:, :, None]
    O += torch.matmul(Q, before) * torch.exp((i + 1) * g[:, None])[None, :, None, :, None]
    out = (O * D ** -0.5).view(n, H, N * C, D)[seq, :, at].to(q.dtype)
    # after the last token: the state before its chunk, decayed over the chunk's tokens, and the chunk's own
    end = ((lens - 1).clamp(min=0) / C).floor().long()
    b = torch.arange(n, device=q.device)
    tail = lens - end * C
    state = before[b, :, end] * torch.exp(tail[:, None] * g)[..., None, None] + U[b, :, end]
    return out, torch.where(lens[:, None, None, None] > 0, state, first)


def _plain_step(s):
    c, q = s["case"], s["q"]
    G, D = c["heads"] // c["kv_heads"], c["dim"]
    K, V = s["k"].float().repeat_interleave(G, 1), s["v"].float().repeat_interleave(G, 1)
    state = torch.exp(s["log_decay"])[:, None, None] * s["state"] + K[..., None] * V[..., None, :]
    out = torch.matmul(q.float()[:, :, None] * D ** -0.5, state)[:, :, 0]
    return out.to(q.dtype), state


# ---------------------------------------------------------------------------
# The package's operators.  A program makes a plan once for a model's heads.
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=None)
def _plan(kind, dtype, heads, kv_heads, dim, causal=None):
    import chip_fusion_amd as cf
    if kind == "attention":
        return cf.Attention(dtype, heads, kv_heads, dim, causal=causal)
    return {"prefix": cf.PrefixAttention, "linear": cf.LinearAttention}[kind](dtype, heads, kv_heads, dim)


def _own(s):
    c = s["case"]
    shape = (c["dtype"], c["heads"], c["kv_heads"], c["dim"])
    if c["op"] == "attention":
        return _plan("attention", *shape, c["causal"]).run(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"],
                                                           lse=c["lse"])
    if c["op"] == "prefix":
        return _plan("prefix", *shape).run(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["lens"])
    if c["op"] == "linear":
        return _plan("linear", *shape).run(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], state=s["state"])
    return _plan("linear", *shape).step(s["q"], s["k"], s["v"], s["log_decay"], s["state"])


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "prefix": _plain_prefix, "linear": _plain_linear,
            "linear_step": _plain_step}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# Bytes and operations that no form of the operator does without.
# ---------------------------------------------------------------------------
def work(case):
    H, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "attention":
        lens, before = _lengths(case)
        pairs = sum(n * b + (n * (n + 1) // 2 if case["causal"] else n * n) for n, b in zip(lens, before))
        rows, keys = sum(lens), sum(lens) + sum(before)
        return {"bytes": 2 * D * (2 * rows * H + 2 * keys * Hkv) + (4 * rows * H if case["lse"] else 0),
                "flops": 4 * D * H * pairs}
    if case["op"] == "prefix":
        keys = sum(_own_lengths(case))
        return {"bytes": 2 * D * (2 * case["batch"] * H + 2 * (case["prefix"] + keys) * Hkv),
                "flops": 4 * D * H * (case["batch"] * case["prefix"] + keys)}
    step = case["op"] == "linear_step"
    rows = case["batch"] if step else case["total"]
    n = case["batch"] if step else case["seqs"]
    states = 2 if step or case["state"] else 1
    return {"bytes": 2 * D * rows * (2 * H + 2 * Hkv) + 4 * D * D * n * H * states, "flops": 4 * D * D * H * rows}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    H, Hkv, D = case["heads"], case["kv_heads"], case["dim"]
    G, scale = H // Hkv, case["dim"] ** -0.5
    if case["op"] == "attention":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
        q0 = k0 = 0
        for n, b in zip(*_lengths(case)):
            see = torch.ones((n, n + b), dtype=torch.bool, device="cuda")
            see = see.tril(b) if case["causal"] else see
            for h in range(H if n else 0):
                K, V = s["k"][k0:k0 + n + b, h // G].double(), s["v"][k0:k0 + n + b, h // G].double()
                x = torch.where(see, s["q"][q0:q0 + n, h].double() @ K.T * scale, float("-inf"))
                lse[q0:q0 + n, h] = torch.logsumexp(x, -1)
                out[q0:q0 + n, h] = torch.softmax(x, -1) @ V
            q0, k0 = q0 + n, k0 + n + b
        return (out, lse) if case["lse"] else out
    if case["op"] == "prefix":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        kp, vp = s["kp"].double().transpose(0, 1), s["vp"].double().transpose(0, 1)
        for b, n in enumerate(_own_lengths(case)):
            K = torch.cat([kp, s["k"][b, :n].double().transpose(0, 1)], 1)
            V = torch.cat([vp, s["v"][b, :n].double().transpose(0, 1)], 1)
            x = s["q"][b].double().view(Hkv, G, D) @ K.transpose(1, 2) * scale
            out[b] = (torch.softmax(x, -1) @ V).reshape(H, D)
        return out
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    Q, K, V = (x.double() if x.shape[1] == H else x.double().repeat_interleave(G, 1) for x in (s["q"], s["k"], s["v"]))
    if case["op"] == "linear_step":
        state = lam * s["state"].double() + K[..., None] * V[..., None, :]
        return (Q[..., None] * state).sum(-2) * scale, state
    lens = _lengths(case)[0]
    out = torch.empty(Q.shape, dtype=torch.float64, device="cuda")
    state = torch.zeros((len(lens), H, D, D), dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        state += s["state"].double()
    starts = s["cu"][:-1].long()
    # token t of every sequence that has one, all of them at once
    for t in range(max(lens)):
        on = [b for b, n in enumerate(lens) if n > t]
        if t == 0 or len(on) != len(which):
            which, at = torch.tensor(on, device="cuda"), starts[on]
            part = state[which]
        row = at + t
        part = torch.addcmul(lam * part, K[row][..., None], V[row][..., None, :])
        out[row] = torch.matmul(Q[row][:, :, None], part)[:, :, 0] * scale
        if any(lens[b] == t + 1 for b in on):
            state[which] = part
    return out, state
