"""The measured cases of the attention-score operators and of the query / key norm and rotation.

qk         RMS norm of every query and key head with the position rotation in the same pass:
           forward ("fwd"), forward and backward ("train"), and one new token per sequence
           written into the KV caches ("append").
attention  attention of the query streams (S = G k, or G k + 1 with the shared stream, which
           reads KV head 0) whose scores may be capped by a tanh, biased by distance, and
           masked by an interval of keys per query: documents packed in a sequence, a
           bidirectional prefix, a sliding window, padded sequences. Forward ("fwd"), forward
           and backward ("train"), one new token per sequence over its KV cache ("decode").

With `own` false, run() is the plain form in elementary torch operations (32 bits, angles in
64); with `own` true it makes the framework's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------
def listed():
    return [
        # a short prompt: 33 tokens of the 16-expert layer (8 groups, top-1, shared head)
        dict(name="qk_short_prompt", op="qk", dir="fwd", dtype="bf16", M=33, G=8, k=1, d=48, rot=48,
             far=0, inter=False, norm=True),
        # prefill of the same layer at 16K tokens
        dict(name="qk_prefill_16k", op="qk", dir="fwd", dtype="bf16", M=16384, G=8, k=1, d=48, rot=48,
             far=0, inter=False, norm=True),
        # a training step of 32K tokens at head dim 128, rotating half of the head, interleaved
        dict(name="qk_train_32k_d128", op="qk", dir="train", dtype="bf16", M=32768, G=8, k=1, d=128,
             rot=64, far=0, inter=True, norm=True),
        # float32 training at an odd token count and far positions
        dict(name="qk_train_f32_far", op="qk", dir="train", dtype="f32", M=5001, G=8, k=2, d=64, rot=64,
             far=1000000, inter=False, norm=True),
        # one generation step of 64 sequences: rotate, and append to the caches
        dict(name="qk_append_64", op="qk", dir="append", dtype="bf16", M=64, G=8, k=1, d=48, rot=48,
             far=1024, inter=False, norm=True),
        # a short ragged prompt with capped scores
        dict(name="attn_short_cap", op="attention", dir="fwd", B=1, T=77, G=8, k=1, d=48, mask="causal",
             docs=0, win=0, cap=30.0, bias=False, sharp=3.0),
        # long-context prefill, 12 documents packed in 16K tokens, capped scores
        dict(name="attn_docs_cap_16k", op="attention", dir="fwd", B=1, T=16384, G=8, k=1, d=48,
             mask="docs", docs=12, win=0, cap=30.0, bias=False, sharp=3.0),
        # bidirectional prefixes with a distance bias, wider groups
        dict(name="attn_prefix_bias_4k", op="attention", dir="fwd", B=2, T=4096, G=8, k=2, d=64,
             mask="prefix", docs=0, win=0, cap=0.0, bias=True, sharp=1.0),
        # a training step on packed documents with capped scores
        dict(name="attn_train_docs_cap_8k", op="attention", dir="train", B=1, T=8192, G=8, k=1, d=48,
             mask="docs", docs=5, win=0, cap=50.0, bias=False, sharp=2.0),
        # a training step with distance bias and a sliding window at head dim 128, odd length
        dict(name="attn_train_window_bias_d128", op="attention", dir="train", B=2, T=2047, G=8, k=1,
             d=128, mask="window", docs=0, win=1000, cap=0.0, bias=True, sharp=1.0),
        # one generation step of 64 sequences of up to 8192 cached tokens, capped and biased
        dict(name="attn_decode_64x8k", op="attention", dir="decode", B=64, T=8192, G=8, k=1, d=48,
             mask="causal", docs=0, win=0, cap=30.0, bias=True, sharp=2.0),
        # one generation step of a single sequence inside a window of its cache
        dict(name="attn_decode_1x2k_window", op="attention", dir="decode", B=1, T=2000, G=8, k=2, d=64,
             mask="window", docs=0, win=1500, cap=0.0, bias=True, sharp=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([16, 32, 48, 64, 80, 96, 112, 128])
    G = rng.choice([1, 2, 4, 8])
    k = rng.choice([1, 1, 2])
    if rng.random() < 0.4:
        direction = rng.choice(["fwd", "train", "append"])
        M = _log_int(rng, 1, 128 if direction == "append" else 16384)
        rot = rng.choice([d, d, 16, 0])
        return dict(op="qk", dir=direction, dtype="bf16" if direction == "append" else
                    rng.choice(["bf16", "bf16", "f32"]), M=M, G=G, k=k, d=d, rot=rot,
                    far=rng.randrange(1, 2048) if direction == "append" else
                    rng.choice([0, 0, rng.randrange(1, 1000000)]),
                    inter=rng.random() < 0.4, norm=rng.random() < 0.8 or rot == 0)
    direction = rng.choice(["fwd", "train", "decode"])
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    bias = rng.random() < 0.5
    sharp = rng.choice([1.0, 2.0, 3.0])
    if direction == "decode":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, 8192)
        mask = rng.choice(["causal", "window"])
        return dict(op="attention", dir=direction, B=B, T=T, G=G, k=k, d=d, mask=mask, docs=0,
                    win=_log_int(rng, 1, T) if mask == "window" else 0, cap=cap, bias=bias, sharp=sharp)
    B = rng.choice([1, 1, 2, 3])
    # a row that sees a single key has no gradient of q and k but roundings: training cases
    # have rows that see more
    few = 4 if direction == "train" else 1
    T = _log_int(rng, 16 if direction == "train" else 1, 4096 // B)
    mask = rng.choice(["causal", "docs", "prefix", "window", "padded"])
    return dict(op="attention", dir=direction, B=B, T=T, G=G, k=k, d=d, mask=mask,
                docs=rng.randrange(1, 9) if mask == "docs" else 0,
                win=_log_int(rng, few, T) if mask == "window" else 0, cap=cap, bias=bias, sharp=sharp)


# ---------------------------------------------------------------------------------------
# What a case's structure is: stream counts, document lengths, key intervals
# ---------------------------------------------------------------------------------------
EPS = 1e-6
ROPE_BASE = 10000.0


def _doc_lengths(T, docs):
    """Uneven document lengths of a sequence of T tokens (some may be empty when T is small)."""
    w = [1.0 + 2.0 * (i % 3) for i in range(docs)]
    edges = [round(T * sum(w[:i]) / sum(w)) for i in range(docs + 1)]
    return [b - a for a, b in zip(edges, edges[1:])]


def _prefix(T, b):
    return min(T, T // 3 + 5 * b)


def _padded(T, b):
    return max(1, T - (b + 1) * T // 5)


def _spans(case, seed):
    """Per sequence the first key and the end of the keys of every query, as lists."""
    B, T, mask = case["B"], case["T"], case["mask"]
    rng = random.Random(seed)
    begins, ends = [], []
    for b in range(B):
        if mask == "docs":
            lens = _doc_lengths(T, case["docs"])
            rng.shuffle(lens)
            be, at = [], 0
            for n in lens:
                be += [at] * n
                at += n
            en = [t + 1 for t in range(T)]
        elif mask == "prefix":
            p = _prefix(T, b)
            be, en = [0] * T, [max(t + 1, p) for t in range(T)]
        elif mask == "window":
            be, en = [max(0, t + 1 - case["win"]) for t in range(T)], [t + 1 for t in range(T)]
        elif mask == "padded":  # both directions inside a sequence; rows behind it see nothing
            n = _padded(T, b)
            be, en = [0] * T, [n if t < n else 0 for t in range(T)]
        else:
            be, en = [0] * T, [t + 1 for t in range(T)]
        begins += be
        ends += en
    return begins, ends


def _positions(case):
    """The new tokens' positions of a decode or append case: ragged, one per sequence."""
    if case["op"] == "qk":
        B, L = case["M"], case["far"]
    else:
        B, L = case["B"], case["T"]
    return [max(0, L - 1 - (b * 37) % (L // 4 + 1)) for b in range(B)]


def _streams(case):
    return case["G"] * case["k"] + 1


def work(case):
    S, G, d = _streams(case), case["G"], case["d"]
    if case["op"] == "qk":
        M, e = case["M"], 2 if case["dtype"] == "bf16" else 4
        elems = (S + G) * M * d
        if case["dir"] == "append":  # q in and out; k and v in, into the caches
            return {"bytes": e * 2 * (S + 2 * G) * M * d, "flops": 8 * elems}
        # the step reads q, k once, and the gradients, and writes the outputs and gradients
        n = 2 if case["dir"] == "fwd" else 4
        return {"bytes": e * n * elems, "flops": (8 if case["dir"] == "fwd" else 24) * elems}
    B, T = case["B"], case["T"]
    if case["dir"] == "decode":
        pos = _positions(case)
        keys = sum(p + 1 if case["mask"] != "window" else min(p + 1, case["win"]) for p in pos)
        return {"bytes": 2 * 2 * G * d * keys + 2 * 2 * S * B * d, "flops": 4 * d * keys * S}
    begin, end = _spans(case, 0)
    pairs = sum(max(0, e - b) for b, e in zip(begin, end))
    M = B * T
    if case["dir"] == "fwd":
        return {"bytes": 2 * M * d * (2 * S + 2 * G), "flops": 4 * d * S * pairs}
    # training: q, k, v, dout in; out, dq, dk, dv out; scores once, and the five products of
    # the backward pass
    return {"bytes": 2 * M * d * (4 * S + 4 * G), "flops": 14 * d * S * pairs}


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------
def _slopes(S):
    return [2.0 ** (-8.0 * (i + 1) / S) for i in range(S)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16
    S, G, d = _streams(case), case["G"], case["d"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dt)

    s = dict(case=case)
    if case["op"] == "qk":
        M = case["M"]
        # rows as a projection gives them: sizes that differ from head to head
        s["q"] = normal(S, M, d, scale=1.7)
        s["k"] = normal(G, M, d, scale=0.6)
        s["qw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        s["kw"] = 1.0 + 0.2 * torch.randn(d, generator=g, device=DEV)
        r = case["rot"]
        s["inv_freq"] = ROPE_BASE ** (-torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / max(r, 1))
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        if case["dir"] == "append":
            L = max(case["far"], 1)
            s["v"] = normal(G, M, d)
            s["kc"], s["vc"] = normal(G, M, L, d), normal(G, M, L, d)
            s["pos"] = torch.tensor(_positions(case), dtype=torch.int32, device=DEV)
        else:
            s["pos"] = torch.arange(M, dtype=torch.int32, device=DEV) + case["far"]
        if case["dir"] == "train":
            s["dqo"], s["dko"] = normal(S, M, d), normal(G, M, d)
            s["dq"], s["dk"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
            s["dqw"], s["dkw"] = torch.empty_like(s["qw"]), torch.empty_like(s["kw"])
        return s
    B, T = case["B"], case["T"]
    s["slopes"] = torch.tensor(_slopes(S), dtype=torch.float32, device=DEV) if case["bias"] else None
    if case["dir"] == "decode":
        s["q"] = normal(S, B, d, scale=case["sharp"])
        s["kc"], s["vc"] = normal(G, B, T, d), normal(G, B, T, d)
        pos = _positions(case)
        random.Random(seed).shuffle(pos)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
        s["begin"] = None
        if case["mask"] == "window":
            s["begin"] = (s["pos"] + 1 - case["win"]).clamp(min=0)
        s["out"] = torch.empty_like(s["q"])
        return s
    M = B * T
    s["q"] = normal(S, M, d, scale=case["sharp"])
    s["k"], s["v"] = normal(G, M, d), normal(G, M, d)
    begin, end = _spans(case, seed)
    s["begin"] = torch.tensor(begin, dtype=torch.int32, device=DEV)
    s["end"] = torch.tensor(end, dtype=torch.int32, device=DEV)
    # a plain causal call passes no intervals, a causal mask only the first keys
    s["causal"] = case["mask"] in ("causal", "docs", "window")
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(S, M, dtype=torch.float32, device=DEV)
    if case["dir"] == "train":
        s["do"] = normal(S, M, d)
        s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
    return s


# ---------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------
def _angles(s):
    """cos and sin of every token's pairs, [M, rot/2]."""
    a = s["pos"].to(torch.float64)[:, None] * s["inv_freq"][None, :]
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(x, rot, inter):
    """The two members of every rotated pair."""
    if inter:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., : rot // 2], x[..., rot // 2: rot]


def _unpair(a, b, rest, inter):
    if inter:
        return torch.cat([torch.stack([a, b], dim=-1).flatten(-2), rest], dim=-1)
    return torch.cat([a, b, rest], dim=-1)


def _rotate(x, c, sn, rot, inter):
    if rot == 0:
        return x
    a, b = _pairs(x, rot, inter)
    return _unpair(a * c - b * sn, a * sn + b * c, x[..., rot:], inter)


def _plain_qk_forward(x, w, c, sn, case):
    x = x.float()
    if case["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _rotate(x, c, sn, case["rot"], case["inter"])


def _plain_qk_backward(x, w, c, sn, dy, case):
    x, gr = x.float(), _rotate(dy.float(), c, -sn, case["rot"], case["inter"])
    if not case["norm"]:
        return gr, torch.zeros_like(w)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    gw = gr * w
    return r * (gw - xh * (gw * xh).mean(-1, keepdim=True)), (gr * xh).sum((0, 1))


def _plain_qk(s):
    case = s["case"]
    c, sn = _angles(s)
    dt = s["q"].dtype
    q = _plain_qk_forward(s["q"], s["qw"], c, sn, case).to(dt)
    k = _plain_qk_forward(s["k"], s["kw"], c, sn, case).to(dt)
    if case["dir"] == "fwd":
        return q, k
    if case["dir"] == "append":
        rows = torch.arange(case["M"], device=DEV)
        s["kc"][:, rows, s["pos"].long()] = k
        s["vc"][:, rows, s["pos"].long()] = s["v"]
        return q, s["kc"], s["vc"]
    dq, dqw = _plain_qk_backward(s["q"], s["qw"], c, sn, s["dqo"], case)
    dk, dkw = _plain_qk_backward(s["k"], s["kw"], c, sn, s["dko"], case)
    return q, k, dq.to(dt), dk.to(dt), dqw, dkw


def _kv_of(case):
    """KV head of every stream."""
    return [i // case["k"] for i in range(case["G"] * case["k"])] + [0]


def _plain_probs(sc, allowed):
    """Softmax over the last axis; a row with no key gives zeros."""
    sc = torch.where(allowed, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    n = p.sum(-1, keepdim=True)
    return p / torch.where(n > 0, n, torch.ones_like(n))


def _plain_attention(s):
    case = s["case"]
    B, T, d, S, G = case["B"], case["T"], case["d"], _streams(case), case["G"]
    of = torch.tensor(_kv_of(case), device=DEV)
    scale, cap = 1.0 / math.sqrt(d), case["cap"]
    q = s["q"].float().view(S, B, T, d)
    k = s["k"].float().view(G, B, T, d)[of]
    v = s["v"].float().view(G, B, T, d)[of]
    t = torch.arange(T, device=DEV)
    allowed = (t >= s["begin"].view(B, T, 1)) & (t < s["end"].view(B, T, 1))
    sc = torch.matmul(q, k.transpose(-1, -2)) * scale
    th = None
    if cap > 0:
        th = torch.tanh(sc / cap)
        sc = cap * th
    if s["slopes"] is not None:
        sc = sc - s["slopes"].view(S, 1, 1, 1) * (t[:, None] - t[None, :]).abs()
    p = _plain_probs(sc, allowed)
    del sc
    o = torch.matmul(p, v)
    out = o.to(torch.bfloat16).view(S, B * T, d)
    if case["dir"] == "fwd":
        return out
    do = s["do"].float().view(S, B, T, d)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True))
    if th is not None:
        ds = ds * (1.0 - th * th)
    dq = torch.matmul(ds, k) * scale
    dk = torch.matmul(ds.transpose(-1, -2), q) * scale
    gk = torch.zeros(G, B, T, d, device=DEV).index_add_(0, of, dk)
    gv = torch.zeros(G, B, T, d, device=DEV).index_add_(0, of, dv)
    bf = torch.bfloat16
    return out, dq.to(bf).view(S, B * T, d), gk.to(bf).view(G, B * T, d), gv.to(bf).view(G, B * T, d)


def _plain_decode(s):
    case = s["case"]
    B, L, d, S = case["B"], case["T"], case["d"], _streams(case)
    of = torch.tensor(_kv_of(case), device=DEV)
    sc = torch.matmul(s["kc"].float()[of], s["q"].float()[..., None])[..., 0] / math.sqrt(d)
    if case["cap"] > 0:
        sc = case["cap"] * torch.tanh(sc / case["cap"])
    u = torch.arange(L, device=DEV)
    pos = s["pos"].view(B, 1)
    if s["slopes"] is not None:
        sc = sc - s["slopes"].view(S, 1, 1) * (pos - u).abs()
    allowed = u <= pos
    if s["begin"] is not None:
        allowed = allowed & (u >= s["begin"].view(B, 1))
    p = _plain_probs(sc, allowed.expand(S, B, L))
    return torch.matmul(p[..., None, :], s["vc"].float()[of])[..., 0, :].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------------------
def _own_qk(s):
    from moe_query_head_b200 import gqe as GQ
    case = s["case"]
    how = dict(norm=case["norm"], q_weight=s["qw"], k_weight=s["kw"], eps=EPS,
               inv_freq=s["inv_freq"] if case["rot"] else None, interleaved=case["inter"])
    if case["dir"] == "append":
        GQ.gqe_qk_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["q_out"], s["kc"], s["vc"], **how)
        return s["q_out"], s["kc"], s["vc"]
    GQ.gqe_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], positions=s["pos"], **how)
    if case["dir"] == "fwd":
        return s["q_out"], s["k_out"]
    GQ.gqe_qk_norm_rope_backward(s["q"], s["k"], s["dqo"], s["dko"], s["dq"], s["dk"], s["dqw"], s["dkw"],
                                 positions=s["pos"], **how)
    return s["q_out"], s["k_out"], s["dq"], s["dk"], s["dqw"], s["dkw"]


def _own_attention(s):
    from moe_query_head_b200 import gqe as GQ
    case = s["case"]
    how = dict(softcap=case["cap"], slopes=s["slopes"])
    if case["dir"] == "decode":
        GQ.gqe_attention_decode(s["q"], s["kc"], s["vc"], s["pos"], s["out"], case["k"],
                                key_begin=s["begin"], **how)
        return s["out"]
    mask = case["mask"]
    how.update(causal=s["causal"], key_begin=s["begin"] if mask in ("docs", "window") else None,
               key_end=s["end"] if mask in ("prefix", "padded") else None)
    B, T = case["B"], case["T"]
    GQ.gqe_attention_forward(s["q"], s["k"], s["v"], s["out"], s["lse"], B, T, case["k"], **how)
    if case["dir"] == "fwd":
        return s["out"]
    GQ.gqe_attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["do"], s["dq"], s["dk"], s["dv"],
                              B, T, case["k"], **how)
    return s["out"], s["dq"], s["dk"], s["dv"]


def run(state):
    case = state["case"]
    if case["op"] == "qk":
        return _own_qk(state) if own else _plain_qk(state)
    if own:
        return _own_attention(state)
    return _plain_decode(state) if case["dir"] == "decode" else _plain_attention(state)


# ---------------------------------------------------------------------------------------
# 64 bits, from the definitions: complex rotations, one sequence and stream at a time, and
# gradients by differentiation
# ---------------------------------------------------------------------------------------
def _exact_qk_one(x, w, turn, case):
    """One tensor's rows in float64 (differentiable): norm, then each pair times exp(i angle)."""
    if case["norm"]:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["d"] + EPS) * w
    r = case["rot"]
    if r == 0:
        return x
    head = x[..., :r]
    if case["inter"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * turn
        y = torch.view_as_real(z).reshape(head.shape)
    else:
        z = torch.complex(head[..., : r // 2], head[..., r // 2:]) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., r:]], -1)


def _exact_qk(s):
    case = s["case"]
    q, k, qw, kw = (s[n].double().requires_grad_() for n in ("q", "k", "qw", "kw"))
    angle = torch.outer(s["pos"].double(), s["inv_freq"])
    turn = torch.polar(torch.ones_like(angle), angle)
    yq, yk = _exact_qk_one(q, qw, turn, case), _exact_qk_one(k, kw, turn, case)
    if case["dir"] == "fwd":
        return yq.detach(), yk.detach()
    if case["dir"] == "append":
        kc, vc = s["kc"].double(), s["vc"].double()
        for b, p in enumerate(s["pos"].tolist()):
            kc[:, b, p], vc[:, b, p] = yk.detach()[:, b], s["v"][:, b].double()
        return yq.detach(), kc, vc
    ((yq * s["dqo"].double()).sum() + (yk * s["dko"].double()).sum()).backward()
    zero = torch.zeros_like(qw)
    return (yq.detach(), yk.detach(), q.grad, k.grad, qw.grad if qw.grad is not None else zero,
            kw.grad if kw.grad is not None else zero)


def _exact_rows(q, k, v, t, u, begin, end, cap, slope):
    """Rows q at positions t over keys k, v at positions u, in float64."""
    z = (q @ k.T) / math.sqrt(q.shape[-1])
    if cap > 0:
        z = torch.tanh(z / cap) * cap
    if slope:
        z = z - slope * (t[:, None] - u[None, :]).abs().double()
    hidden = (u[None, :] < begin[:, None]) | (u[None, :] >= end[:, None])
    empty = hidden.all(-1)
    z = z.masked_fill(hidden, -math.inf).masked_fill(empty[:, None], 0.0)
    w = (z - torch.logsumexp(z, -1, keepdim=True)).exp().masked_fill(empty[:, None], 0.0)
    return w @ v


def _exact_attention(s):
    case = s["case"]
    B, T, d, S, G = case["B"], case["T"], case["d"], _streams(case), case["G"]
    of = _kv_of(case)
    train = case["dir"] == "train"
    q, k, v = (s[n].double().view(-1, B, T, d).requires_grad_(train) for n in ("q", "k", "v"))
    begin, end = s["begin"].view(B, T), s["end"].view(B, T)
    slopes = s["slopes"].double().tolist() if s["slopes"] is not None else [0.0] * S
    u = torch.arange(T, device=DEV)
    out = torch.empty(S, B, T, d, dtype=torch.float64, device=DEV)
    step = 4096
    for b in range(B):
        for i in range(S):
            for t0 in range(0, T, step):
                rows = slice(t0, min(T, t0 + step))
                o = _exact_rows(q[i, b, rows], k[of[i], b], v[of[i], b], u[rows], u, begin[b, rows],
                                end[b, rows], case["cap"], slopes[i])
                if train:
                    (o * s["do"].double().view(S, B, T, d)[i, b, rows]).sum().backward()
                out[i, b, rows] = o.detach()
    out = out.view(S, B * T, d)
    return (out, q.grad.view(S, B * T, d), k.grad.view(G, B * T, d), v.grad.view(G, B * T, d)) if train else out


def _exact_decode(s):
    case = s["case"]
    S, B = _streams(case), case["B"]
    of = _kv_of(case)
    slopes = s["slopes"].double().tolist() if s["slopes"] is not None else [0.0] * S
    out = torch.zeros(S, B, case["d"], dtype=torch.float64, device=DEV)
    first = s["begin"].tolist() if s["begin"] is not None else [0] * B
    for b, p in enumerate(s["pos"].tolist()):
        u = torch.arange(first[b], p + 1, device=DEV)
        one = torch.tensor([0], device=DEV)
        for i in range(S):
            out[i, b] = _exact_rows(s["q"][i, b: b + 1].double(), s["kc"][of[i], b, u].double(),
                                    s["vc"][of[i], b, u].double(), one + p, u, one, one + p + 1,
                                    case["cap"], slopes[i])[0]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(state)
    return _exact_decode(state) if case["dir"] == "decode" else _exact_attention(state)
