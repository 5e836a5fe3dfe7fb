"""Attention with capped, biased and masked scores against its 64-bit form: outputs and
gradients within the bounds of their roundings (tests/scores_ref.py)."""
import math

import pytest
import torch

from tests import scores_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


def rows(H, M, d, seed, scale=1.0, major="heads"):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(H, M, d, generator=g) * scale).to(BF).cuda()
    if major == "tokens":
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    return x


def documents(T, cuts):
    """First key and end of every token's document, for documents that begin at `cuts`."""
    edges = sorted({0, T, *[c for c in cuts if 0 < c < T]})
    b, e = torch.zeros(T, dtype=torch.int32), torch.zeros(T, dtype=torch.int32)
    for lo, hi in zip(edges, edges[1:]):
        b[lo:hi], e[lo:hi] = lo, hi
    return b, e


def mask(kind, B, T, seed):
    """causal, key_begin, key_end of a named mask."""
    t = torch.arange(T, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed)
    if kind == "causal":
        return 1, None, None
    if kind == "full":
        return 0, None, None
    if kind in ("docs", "docs_both"):
        cuts = [torch.randint(1, max(T, 2), (5,), generator=g).tolist() for _ in range(B)]
        d = [documents(T, c) for c in cuts]
        begin, end = torch.cat([x[0] for x in d]), torch.cat([x[1] for x in d])
        return (1, begin, None) if kind == "docs" else (0, begin, end)
    if kind == "prefix":
        return 0, None, torch.cat([torch.clamp(t + 1, min=min(T, T // 3 + b)) for b in range(B)])
    if kind == "window":
        return 1, torch.cat([t + 1 - max(1, T // 4)] * B), None  # negative begins are cut to 0
    if kind == "padded":  # rows behind each sequence see nothing
        n = [max(0, T - (b * T) // 3 - 1) for b in range(B)]
        return 0, None, torch.cat([torch.where(t < m, m, 0).to(torch.int32) for m in n])
    if kind == "random":  # any intervals, empty and reversed ones and ends behind T among them
        b = torch.randint(-3, T + 2, (B * T,), generator=g, dtype=torch.int32)
        return 0, b, b + torch.randint(-20, T, (B * T,), generator=g, dtype=torch.int32)
    if kind == "nothing":
        return 0, torch.full((B * T,), 5, dtype=torch.int32), torch.full((B * T,), 5, dtype=torch.int32)
    raise ValueError(kind)


class Run:
    """One forward and backward on the GPU, and their 64-bit forms."""

    def __init__(self, G, B, T, Gk, k, shared, d, kind, cap, bias, *, sharp=1.5, major="heads",
                 scale=0.0, seed=0, slopes=None, poison=None, grad=True):
        S, M = Gk * k + shared, B * T
        self.q, self.k = rows(S, M, d, seed, sharp, major), rows(Gk, M, d, seed + 1, 1.0, major)
        self.v, self.do = rows(Gk, M, d, seed + 2, 1.0, major), rows(S, M, d, seed + 3, 1.0, major)
        clean = [x.double().cpu() for x in (self.q, self.k, self.v, self.do)]
        if poison is not None:
            for x in (self.q, self.k, self.v, self.do):
                x[:, poison] = float("nan")
        causal, kb, ke = mask(kind, B, T, seed)
        if bias and slopes is None:
            slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / S) for i in range(S)])
        on = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.how = dict(causal=causal, scale=scale, softcap=cap, slopes=on(slopes), key_begin=on(kb),
                        key_end=on(ke))
        nan = float("nan")
        self.out, self.dq = torch.full_like(self.q, nan), torch.full_like(self.q, nan)
        self.dk, self.dv = torch.full_like(self.k, nan), torch.full_like(self.v, nan)
        self.lse = torch.full((S, M), nan, device="cuda")
        self.args = (B, T, k)
        G.gqe_attention_forward(self.q, self.k, self.v, self.out, self.lse, *self.args, **self.how)
        if grad:
            G.gqe_attention_backward(self.q, self.k, self.v, self.out, self.lse, self.do, self.dq,
                                     self.dk, self.dv, *self.args, **self.how)
        assert G.gqe_check_op_status() == G.GQE_OK
        self.ref = R.attention_all(clean[0], clean[1], clean[2], B, T, Gk, k, causal, kb, ke, cap,
                                   slopes, scale, clean[3] if grad else None)
        self.begin, self.end = R.spans(B, T, causal, kb, ke)

    def check(self, grad=True, skip=None):
        out, mag, g = self.ref
        keep = torch.ones(out.shape[1], dtype=torch.bool)
        if skip is not None:
            keep[skip] = False
        # weights in bf16 and exponentials to 2^-9: 3 half steps in the numerator and the row's
        # sum together; one more in the output
        pairs = [("out", self.out, out, 3 * R.BF16 * mag + R.BF16 * out.abs())]
        if grad:
            for n in ("dq", "dk", "dv"):
                pairs.append((n, getattr(self, n), g[n], g["e" + n] + R.BF16 * g[n].abs()))
        for n, got, want, tol in pairs:
            x = got.double().cpu()
            if n in ("out", "dq"):
                x, want, tol = x[:, keep], want[:, keep], tol[:, keep]
            else:
                x, want, tol = x[:, keep], want[:, keep], tol[:, keep]
            err = (x - want).abs()
            assert not x.isnan().any(), n
            assert (err <= tol + 1e-6).all(), (n, float((err - tol).max()), float(err.max()))
        empty = (self.begin >= self.end).view(-1) & keep
        assert (self.out[:, empty.cuda()] == 0).all()
        assert (self.lse.cpu()[:, empty] == -math.inf).all()
        if grad:
            assert (self.dq[:, empty.cuda()] == 0).all()


SHAPES = [  # B, T, G, k, shared, d
    (1, 1, 1, 1, 0, 16),
    (2, 2, 2, 1, 1, 48),
    (1, 64, 1, 2, 1, 32),
    (3, 127, 2, 1, 1, 64),
    (1, 128, 1, 1, 1, 80),
    (2, 129, 2, 2, 1, 96),
    (1, 300, 2, 1, 1, 48),
    (1, 333, 1, 3, 0, 112),
    (2, 257, 1, 1, 1, 128),
    (1, 700, 1, 1, 1, 16),
]
MASKS = ["causal", "full", "docs", "docs_both", "prefix", "window", "padded", "random", "nothing"]


@pytest.mark.parametrize("kind", MASKS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_masks(G, shape, kind):
    """Every mask at every shape; cap and bias alternate over the pairs so that each mask and
    each shape meets all four forms of the score."""
    form = (SHAPES.index(shape) + MASKS.index(kind)) % 4
    r = Run(G, *shape, kind, 20.0 if form & 1 else 0.0, bool(form & 2), seed=SHAPES.index(shape))
    r.check()


@pytest.mark.parametrize("kind", ["causal", "full", "docs", "padded", "random", "nothing"])
@pytest.mark.parametrize("T,d", [(1030, 16), (1100, 48), (2060, 64), (2050, 48)])
def test_split_gradients(G, T, d, kind):
    """Lengths at which two or four CTAs share a query tile's steps (and a key tile's jobs), some
    of them with none."""
    Run(G, 1, T, 1, 1, 1, d, kind, 0.0, False, seed=T).check()


@pytest.mark.parametrize("cap", [2.0 ** -13, 2.0 ** 13])
def test_smallest_and_largest_cap(G, cap):
    """At the largest cap a score is off by 8e-4 (the tanh's error times the cap), a fifth of a half
    step of its weight: inside the three that the bound of check() counts."""
    Run(G, 1, 200, 2, 1, 1, 48, "docs", cap, False).check()


@pytest.mark.parametrize("d", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True), (50.0, True)])
def test_head_dims(G, d, cap, bias):
    Run(G, 1, 260, 2, 1, 1, d, "docs", cap, bias, seed=d, sharp=2.0).check()


def test_token_major_strides(G):
    Run(G, 2, 150, 2, 2, 1, 48, "docs", 30.0, True, major="tokens", seed=4).check()


def test_scale_and_steep_bias(G):
    """A given scale; slopes so steep that far keys vanish and first tiles lie far below zero."""
    Run(G, 1, 400, 2, 1, 1, 48, "full", 0.0, True, scale=0.05, seed=5,
        slopes=torch.tensor([4.0, 0.0, -0.01])).check()


def test_rows_far_below_zero(G):
    """Scores near -300 in rows whose first key tiles are masked: nothing is lost to the
    reference of a masked tile."""
    B, T, d = 1, 300, 48
    q, k, v = rows(1, T, d, 1), rows(1, T, d, 2), rows(1, T, d, 3)
    q[:] = 8.0
    k[:] = -(43.0 + 0.02 * torch.randn(1, T, d, generator=torch.Generator().manual_seed(9)).cuda()).to(BF)
    begin = torch.full((T,), 200, dtype=torch.int32)
    out, lse = torch.empty_like(q), torch.empty(1, T, device="cuda")
    G.gqe_attention_forward(q, k, v, out, lse, B, T, 1, causal=0, key_begin=begin.cuda())
    ref, mag, _ = R.attention_all(*[x.double().cpu() for x in (q, k, v)], B, T, 1, 1, 0, begin, None,
                                  0.0, None, 0.0)
    err = (out.double().cpu() - ref).abs()
    # scores of size 2380 in float32 products: 2^-24 x 2380 x 8 relative in a weight
    assert (err <= (4 * R.BF16 + 2.0 ** -24 * 2380 * 8) * mag).all()


@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("kind", ["padded", "docs_both", "window"])
def test_masked_places_hold_anything(G, d, kind):
    """NaN in the rows that others cannot see reaches nobody else, forward or backward."""
    B, T = 2, 200
    if kind == "padded":
        poison = [i for b in range(B) for i in range(b * T + max(0, T - (b * T) // 3 - 1), b * T + T)]
        r = Run(G, B, T, 2, 1, 1, d, kind, 0.0, False, poison=poison, seed=1)
        r.check(skip=poison)
    elif kind == "docs_both":
        # one document of the first sequence is NaN: its rows are NaN, all others clean
        _, kb, ke = mask(kind, B, T, 2)
        lo, hi = int(kb[100]), int(ke[100])
        poison = list(range(lo, hi))
        r = Run(G, B, T, 2, 1, 1, d, kind, 30.0, True, poison=poison, seed=2)
        r.check(skip=poison)
        for x in (r.out, r.dq, r.dk, r.dv):
            assert x[:, poison].isnan().all()
    else:
        # token 0 leaves the windows of rows 50 and later
        r = Run(G, B, T, 2, 1, 1, d, kind, 0.0, True, poison=[0], seed=3)
        far = torch.ones(B * T, dtype=torch.bool)
        far[:100] = False  # rows that see token 0, and the keys whose gradients they feed
        got, (want, mag, _) = r.out.double().cpu(), r.ref
        assert ((got - want).abs() <= 4 * R.BF16 * mag + 1e-6)[:, far].all()
        assert r.out[:, :50].isnan().all()
        for n in ("dq", "dk", "dv"):
            assert not getattr(r, n)[:, far.cuda()].isnan().any()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_one_bad_value(G, bad):
    """One infinity or NaN in a value row: the rows that see it are NaN in that column (whether
    their tile is seen whole or in part), the others are untouched."""
    B, T, d, at, col = 1, 300, 48, 140, 7
    q, k, v = rows(2, T, d, 1), rows(1, T, d, 2), rows(1, T, d, 3)
    out = torch.empty_like(q)
    G.gqe_attention_forward(q, k, v, out, None, B, T, 1)
    v2 = v.clone()
    v2[0, at, col] = bad
    out2 = torch.empty_like(q)
    G.gqe_attention_forward(q, k, v2, out2, None, B, T, 1)
    assert not torch.isfinite(out2[:, at:, col]).any()
    out2[:, at:, col] = out[:, at:, col]
    assert torch.equal(out, out2)


@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("at", [3, 200, 333])
def test_one_nan_key(G, d, cap, at):
    """A NaN in one key row: every row that sees the key is NaN throughout, wherever the key lies
    in its tile, with a log-sum-exp of NaN; rows before it keep their bits. The gradients of
    the rows that see it are NaN."""
    B, T = 1, 400
    q, k, v = rows(2, T, d, 1), rows(1, T, d, 2), rows(1, T, d, 3)
    outs = []
    for key in (k, k.clone()):
        if outs:
            key[0, at, 5] = float("nan")
        out, lse = torch.empty_like(q), torch.empty(2, T, device="cuda")
        G.gqe_attention_forward(q, key, v, out, lse, B, T, 1, softcap=cap)
        outs.append((out, lse))
    (o0, l0), (o1, l1) = outs
    assert o1[:, at:].isnan().all() and l1[:, at:].isnan().all()
    assert torch.equal(o0[:, :at], o1[:, :at]) and torch.equal(l0[:, :at], l1[:, :at])
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    k[0, at, 5] = float("nan")
    G.gqe_attention_backward(q, k, v, o1, l1, q, dq, dk, dv, B, T, 1, softcap=cap)
    assert dq[:, at:].isnan().all() and not dq[:, :at].isnan().any()


def test_same_bits_streams_and_graph(G):
    """The same bits from run to run, on another stream, and from graphs replayed together."""
    B, T, Gk, k, d = 2, 300, 2, 1, 48
    r = Run(G, B, T, Gk, k, 1, d, "docs", 30.0, True, seed=7)
    first = [x.clone() for x in (r.out, r.lse, r.dq, r.dk, r.dv)]

    def call(t):
        G.gqe_attention_forward(r.q, r.k, r.v, t[0], t[1], *r.args, **r.how)
        G.gqe_attention_backward(r.q, r.k, r.v, t[0], t[1], r.do, t[2], t[3], t[4], *r.args, **r.how)

    outs = [[torch.empty_like(x) for x in first] for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs[0])
    torch.cuda.synchronize()
    graphs = []
    for o in outs[1:]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert G.gqe_check_op_status() == G.GQE_OK
    for o in outs:
        for a, b in zip(first, o):
            assert torch.equal(a, b)


def test_no_tokens(G):
    q, k = rows(2, 0, 48, 1), rows(1, 0, 48, 2)
    lse = torch.empty(2, 0, device="cuda")
    for B, T in ((0, 5), (3, 0)):
        G.gqe_attention_forward(q, k, k, q, lse, B, T, 2)
        G.gqe_attention_backward(q, k, k, q, lse, q, q, k, k, B, T, 2)


# ---------------------------------------------------------------------------------------
# One new token per sequence
# ---------------------------------------------------------------------------------------
def decode_ref(q, kc, vc, pos, begin, k, cap, slopes):
    S, B, d = q.shape
    of = R.kv_of(kc.shape[0], k, S)
    out, mag = torch.zeros(S, B, d, dtype=torch.float64), torch.zeros(S, B, d, dtype=torch.float64)
    for b in range(B):
        p = int(pos[b])
        lo = max(0, int(begin[b])) if begin is not None else 0
        if p < lo:
            continue
        for s in range(S):
            kk, vv = (c[of[s], b, lo:p + 1].double().cpu() for c in (kc, vc))
            sl = 0.0 if slopes is None else float(slopes[s])
            n = p + 1 - lo
            o, w = R.attention(q[s, b:b + 1].double().cpu(), kk, vv, torch.tensor([0]),
                               torch.tensor([n]), cap, sl, 1 / math.sqrt(d), torch.tensor([n - 1]))
            out[s, b], mag[s, b] = o[0], (w @ vv.abs())[0]
    return out, mag


@pytest.mark.parametrize("d,Gk,k,shared", [(16, 1, 1, 0), (32, 2, 2, 1), (48, 8, 1, 1), (64, 2, 4, 1),
                                           (80, 1, 8, 1), (96, 2, 1, 1), (112, 1, 3, 0), (128, 2, 2, 1)])
@pytest.mark.parametrize("cap,bias,window", [(0.0, False, False), (20.0, True, True)])
def test_decode(G, d, Gk, k, shared, cap, bias, window):
    B, L = 6, 700
    S = Gk * k + shared
    q = rows(S, B, d, 1, 2.0, "tokens")
    kc, vc = rows(Gk, B * L, d, 2).view(Gk, B, L, d), rows(Gk, B * L, d, 3).view(Gk, B, L, d)
    pos = torch.tensor([0, 63, 64, 699, -1, 300], dtype=torch.int32)
    for b in range(B):  # rows behind the position hold anything
        kc[:, b, int(pos[b]) + 1:] = float("nan")
        vc[:, b, int(pos[b]) + 1:] = float("inf")
    begin = None
    if window:
        begin = torch.tensor([-4, 60, 65, 500, 0, 300], dtype=torch.int32)  # sequence 2 sees nothing
        kc[:, 3, :500], vc[:, 3, :500] = float("nan"), float("nan")
    slopes = torch.tensor([2.0 ** (-i - 1) for i in range(S)]) if bias else None
    out = torch.full_like(q, float("nan"))
    on = lambda x: None if x is None else x.cuda()  # noqa: E731
    G.gqe_attention_decode(q, kc, vc, pos.cuda(), out, k, softcap=cap, slopes=on(slopes), key_begin=on(begin))
    assert G.gqe_check_op_status() == G.GQE_OK
    ref, mag = decode_ref(q, kc, vc, pos, begin, k, cap, slopes)
    # float32 throughout, one rounding: scores of size 8 carry 64 roundings of 2^-24
    err = (out.double().cpu() - ref).abs()
    assert (err <= R.BF16 * ref.abs() + 2.0 ** -15 * mag).all(), float(err.max())
    assert (out[:, 4] == 0).all()


def test_decode_bad_position(G):
    q, kc = rows(2, 3, 48, 1), rows(1, 3 * 10, 48, 2).view(1, 3, 10, 48)
    out = torch.full_like(q, 7.0)
    pos = torch.tensor([4, 10, -2], dtype=torch.int32, device="cuda")
    G.gqe_attention_decode(q, kc, kc, pos, out, 2)
    assert G.gqe_check_op_status() == G.GQE_ERR_INVALID_ARG
    assert G.gqe_check_op_status() == G.GQE_OK
    assert (out[:, 1:] == 7.0).all() and not (out[:, 0] == 7.0).all()


def test_decode_far_offsets(G):
    """A cache of more than 2^31 values per head: the last rows of the last sequence."""
    B, L, d = 2, (1 << 23) + 77, 128
    kc = torch.zeros(1, B, L, d, dtype=BF, device="cuda")
    vc = torch.zeros(1, B, L, d, dtype=BF, device="cuda")
    kc[0, 1, L - 300:], vc[0, 1, L - 300:] = rows(1, 300, d, 5)[0], rows(1, 300, d, 6)[0]
    q = rows(1, B, d, 7)
    pos = torch.tensor([0, L - 1], dtype=torch.int32)
    begin = torch.tensor([0, L - 290], dtype=torch.int32)
    out = torch.empty_like(q)
    G.gqe_attention_decode(q, kc, vc, pos.cuda(), out, 1, key_begin=begin.cuda(),
                           slopes=torch.tensor([0.01], device="cuda"))
    ref, mag = decode_ref(q, kc, vc, pos, begin, 1, 0.0, torch.tensor([0.01]))
    assert ((out.double().cpu() - ref).abs() <= R.BF16 * ref.abs() + 2.0 ** -15 * mag + 1e-30).all()


def test_append_decode_and_prefill_agree(G):
    """The operators together, as a user runs them: prefill of T tokens by norm, rotation and
    attention; the last token again by append and decode over the caches."""
    B, T, Gk, k, d = 3, 150, 2, 1, 48
    S = Gk * k + 1
    q, kx, v = rows(S, B * T, d, 1), rows(Gk, B * T, d, 2), rows(Gk, B * T, d, 3)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    f = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    tr = dict(q_weight=w, k_weight=w, inv_freq=f)
    sc = dict(softcap=15.0, slopes=torch.tensor([0.1, 0.02, 0.3], device="cuda"))
    qn, kn = torch.empty_like(q), torch.empty_like(kx)
    G.gqe_qk_norm_rope(q, kx, qn, kn, T=T, **tr)
    out = torch.empty_like(q)
    G.gqe_attention_forward(qn, kn, v, out, None, B, T, k, **sc)
    kc = torch.zeros(Gk, B, T + 5, d, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    kc[:, :, :T - 1], vc[:, :, :T - 1] = kn.view(Gk, B, T, d)[:, :, :T - 1], v.view(Gk, B, T, d)[:, :, :T - 1]
    last = lambda x: x.view(x.shape[0], B, T, d)[:, :, T - 1]  # noqa: E731
    pos = torch.full((B,), T - 1, dtype=torch.int32, device="cuda")
    q1 = torch.empty(S, B, d, dtype=BF, device="cuda")
    G.gqe_qk_norm_rope_append(last(q), last(kx), last(v), pos, q1, kc, vc, **tr)
    assert torch.equal(kc[:, :, T - 1], last(kn)) and torch.equal(q1, last(qn))
    o1 = torch.empty_like(q1)
    G.gqe_attention_decode(q1, kc, vc, pos, o1, k, **sc)
    assert G.gqe_check_op_status() == G.GQE_OK
    _, mag, _ = R.attention_all(*[x.double().cpu() for x in (qn, kn, v)], B, T, Gk, k, 1, None, None, 15.0,
                                sc["slopes"].cpu(), 0.0)
    assert ((o1.double() - last(out).double()).abs().cpu() <= 5 * R.BF16 * last(mag)).all()
