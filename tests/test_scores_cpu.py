"""Operators without a handle, on the CPU: the library's refusals (nothing is launched), and the
64-bit forms the GPU tests compare with, against finite differences."""
import ctypes

import pytest
import torch

from tests import scores_ref as R

P = 4096  # an aligned address that is never read


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


def heads(G, H, d=48, M=8, data=P, hs=None, ts=None):
    return G.Heads(data, H, M * d if hs is None else hs, d if ts is None else ts)


def transform(G, **kw):
    a = dict(d_h=48, dtype=G.GQE_BF16, norm=1, eps=1e-6, q_weight=None, k_weight=None, rot_dim=48,
             interleaved=0, inv_freq=P)
    a.update(kw)
    return G.QkTransform(**a)


INV, UNS, WS = 1, 2, 3


@pytest.mark.parametrize("kw,want", [
    (dict(d_h=40, rot_dim=0), UNS), (dict(d_h=144, rot_dim=0), UNS), (dict(d_h=0, rot_dim=0), UNS),
    (dict(dtype=2), INV), (dict(norm=2), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(rot_dim=8), INV), (dict(rot_dim=64), INV), (dict(rot_dim=-16), INV),
    (dict(inv_freq=None), INV), (dict(inv_freq=P + 4), INV), (dict(interleaved=3), INV),
    (dict(q_weight=P + 1), INV)])
def test_transform_refusals(G, kw, want):
    r = ctypes.byref
    tr, q, k = transform(G, **kw), heads(G, 9), heads(G, 8)
    assert G.lib.gqe_qk_norm_rope(r(tr), 8, r(q), r(k), P, 0, r(q), r(k), None) == want
    assert G.lib.gqe_qk_norm_rope_backward(r(tr), 8, r(q), r(k), P, 0, r(q), r(k), r(q), r(k), None,
                                           None, None, 0, None) == want
    c = heads(G, 8, ts=20 * 48, hs=8 * 20 * 48)
    assert G.lib.gqe_qk_norm_rope_append(r(tr), 8, r(q), r(k), r(k), P, 20, r(q), r(c), r(c), None) == want


def test_tensor_refusals(G):
    r, tr = ctypes.byref, transform(G)
    q, k = heads(G, 9), heads(G, 8)

    def call(q=q, k=k, qo=q, ko=k, M=8, pos=P, T=0):
        return G.lib.gqe_qk_norm_rope(r(tr), M, r(q), r(k), pos, T, r(qo), r(ko), None)

    assert call(M=-1) == INV
    assert call(pos=None) == INV and call(pos=P + 2) == INV
    assert call(qo=heads(G, 8)) == INV  # head counts differ
    for bad in (heads(G, 9, data=None), heads(G, 9, data=P + 8), heads(G, 9, hs=4), heads(G, 9, ts=47),
                heads(G, 9, ts=52), heads(G, 9, hs=0), heads(G, -1), heads(G, 9, hs=1 << 40)):
        assert call(q=bad) == INV and call(qo=bad) == INV
    many = heads(G, 513)
    assert call(q=many, qo=many) == UNS
    assert G.lib.gqe_qk_norm_rope(None, 8, r(q), r(k), P, 0, r(q), r(k), None) == INV
    assert G.lib.gqe_qk_norm_rope(r(tr), 8, None, r(k), P, 0, r(q), r(k), None) == INV
    assert G.lib.gqe_qk_norm_rope(r(tr), 8, r(q), r(k), P, 0, None, r(k), None) == INV
    assert call(M=0, q=heads(G, 9, data=None), qo=heads(G, 9, data=None)) == 0


def test_backward_workspace(G):
    r, tr = ctypes.byref, transform(G)
    q, k = heads(G, 9), heads(G, 8)
    n = G.lib.gqe_qk_norm_rope_workspace_bytes(48)
    assert n > 0 and G.lib.gqe_qk_norm_rope_workspace_bytes(40) == -1

    def call(ws, size):
        return G.lib.gqe_qk_norm_rope_backward(r(tr), 8, r(q), r(k), P, 0, r(q), r(k), r(q), r(k), P, None,
                                               ws, size, None)

    assert call(None, n) == INV and call(P + 8, n) == INV and call(P, n - 1) == WS


def test_append_refusals(G):
    r, tr = ctypes.byref, transform(G)
    q, k, c = heads(G, 9), heads(G, 8), heads(G, 8, ts=20 * 48, hs=8 * 20 * 48)

    def call(v=k, pos=P, L=20, kc=c, vc=c, B=8):
        return G.lib.gqe_qk_norm_rope_append(r(tr), B, r(q), r(k), r(v), pos, L, r(q), r(kc), r(vc), None)

    assert call(v=heads(G, 7)) == INV and call(pos=None) == INV and call(pos=P + 1) == INV
    assert call(L=0) == INV and call(L=21) == INV  # sequences closer than L rows
    assert call(kc=heads(G, 7, ts=960)) == INV and call(B=-1) == INV and call(B=0) == 0


def scores(gqe, **kw):
    a = dict(B=2, T=4, G=8, k=1, S=9, d_h=48, causal=1, scale=0.0, softcap=0.0, slopes=None,
             key_begin=None, key_end=None)
    a.update(kw)
    return gqe.Scores(**a)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(G=0), INV), (dict(k=0), INV), (dict(S=10), INV),
    (dict(S=7), INV), (dict(causal=2), INV), (dict(scale=-1.0), INV), (dict(scale=float("inf")), INV),
    (dict(softcap=-2.0), INV), (dict(softcap=float("nan")), INV), (dict(slopes=P + 2), INV),
    (dict(key_begin=P + 1), INV), (dict(key_end=P + 3), INV), (dict(d_h=72), UNS), (dict(d_h=256), UNS),
    (dict(B=1 << 14, T=1 << 14), UNS), (dict(B=1, T=1 << 28), UNS)])
def test_attention_refusals(G, kw, want):
    r = ctypes.byref
    a, q, k = scores(G, **kw), heads(G, 9), heads(G, 8)
    assert G.lib.gqe_attention_forward(r(a), r(q), r(k), r(k), r(q), P, None) == want
    assert G.lib.gqe_attention_backward(r(a), r(q), r(k), r(k), r(q), P, r(q), r(q), r(k), r(k), P, 1 << 40,
                                        None) == want
    assert G.lib.gqe_attention_workspace_bytes(r(a)) == -1


def test_attention_tensor_refusals(G):
    r, a = ctypes.byref, scores(G)
    q, k = heads(G, 9), heads(G, 8)
    n = G.lib.gqe_attention_workspace_bytes(r(a))
    assert n >= 9 * 8 * 4

    def fwd(q=q, k=k, v=k, o=q, lse=P):
        return G.lib.gqe_attention_forward(r(a), r(q), r(k), r(v), r(o), lse, None)

    def bwd(lse=P, ws=P, size=n, dq=q, dk=k):
        return G.lib.gqe_attention_backward(r(a), r(q), r(k), r(k), r(q), lse, r(q), r(dq), r(dk), r(k), ws,
                                            size, None)

    for bad in (heads(G, 8), heads(G, 9, data=None), heads(G, 9, data=P + 2), heads(G, 9, ts=44)):
        assert fwd(q=bad) == INV and fwd(o=bad) == INV and bwd(dq=bad) == INV
    assert fwd(k=heads(G, 9)) == INV and fwd(v=heads(G, 7)) == INV and bwd(dk=heads(G, 7)) == INV
    assert fwd(lse=P + 2) == INV and bwd(lse=None) == INV
    assert bwd(ws=None) == INV and bwd(ws=P + 8) == INV and bwd(size=n - 1) == WS
    assert G.lib.gqe_attention_forward(None, r(q), r(k), r(k), r(q), P, None) == INV


def test_decode_refusals(G):
    r = ctypes.byref
    q, c = heads(G, 9, M=2), heads(G, 8, ts=20 * 48, hs=2 * 20 * 48)

    def call(pos=P, L=20, qq=q, o=q, kc=c, **kw):
        a = scores(G, **kw)
        return G.lib.gqe_attention_decode(r(a), r(qq), r(kc), r(c), L, pos, r(o), P, 0, None)

    assert call(pos=None) == INV and call(pos=P + 1) == INV and call(L=0) == INV and call(L=21) == INV
    assert call(qq=heads(G, 8)) == INV and call(o=heads(G, 9, data=P + 2)) == INV
    assert call(kc=heads(G, 7, ts=960)) == INV
    assert call(G=1, k=9, S=9) == UNS and call(B=65536) == UNS and call(d_h=20) == UNS
    assert call(L=(1 << 30) + 1) == UNS and call(scale=-1.0) == INV and call(key_begin=P + 1) == INV
    assert G.lib.gqe_attention_decode_workspace_bytes(r(scores(G, G=0)), 20) == -1
    assert G.lib.gqe_attention_decode_workspace_bytes(r(scores(G)), 0) == -1
    assert call(B=0) == 0


def test_binding_refuses_mismatched_tensors(G):
    """Sizes, types and devices that the library cannot see."""
    bf = torch.bfloat16
    q, k = torch.zeros(9, 8, 48, dtype=bf), torch.zeros(8, 8, 48, dtype=bf)
    f = torch.zeros(24, dtype=torch.float64)
    lse = torch.zeros(9, 8)

    def refused(fn, *a, **kw):
        with pytest.raises(G.GQEError) as e:
            fn(*a, **kw)
        assert e.value.status == G.GQE_ERR_INVALID_ARG

    refused(G.gqe_qk_norm_rope, q, k, q, k, inv_freq=f)  # not on a GPU
    refused(G.gqe_qk_norm_rope, q, k, q.float(), k)
    refused(G.gqe_qk_norm_rope, q, k[:, :4], q, k)
    refused(G.gqe_qk_norm_rope, q, k, q, k, q_weight=torch.ones(47))
    refused(G.gqe_qk_norm_rope, q, k, q, k, inv_freq=f.float())
    refused(G.gqe_qk_norm_rope, q, k, q, k, positions=torch.zeros(8, dtype=torch.int64))
    refused(G.gqe_qk_norm_rope, q.half(), k, q, k)
    refused(G.gqe_attention_forward, q, k, k, q, lse, 2, 5, 1)  # B T is not the rows
    refused(G.gqe_attention_forward, q, k, k, q, lse[:4], 2, 4, 1)
    refused(G.gqe_attention_forward, q, k, k, q, lse, 2, 4, 1)  # not on a GPU
    refused(G.gqe_attention_forward, q, k, k, q, lse, 2, 4, 1, key_begin=torch.zeros(7, dtype=torch.int32))
    refused(G.gqe_attention_forward, q[..., ::2], k, k, q, lse, 2, 4, 1)
    refused(G.gqe_attention_decode, q, k, k, torch.zeros(8, dtype=torch.int32), q, 1)


def difference(f, x, h=1e-5):
    """Central differences of a scalar function of every element of x."""
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        e = torch.zeros_like(x).view(-1)
        e[i] = h
        e = e.view_as(x)
        g.view(-1)[i] = (f(x + e) - f(x - e)) / (2 * h)
    return g


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_attention_form_against_differences(cap):
    g = torch.Generator().manual_seed(0)
    B, T, Gk, k, d = 1, 6, 1, 1, 4
    q, kk, v, do = (torch.randn(n, T, d, generator=g, dtype=torch.float64) for n in (2, 1, 1, 2))
    sl = torch.tensor([0.3, 0.05])
    b = torch.tensor([0, 0, 2, 2, 4, 9])
    _, _, grads = R.attention_all(q, kk, v, B, T, Gk, k, 1, b, None, cap, sl, 0.0, do)

    def loss(q_, k_, v_):
        out = torch.zeros_like(q)
        # the definition once more, term by term
        for s in range(2):
            for t in range(T):
                us = [u for u in range(T) if int(b[t]) <= u <= t]
                if not us:
                    continue
                z = torch.stack([(q_[s, t] * k_[0, u]).sum() / 2.0 for u in us])
                z = cap * torch.tanh(z / cap) if cap else z
                z = z - sl[s].double() * torch.tensor([float(t - u) for u in us])
                w = torch.exp(z - z.max())
                out[s, t] = sum(wi * v_[0, u] for wi, u in zip(w / w.sum(), us))
        return (out * do).sum()

    for n, x, f in (("dq", q, lambda x: loss(x, kk, v)), ("dk", kk, lambda x: loss(q, x, v)),
                    ("dv", v, lambda x: loss(q, kk, x))):
        # differences of step 1e-5: h^2 and 1e-16 / h both near 1e-10 of values of size 10
        assert (difference(f, x) - grads[n]).abs().max() < 1e-7


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_form_against_differences(inter):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 3, 32, generator=g, dtype=torch.float64)
    w = torch.randn(32, generator=g, dtype=torch.float64)
    gy = torch.randn(2, 3, 32, generator=g, dtype=torch.float64)
    ang = torch.randn(3, 8, generator=g, dtype=torch.float64) * 5
    f = lambda x, w: (R.norm_rope(x, w, ang, True, 1e-6, 16, inter) * gy).sum()  # noqa: E731
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    f(xg, wg).backward()
    assert (difference(lambda t: f(t, w), x) - xg.grad).abs().max() < 1e-7
    assert (difference(lambda t: f(x, t), w) - wg.grad).abs().max() < 1e-7
    # a rotation keeps every pair's length
    y = R.norm_rope(x, w, ang, False, 0.0, 16, inter)
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))


def test_layer_options_without_a_handle(G):
    assert G.lib.gqe_set_qk_transform(None, ctypes.byref(transform(G)), None, None, None) == INV
    assert G.lib.gqe_set_qk_transform(None, None, None, None, None) == INV
    assert G.lib.gqe_set_scores(None, 0.0, 1.0, None, None, None) == INV


@pytest.mark.parametrize("kw", [dict(softcap=2.0 ** -14), dict(softcap=1e4), dict(softcap=1.0, scale=2.0 ** 61)])
def test_caps_out_of_range(G, kw):
    """Caps whose tanh float32 cannot give (its error is 1e-7 of the cap) are refused."""
    r = ctypes.byref
    a, q, k = scores(G, **kw), heads(G, 9), heads(G, 8)
    c = heads(G, 8, ts=20 * 48, hs=2 * 20 * 48)
    assert G.lib.gqe_attention_forward(r(a), r(q), r(k), r(k), r(q), P, None) == UNS
    assert G.lib.gqe_attention_backward(r(a), r(q), r(k), r(k), r(q), P, r(q), r(q), r(k), r(k), P, 1 << 40,
                                        None) == UNS
    assert G.lib.gqe_attention_workspace_bytes(r(a)) == -1
    q = heads(G, 9, M=2)
    assert G.lib.gqe_attention_decode(r(a), r(q), r(c), r(c), 20, P, r(q), P, 0, None) == UNS
    assert G.lib.gqe_attention_decode_workspace_bytes(r(a), 20) == -1


@pytest.mark.parametrize("kw", [dict(softcap=-1.0), dict(softcap=float("nan")), dict(norm_eps=-1e-6),
                                dict(rope_dim=32), dict(rope_base=0.0), dict(rope_base=-1e4),
                                dict(rope_base=1e4, rope_dim=-16)])
def test_module_option_values(kw):
    from moe_query_head_b200.module import GQEAttention
    with pytest.raises(ValueError):
        GQEAttention(64, 4, 2, head_dim=32, **kw)


def test_module_options_are_checked():
    from moe_query_head_b200.module import GQEAttention, document_spans, prefix_spans
    with pytest.raises(ValueError):
        GQEAttention(64, 4, 2, head_dim=32, rope_base=1e4, rope_dim=24)
    with pytest.raises(ValueError):
        GQEAttention(64, 4, 2, head_dim=32, rope_base=1e4, rope_dim=48)
    with pytest.raises(ValueError):
        GQEAttention(64, 4, 2, slopes=[0.1, 0.2])  # three streams
    with pytest.raises(ValueError):
        GQEAttention(64, 4, 2, slopes="other")
    m = GQEAttention(64, 4, 2, qk_norm=True, rope_base=1e4, slopes="geometric")
    assert {n for n, _ in m.named_parameters()} >= {"q_norm", "k_norm"}
    with pytest.raises(ValueError):
        m._ints(torch.zeros(3), 4, "cpu")
    for bad in (torch.zeros(3, dtype=torch.int32), torch.zeros(2)):  # size, type
        with pytest.raises(ValueError):
            m.decode_step(torch.zeros(2, 64), None, None, None, bad)
    b, e = document_spans([2, 0, 3], 7)
    assert b.tolist() == [0, 0, 2, 2, 2, 0, 0] and e.tolist() == [2, 2, 5, 5, 5, 0, 0]
    with pytest.raises(ValueError):
        document_spans([5, 3], 7)
    assert prefix_spans(3, 5).tolist() == [3, 3, 3, 4, 5] and prefix_spans(9, 2).tolist() == [2, 2]
