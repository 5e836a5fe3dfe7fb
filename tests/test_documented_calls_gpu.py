"""Calls of the operators that their documentation allows beside the ordinary ones: in place, other
cache layouts, many streams a KV head, many short sequences, offsets past 2^31."""
import pytest
import torch

from tests import scores_ref as R
from tests.test_attention_scores_gpu import Run, decode_ref, rows

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("d", [48, 112, 128])
@pytest.mark.parametrize("major", ["heads", "tokens"])
def test_in_place(G, d, dt, major):
    """Forward and gradients written over their inputs."""
    M = 150
    q, k, gq, gk = (rows(h, M, d, i, 1.0, major).to(dt) for i, h in enumerate((5, 3, 5, 3)))
    f = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    for norm in (True, False):
        how = dict(norm=norm, q_weight=w, k_weight=w, inv_freq=f)
        out = [torch.empty_like(x) for x in (q, k, gq, gk)]
        dw = torch.empty(4, d, device="cuda")
        G.gqe_qk_norm_rope(q, k, out[0], out[1], **how)
        G.gqe_qk_norm_rope_backward(q, k, gq, gk, out[2], out[3], dw[0], dw[1], **how)
        same = [x.clone() for x in (q, k, gq, gk)]
        G.gqe_qk_norm_rope_backward(q, k, same[2], same[3], same[2], same[3], dw[2], dw[3], **how)
        G.gqe_qk_norm_rope(same[0], same[1], same[0], same[1], **how)
        for a, b in zip(out, same):
            assert torch.equal(a, b)
        assert torch.equal(dw[:2], dw[2:])


@pytest.mark.parametrize("window", [False, True])
def test_caches_by_sequence(G, window):
    """Caches stored [B, G, L_max, d_h] and inside larger ones."""
    B, L, Gk, k, d = 4, 200, 2, 1, 48
    q = rows(Gk * k + 1, B, d, 1)
    kn, vn = rows(Gk, B, d, 2), rows(Gk, B, d, 3)
    pos = torch.tensor([0, 199, 77, 130], dtype=torch.int32)
    begin = torch.tensor([0, 150, 70, 131], dtype=torch.int32).cuda() if window else None
    big = [rows(B * (Gk + 1), L + 9, d, s).view(B, Gk + 1, L + 9, d) for s in (4, 5)]
    kc, vc = (c[:, 1:, :L].transpose(0, 1) for c in big)
    before = [c.clone() for c in big]
    qo = torch.empty_like(q)
    G.gqe_qk_norm_rope_append(q, kn, vn, pos.cuda(), qo, kc, vc, norm=False)
    for b in range(B):
        assert torch.equal(kc[:, b, int(pos[b])], kn[:, b]) and torch.equal(vc[:, b, int(pos[b])], vn[:, b])
        for c, x in zip(before, (kn, vn)):
            c[b, 1:, int(pos[b])] = x[:, b]
    for a, b in zip(before, big):
        assert torch.equal(a, b)
    out = torch.empty_like(q)
    G.gqe_attention_decode(qo, kc, vc, pos.cuda(), out, k, key_begin=begin)
    assert G.gqe_check_op_status() == G.GQE_OK
    ref, mag = decode_ref(qo, kc, vc, pos, begin, k, 0.0, None)
    # float32 throughout, one rounding: scores of size 8 carry 64 roundings of 2^-24
    assert ((out.double().cpu() - ref).abs() <= R.BF16 * ref.abs() + 2.0 ** -15 * mag).all()


@pytest.mark.parametrize("shape,kind", [((1, 140, 1, 17, 1, 48), "causal"), ((1, 90, 2, 9, 0, 128), "docs"),
                                        ((70, 3, 2, 1, 1, 64), "causal"), ((60, 5, 1, 2, 1, 96), "padded")])
def test_many_streams_and_short_sequences(G, shape, kind):
    Run(G, *shape, kind, 20.0, True, seed=3).check()


@pytest.mark.parametrize("d,S,Gk,k", [(128, 17, 16, 1), (48, 45, 4, 11)])
def test_offsets_past_32_bits(G, d, S, Gk, k):
    """2^20 and one tokens in windows of 40, more than 2^31 values in q: the last rows of the last
    streams, forward and gradients, against the same rows alone (a window only sees its own)."""
    T, w, n = (1 << 20) + 1, 40, 600
    g = torch.Generator(device="cuda").manual_seed(1)
    assert S * T * d > 1 << 31
    q, do = (torch.empty(S, T, d, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))
    kk, v = (torch.empty(Gk, T, d, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))

    def run(q, kk, v, do, T):
        begin = torch.arange(T, dtype=torch.int32, device="cuda") + 1 - w
        out, lse = torch.empty_like(q), torch.empty(S, T, device="cuda")
        dq, dk, dv = torch.empty_like(q), torch.empty_like(kk), torch.empty_like(v)
        G.gqe_attention_forward(q, kk, v, out, lse, 1, T, k, key_begin=begin, softcap=30.0)
        G.gqe_attention_backward(q, kk, v, out, lse, do, dq, dk, dv, 1, T, k, key_begin=begin, softcap=30.0)
        assert G.gqe_check_op_status() == G.GQE_OK
        return out, lse, dq, dk, dv

    big = run(q, kk, v, do, T)
    part = run(*(x[:, T - n:].contiguous() for x in (q, kk, v, do)), n)
    # rows whose whole window, and keys whose queries, are in the part. Key tiles start elsewhere in
    # it, so sums are taken in another order: bf16 weights (2^-8) and exponentials (2^-9) of the same
    # values either way. Weights of 40 keys and gradients of 12 streams in the 2-norm.
    for a, b in zip(big, part):
        a, b = a[:, T - n + 2 * w:].double(), b[:, 2 * w:].double()
        assert ((a - b).norm() / b.norm()) <= 2 * 3 * R.BF16
        assert ((a[-1] - b[-1]).norm() / b[-1].norm()) <= 2 * 3 * R.BF16
    del big, part
    f = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    a = [torch.empty_like(q), torch.empty_like(kk)]
    G.gqe_qk_norm_rope(q, kk, *a, positions=pos, inv_freq=f)
    b = [torch.empty_like(x[:, T - n:]).contiguous() for x in (q, kk)]
    G.gqe_qk_norm_rope(q[:, T - n:].contiguous(), kk[:, T - n:].contiguous(), *b, positions=pos[T - n:], inv_freq=f)
    for x, y in zip(a, b):
        assert torch.equal(x[:, T - n:], y)
    G.gqe_qk_norm_rope_backward(q, kk, do, v, *a, positions=pos, inv_freq=f)
    G.gqe_qk_norm_rope_backward(*(x[:, T - n:].contiguous() for x in (q, kk, do, v)), *b, positions=pos[T - n:],
                                inv_freq=f)
    for x, y in zip(a, b):
        assert torch.equal(x[:, T - n:], y)
