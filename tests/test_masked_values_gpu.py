"""Finite values of any size in masked places: the rows that do not see them keep their bits,
forward and backward. (A weight that is only nearly zero, times the largest bf16, is not.)"""
import pytest
import torch

from tests.test_attention_scores_gpu import mask, rows

pytestmark = pytest.mark.gpu
LARGEST = torch.finfo(torch.bfloat16).max


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


def run(G, t, B, T, k, grad=True, **how):
    """out, lse, dq, dk, dv of the tensors t = (q, k, v, dout)."""
    q, kk, v, do = t
    out, lse = torch.empty_like(q), torch.empty(q.shape[0], B * T, device="cuda")
    G.gqe_attention_forward(q, kk, v, out, lse, B, T, k, **how)
    g = [torch.empty_like(x) for x in (q, kk, v)]
    if grad:
        G.gqe_attention_backward(q, kk, v, out, lse, do, *g, B, T, k, **how)
    assert G.gqe_check_op_status() == G.GQE_OK
    return [out, lse, *g]


def tensors(S, Gk, M, d):
    return [rows(S, M, d, 1, 1.5), rows(Gk, M, d, 2), rows(Gk, M, d, 3), rows(S, M, d, 4)]


def signs(n, d):
    """+-1 in every combination of a row's and a column's parity."""
    return (1.0 - 2.0 * ((torch.arange(n)[:, None] + torch.arange(d)) % 2)).cuda().bfloat16()


@pytest.mark.parametrize("d", [32, 48, 64, 128])
@pytest.mark.parametrize("what", ["v", "kv"])
def test_future_token(G, d, what):
    """A later token's key and value at every place of sixteen neighbours: the rows before it see
    a causal mask end inside their tile."""
    T = 170
    clean = tensors(2, 1, T, d)
    want = run(G, clean, 1, T, 2)
    for at in range(130, 146):
        t = [x.clone() for x in clean]
        for x in t[1 if what == "kv" else 2:3]:
            x[:, at] = LARGEST * signs(1, d)
        got = run(G, t, 1, T, 2)
        for a, b in zip(want[:3], got[:3]):  # out, lse, dq
            assert torch.equal(a[:, :at], b[:, :at]), at


@pytest.mark.parametrize("d", [16, 48, 64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("kind", ["docs_both", "padded"])
def test_other_documents_and_padding(G, d, bias, kind):
    """A whole document, or the rows behind a sequence, of the largest values in q, k, v and
    dout: every other row's output and gradients keep their bits."""
    B, T, S = 2, 200, 3
    causal, kb, ke = mask(kind, B, T, 2)
    if kind == "padded":
        bad = [i for b in range(B) for i in range(b * T + max(0, T - (b * T) // 3 - 1), b * T + T)]
    else:
        bad = list(range(int(kb[100]), int(ke[100])))
    keep = torch.ones(B * T, dtype=torch.bool)
    keep[bad] = False
    on = lambda x: None if x is None else x.cuda()  # noqa: E731
    how = dict(causal=causal, key_begin=on(kb), key_end=on(ke))
    if bias:
        how["slopes"] = torch.tensor([0.5, 0.1, 0.02], device="cuda")
    clean = tensors(S, 2, B * T, d)
    want = run(G, clean, B, T, 1, **how)
    t = [x.clone() for x in clean]
    for x in t:
        x[:, bad] = LARGEST * signs(len(bad), d)
    got = run(G, t, B, T, 1, **how)
    for a, b in zip(want, got):
        assert torch.equal(a[:, keep.cuda()], b[:, keep.cuda()])


@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("at", [5, 11, 14])
def test_behind_a_window(G, d, cap, at):
    """A value row that has left the window of later queries."""
    T, w = 300, 60
    begin = (torch.arange(T, dtype=torch.int32) + 1 - w).cuda()
    clean = tensors(2, 1, T, d)
    want = run(G, clean, 1, T, 2, softcap=cap, key_begin=begin)
    for sign in (1.0, -1.0):
        t = [x.clone() for x in clean]
        t[2][:, at] = sign * LARGEST
        got = run(G, t, 1, T, 2, softcap=cap, key_begin=begin)
        for a, b in zip(want[:3], got[:3]):
            assert torch.equal(a[:, at + w:], b[:, at + w:])
