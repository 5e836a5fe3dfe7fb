"""Rows all of whose scores are -infinity."""
import pytest
import torch

from tests.test_attention_scores_gpu import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


@pytest.mark.parametrize("d", [16, 48, 64, 128])
@pytest.mark.parametrize("T", [1, 70, 700])
def test_only_minus_infinity(G, d, T):
    """A row that sees keys, all with a score of -infinity: no softmax, NaN; in the forward and
    in the single-token form alike. A row without keys stays zeros."""
    q, k, v = rows(1, T, d, 1), rows(1, T, d, 2), rows(1, T, d, 3)
    q[..., 3], k[..., 3] = float("inf"), -1.0
    out = torch.empty_like(q)
    G.gqe_attention_forward(q, k, v, out, None, 1, T, 1)
    assert out.isnan().all()
    B = 2
    kc, vc = k.view(1, 1, T, d).repeat(1, B, 1, 1), v.view(1, 1, T, d).repeat(1, B, 1, 1)
    q1 = q[:, :1].repeat(1, B, 1)
    pos = torch.tensor([T - 1, -1], dtype=torch.int32, device="cuda")
    o1 = torch.empty_like(q1)
    G.gqe_attention_decode(q1, kc, vc, pos, o1, 1)
    assert G.gqe_check_op_status() == G.GQE_OK
    assert o1[:, 0].isnan().all() and (o1[:, 1] == 0).all()


@pytest.mark.parametrize("d", [48, 64])
def test_scores_past_float32_steps(G, d):
    """Scores of 10^8, where float32 steps by 8: the largest one's weight may be 2^-8 of the
    reference's, and the row is still its value."""
    T = 300
    q, k, v = torch.zeros(1, T, d).bfloat16().cuda(), torch.zeros(1, T, d).bfloat16().cuda(), rows(1, T, d, 3)
    q[..., 0] = torch.linspace(300.0, 500.0, T).bfloat16().cuda()
    k[..., 0] = 1.0
    k[0, 50, 0] = 1.25
    out = torch.empty_like(q)
    G.gqe_attention_forward(q, k, v, out, None, 1, T, 1, causal=0, scale=333333.0)
    # one weight of one half step and a sum of it, the output's rounding
    assert ((out.double() - v[:, 50:51].double()).abs() <= 3 * 2.0 ** -8 * v[:, 50:51].double().abs()).all()
