"""The norm without an epsilon: places of a block without a token add nothing to the weights'
gradients."""
import pytest
import torch

from tests import scores_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dt", [(48, torch.bfloat16), (64, torch.float32), (112, torch.bfloat16),
                                  (128, torch.bfloat16)])
@pytest.mark.parametrize("M", [1, 33, 50001])
def test_weight_gradients_without_eps(d, dt, M):
    """One token, one block with places left, and several rounds of blocks with a remainder."""
    from moe_query_head_b200 import gqe as G
    g = torch.Generator().manual_seed(M)
    x = [torch.randn(h, M, d, generator=g).to(dt) for h in (2, 1, 2, 1)]  # q, k and their gradients
    q, k, gq, gk = (t.cuda() for t in x)
    w = [(1 + 0.3 * torch.randn(d, generator=g)) for _ in range(2)]
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dw = [torch.empty(d, device="cuda") for _ in range(2)]
    G.gqe_qk_norm_rope_backward(q, k, gq, gk, dq, dk, *dw, q_weight=w[0].cuda(), k_weight=w[1].cuda(),
                                eps=0.0)
    assert torch.isfinite(dq).all() and torch.isfinite(dk).all()
    for xs, gs, got in ((x[0], x[2], dw[0]), (x[1], x[3], dw[1])):
        xs, gs = xs.double(), gs.double()
        terms = gs * xs / (xs * xs).mean(-1, keepdim=True).sqrt()
        # roundings of a term (16, the row's factor included) and of the sums on its way: a thread's
        # rows (some 9), its block's (at most 64 of 128 / lanes, in 4 warps 128), the blocks' (10
        # and 64): each at most 2^-24 of the sum of magnitudes
        tol = (16 + 9 + 128 + 74) * R.F32 * terms.abs().sum((0, 1))
        assert ((got.double().cpu() - terms.sum((0, 1))).abs() <= tol).all()
