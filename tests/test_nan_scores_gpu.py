"""A NaN score makes its whole row NaN whatever the scores that follow it."""
import pytest
import torch

from tests.test_attention_scores_gpu import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("col", [3, 12, 70])
@pytest.mark.parametrize("cap", [0.0, 100.0])
def test_nan_before_larger_scores(G, d, bias, col, cap):
    """The NaN lies in the tile that is taken first (the last one with a bias), and later tiles
    hold scores 50 and more above it."""
    T = 400
    q, k, v = torch.ones(2, T, d).bfloat16().cuda(), rows(1, T, d, 2, 0.1), rows(1, T, d, 3)
    at, high = (col, slice(256, 384)) if not bias else (384 + col % 16, slice(0, 128))
    k[:, high] = 64.0 / d ** 0.5
    k[0, at, 5] = float("nan")
    how = dict(causal=0, softcap=cap)
    if bias:
        how["slopes"] = torch.tensor([0.0, 1e-3], device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, T, device="cuda")
    G.gqe_attention_forward(q, k, v, out, lse, 1, T, 2, **how)
    assert G.gqe_check_op_status() == G.GQE_OK
    assert out.isnan().all() and lse.isnan().all()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
    G.gqe_attention_backward(q, k, v, out, lse, q, dq, dk, dv, 1, T, 2, **how)
    assert dq.isnan().all()
