"""Keys with infinities."""
import pytest
import torch

from tests.test_attention_scores_gpu import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("T,at", [(300, 140), (300, 299), (2060, 1000), (2060, 2055)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
def test_query_gradients_of_an_infinite_key(G, d, T, at, bad):
    """A key with an infinity, seen by the rows from `at` on under a causal mask: each has a score of
    +-infinity for it, a weight of 0 or NaN, and 0 or NaN times infinity in dq. The rows before it
    keep their bits."""
    q, k, v, do = rows(2, T, d, 1), rows(1, T, d, 2), rows(1, T, d, 3), rows(2, T, d, 4)
    got = []
    for key in (k, k.clone()):
        if got:
            key[0, at, 7] = bad
        out, lse = torch.empty_like(q), torch.empty(2, T, device="cuda")
        g = [torch.empty_like(x) for x in (q, k, v)]
        G.gqe_attention_forward(q, key, v, out, lse, 1, T, 2)
        G.gqe_attention_backward(q, key, v, out, lse, do, *g, 1, T, 2)
        got.append((out, lse, g[0]))
    assert G.gqe_check_op_status() == G.GQE_OK
    (o0, l0, dq0), (o1, l1, dq1) = got
    for a, b in ((o0, o1), (l0, l1), (dq0, dq1)):
        assert torch.equal(a[:, :at], b[:, :at])
    sign = q[:, at:, 7].sign() * (1 if bad > 0 else -1)
    assert o1[:, at:][sign > 0].isnan().all()
    assert torch.isfinite(o1[:, at:][sign < 0]).all()
    assert dq1[:, at:, 7].isnan().all()
