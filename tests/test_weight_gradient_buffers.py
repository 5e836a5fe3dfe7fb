"""One buffer for both weights' gradients would be written by two sums at once: refused."""
import ctypes

import pytest

from tests.test_scores_cpu import INV, P, heads, transform


def test_operator_refuses_one_buffer():
    from moe_query_head_b200 import gqe as G
    r, tr = ctypes.byref, transform(G)
    q, k = heads(G, 9), heads(G, 8)
    n = G.lib.gqe_qk_norm_rope_workspace_bytes(48)

    def call(dq, dk, M=8):
        return G.lib.gqe_qk_norm_rope_backward(r(tr), M, r(q), r(k), P, 0, r(q), r(k), r(q), r(k), dq, dk, P, n,
                                               None)

    assert call(P, P) == INV and call(P, P, M=0) == INV
    assert call(None, None, M=0) == 0


@pytest.mark.gpu
def test_handle_refuses_one_buffer():
    import torch
    from moe_query_head_b200 import gqe as G
    h = G.gqe_create(64, 4, 2, 1, 32, G.GQE_BF16, 64)
    dw = torch.empty(2, 32, device="cuda")
    with pytest.raises(G.GQEError) as e:
        G.gqe_set_qk_transform(h, 32, dq_weight=dw[0], dk_weight=dw[0])
    assert e.value.status == INV
    G.gqe_set_qk_transform(h, 32, dq_weight=dw[0], dk_weight=dw[1])
    G.gqe_set_qk_transform(h, 32)
    G.gqe_destroy(h)
