"""The device's status word of the operators without a handle."""
import pytest
import torch

from tests.test_attention_scores_gpu import rows

pytestmark = pytest.mark.gpu


def test_reports_of_two_streams():
    """A report is seen once, on whichever stream it was made and is asked for; a later report
    is seen again."""
    from moe_query_head_b200 import gqe as G
    d = 48
    q, kc = rows(2, 3, d, 1), rows(1, 3 * 10, d, 2).view(1, 3, 10, d)
    k = rows(1, 3, d, 3)
    out = torch.empty_like(q)
    good = torch.tensor([4, 9, -1], dtype=torch.int32, device="cuda")
    bad = torch.tensor([4, 10, -2], dtype=torch.int32, device="cuda")
    kc2, vc2, out2 = kc.clone(), kc.clone(), torch.empty_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert G.gqe_check_op_status() == G.GQE_OK
    for check in (None, side):
        G.gqe_attention_decode(q, kc, kc, good, out, 2)
        G.gqe_qk_norm_rope_append(q, k, k, bad, out2, kc2, vc2, stream=side)
        side.synchronize()
        assert G.gqe_check_op_status(check) == G.GQE_ERR_INVALID_ARG
        assert G.gqe_check_op_status() == G.GQE_OK and G.gqe_check_op_status(side) == G.GQE_OK
        G.gqe_attention_decode(q, kc, kc, bad, out, 2)
        assert G.gqe_check_op_status() == G.GQE_ERR_INVALID_ARG
        assert G.gqe_check_op_status() == G.GQE_OK
