"""Scales that a distance bias is served with."""
import ctypes

import pytest
import torch

from tests import scores_ref as R
from tests.test_attention_scores_gpu import rows
from tests.test_scores_cpu import P, UNS, heads, scores


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


@pytest.mark.parametrize("scale", [1e-37, 2.0 ** -61, 2.0 ** 61])
def test_scales_out_of_range_are_refused(G, scale):
    """slope / scale would leave float32's range."""
    r = ctypes.byref
    a, q, k = scores(G, scale=scale, slopes=P), heads(G, 9), heads(G, 8)
    assert G.lib.gqe_attention_forward(r(a), r(q), r(k), r(k), r(q), P, None) == UNS
    assert G.lib.gqe_attention_backward(r(a), r(q), r(k), r(k), r(q), P, r(q), r(q), r(k), r(k), P, 1 << 40,
                                        None) == UNS
    assert G.lib.gqe_attention_workspace_bytes(r(a)) == -1
    c, q = heads(G, 8, ts=20 * 48, hs=2 * 20 * 48), heads(G, 9, M=2)
    assert G.lib.gqe_attention_decode(r(a), r(q), r(c), r(c), 20, P, r(q), P, 0, None) == UNS
    # the same scale without slopes, and no scale with them, are served
    assert G.lib.gqe_attention_workspace_bytes(r(scores(G, scale=scale))) > 0
    assert G.lib.gqe_attention_workspace_bytes(r(scores(G, slopes=P))) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("d", [48, 128])
@pytest.mark.parametrize("causal", [0, 1])
def test_smallest_scale(G, d, causal):
    """At a scale of 2^-60 the bias alone is left of the scores."""
    T, slopes = 200, torch.tensor([1.0, 0.03])
    q, k, v = rows(2, T, d, 1), rows(1, T, d, 2), rows(1, T, d, 3)
    out = torch.empty_like(q)
    G.gqe_attention_forward(q, k, v, out, None, 1, T, 2, causal=causal, scale=2.0 ** -60, slopes=slopes.cuda())
    ref, mag, _ = R.attention_all(*[x.double().cpu() for x in (q, k, v)], 1, T, 1, 2, causal, None, None, 0.0,
                                  slopes, 2.0 ** -60)
    # three half steps of the weights, one of the output
    assert ((out.double().cpu() - ref).abs() <= 3 * R.BF16 * mag + R.BF16 * ref.abs()).all()
