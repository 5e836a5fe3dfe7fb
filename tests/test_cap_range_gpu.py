"""Caps above the ordinary ones with scores up to the cap, where some tiles of a row take the
cap's polynomial and others its exponential."""
import math

import pytest
import torch

from tests import scores_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LOG2E = 1.0 / math.log(2.0)


@pytest.mark.parametrize("d", [48, 64, 128])
@pytest.mark.parametrize("cap", [30.0, 200.0, 500.0, 1000.0, 1900.0, 4000.0, 8192.0])
@pytest.mark.parametrize("part", [0.3, 0.745])
def test_near_ties_close_to_the_cap(d, cap, part):
    """Scores near `part` of the cap a few units apart; one key of the second tile lies at -0.9
    of it, so that tile is not the polynomial's. Values of +1 in the first and last tile and -1 in
    the second turn a difference between the forms into an output."""
    from moe_query_head_b200 import gqe as G
    T = 384
    g = torch.Generator().manual_seed(int(cap))
    q, k = torch.zeros(1, T, d), torch.zeros(1, T, d)
    q[..., 0], q[..., 1] = 32.0, torch.randn(T, generator=g)
    k[..., 0], k[..., 1] = part * cap / 32.0, 1.5 * torch.randn(T, generator=g)
    k[0, 200, 0] = -0.9 * cap / 32.0
    v = torch.ones(1, T, d)
    v[:, 128:256] = -1.0
    do = torch.randn(1, T, d, generator=g)
    host = [x.to(BF) for x in (q, k, v, do)]
    q, k, v, do = (x.cuda() for x in host)
    out, lse = torch.empty_like(q), torch.empty(1, T, device="cuda")
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    how = dict(causal=0, scale=1.0, softcap=cap)
    G.gqe_attention_forward(q, k, v, out, lse, 1, T, 1, **how)
    G.gqe_attention_backward(q, k, v, out, lse, do, dq, dk, dv, 1, T, 1, **how)
    assert G.gqe_check_op_status() == G.GQE_OK
    x = [h.double() for h in host]
    ref, mag, gr = R.attention_all(x[0], x[1], x[2], 1, T, 1, 1, 0, None, None, cap, None, 1.0, x[3])
    # A score's error: 2^-11 where the polynomial serves it, and float32's in the form with the
    # exponential: 1e-7 of the cap in the tanh, a rounding each of the product, the argument, the
    # cap's product, the reference's difference and the log-sum-exp (magnitudes up to 1.45 cap).
    ez = 2.0 ** -11 + (1e-7 + 5 * R.F32 * 1.45) * cap
    z = cap * torch.tanh(x[0][0] @ x[1][0].T / cap)
    want = torch.logsumexp(z, -1) * LOG2E
    # 2^x on the FMA pipe to 2^-9, and the weights' bf16 rounding where their sum is taken of those
    tol = LOG2E * (2.0 ** -9 + (R.BF16 if d <= 48 else 0.0) + ez)
    err = (lse[0].double().cpu() - want).abs().max()
    assert err <= tol, (float(err), tol)
    err = (out.double().cpu() - ref).abs()
    assert (err <= (3 * R.BF16 + 2 * ez) * mag + R.BF16 * ref.abs()).all(), float(err.max())
    # Gradients: the bounds of scores_ref count four half steps of p and dz; the scores' error, once
    # in the weight and once in the log-sum-exp, is at most another 2 ez / 2^-8 of them.
    more = 1.0 + 2 * ez / (4 * R.BF16)
    for n, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        err = (got.double().cpu() - gr[n]).abs()
        bound = more * gr["e" + n] + R.BF16 * gr[n].abs() + 1e-6
        assert (err <= bound).all(), (n, float((err - bound).max()))
