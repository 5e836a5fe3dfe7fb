"""The norm and rotation of queries and keys against its 64-bit form."""
import pytest
import torch

from tests import scores_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def G():
    from moe_query_head_b200 import gqe
    return gqe


def inv_freq(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))


def rows(H, M, d, dt, seed, major="heads"):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(H, M, d, generator=g) * (1.0 + torch.arange(H).view(H, 1, 1))).to(dt).cuda()
    if major == "tokens":  # a [M, H, d] tensor seen as [H, M, d]
        x = x.transpose(0, 1).contiguous().transpose(0, 1)
    elif major == "wide":  # rows inside wider ones
        x = torch.cat([x, torch.full_like(x, float("nan"))], -1)[..., :d]
    return x


def close(got, want, dt, scale):
    """Half a step of the type, and 16 float32 roundings of the row's size: the sum of squares
    and its root (3), the weight, the row factor and the rotation's sines and products."""
    tol = want.abs() * (R.BF16 if dt is torch.bfloat16 else R.F32) + 16 * R.F32 * scale
    bad = (got.double().cpu() - want).abs() > tol
    assert not bad.any(), (got.double().cpu() - want).abs().max()


CASES = [  # d, rot, interleaved, norm, Hq, Hk, M, dtype, layout
    (16, 16, False, True, 3, 2, 1, torch.bfloat16, "heads"),
    (32, 16, True, True, 2, 1, 7, torch.float32, "heads"),
    (48, 48, False, True, 9, 8, 130, torch.bfloat16, "tokens"),
    (48, 32, True, True, 9, 8, 65, torch.bfloat16, "wide"),
    (64, 64, True, False, 5, 4, 33, torch.float32, "tokens"),
    (80, 80, False, True, 4, 4, 100, torch.bfloat16, "heads"),
    (96, 0, False, True, 1, 1, 257, torch.float32, "wide"),
    (112, 112, True, True, 17, 3, 50, torch.bfloat16, "heads"),
    (128, 128, False, True, 33, 8, 1000, torch.bfloat16, "heads"),
    (128, 64, False, False, 2, 0, 64, torch.float32, "heads"),
    (64, 64, False, True, 0, 6, 300, torch.bfloat16, "tokens"),
    (48, 48, False, True, 9, 8, 5000, torch.float32, "heads"),
]


@pytest.mark.parametrize("d,rot,inter,norm,Hq,Hk,M,dt,layout", CASES)
@pytest.mark.parametrize("far", [0, 1_000_003])
def test_forward_and_gradients(G, d, rot, inter, norm, Hq, Hk, M, dt, layout, far):
    q, k = rows(Hq, M, d, dt, 1, layout), rows(Hk, M, d, dt, 2, layout)
    gq, gk = rows(Hq, M, d, dt, 3, layout), rows(Hk, M, d, dt, 4, layout)
    w = [(1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i))).cuda() for i in (5, 6)]
    pos = (torch.arange(M, dtype=torch.int32) * 3 - 5 + far).cuda()
    f = inv_freq(rot).cuda() if rot else None
    how = dict(positions=pos, norm=norm, q_weight=w[0], k_weight=w[1], eps=EPS, inv_freq=f,
               interleaved=inter)
    outs = [torch.full_like(x, float("nan")) for x in (q, k, q, k)]
    dw = [torch.full((d,), float("nan"), device="cuda") for _ in range(2)]
    G.gqe_qk_norm_rope(q, k, outs[0], outs[1], **how)
    G.gqe_qk_norm_rope_backward(q, k, gq, gk, outs[2], outs[3], dw[0], dw[1], **how)
    assert G.gqe_check_op_status() == G.GQE_OK
    angle = pos.cpu().double()[:, None] * inv_freq(rot)
    for x, wt, gy, y, dx, dwt in ((q, w[0], gq, outs[0], outs[2], dw[0]),
                                  (k, w[1], gk, outs[1], outs[3], dw[1])):
        x64, w64 = x.double().cpu().requires_grad_(), wt.double().cpu().requires_grad_()
        ref = R.norm_rope(x64, w64, angle, norm, EPS, rot, inter)
        if x.numel() == 0:
            assert torch.equal(dwt.cpu(), torch.zeros(d))
            continue
        size = ref.detach().abs().amax(-1, keepdim=True)
        close(y, ref.detach(), dt, size)
        ref.backward(gy.double().cpu())
        # the row's factor 1 / rms times the largest weighted gradient bounds every term of dx
        gsize = gy.double().cpu().abs().amax(-1, keepdim=True) * 2.0
        if norm:
            gsize = gsize * 2 * wt.abs().max().cpu() / torch.sqrt((x64.detach() ** 2).mean(-1, keepdim=True) + EPS)
            gsize = gsize * (1 + (d ** 0.5))
        close(dx, x64.grad, dt, gsize)
        want = w64.grad if norm else torch.zeros(d, dtype=torch.float64)
        # a sum of n products in float32: 2 log2(n) + 40 roundings of the sum of magnitudes
        tol = 80 * R.F32 * (gy.double().cpu().abs().amax() * d ** 0.5 * 2) * (x.shape[0] * M) ** 0.5 * 4
        assert ((dwt.double().cpu() - want).abs() <= tol + 1e-30).all()


def test_period_positions_and_in_place(G):
    T, B, d = 37, 3, 48
    q, k = rows(9, B * T, d, torch.bfloat16, 1), rows(8, B * T, d, torch.bfloat16, 2)
    f = inv_freq(d).cuda()
    a = [torch.empty_like(q), torch.empty_like(k)]
    pos = torch.arange(T, dtype=torch.int32).repeat(B).cuda()
    G.gqe_qk_norm_rope(q, k, *a, positions=pos, inv_freq=f)
    G.gqe_qk_norm_rope(q, k, q, k, T=T, inv_freq=f)
    assert torch.equal(q, a[0]) and torch.equal(k, a[1])


def test_same_bits_and_graph(G):
    """Weight gradients have the same bits from run to run, also from a captured graph."""
    d, M = 64, 3000
    q, k = rows(9, M, d, torch.bfloat16, 1), rows(8, M, d, torch.bfloat16, 2)
    f = inv_freq(d).cuda()
    dx = [torch.empty_like(q), torch.empty_like(k)]
    dw = [[torch.empty(d, device="cuda") for _ in range(2)] for _ in range(3)]

    def call(w):
        G.gqe_qk_norm_rope_backward(q, k, q, k, *dx, *w, inv_freq=f)

    call(dw[0])
    call(dw[1])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(dw[2])
    dw[2][0].zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(dw[0][0], dw[i][0]) and torch.equal(dw[0][1], dw[i][1])


def test_no_tokens(G):
    d = 32
    q, k = rows(2, 0, d, torch.bfloat16, 1), rows(1, 0, d, torch.bfloat16, 2)
    dw = [torch.full((d,), 7.0, device="cuda") for _ in range(2)]
    G.gqe_qk_norm_rope(q, k, q, k)
    G.gqe_qk_norm_rope_backward(q, k, q, k, q, k, *dw)
    assert all((x == 0).all() for x in dw)


@pytest.mark.parametrize("d,dt", [(48, torch.bfloat16), (128, torch.bfloat16), (64, torch.float32)])
def test_append(G, d, dt):
    """Keys are normed, rotated and written to their rows, values copied; idle slots and every
    other row stay as they were, and a bad position is reported."""
    B, L, Hk, Hq = 5, 20, 4, 9
    q, k, v = rows(Hq, B, d, dt, 1), rows(Hk, B, d, dt, 2), rows(Hk, B, d, dt, 3, "tokens")
    kc, vc = rows(Hk, B * L, d, dt, 4).view(Hk, B, L, d), rows(Hk, B * L, d, dt, 5).view(Hk, B, L, d)
    kc0, vc0 = kc.clone(), vc.clone()
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    pos = torch.tensor([0, 19, -1, 7, 3], dtype=torch.int32, device="cuda")
    f = inv_freq(d).cuda()
    out = torch.full_like(q, 3.0)
    G.gqe_qk_norm_rope_append(q, k, v, pos, out, kc, vc, q_weight=w, k_weight=w, eps=EPS, inv_freq=f)
    assert G.gqe_check_op_status() == G.GQE_OK
    angle = pos.cpu().double()[:, None] * inv_freq(d)
    rq = R.norm_rope(q.double().cpu(), w.double().cpu(), angle, True, EPS, d, False)
    rk = R.norm_rope(k.double().cpu(), w.double().cpu(), angle, True, EPS, d, False)
    live = [b for b in range(B) if pos[b] >= 0]
    close(out[:, live], rq[:, live], dt, rq[:, live].abs().amax(-1, keepdim=True))
    assert (out[:, 2] == 3.0).all()
    for b in live:
        p = int(pos[b])
        close(kc[:, b, p], rk[:, b], dt, rk[:, b].abs().amax(-1, keepdim=True))
        assert torch.equal(vc[:, b, p], v[:, b])
        kc[:, b, p], vc[:, b, p] = kc0[:, b, p], vc0[:, b, p]
    assert torch.equal(kc, kc0) and torch.equal(vc, vc0)
    pos[1] = L  # behind the cache
    pos[3] = -2
    out.fill_(3.0)
    G.gqe_qk_norm_rope_append(q, k, v, pos, out, kc, vc, inv_freq=f)
    assert G.gqe_check_op_status() == G.GQE_ERR_INVALID_ARG
    assert G.gqe_check_op_status() == G.GQE_OK
    assert (out[:, 1] == 3.0).all() and (out[:, 3] == 3.0).all()
    assert torch.equal(kc[:, 1], kc0[:, 1]) and torch.equal(vc[:, 3], vc0[:, 3])
