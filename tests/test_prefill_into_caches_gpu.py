"""A layer with norm and rotation: the caches filled from a forward's K and V, and generation from
there."""
import pytest
import torch

from moe_query_head_b200 import workloads as W
from tests.gqe_testlib import BF16_REL_L2, rel_l2, to_host_f64
from tests.test_layer_options_gpu import EPS, MAIN, build, layer_ref, load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["norm_rope", "all"])
def test_decode_after_a_forward(name):
    from moe_query_head_b200 import gqe as G
    wl = MAIN.with_(B=2, T=60)
    n = 55  # tokens of the prompt
    inp = W.generate(wl)
    o, m, _, _ = build(wl, name)
    w = load(m, inp, o)
    x = torch.from_numpy(inp.f64("x")).float().view(wl.B, wl.T, wl.dim).cuda()
    with torch.no_grad():
        y = [m(x[:, :n])]
    K, V = (torch.empty(wl.G, wl.B * n, wl.d_h, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    G.gqe_get_tensor(m._h, "K", K)
    G.gqe_get_tensor(m._h, "V", V)
    freq, _ = m._tables_on(x.device)
    how = dict(q_weight=m.q_norm.detach(), k_weight=m.k_norm.detach(), eps=EPS, inv_freq=freq,
               interleaved=o["inter"])
    G.gqe_qk_norm_rope(K[:0], K, K[:0], K, T=n, **how)
    kc, vc = m.allocate_cache(wl.B, wl.T)
    kc[:, :, :n], vc[:, :, :n] = K.view(wl.G, wl.B, n, -1), V.view(wl.G, wl.B, n, -1)
    lengths = torch.full((wl.B,), n, dtype=torch.int32, device="cuda")
    for t in range(n, wl.T):
        y.append(m.decode_step(x[:, t], kc, vc, lengths)[:, None])
        lengths += 1
    assert G.gqe_check_device_status(m._h) == G.GQE_OK
    # the same prompt by single steps: the same rows of the caches
    kc2, vc2 = m.allocate_cache(wl.B, wl.T)
    lengths.zero_()
    for t in range(n):
        m.decode_step(x[:, t], kc2, vc2, lengths)
        lengths += 1
    assert torch.equal(kc[:, :, :n], kc2[:, :, :n]) and torch.equal(vc[:, :, :n], vc2[:, :, :n])
    t = torch.arange(wl.T)
    ref = layer_ref(wl, torch.from_numpy(inp.f64("x")), {k: p.detach() for k, p in w.items()}, o,
                    torch.zeros(wl.B, wl.T, dtype=torch.long), (t + 1).expand(wl.B, -1), t.repeat(wl.B))
    got = torch.cat(y, 1)
    assert rel_l2(to_host_f64(got).reshape(wl.M, -1), ref.numpy()) <= BF16_REL_L2
