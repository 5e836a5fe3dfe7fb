"""The layer with options: norm and rotation of its queries and keys, capped, biased and masked
scores, in gqe_forward, gqe_decode, the backward pass, on a group range and through the module,
against a float64 form of the whole layer (rel-L2 1e-2, the layer tests' tolerance in bf16)."""
import math

import pytest
import torch

from moe_query_head_b200 import group_parallel as GP
from moe_query_head_b200 import workloads as W
from moe_query_head_b200.module import GQEAttention, document_spans, prefix_spans
from tests import scores_ref as R
from tests.gqe_testlib import BF16_REL_L2, GpuRun, rel_l2, to_device, to_host_f64

pytestmark = pytest.mark.gpu
MAIN = W.WORKLOADS["main_b8_t2048"]
WIDE = W.WORKLOADS["wide_k2"]
TINY = W.WORKLOADS["tiny_f32"]
NAMES = ("W_r", "W_q", "W_k", "W_v", "W_shared", "W_o")
EPS = 1e-6


def layer_ref(wl, x, w, opt, begin, end, pos):
    """The layer on x [B T, dim] in float64 (differentiable). w: the weights and, where the
    options have a norm, q_norm and k_norm; begin, end [B, T], pos [B T]."""
    B, T, M, G, k, E, dh = wl.B, wl.T, wl.M, wl.G, wl.k, wl.E, wl.d_h
    p = torch.softmax((x @ w["W_r"].T).view(M, G, E), -1)
    sel = torch.sort(torch.topk(p.detach(), k, -1).indices, -1).values  # margins rule out ties
    ps = torch.gather(p, 2, sel)
    q = torch.einsum("md,gehd->mgeh", x, w["W_q"].view(G, E, dh, -1))
    q = torch.gather(q, 2, sel[..., None].expand(-1, -1, -1, dh)).reshape(M, G * k, dh).transpose(0, 1)
    if wl.shared:
        q = torch.cat([q, (x @ w["W_shared"].T)[None]])
    kk = (x @ w["W_k"].T).view(M, G, dh).transpose(0, 1)
    v = (x @ w["W_v"].T).view(M, G, dh).transpose(0, 1)
    if opt.get("norm") or opt.get("rot"):
        f = opt["base"] ** (-torch.arange(0, opt["rot"], 2, dtype=torch.float64) / max(opt["rot"], 1))
        ang = pos.double()[:, None] * f
        q, kk = (R.norm_rope(t, n, ang, opt["norm"], EPS, opt["rot"], opt["inter"])
                 for t, n in ((q, w.get("q_norm")), (kk, w.get("k_norm"))))
    S = q.shape[0]
    of = R.kv_of(G, k, S)
    outs = []
    for s in range(S):
        sl = opt["slopes"][s] if opt.get("slopes") else 0.0
        outs.append(torch.cat([R.attention(q[s, r], kk[of[s], r], v[of[s], r], begin[b], end[b],
                                           opt.get("cap", 0.0), sl, 1 / math.sqrt(dh))[0]
                               for b, r in ((b, slice(b * T, b * T + T)) for b in range(B))]))
    ps = ps.reshape(M, G * k)
    blocks = [o * ps[:, s:s + 1] if wl.variant == "weighted_concat" and s < G * k else o
              for s, o in enumerate(outs[:G * k])]
    if wl.variant == "gqe":
        ws = ps / ps.sum(-1, keepdim=True)
        blocks.append(sum(ws[:, s:s + 1] * o for s, o in enumerate(outs[:G * k])))
    if wl.shared:
        blocks.append(outs[-1])
    return torch.cat(blocks, -1) @ w["W_o"].T


OPTS = {
    "norm_rope": dict(norm=True, rot=48, base=10000.0, inter=False),
    "rope_part": dict(norm=False, rot=32, base=500.0, inter=True, positions=True),
    "cap": dict(cap=2.0),
    "bias_docs": dict(bias=True, docs=True),
    "all": dict(norm=True, rot=16, base=10000.0, inter=False, cap=5.0, bias=True, docs=True, positions=True),
    "prefix": dict(prefix=True, cap=3.0),
}


def build(wl, name):
    """The reference's options and the module of a case, with the call's index tensors."""
    o = dict(norm=False, rot=0, inter=False, base=1.0)
    o.update(OPTS[name])
    S = wl.G * wl.k + wl.shared
    o["slopes"] = [2.0 ** (-8.0 * (s + 1) / S) for s in range(S)] if o.get("bias") else None
    m = GQEAttention(wl.dim, wl.N, wl.G, wl.k, wl.d_h, wl.variant, shared=wl.shared,
                     causal=not o.get("prefix"), qk_norm=o["norm"], norm_eps=EPS,
                     rope_base=o["base"] if o["rot"] else None, rope_dim=o["rot"] or None,
                     rope_interleaved=o["inter"], softcap=o.get("cap", 0.0),
                     slopes="geometric" if o.get("bias") else None).cuda()
    call = {}
    if o.get("docs"):
        d = [document_spans([wl.T // 3 + b, wl.T // 2], wl.T) for b in range(wl.B)]  # the rest: padding
        call["key_begin"] = torch.stack([x[0] for x in d]).cuda()
        call["key_end"] = torch.stack([x[1] for x in d]).cuda()
    if o.get("prefix"):
        call["key_end"] = torch.stack([prefix_spans(wl.T // 4 + b, wl.T) for b in range(wl.B)]).cuda()
    pos = torch.arange(wl.T).repeat(wl.B)
    if o.get("positions"):
        pos = pos * 2 + 7
        call["positions"] = pos.view(wl.B, wl.T).cuda()
    b0, e0 = R.spans(wl.B, wl.T, m.causal, *(call[n].cpu().view(-1) if n in call else None
                                             for n in ("key_begin", "key_end")))
    return o, m, call, (b0, e0, pos)


def load(m, inp, o):
    """The workload's weights in the module, and all weights as float64 leaves."""
    g = torch.Generator().manual_seed(3)
    with torch.no_grad():
        for n in NAMES:
            if getattr(m, n) is not None:
                getattr(m, n).copy_(torch.from_numpy(inp.f64(n)).float())
        if o["norm"]:
            for p in (m.q_norm, m.k_norm):
                p.copy_(1 + 0.2 * torch.randn(p.shape, generator=g))
    names = [n for n in NAMES + ("q_norm", "k_norm") if getattr(m, n, None) is not None]
    return {n: getattr(m, n).detach().double().cpu().requires_grad_() for n in names}


@pytest.mark.parametrize("name", list(OPTS))
@pytest.mark.parametrize("wl", [MAIN.with_(B=2, T=150), WIDE.with_(B=1, T=200, variant="weighted_concat"),
                                MAIN.with_(B=1, T=140, shared=False, variant="hard_concat")],
                         ids=["main_gqe", "wide_weighted", "hard_no_shared"])
def test_module_forward_and_gradients(wl, name):
    inp = W.generate(wl)
    o, m, call, ref_args = build(wl, name)
    w = load(m, inp, o)
    x64 = torch.from_numpy(inp.f64("x")).requires_grad_()
    x = x64.detach().float().view(wl.B, wl.T, wl.dim).cuda().requires_grad_()
    dy = torch.randn(wl.M, wl.dim, generator=torch.Generator().manual_seed(5)).bfloat16()
    y = m(x, **call)
    y.backward(dy.view_as(y).cuda())
    ref = layer_ref(wl, x64, w, o, *ref_args)
    ref.backward(dy.double())
    assert rel_l2(to_host_f64(y.detach()).reshape(wl.M, -1), ref.detach().numpy()) <= BF16_REL_L2
    errs = {"x": rel_l2(x.grad.cpu().double().view(wl.M, -1).numpy(), x64.grad.numpy())}
    for n in w:
        g = getattr(m, n).grad.cpu().double()
        if w[n].grad is None:  # hard_concat: the selection alone, the router has no gradient
            assert not g.any()
        else:
            errs[n] = rel_l2(g.numpy(), w[n].grad.numpy())
    assert all(e <= BF16_REL_L2 for e in errs.values()), errs


def test_backward_after_another_call():
    """A backward whose options and state another call has replaced runs its forward again."""
    wl = MAIN.with_(B=1, T=130)
    inp = W.generate(wl)
    o, m, call, _ = build(wl, "all")
    load(m, inp, o)
    x = torch.from_numpy(inp.f64("x")).float().view(1, wl.T, wl.dim).cuda()

    def grads(between):
        m.zero_grad()
        y = m(x, **call)
        if between:
            with torch.no_grad():
                m(x[:, :50])  # no intervals, other positions
        y.float().square().sum().backward()
        return [p.grad.clone() for p in m.parameters()]

    for a, b in zip(grads(False), grads(True)):
        assert torch.equal(a, b)


def test_norm_weights_changed_before_the_backward():
    """The backward uses the weights its forward had, as it does the projections'."""
    wl = MAIN.with_(B=1, T=70)
    inp = W.generate(wl)
    o, m, call, _ = build(wl, "norm_rope")
    load(m, inp, o)
    x = torch.from_numpy(inp.f64("x")).float().view(1, wl.T, wl.dim).cuda()

    def grads(change):
        m.zero_grad()
        y = m(x, **call)
        if change:
            with torch.no_grad():
                for p in (m.q_norm, m.k_norm, m.W_q):
                    p.mul_(-3.0)
        y.float().square().sum().backward()
        return [p.grad.clone() for p in m.parameters()]

    for a, b in zip(grads(False), grads(True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["norm_rope", "cap", "all"])
@pytest.mark.parametrize("variant", ["gqe", "weighted_concat"])
def test_decode_continues_the_forward(name, variant):
    """Decode steps over a cache give the rows of a forward over the whole sequence (the
    reference's rows), also as a captured graph; a window of the cache is read as one."""
    wl = MAIN.with_(B=3, T=70, variant=variant)
    inp = W.generate(wl)
    o, m, _, _ = build(wl, name)
    w = load(m, inp, o)
    x = torch.from_numpy(inp.f64("x")).float().view(wl.B, wl.T, wl.dim).cuda()
    kc, vc = m.allocate_cache(wl.B, wl.T + 3)
    kc.fill_(float("nan"))
    vc.fill_(float("nan"))
    lengths = torch.zeros(wl.B, dtype=torch.int32, device="cuda")
    begin = torch.zeros(wl.B, dtype=torch.int32, device="cuda")
    ys = []
    step_x = x[:, 0].clone()
    for t in range(wl.T - 2):
        begin.copy_((lengths - 40).clamp(min=0))
        ys.append(m.decode_step(x[:, t], kc, vc, lengths, begin))
        lengths += 1
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m.decode_step(step_x, kc, vc, lengths, begin)
    for t in range(wl.T - 2, wl.T):
        step_x.copy_(x[:, t])
        begin.copy_((lengths - 40).clamp(min=0))
        g.replay()
        ys.append(y.clone())
        lengths += 1
    got = torch.stack(ys, 1)
    t = torch.arange(wl.T)
    b0 = (t - 40).clamp(min=0).expand(wl.B, -1)
    ref = layer_ref(wl, torch.from_numpy(inp.f64("x")), {n: p.detach() for n, p in w.items()},
                    o, b0, (t + 1).expand(wl.B, -1), t.repeat(wl.B))
    assert rel_l2(to_host_f64(got).reshape(wl.M, -1), ref.numpy()) <= BF16_REL_L2
    from moe_query_head_b200 import gqe as GQ
    assert GQ.gqe_check_device_status(m._h) == GQ.GQE_OK
    lengths.fill_(-1)  # a step's position must lie in the cache
    m.decode_step(x[:, 0], kc, vc, lengths)
    assert GQ.gqe_check_device_status(m._h) == GQ.GQE_ERR_INVALID_ARG


def test_group_ranges_sum_to_the_layer():
    """Forward and backward of two group ranges with options: outputs, gradients and the norm
    weights' gradients sum to the layer's."""
    from moe_query_head_b200 import gqe as GQ
    wl = MAIN.with_(B=1, T=150)
    inp = W.generate(wl)
    o, m, call, ref_args = build(wl, "all")
    w = load(m, inp, o)
    d = {n: to_device(inp, n) for n in ("x",) + NAMES}
    dy = torch.randn(wl.M, wl.dim, generator=torch.Generator().manual_seed(5)).bfloat16()
    freq, slopes = m._tables_on(torch.device("cuda", 0))
    call = {n: t.int().reshape(-1).contiguous() for n, t in call.items()}
    total, dx = torch.zeros(wl.M, wl.dim, device="cuda"), torch.zeros(wl.M, wl.dim, device="cuda")
    shards, dots, dn = [], [], torch.zeros(2, wl.d_h, device="cuda")
    keep = []
    for g0, g1 in GP.group_ranges(wl.G, 2):
        sh = GP.GroupShard(dim=wl.dim, N=wl.N, G=wl.G, k=wl.k, d_h=wl.d_h, variant=wl.variant, causal=True,
                           max_tokens=wl.M, g0=g0, g1=g1, W_r=d["W_r"], W_q=d["W_q"], W_k=d["W_k"],
                           W_v=d["W_v"], W_shared=d["W_shared"], W_o=d["W_o"])
        sh.enable_backward()
        sl = torch.cat([slopes[g0 * wl.k:g1 * wl.k], slopes[-1:]]) if g0 == 0 else slopes[g0 * wl.k:g1 * wl.k]
        part = [torch.empty(wl.d_h, device="cuda") for _ in range(2)]
        keep.append((sl, part))
        GQ.gqe_set_qk_transform(sh.h, wl.d_h, norm=True, q_weight=m.q_norm.detach(), k_weight=m.k_norm.detach(),
                                eps=EPS, inv_freq=freq, positions=call["positions"], dq_weight=part[0],
                                dk_weight=part[1])
        GQ.gqe_set_scores(sh.h, softcap=o["cap"], slopes=sl, key_begin=call["key_begin"],
                          key_end=call["key_end"])
        out = torch.empty(wl.M, wl.dim, dtype=torch.bfloat16, device="cuda")
        sh.forward(d["x"], wl.B, wl.T, out)
        total += out.float()
        dots.append(torch.empty(wl.M, device="cuda"))
        sh.backward_begin(d["x"], wl.B, wl.T, dy.cuda(), dots[-1])
        shards.append(sh)
    for sh, (_, part) in zip(shards, keep):
        g = sh.backward_finish(d["x"], wl.B, wl.T, dy.cuda(), 0.0, sum(dots))
        dx += g["x"]
        dn += torch.stack(part)
        assert GQ.gqe_check_device_status(sh.h) == GQ.GQE_OK
        sh.close()
    x64 = torch.from_numpy(inp.f64("x")).requires_grad_()
    ref = layer_ref(wl, x64, w, o, *ref_args)
    ref.backward(dy.double())
    assert rel_l2(total.cpu().double().numpy(), ref.detach().numpy()) <= BF16_REL_L2
    assert rel_l2(dx.cpu().double().numpy(), x64.grad.numpy()) <= BF16_REL_L2
    for i, n in enumerate(("q_norm", "k_norm")):
        assert rel_l2(dn[i].cpu().double().numpy(), w[n].grad.numpy()) <= BF16_REL_L2


def test_float32_handle_transform():
    """A float32 handle norms and rotates too (its attention stays exact); scores are refused."""
    from moe_query_head_b200 import gqe as GQ
    wl = TINY.with_(T=50)
    inp = W.generate(wl)
    run = GpuRun(inp)
    f = (100.0 ** (-torch.arange(0, 16, 2, dtype=torch.float64) / 16)).cuda()
    n = torch.linspace(0.5, 1.5, 16, device="cuda")
    GQ.gqe_set_qk_transform(run.h, 16, GQ.GQE_F32, q_weight=n, k_weight=n, eps=EPS, inv_freq=f)
    run.forward()
    w = {x: torch.from_numpy(inp.f64(x)) for x in NAMES}
    w["q_norm"] = w["k_norm"] = n.double().cpu()
    b0, e0 = R.spans(1, 50, 1, None, None)
    ref = layer_ref(wl, torch.from_numpy(inp.f64("x")), w, dict(norm=True, rot=16, base=100.0, inter=False),
                    b0, e0, torch.arange(50))
    assert rel_l2(run.out.double().cpu().numpy(), ref.numpy()) <= 1e-5
    with pytest.raises(GQ.GQEError) as e:
        GQ.gqe_set_scores(run.h, softcap=3.0)
    assert e.value.status == GQ.GQE_ERR_UNSUPPORTED
    run.close()


def test_options_of_the_forward_and_back_to_none():
    """A backward with other options than its forward's is refused; options turned off leave the
    layer's bits as they were before."""
    from moe_query_head_b200 import gqe as GQ
    wl = MAIN.with_(B=1, T=100)
    inp = W.generate(wl)
    run = GpuRun(inp).forward()
    plain = run.out.clone()
    GQ.gqe_enable_backward(run.h)
    d = run.dev
    f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    g = [f32(wl.M, wl.dim), f32(wl.N, wl.dim), f32(wl.N * wl.d_h, wl.dim), f32(wl.G * wl.d_h, wl.dim),
         f32(wl.G * wl.d_h, wl.dim), f32(wl.d_h, wl.dim), f32(wl.dim, wl.D_o)]
    dy = torch.ones(wl.M, wl.dim, dtype=torch.bfloat16, device="cuda")

    def backward():
        GQ.gqe_backward(run.h, d["x"], wl.B, wl.T, d["W_r"], d["W_q"], d["W_k"], d["W_v"], d["W_shared"],
                        d["W_o"], wl.N, wl.G, wl.k, wl.d_h, 0, 1, dy, 0.0, *g)

    backward()
    GQ.gqe_set_scores(run.h, softcap=1.0)
    with pytest.raises(GQ.GQEError):
        backward()
    run.forward()
    assert not torch.equal(run.out, plain)
    backward()
    GQ.gqe_set_scores(run.h, softcap=1.0)  # the same again changes nothing
    backward()
    GQ.gqe_set_scores(run.h)
    GQ.gqe_set_qk_transform(run.h, wl.d_h, norm=True)
    run.forward()
    assert not torch.equal(run.out, plain)
    GQ.gqe_set_qk_transform(run.h)
    run.forward()
    assert torch.equal(run.out, plain)
    with pytest.raises(GQ.GQEError):
        GQ.gqe_set_qk_transform(run.h, 64)  # not the handle's head dim
    run.close()


def test_training_step_captured():
    """A forward and backward with options captured as one graph replay to the eager bits."""
    from moe_query_head_b200 import gqe as GQ
    wl = MAIN.with_(B=1, T=140)
    inp = W.generate(wl)
    run = GpuRun(inp)
    GQ.gqe_enable_backward(run.h)
    kb, ke = (t.cuda() for t in document_spans([60, 50], wl.T))
    n = torch.linspace(0.5, 1.5, wl.d_h, device="cuda")
    dn = torch.empty(2, wl.d_h, device="cuda")
    GQ.gqe_set_qk_transform(run.h, wl.d_h, q_weight=n, k_weight=n, dq_weight=dn[0], dk_weight=dn[1])
    GQ.gqe_set_scores(run.h, softcap=4.0, key_begin=kb, key_end=ke)
    d = run.dev
    f32 = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    g = [f32(wl.M, wl.dim), f32(wl.N, wl.dim), f32(wl.N * wl.d_h, wl.dim), f32(wl.G * wl.d_h, wl.dim),
         f32(wl.G * wl.d_h, wl.dim), f32(wl.d_h, wl.dim), f32(wl.dim, wl.D_o), dn]
    dy = torch.randn(wl.M, wl.dim, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()

    def step():
        GQ.gqe_forward(run.h, d["x"], wl.B, wl.T, d["W_r"], d["W_q"], d["W_k"], d["W_v"], d["W_shared"],
                       d["W_o"], wl.N, wl.G, wl.k, wl.d_h, 0, 1, run.out, run.aux)
        GQ.gqe_backward(run.h, d["x"], wl.B, wl.T, d["W_r"], d["W_q"], d["W_k"], d["W_v"], d["W_shared"],
                        d["W_o"], wl.N, wl.G, wl.k, wl.d_h, 0, 1, dy, 0.01, *g[:7])

    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in g] + [run.out.clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in g:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert GQ.gqe_check_device_status(run.h) == GQ.GQE_OK
    for a, b in zip(want, g + [run.out]):
        assert torch.equal(a, b)
    run.close()
