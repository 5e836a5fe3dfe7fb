"""Plain 64-bit forms of the operators without a handle, with the error bounds their kernels'
roundings allow. Written from the definitions in include/gqe.h, one step at a time."""
import math

import torch

BF16 = 2.0 ** -8   # half a step, relative
F32 = 2.0 ** -24


def norm_rope(x, w, angle, norm, eps, rot, interleaved):
    """x [H, M, d] float64, w [d], angle [M, rot/2] -> [H, M, d]."""
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if rot == 0:
        return x
    c, s = torch.cos(angle), torch.sin(angle)
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ya, yb = a * c - b * s, a * s + b * c
    y = torch.stack([ya, yb], -1).flatten(-2) if interleaved else torch.cat([ya, yb], -1)
    return torch.cat([y, x[..., rot:]], -1)


def kv_of(G, k, S):
    return [i // k for i in range(G * k)] + [0] * (S - G * k)


def spans(B, T, causal, key_begin, key_end):
    """begin, end [B, T] of the keys each row sees."""
    t = torch.arange(T)
    b = torch.zeros(B, T, dtype=torch.long) if key_begin is None else key_begin.long().view(B, T).clamp(min=0)
    e = torch.full((B, T), T) if key_end is None else key_end.long().view(B, T).clamp(max=T)
    if causal:
        e = torch.minimum(e, (t + 1).expand(B, T))
    return b, e


def attention(q, k, v, begin, end, cap, slopes, scale, pos=None):
    """One stream of one sequence in float64: q [R, d], k, v [U, d], begin, end [R], pos [R].
    Returns out, p, and the cap's derivative (all differentiable in q, k, v)."""
    u = torch.arange(k.shape[0])
    pos = torch.arange(q.shape[0]) if pos is None else pos
    z = scale * (q @ k.T)
    if cap > 0:
        z = cap * torch.tanh(z / cap)
    z = z - slopes * (pos[:, None] - u[None, :]).abs()
    see = (u[None, :] >= begin[:, None]) & (u[None, :] < end[:, None])
    empty = ~see.any(-1, keepdim=True)
    z = z.masked_fill(~see, -math.inf).masked_fill(empty, 0.0)
    p = torch.softmax(z, -1).masked_fill(~see, 0.0)
    return p @ v, p


def attention_all(q, k, v, B, T, G, kk, causal, key_begin, key_end, cap, slopes, scale, dout=None):
    """All streams: q [S, B T, d], k, v [G, B T, d] (float64, CPU). Returns out, its absolute
    weight sum sum p |v|, and with dout the gradients and their error bounds."""
    S, M, d = q.shape
    scale = scale or 1.0 / math.sqrt(d)
    of = kv_of(G, kk, S)
    b0, e0 = spans(B, T, causal, key_begin, key_end)
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    g = None
    if dout is not None:
        g = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        g.update({"e" + n: torch.zeros_like(x) for n, x in list(g.items())})
    for b in range(B):
        r = slice(b * T, b * T + T)
        for s in range(S):
            h = of[s]
            sl = 0.0 if slopes is None else float(slopes[s])
            leaves = [x.clone().requires_grad_(dout is not None) for x in (q[s, r], k[h, r], v[h, r])]
            o, p = attention(*leaves, b0[b], e0[b], cap, sl, scale)
            out[s, r], mag[s, r] = o.detach(), p.detach() @ v[h, r].abs()
            if dout is None:
                continue
            o.backward(dout[s, r])
            p = p.detach()
            for n, x, i in (("dq", leaves[0], s), ("dk", leaves[1], h), ("dv", leaves[2], h)):
                g[n][i, r] += x.grad
            # roundings of p (its own, and the log-sum-exp's, 3 half steps together), of dz, and
            # of out inside D = <dout, out> (5 half steps of sum p |v|)
            D = (dout[s, r] * o.detach()).sum(-1, keepdim=True)
            eD = 5 * BF16 * (dout[s, r].abs() * mag[s, r]).sum(-1, keepdim=True)
            dP = dout[s, r] @ v[h, r].T
            ez = p * (4 * BF16 * (dP - D).abs() + eD)
            g["edq"][s, r] += scale * (ez @ k[h, r].abs())
            g["edk"][h, r] += scale * (ez.T @ q[s, r].abs())
            g["edv"][h, r] += 4 * BF16 * (p.T @ dout[s, r].abs())
    return out, mag, g
