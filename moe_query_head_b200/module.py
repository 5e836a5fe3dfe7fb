"""A PyTorch module over the C ABI with the interface of the "GQE: Grouped Query Experts"
README (Usage, Parameters): ``GQEAttention(dim, num_query_experts=16, num_kv_heads=8,
top_k=1, head_dim=None, variant="gqe")``, ``y = attn(x)`` and ``collect_aux_loss(model)``, the
layer trained with ``loss.backward()`` after adding 0.01 times the aux loss to the task loss.

The module owns its weights as float32 parameters in nn.Linear layout ([out, in], no
biases): W_r [N, dim], W_q [N d_h, dim], W_k, W_v [G d_h, dim], W_shared [d_h, dim] and W_o
[dim, D_o]. Each call casts them and the input to bf16 and runs gqe_forward; the backward
runs gqe_backward (the whole layer's gradients in float32). This file only marshals
arguments: every step of the layer runs in the library's kernels.

Options beyond the README's interface, for use in a model: RMS norm of every query and key head
(qk_norm) and rotation by position (rope_base) between the projections and the attention, and
scores capped by a tanh (softcap), biased by distance (slopes) and masked by an interval of
keys per token (key_begin, key_end of a call; `document_spans` and `prefix_spans` make them).
They are set on the handle before each call (gqe_set_qk_transform, gqe_set_scores).

The library keeps one layer's forward state per handle. A backward whose forward is no longer
the handle's last (another call of the same module in between) runs that forward again
before gqe_backward. Reading the aux loss's gradient coefficient synchronises the stream.
"""
from __future__ import annotations

import math

import torch
from torch import nn

from . import gqe as G


class _GQEFunction(torch.autograd.Function):
    """y, aux = the layer of `mod` on x; backward through gqe_backward."""

    @staticmethod
    def forward(ctx, x, W_r, W_q, W_k, W_v, W_shared, W_o, q_norm, k_norm, mod, call):
        B, T, dim = x.shape
        bf = torch.bfloat16
        xb = x.reshape(B * T, dim).to(bf).contiguous()
        w = [W.detach().to(bf).contiguous() for W in (W_r, W_q, W_k, W_v)]
        ws = W_shared.detach().to(bf).contiguous() if W_shared is not None else None
        wo = W_o.detach().to(bf).contiguous()
        h = mod._handle_for(B * T)
        out = torch.empty((B * T, dim), dtype=bf, device=x.device)
        aux = torch.zeros(1, dtype=torch.float32, device=x.device)
        # copies: the backward reads them after the caller may have changed the parameters
        norms = [n.detach().to(torch.float32, copy=True) if n is not None else None
                 for n in (q_norm, k_norm)]
        mod._set_options(h, norms, call, x.device)
        mod._forward_call(h, xb, B, T, w, ws, wo, out, aux)
        ctx.mod, ctx.B, ctx.T, ctx.call = mod, B, T, mod._calls
        ctx.norms, ctx.options = norms, call  # alive until the backward has read them
        ctx.has_shared = ws is not None
        ctx.x_dtype = x.dtype
        ctx.save_for_backward(xb, *w, wo, *([ws] if ws is not None else []))
        return out.view(B, T, dim), aux[0]

    @staticmethod
    def backward(ctx, dy, daux):
        mod, B, T = ctx.mod, ctx.B, ctx.T
        saved = ctx.saved_tensors
        xb, W_r, W_q, W_k, W_v, W_o = saved[:6]
        W_s = saved[6] if ctx.has_shared else None
        h = mod._h
        if mod._calls != ctx.call:
            # another forward ran on the handle since: restore this call's state
            out = torch.empty((B * T, mod.dim), dtype=torch.bfloat16, device=xb.device)
            aux = torch.zeros(1, dtype=torch.float32, device=xb.device)
            mod._set_options(h, ctx.norms, ctx.options, xb.device)
            mod._forward_call(h, xb, B, T, [W_r, W_q, W_k, W_v], W_s, W_o, out, aux)
            ctx.call = mod._calls
        G.gqe_enable_backward(h)
        dn = [torch.empty_like(n) if n is not None else None for n in ctx.norms]
        mod._set_options(h, ctx.norms, ctx.options, xb.device, dn)
        aux_grad = 0.0 if daux is None else float(daux)
        if dy is None:
            dy = torch.zeros((B, T, mod.dim), dtype=torch.bfloat16, device=xb.device)
        dyb = dy.reshape(B * T, mod.dim).to(torch.bfloat16).contiguous()
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=xb.device)  # noqa: E731
        g = [f32(B * T, mod.dim), f32(*W_r.shape), f32(*W_q.shape), f32(*W_k.shape),
             f32(*W_v.shape), f32(*W_s.shape) if W_s is not None else None, f32(*W_o.shape)]
        G.gqe_backward(h, xb, B, T, W_r, W_q, W_k, W_v, W_s, W_o, mod.N, mod.G, mod.k, mod.d_h,
                       G.VARIANTS[mod.variant], int(mod.causal), dyb, aux_grad, *g)
        dx = g[0].view(B, T, mod.dim).to(ctx.x_dtype)
        return dx, g[1], g[2], g[3], g[4], g[5], g[6], dn[0], dn[1], None, None


class GQEAttention(nn.Module):
    """GQE attention ("GQE: Grouped Query Experts" README, Parameters): N query-head experts in
    G groups (num_kv_heads, one dense KV head each), the top k of each group per token plus
    the always-on shared head, output construction `variant` ("gqe", "weighted_concat",
    "hard_concat"); head_dim defaults to dim // num_query_experts. Input [B, T, dim], output
    [B, T, dim] in bf16; causal unless causal=False.

    qk_norm: RMS norm of every query and key head with weights q_norm, k_norm [head_dim].
    rope_base: rotate queries and keys by position, pair i of rope_dim values (head_dim unless
    given) by position * rope_base^(-2i/rope_dim); rope_interleaved pairs neighbours instead of
    halves. softcap: scores z become softcap tanh(z / softcap). slopes: one value per query
    stream (num_kv_heads * top_k routed ones, then the shared one), scores lose slope times
    distance; "geometric" for 2^(-8 (s+1) / streams)."""

    def __init__(self, dim: int, num_query_experts: int = 16, num_kv_heads: int = 8,
                 top_k: int = 1, head_dim: int | None = None, variant: str = "gqe",
                 shared: bool = True, causal: bool = True, qk_norm: bool = False,
                 norm_eps: float = 1e-6, rope_base: float | None = None,
                 rope_dim: int | None = None, rope_interleaved: bool = False,
                 softcap: float = 0.0, slopes=None):
        super().__init__()
        if num_query_experts % num_kv_heads != 0:
            raise ValueError("num_query_experts must be divisible by num_kv_heads")
        if variant not in G.VARIANTS:
            raise ValueError(f"variant must be one of {sorted(G.VARIANTS)}")
        self.dim, self.N, self.G, self.k = dim, num_query_experts, num_kv_heads, top_k
        self.d_h = head_dim if head_dim is not None else dim // num_query_experts
        self.variant, self.shared, self.causal = variant, shared, causal
        d, dh = dim, self.d_h
        self.W_r = nn.Parameter(torch.empty(self.N, d))
        self.W_q = nn.Parameter(torch.empty(self.N * dh, d))
        self.W_k = nn.Parameter(torch.empty(self.G * dh, d))
        self.W_v = nn.Parameter(torch.empty(self.G * dh, d))
        self.W_shared = nn.Parameter(torch.empty(dh, d)) if shared else None
        self.W_o = nn.Parameter(torch.empty(d, self.D_o))
        for p in self.parameters():  # nn.Linear's default: U(-1/sqrt(in), 1/sqrt(in))
            bound = 1.0 / math.sqrt(p.shape[1])
            nn.init.uniform_(p, -bound, bound)
        self.q_norm = nn.Parameter(torch.ones(dh)) if qk_norm else None
        self.k_norm = nn.Parameter(torch.ones(dh)) if qk_norm else None
        self.qk_norm, self.norm_eps, self.softcap = qk_norm, norm_eps, float(softcap)
        self.rope_interleaved = rope_interleaved
        if not self.softcap >= 0:
            raise ValueError("softcap must be positive, or 0 for none")
        if not norm_eps >= 0:
            raise ValueError("norm_eps must not be negative")
        if rope_base is None and rope_dim is not None:
            raise ValueError("rope_dim needs a rope_base")
        if rope_base is not None and not rope_base > 0:
            raise ValueError("rope_base must be positive")
        rot = (rope_dim if rope_dim is not None else dh) if rope_base is not None else 0
        if rot % 16 != 0 or not 0 <= rot <= dh:
            raise ValueError("rope_dim must be a multiple of 16 up to head_dim")
        self._freq = [float(rope_base) ** (-2.0 * i / rot) for i in range(rot // 2)] if rot else None
        streams = self.G * self.k + bool(shared)
        if isinstance(slopes, str):
            if slopes != "geometric":
                raise ValueError('slopes must be "geometric" or one value per query stream')
            slopes = [2.0 ** (-8.0 * (s + 1) / streams) for s in range(streams)]
        self._slopes = None if slopes is None else [float(s) for s in slopes]
        if self._slopes is not None and len(self._slopes) != streams:
            raise ValueError(f"expected {streams} slopes, one per query stream")
        self._tables = {}  # per device: frequencies (float64) and slopes (float32)
        self._options_set = False
        self._h = None
        self._max_tokens = 0
        self._device = None
        self._calls = 0
        self._aux = None

    @property
    def D_o(self) -> int:
        return (self.G * self.k + (self.variant == "gqe") + self.shared) * self.d_h

    def _handle_for(self, M: int):
        dev = torch.cuda.current_device()
        if self._h is None or M > self._max_tokens or dev != self._device:
            self._release()
            self._h = G.gqe_create(self.dim, self.N, self.G, self.k, self.d_h, G.GQE_BF16, M)
            self._max_tokens, self._device = M, dev
            self._options_set = False
        return self._h

    def _tables_on(self, device):
        if device not in self._tables:
            make = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device=device)  # noqa: E731
            self._tables[device] = (make(self._freq, torch.float64),
                                    make(self._slopes, torch.float32))
        return self._tables[device]

    def _set_options(self, h, norms, call, device, dnorms=(None, None)):
        """Sets the norm, rotation and scores of one call on the handle; call: its positions,
        key_begin and key_end. Modules without options never touch the handle."""
        positions, key_begin, key_end = call
        transform = self.qk_norm or self._freq is not None
        scores = (self.softcap > 0 or self._slopes is not None or key_begin is not None
                  or key_end is not None)
        if not (transform or scores or self._options_set):
            return
        freq, slopes = self._tables_on(device)
        if transform:
            G.gqe_set_qk_transform(h, self.d_h, norm=self.qk_norm, q_weight=norms[0],
                                   k_weight=norms[1], eps=self.norm_eps, inv_freq=freq,
                                   interleaved=self.rope_interleaved, positions=positions,
                                   dq_weight=dnorms[0], dk_weight=dnorms[1])
        G.gqe_set_scores(h, softcap=self.softcap, slopes=slopes, key_begin=key_begin,
                         key_end=key_end)
        self._options_set = True

    def _forward_call(self, h, xb, B, T, w, ws, wo, out, aux):
        G.gqe_forward(h, xb, B, T, w[0], w[1], w[2], w[3], ws, wo, self.N, self.G, self.k,
                      self.d_h, G.VARIANTS[self.variant], int(self.causal), out, aux)
        self._calls += 1

    def forward(self, x: torch.Tensor, positions: torch.Tensor | None = None,
                key_begin: torch.Tensor | None = None,
                key_end: torch.Tensor | None = None) -> torch.Tensor:
        """positions: of every token for the rotation ([B, T], or None for 0 .. T-1); key_begin,
        key_end: the keys [begin, end) every token sees ([B, T] positions in its sequence, on
        top of the causal mask), or None for all."""
        if x.dim() != 3 or x.shape[2] != self.dim:
            raise ValueError(f"expected input [B, T, {self.dim}]")
        call = tuple(self._ints(t, x.shape[0] * x.shape[1], x.device)
                     for t in (positions, key_begin, key_end))
        y, aux = _GQEFunction.apply(x, self.W_r, self.W_q, self.W_k, self.W_v, self.W_shared,
                                    self.W_o, self.q_norm, self.k_norm, self, call)
        self._aux = aux
        return y

    @staticmethod
    def _ints(t, n, device):
        """A private int32 copy of an index tensor: the backward reads it after the caller may
        have changed its own."""
        if t is None:
            return None
        if t.numel() != n:
            raise ValueError(f"expected {n} positions, one per token")
        return t.detach().to(device=device, dtype=torch.int32).reshape(-1).clone()

    def allocate_cache(self, B: int, L_max: int, device=None):
        """Empty KV caches for generation: k_cache, v_cache [G, B, L_max, d_h] in bf16."""
        shape = (self.G, B, L_max, self.d_h)
        dev = device if device is not None else self.W_r.device
        return (torch.zeros(shape, dtype=torch.bfloat16, device=dev),
                torch.zeros(shape, dtype=torch.bfloat16, device=dev))

    @torch.no_grad()
    def decode_step(self, x_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    lengths: torch.Tensor,
                    key_begin: torch.Tensor | None = None) -> torch.Tensor:
        """One generation step (gqe_decode): x_new [B, dim], one new token per sequence at
        position lengths[b] (int32, on the device); its K / V are written into the caches at
        that row and y_new [B, dim] (bf16) is returned. The caller advances `lengths`.
        key_begin: [B] first visible rows of the caches (int32, on the device), or None. A
        rotated key has its row as its position: a forward with `positions` of its own is not
        continued."""
        B = x_new.shape[0]
        if key_begin is not None and (key_begin.numel() != B or key_begin.dtype != torch.int32
                                      or key_begin.device != x_new.device):
            raise ValueError(f"expected {B} first rows (int32, on the device), one per sequence")
        bf = torch.bfloat16
        h = self._handle_for(B)
        w = [W.to(bf).contiguous() for W in (self.W_r, self.W_q, self.W_k, self.W_v)]
        ws = self.W_shared.to(bf).contiguous() if self.W_shared is not None else None
        out = torch.empty((B, self.dim), dtype=bf, device=x_new.device)
        aux = torch.zeros(1, dtype=torch.float32, device=x_new.device)
        # (no copy of key_begin: a captured step reads the caller's, as it does `lengths`)
        norms = [n.float().contiguous() if n is not None else None
                 for n in (self.q_norm, self.k_norm)]
        self._set_options(h, norms, (None, key_begin, None), x_new.device)
        G.gqe_decode(h, x_new.to(bf).contiguous(), B, k_cache, v_cache, k_cache.shape[2],
                     lengths, w[0], w[1], w[2], w[3], ws, self.W_o.to(bf).contiguous(), self.N,
                     self.G, self.k, self.d_h, G.VARIANTS[self.variant], out, aux)
        self._calls += 1  # the handle's saved state is no longer a forward's
        return out

    def aux_loss(self) -> torch.Tensor | None:
        """The Switch load-balancing loss of the last call (a differentiable scalar)."""
        return self._aux

    def _release(self):
        if self._h is not None:
            G.gqe_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self._release()
        except Exception:
            pass


def collect_aux_loss(model: nn.Module) -> torch.Tensor:
    """The sum of the aux losses of the last calls of every GQEAttention in `model` (the
    README's collect_aux_loss; the caller applies its coefficient, 0.01 in the README)."""
    total = None
    for m in model.modules():
        if isinstance(m, GQEAttention) and m._aux is not None:
            total = m._aux if total is None else total + m._aux
    if total is None:
        p = next(model.parameters(), None)
        return torch.zeros((), device=p.device if p is not None else None)
    return total


def document_spans(lengths, T: int, device=None):
    """key_begin, key_end [T] (int32) of one sequence of T tokens packed with documents of these
    lengths: every token sees its own document (with causal=True, up to itself). Tokens behind
    the last document see nothing."""
    begin = torch.zeros(T, dtype=torch.int32)
    end = torch.zeros(T, dtype=torch.int32)
    at = 0
    for n in lengths:
        n = int(n)
        if n < 0 or at + n > T:
            raise ValueError("document lengths must not be negative or exceed the sequence")
        begin[at:at + n], end[at:at + n] = at, at + n
        at += n
    return begin.to(device), end.to(device)


def prefix_spans(prefix: int, T: int, device=None):
    """key_end [T] (int32) of one sequence whose first `prefix` tokens every token sees, and which
    is causal behind them (for a module with causal=False)."""
    return torch.clamp(torch.arange(1, T + 1, dtype=torch.int32), min=min(prefix, T)).to(device)
