"""A small sequence model of two layers -- one with the selective scan, one with
the SSD scan, and with --delta a third with the gated delta rule -- trained for a few
steps and then used to generate.

    python examples/layer_stack.py [--steps 30] [--dtype f32|bf16] [--delta]

Training runs the convolution, the scans, the norm of queries and keys, the gated norm
and the block norm forward and backward (each wrapped as an autograd function below; the
projections are plain matrix products).  Generation takes a batch of prompts of
unequal lengths (one of them empty) through the prompt forms, which leave every
layer's convolution and scan states, and goes on token by token with the
single-token forms over a cache of slots.  The generated logits are compared
with those of a full pass over the same tokens.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import state_space_model_sm_gb300 as ssd  # noqa: E402

CHUNK = 64


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        ctx.save_for_backward(x, w, bias)
        return ssd.causal_conv_fwd(x, w, bias, return_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        g = ssd.causal_conv_bwd(*ctx.saved_tensors, dy.contiguous())
        return g["dx"], g["dw"], g["dbias"]


class SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, dt_bias, A, B, C, D, z):
        ctx.save_for_backward(x, dt, dt_bias, A, B, C, D, z)
        return ssd.selective_scan_fwd(x, dt, dt_bias, A, B, C, D, z, return_final_states=False)[0]

    @staticmethod
    def backward(ctx, dout):
        g = ssd.selective_scan_bwd(*ctx.saved_tensors, dout.contiguous())
        t = dout.dtype
        return (g["dx"], g["ddt"], g["ddt_bias"], g["dA"], g["dB"].to(t), g["dC"].to(t), g["dD"],
                g["dz"])


class SSDScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, dt_bias, A, B, C, D):
        ctx.save_for_backward(x, dt, dt_bias, A, B, C, D)
        return ssd.ssd_fwd(x, dt, dt_bias, A, B, C, D, CHUNK, out_dtype=x.dtype,
                           return_final_states=False)[0]

    @staticmethod
    def backward(ctx, dy):
        g = ssd.ssd_bwd(*ctx.saved_tensors, CHUNK, None, dy.contiguous())
        t = dy.dtype
        return (g["dx"].to(t), g["ddt"].to(t), g["ddt_bias"], g["dA"], g["dB"].to(t),
                g["dC"].to(t), g["dD"])


class QkNorm(torch.autograd.Function):
    """Unit queries and keys, turned by their positions."""

    @staticmethod
    def forward(ctx, q, k, w_q, w_k, freq):
        ctx.save_for_backward(q, k, w_q, w_k, freq)
        return ssd.qk_norm_fwd(q, k, w_q, w_k, freq, l2=True)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, w_q, w_k, freq = ctx.saved_tensors
        g = ssd.qk_norm_bwd(q, k, w_q, w_k, freq, None, dq.contiguous(), dk.contiguous(), l2=True)
        return g["dq"], g["dk"], g["dw_q"], g["dw_k"], None


class GatedDelta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, dt, dt_bias, A, beta):
        ctx.save_for_backward(q, k, v, dt, dt_bias, A, beta)
        return ssd.gated_delta_fwd(q, k, v, dt, dt_bias, A, beta, return_final_states=False)[0]

    @staticmethod
    def backward(ctx, dy):
        g = ssd.gated_delta_bwd(*ctx.saved_tensors, dy.contiguous())
        return g["dq"], g["dk"], g["dv"], g["ddt"], g["ddt_bias"], g["dA"], g["dbeta"]


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, z, w):
        out, rstd = ssd.gated_norm_fwd(y, z, w, y.shape[-1])
        ctx.save_for_backward(y, z, w, rstd)
        return out

    @staticmethod
    def backward(ctx, dout):
        y, z, w, rstd = ctx.saved_tensors
        g = ssd.gated_norm_bwd(y, z, w, dout.contiguous(), y.shape[-1], rstd=rstd)
        return g["dy"], g["dz"], g["dw"]


class BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, o, w_pre, w_post, gate, scale):
        ctx.save_for_backward(residual, o, w_pre, w_post, gate)
        ctx.scale = scale
        return ssd.block_norm_fwd(residual, o, w_pre, w_post, gate, scale=scale)

    @staticmethod
    def backward(ctx, dresidual, dh):
        g = ssd.block_norm_bwd(*ctx.saved_tensors, dh.contiguous(), dresidual.contiguous(),
                               scale=ctx.scale)
        return g["dresidual"], g["do"], g["dw_pre"], g["dw_post"], g["dgate"], None


def _dt_bias(n, gen):
    step = torch.exp(torch.rand(n, generator=gen) * 4.6 - 6.9)  # 1e-3 .. 1e-1
    return torch.log(torch.expm1(step))


class SelectiveLayer:
    """in-projection -> convolution -> selective scan (gated by z) -> out-projection."""

    def __init__(self, width, inner, state, rank, gen, dtype):
        n = lambda *s: torch.randn(*s, generator=gen) * s[0] ** -0.5  # noqa: E731
        self.inner, self.state, self.rank, self.K = inner, state, rank, 4
        self.p = dict(w_in=n(width, 2 * inner).to(dtype), conv=torch.rand(inner, 4, generator=gen) - 0.5,
                      conv_bias=torch.zeros(inner), w_x=n(inner, rank + 2 * state).to(dtype),
                      w_dt=n(rank, inner).to(dtype), dt_bias=_dt_bias(inner, gen),
                      A_log=torch.log(torch.arange(1.0, state + 1)).repeat(inner, 1),
                      D=torch.ones(inner), w_out=n(inner, width).to(dtype))

    def _scan_inputs(self, x):
        p, r, s = self.p, self.rank, self.state
        low, B, C = (x @ p["w_x"]).split([r, s, s], -1)
        return low @ p["w_dt"], B.unsqueeze(-2), C.unsqueeze(-2)

    def train(self, h):
        p = self.p
        x, z = (h @ p["w_in"]).split(self.inner, -1)
        x = Conv.apply(x, p["conv"], p["conv_bias"])
        dt, B, C = self._scan_inputs(x)
        y = SelectiveScan.apply(x, dt, p["dt_bias"], -torch.exp(p["A_log"]), B, C, p["D"], z)
        return y @ p["w_out"]

    def cache(self, slots, dtype):
        return [torch.zeros(slots, self.K - 1, self.inner, dtype=dtype, device="cuda"),
                torch.zeros(slots, self.inner, self.state, device="cuda")]

    def prompt(self, h, lengths, cache, slots):
        p = self.p
        x, z = (h @ p["w_in"]).split(self.inner, -1)
        x, conv = ssd.causal_conv_fwd(x, p["conv"], p["conv_bias"], lengths=lengths)
        dt, B, C = self._scan_inputs(x)
        y, state = ssd.selective_scan_fwd(x, dt, p["dt_bias"], -torch.exp(p["A_log"]), B, C, p["D"],
                                          z, lengths=lengths)
        cache[0][slots.long()], cache[1][slots.long()] = conv, state
        return y @ p["w_out"]

    def token(self, h, cache, slots):
        p = self.p
        x, z = (h @ p["w_in"]).split(self.inner, -1)
        x = ssd.causal_conv_step(x, cache[0], p["conv"], p["conv_bias"], slots=slots)
        dt, B, C = self._scan_inputs(x)
        y = ssd.selective_step(x, dt, p["dt_bias"], -torch.exp(p["A_log"]), B, C, cache[1], p["D"], z,
                               slots=slots)
        return y @ p["w_out"]


class SSDLayer:
    """in-projection -> convolution of x, B, C -> SSD scan -> gated norm -> out-projection."""

    def __init__(self, width, heads, headdim, state, gen, dtype):
        n = lambda *s: torch.randn(*s, generator=gen) * s[0] ** -0.5  # noqa: E731
        self.H, self.P, self.N, self.K = heads, headdim, state, 4
        self.inner = heads * headdim
        self.ch = self.inner + 2 * state
        self.p = dict(w_in=n(width, self.inner + self.ch + heads).to(dtype),
                      conv=torch.rand(self.ch, 4, generator=gen) - 0.5, conv_bias=torch.zeros(self.ch),
                      dt_bias=_dt_bias(heads, gen),
                      A_log=torch.log(1 + 15 * torch.rand(heads, generator=gen)),
                      D=torch.ones(heads), norm=torch.ones(self.inner),
                      w_out=n(self.inner, width).to(dtype))

    def _split(self, h):
        return (h @ self.p["w_in"]).split([self.inner, self.ch, self.H], -1)

    def _xbc(self, u):
        x, B, C = u.split([self.inner, self.N, self.N], -1)
        return (x.unflatten(-1, (self.H, self.P)).contiguous(), B.unsqueeze(-2).contiguous(),
                C.unsqueeze(-2).contiguous())

    def train(self, h):
        p = self.p
        z, u, dt = self._split(h)
        x, B, C = self._xbc(Conv.apply(u, p["conv"], p["conv_bias"]))
        y = SSDScan.apply(x, dt.contiguous(), p["dt_bias"], -torch.exp(p["A_log"]), B, C, p["D"])
        return GatedNorm.apply(y.flatten(-2), z.contiguous(), p["norm"]) @ p["w_out"]

    def cache(self, slots, dtype):
        return [torch.zeros(slots, self.K - 1, self.ch, dtype=dtype, device="cuda"),
                torch.zeros(slots, self.H, self.P, self.N, device="cuda")]

    def prompt(self, h, lengths, cache, slots):
        p = self.p
        z, u, dt = self._split(h)
        u, conv = ssd.causal_conv_fwd(u, p["conv"], p["conv_bias"], lengths=lengths)
        x, B, C = self._xbc(u)
        # a step of softplus(-inf) = 0 keeps the state over the padding
        pad = torch.arange(h.shape[1], device="cuda")[None, :] >= lengths[:, None]
        dt = dt.masked_fill(pad[..., None], float("-inf")).contiguous()
        y, state = ssd.ssd_fwd(x, dt, p["dt_bias"], -torch.exp(p["A_log"]), B, C, p["D"], CHUNK,
                               out_dtype=x.dtype)
        cache[0][slots.long()], cache[1][slots.long()] = conv, state
        return ssd.gated_norm_fwd(y.flatten(-2), z.contiguous(), p["norm"], self.inner,
                                  return_rstd=False)[0] @ p["w_out"]

    def token(self, h, cache, slots):
        p = self.p
        z, u, dt = self._split(h)
        u = ssd.causal_conv_step(u, cache[0], p["conv"], p["conv_bias"], slots=slots)
        x, B, C = self._xbc(u)
        y = ssd.ssd_step(x, dt.contiguous(), p["dt_bias"], -torch.exp(p["A_log"]), B, C, cache[1],
                         p["D"], slots=slots)
        return ssd.gated_norm_fwd(y.flatten(-2), z.contiguous(), p["norm"], self.inner,
                                  return_rstd=False)[0] @ p["w_out"]


class DeltaLayer:
    """in-projection -> convolution of q, k, v -> unit, turned queries and keys -> gated
    delta rule -> gated norm -> out-projection."""

    def __init__(self, width, heads, headdim, groups, state, gen, dtype):
        n = lambda *s: torch.randn(*s, generator=gen) * s[0] ** -0.5  # noqa: E731
        self.H, self.P, self.G, self.N, self.K = heads, headdim, groups, state, 4
        self.inner, self.gn = heads * headdim, groups * state
        self.ch = 2 * self.gn + self.inner
        self.freq = (100.0 ** (-torch.arange(state // 4) / (state // 4))).cuda()  # half of each key
        self.p = dict(w_in=n(width, self.inner + self.ch + 2 * heads).to(dtype),
                      conv=torch.rand(self.ch, 4, generator=gen) - 0.5, conv_bias=torch.zeros(self.ch),
                      w_q=torch.ones(state), w_k=torch.ones(state), dt_bias=_dt_bias(heads, gen),
                      A_log=torch.log(1 + 15 * torch.rand(heads, generator=gen)),
                      norm=torch.ones(self.inner), w_out=n(self.inner, width).to(dtype))

    def _split(self, h):
        return (h @ self.p["w_in"]).split([self.inner, self.ch, self.H, self.H], -1)

    def _qkv(self, u):
        q, k, v = u.split([self.gn, self.gn, self.inner], -1)
        return (q.unflatten(-1, (self.G, self.N)), k.unflatten(-1, (self.G, self.N)),
                v.unflatten(-1, (self.H, self.P)))

    def train(self, h):
        p = self.p
        z, u, dt, beta = self._split(h)
        q, k, v = self._qkv(Conv.apply(u, p["conv"], p["conv_bias"]))
        q, k = QkNorm.apply(q, k, p["w_q"], p["w_k"], self.freq)
        y = GatedDelta.apply(q, k, v, dt.contiguous(), p["dt_bias"], -torch.exp(p["A_log"]),
                             beta.contiguous())
        return GatedNorm.apply(y.flatten(-2), z.contiguous(), p["norm"]) @ p["w_out"]

    def cache(self, slots, dtype):
        """Convolution inputs, states, and the position of the next token of each slot."""
        return [torch.zeros(slots, self.K - 1, self.ch, dtype=dtype, device="cuda"),
                torch.zeros(slots, self.H, self.P, self.N, device="cuda"),
                torch.zeros(slots, dtype=torch.int32, device="cuda")]

    def prompt(self, h, lengths, cache, slots):
        p = self.p
        z, u, dt, beta = self._split(h)
        u, conv = ssd.causal_conv_fwd(u, p["conv"], p["conv_bias"], lengths=lengths)
        q, k, v = self._qkv(u)
        q, k = ssd.qk_norm_fwd(q, k, p["w_q"], p["w_k"], self.freq, l2=True)
        y, state = ssd.gated_delta_fwd(q, k, v, dt.contiguous(), p["dt_bias"], -torch.exp(p["A_log"]),
                                       beta.contiguous(), lengths=lengths)
        for c, new in zip(cache, (conv, state, lengths)):
            c[slots.long()] = new
        return ssd.gated_norm_fwd(y.flatten(-2), z.contiguous(), p["norm"], self.inner,
                                  return_rstd=False)[0] @ p["w_out"]

    def token(self, h, cache, slots):
        p = self.p
        z, u, dt, beta = self._split(h)
        u = ssd.causal_conv_step(u, cache[0], p["conv"], p["conv_bias"], slots=slots)
        q, k, v = self._qkv(u)
        row = slots.clamp(min=0).long()  # an empty row reads slot 0's position and moves none
        q, k = ssd.qk_norm_fwd(q, k, p["w_q"], p["w_k"], self.freq, cache[2][row], l2=True)
        y = ssd.gated_delta_step(q, k, v, dt.contiguous(), p["dt_bias"], -torch.exp(p["A_log"]),
                                 beta.contiguous(), cache[1], slots=slots)
        cache[2].index_add_(0, row, (slots >= 0).int())
        return ssd.gated_norm_fwd(y.flatten(-2), z.contiguous(), p["norm"], self.inner,
                                  return_rstd=False)[0] @ p["w_out"]


class Stack:
    """Embedding, the layers with a block norm after each, and a head.  The residual
    stream is fp32; h is in the layers' type."""

    def __init__(self, vocab=64, width=64, dtype=torch.float32, seed=0, delta=False):
        gen = torch.Generator().manual_seed(seed)
        self.dtype, self.scale = dtype, 0.5
        self.layers = [SelectiveLayer(width, 2 * width, 16, 8, gen, dtype),
                       SSDLayer(width, 8, 16, 16, gen, dtype)]
        self.p = dict(embed=torch.randn(vocab, width, generator=gen),
                      head=(torch.randn(width, vocab, generator=gen) * width ** -0.5).to(dtype))
        if delta:
            self.layers.append(DeltaLayer(width, 8, 16, 4, 32, gen, dtype))
        for i in range(len(self.layers)):
            self.p.update({f"pre{i}": torch.ones(width), f"post{i}": torch.ones(width),
                           f"gate{i}": torch.ones(1, width)})
        for d in [self.p] + [l.p for l in self.layers]:
            for k in d:
                d[k] = d[k].cuda().requires_grad_()

    def parameters(self):
        return [v for d in [self.p] + [l.p for l in self.layers] for v in d.values()]

    def _run(self, tokens, layer, norm):
        p = self.p
        r = p["embed"][tokens]
        h = torch.nn.functional.normalize(r, dim=-1) * r.shape[-1] ** 0.5
        h = h.to(self.dtype)
        for i, l in enumerate(self.layers):
            r, h = norm(r, layer(i, l, h), p[f"pre{i}"], p[f"post{i}"], p[f"gate{i}"])
        return (h @ p["head"]).float()

    def train_logits(self, tokens):
        return self._run(tokens, lambda i, l, h: l.train(h),
                         lambda *a: BlockNorm.apply(*a, self.scale))

    def _norm(self, r, o, pre, post, gate):
        return ssd.block_norm_fwd(r, o, pre, post, gate, scale=self.scale)

    def cache(self, slots):
        return [l.cache(slots, self.dtype) for l in self.layers]

    @torch.no_grad()
    def prompt_logits(self, tokens, lengths, cache, slots):
        return self._run(tokens, lambda i, l, h: l.prompt(h, lengths, cache[i], slots), self._norm)

    @torch.no_grad()
    def token_logits(self, tokens, cache, slots):
        return self._run(tokens, lambda i, l, h: l.token(h, cache[i], slots), self._norm)


def train(model, steps, batch=16, length=96, lr=1e-2, seed=0):
    """Learns a fixed order of the vocabulary: each token has one successor, and every
    third position holds a random token instead.  The losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    vocab, losses = model.p["embed"].shape[0], []
    after = torch.randperm(vocab, generator=gen, device="cuda")
    for _ in range(steps):
        first = torch.randint(0, vocab, (batch, length // 3 + 1), generator=gen, device="cuda")
        tokens = torch.stack([first, after[first], after[after[first]]], 2).flatten(1)
        tokens = tokens[:, :length + 1].contiguous()
        logits = model.train_logits(tokens[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def generate(model, lengths=(40, 0, 7, 23), new=12, seed=1):
    """Prompts of the given lengths, then `new` given tokens; the largest difference
    of the token-by-token logits from a full pass's, and the scale of the logits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, T = len(lengths), max(lengths)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    vocab = model.p["embed"].shape[0]
    text = torch.randint(0, vocab, (B, T + new), generator=gen, device="cuda")
    slots = torch.tensor([2 * b + 1 for b in range(B)], dtype=torch.int32, device="cuda")
    cache = model.cache(2 * B + 1)
    model.prompt_logits(text[:, :T].contiguous(), n, cache, slots)
    rows = torch.arange(B, device="cuda")
    step = torch.stack([model.token_logits(text[rows, n.long() + i], cache, slots)
                        for i in range(new)], 1)
    with torch.no_grad():
        full = model.train_logits(text)
    want = torch.stack([full[rows, n.long() + i] for i in range(new)], 1)
    return float((step - want).abs().max()), float(want.abs().max())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--dtype", choices=["f32", "bf16"], default="f32")
    ap.add_argument("--delta", action="store_true", help="a third layer with the gated delta rule")
    a = ap.parse_args()
    model = Stack(dtype=torch.float32 if a.dtype == "f32" else torch.bfloat16, delta=a.delta)
    losses = train(model, a.steps)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    d, top = generate(model)
    print(f"generated logits differ from a full pass by {d:.2e} (largest logit {top:.2f})")


if __name__ == "__main__":
    main()
