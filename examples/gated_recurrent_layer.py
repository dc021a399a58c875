"""A gated recurrent layer, trained and then served.

    c = SiLU(causal convolution of u W_x);  i, r = c W_gates
    h = gated recurrence of c with the gates i, r and the rates A = -exp(log_rate)
    y = h W_out;  t' = t + scale * SiLU(u W_z) * RMS(y) * post;  u' = RMS(t') * w

Training: two layers and a head predict the token seen `lag` tokens ago from batches of
packed documents of different lengths; the gradients come from causal_conv1d_bwd,
gated_recurrence_bwd and residual_norm_bwd through torch.autograd.  Serving: a packed prompt
pass in two pieces, the second from the states of the first, then tokens one by one, in a
HIP graph; they must give what one prompt pass over the longer documents gives.

    python examples/gated_recurrent_layer.py [--steps 150] [--dtype bf16|fp32]
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from selective_state_space_54_amd import mssm  # noqa: E402


class CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, weight, bias, offsets):
        ctx.save_for_backward(u, weight, bias, offsets)
        return mssm.causal_conv1d(u, weight, bias, seq_offsets=offsets)

    @staticmethod
    def backward(ctx, dy):
        u, weight, bias, offsets = ctx.saved_tensors
        g = mssm.causal_conv1d_bwd(u, weight, bias, dy.contiguous(), seq_offsets=offsets)
        return g["du"], g["dweight"], g["dbias"], None


class GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, input_gate, decay_gate, A, offsets):
        h, saved = mssm.gated_recurrence(x, input_gate, decay_gate, A, seq_offsets=offsets,
                                         return_saved=True)
        ctx.save_for_backward(x, input_gate, decay_gate, A, offsets, saved)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, input_gate, decay_gate, A, offsets, saved = ctx.saved_tensors
        g = mssm.gated_recurrence_bwd(x, input_gate, decay_gate, A, dh.contiguous(), saved=saved,
                                      seq_offsets=offsets)
        return g["dx"], g["dinput_gate"], g["ddecay_gate"], g["dA"], None


class ResidualNorm(torch.autograd.Function):
    """u, t = the normalised sum and the sum itself."""

    @staticmethod
    def forward(ctx, y, residual, weight, post_weight, gate, scale):
        u, t, rstd, post_rstd = mssm.residual_norm(y, residual, weight, post_weight=post_weight,
                                                   gate=gate, scale=scale, return_stats=True)
        ctx.save_for_backward(y, t, weight, rstd, post_weight, post_rstd, gate, scale)
        return u, t

    @staticmethod
    def backward(ctx, du, dt):
        y, t, weight, rstd, post_weight, post_rstd, gate, scale = ctx.saved_tensors
        g = mssm.residual_norm_bwd(du.contiguous(), y, t, weight, rstd, dtotal=dt.contiguous(),
                                   post_weight=post_weight, post_rstd=post_rstd, gate=gate,
                                   scale=scale)
        return (g["dy"], g["dresidual"], g["dweight"], g["dpost_weight"], g["dgate"], g["dscale"])


class Layer(torch.nn.Module):
    def __init__(self, width, inner, taps, dtype):
        super().__init__()
        p = lambda *s: torch.nn.Parameter((torch.randn(*s) * s[0] ** -0.5).to(dtype))
        self.w_x, self.w_z = p(width, inner), p(width, width)
        self.conv = torch.nn.Parameter(torch.randn(inner, taps) * taps ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(inner))
        self.w_gates = p(inner, 2 * inner)
        self.log_rate = torch.nn.Parameter(torch.linspace(-4.0, 1.5, inner))
        self.w_out = p(inner, width)
        self.post = torch.nn.Parameter(torch.ones(width))
        self.scale = torch.nn.Parameter(torch.full((width,), 0.7))
        self.w = torch.nn.Parameter(torch.ones(width))    # of the norm before the next block

    def gates(self, c):
        """The input's and the decay's gate, views of one projection, and the rates."""
        return *(c @ self.w_gates).chunk(2, dim=-1), -self.log_rate.exp()

    def forward(self, u, t, offsets):
        c = CausalConv.apply(u @ self.w_x, self.conv, self.conv_bias, offsets)
        h = GatedRecurrence.apply(c, *self.gates(c), offsets)
        return ResidualNorm.apply(h @ self.w_out, t, self.w, self.post, u @ self.w_z, self.scale)

    def join(self, h, u, t):
        return mssm.residual_norm(h @ self.w_out, t, self.w, post_weight=self.post,
                                  gate=u @ self.w_z, scale=self.scale)

    def prompt(self, u, t, offsets, states):
        """states: the convolution's and the recurrence's, or None; returns the new ones."""
        conv, rec = states or (None, None)
        c, conv = mssm.causal_conv1d(u @ self.w_x, self.conv, self.conv_bias, state=conv,
                                     seq_offsets=offsets, return_state=True)
        h, rec = mssm.gated_recurrence(c, *self.gates(c), state=rec, seq_offsets=offsets,
                                       return_state=True)
        return *self.join(h, u, t), (conv, rec)

    def token(self, u, t, states):
        """One token for each sequence; the states are updated in place."""
        conv, rec = states
        c = mssm.causal_conv1d_step(u @ self.w_x, self.conv, self.conv_bias, conv)
        h = mssm.gated_recurrence_step(c, *self.gates(c), rec)
        return self.join(h, u, t)


class Model(torch.nn.Module):
    def __init__(self, vocab, width, layers, inner, taps, dtype):
        super().__init__()
        self.embed = torch.nn.Parameter(torch.randn(vocab, width).to(dtype))
        self.layers = torch.nn.ModuleList(Layer(width, inner, taps, dtype) for _ in range(layers))
        self.head = torch.nn.Parameter((torch.randn(width, vocab) * width ** -0.5).to(dtype))

    def forward(self, ids, offsets):
        u = t = self.embed[ids]
        for layer in self.layers:
            u, t = layer(u, t, offsets)
        return (u @ self.head).float()

    @torch.no_grad()
    def prompt(self, ids, offsets, states=None):
        u = t = self.embed[ids]
        new = []
        for n, layer in enumerate(self.layers):
            u, t, state = layer.prompt(u, t, offsets, states and states[n])
            new.append(state)
        return (u @ self.head).float(), new

    @torch.no_grad()
    def token(self, ids, states):
        u = t = self.embed[ids]
        for layer, state in zip(self.layers, states):
            u, t = layer.token(u, t, state)
        return (u @ self.head).float()


def offsets_of(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0)


def serve(model, ids, first, cut, new):
    """Logits of each document's last `new` tokens: the first `cut` tokens of each (as many as
    `first` has) and the rest of the prompt in two passes, then `new` tokens through a graph."""
    pieces = [[i[:c] for i, c in zip(ids, first)], [i[c:n] for i, c, n in zip(ids, first, cut)]]
    states = None
    for p in pieces:
        _, states = model.prompt(torch.cat(p), offsets_of([len(i) for i in p]), states)
    token = torch.stack([i[n] for i, n in zip(ids, cut)])
    flat = [s for pair in states for s in pair]
    kept = [s.clone() for s in flat]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        model.token(token, states)                       # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model.token(token, states)
    for s, k in zip(flat, kept):
        s.copy_(k)
    served = []
    for j in range(new):
        token.copy_(torch.stack([i[n + j] for i, n in zip(ids, cut)]))
        graph.replay()
        served.append(out.clone())
    return torch.stack(served)


def main(steps=150, dtype="bf16", lag=3, new=8, quiet=False):
    """Returns the largest difference of the served tokens' logits from the prompt pass's, in their
    own root mean square."""
    torch.manual_seed(0)
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    model = Model(16, 128, 2, inner=192, taps=4, dtype=dt).cuda()
    opt = torch.optim.Adam(model.parameters(), lr=3e-3, foreach=False)
    lengths = [200, 1, 64, 0, 391]                       # documents of a packed batch
    offsets = offsets_of(lengths)
    for step in range(steps):
        ids = torch.randint(16, (sum(lengths),), device="cuda")
        wanted, known = ids.roll(lag), torch.ones_like(ids, dtype=torch.bool)
        for a in offsets[:-1].tolist():
            known[a:a + lag] = False
        loss = F.cross_entropy(model(ids, offsets)[known], wanted[known])
        opt.zero_grad()
        loss.backward()
        opt.step()
        if not quiet and (step % 25 == 0 or step == steps - 1):
            print(f"step {step}: loss {loss.item():.4f}", flush=True)

    cut = [50, 1, 130]
    ids = [torch.randint(16, (n + new,), device="cuda") for n in cut]
    served = serve(model, ids, [20, 0, 128], cut, new)
    whole, _ = model.prompt(torch.cat(ids), offsets_of([n + new for n in cut]))
    ends = offsets_of([n + new for n in cut])[1:]
    want = torch.stack([whole[ends - new + j] for j in range(new)])
    diff = float((served - want).abs().max() / want.square().mean().sqrt())
    if not quiet:
        print(f"served tokens against the prompt pass: {diff:.2g} of the logits' size")
    return diff


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--dtype", choices=("bf16", "fp32"), default="bf16")
    main(**vars(ap.parse_args()))
