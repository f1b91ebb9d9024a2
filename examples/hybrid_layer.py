"""A small hybrid model, layers of linear attention with a decay in turn with layers of window attention, trained, then
run as it is served: a packed prefill of prompts of different lengths, and generation one token at a time from the
states and ring caches that it left.

A layer, from the normed residual stream x (tokens, d_model):
    linear:  q, k, v, z = projections of x;  a = a small one, a number per head
             q, k = norm per head                                  (mamba_qk_norm_rope_fwd without a rotation)
             y    = linear attention(q, k, v, g = -softplus(a))    (mamba_linear_attn_fwd)
             y    = norm(y) silu(z) per head                       (mamba_gated_norm_fwd)
    window:  q, k, v = projections of x
             q, k = norm per head, rotated by position             (mamba_qk_norm_rope_fwd)
             y    = attention to the last keys and the first few   (mamba_window_attn_fwd)
    stream, x = join of the output projection of y                 (mamba_add_norm_fwd)
Projections are mamba_gemm_bf16, the residual stream is fp32.  The gradients are the same calls' _bwd and two products
per projection.

    python examples/hybrid_layer.py [--steps 40] [--tokens 256]

needs a GPU and the built library; prints the loss, and how far generation is from the prefill.
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_47_amd as ssm  # noqa: E402

BF = torch.bfloat16


def project(x, w):
    """x (tokens, in) w^T for w (out, in)."""
    return ssm.mamba_gemm_bf16(w, x[None], c_trans=True)[0]


def project_bwd(x, w, dy):
    """Gradients of project with respect to x and w."""
    dx = ssm.mamba_gemm_bf16(w.t().contiguous(), dy[None], c_trans=True)[0]
    dw = ssm.mamba_gemm_bf16(dy.t().contiguous(), x[None], b_kcontig=False)[0]
    return dx, dw


def token_positions(offsets, tokens):
    """The position of every token in its sequence."""
    t = torch.arange(tokens, device=offsets.device)
    return t - offsets[torch.searchsorted(offsets, t, right=True) - 1]


class Layer:
    """What both kinds share: the projections, the norms of queries and keys, the join."""

    def __init__(self, sizes, d_model, d_y, dim, gen, dev):
        def rand(*shape):
            return torch.randn(*shape, generator=gen, device=dev) * shape[-1] ** -0.5

        self.sizes = sizes
        self.w = dict(w_in=rand(sum(sizes), d_model), w_out=rand(d_model, d_y), q=torch.ones(dim, device=dev),
                      k=torch.ones(dim, device=dev), scale=torch.full((d_model,), 0.5, device=dev),
                      norm=torch.ones(d_model, device=dev))
        self.freq = None

    def inputs(self, x, positions):
        self.w_in, self.w_out = (self.w[n].to(BF) for n in ("w_in", "w_out"))
        parts = project(x, self.w_in).split(self.sizes, dim=1)
        q, k = (t.unflatten(1, (h, -1)) for t, h in zip(parts, (self.hq, self.hk)))
        qn, kn = ssm.mamba_qk_norm_rope_fwd(q, k, self.w["q"], self.w["k"], positions, self.freq)
        return dict(x=x, positions=positions, q=q, k=k, qn=qn, kn=kn), parts[2:]

    def join(self, s, y, stream):
        s.update(n=y.flatten(1), stream=stream)
        s["o"] = project(s["n"], self.w_out)
        return ssm.mamba_add_norm_fwd(s["o"], stream, self.w["norm"], scale=self.w["scale"])

    def backward(self, s, dx, dstream):
        """Gradients for the next x and stream; returns those of x, of the stream and of the weights."""
        j = ssm.mamba_add_norm_bwd(s["o"], s["stream"], self.w["norm"], dx, dresidual_out=dstream,
                                   scale=self.w["scale"])
        dy, dw_out = project_bwd(s["n"], self.w_out, j["dx"])
        dqn, dkn, rest, dw = self.mixer_bwd(s, dy)
        d = ssm.mamba_qk_norm_rope_bwd(s["q"], s["k"], self.w["q"], self.w["k"], s["positions"], self.freq, dqn, dkn)
        dp = torch.cat([d["dq"].flatten(1), d["dk"].flatten(1), *rest], dim=1)
        dx, dw_in = project_bwd(s["x"], self.w_in, dp)
        dw.update(w_in=dw_in, w_out=dw_out, q=d["dq_weight"], k=d["dk_weight"], scale=j["dscale"], norm=j["dweight"])
        return dx, j["dresidual"], dw


class LinearLayer(Layer):
    """Hk key heads of dk, Hv value heads of dv; what generation keeps is the state of every head."""

    def __init__(self, d_model, hk, hv, dk, dv, gen, dev):
        super().__init__([hk * dk, hk * dk, hv * dv, hv * dv, 16], d_model, hv * dv, dk, gen, dev)
        self.hq, self.hk, self.hv = hk, hk, hv
        self.w["gate"] = torch.ones(dv, device=dev)

    def mixer_inputs(self, x, positions):
        s, (v, z, a) = self.inputs(x, positions if self.freq is not None else None)
        v, z = (t.unflatten(1, (self.hv, -1)) for t in (v, z))
        a = a[:, :self.hv].float()
        s.update(v=v, z=z, a=a, g=-F.softplus(a))
        return s

    def forward(self, x, stream, offsets, positions):
        """Packed sequences: x, stream (tokens, d_model).  Returns the next x and stream, what the gradients need, and
        what generation needs."""
        s = self.mixer_inputs(x, positions)
        s["offsets"] = offsets
        s["y"], last = ssm.mamba_linear_attn_fwd(s["qn"], s["kn"], s["v"], s["g"], seq_offsets=offsets,
                                                 return_last_state=True)
        return *self.join(s, ssm.mamba_gated_norm_fwd(s["y"], s["z"], self.w["gate"]), stream), s, last

    def step(self, x, stream, positions, state):
        """One token for each sequence; the states are updated in place."""
        s = self.mixer_inputs(x, positions)
        y = ssm.mamba_linear_attn_update(state, s["qn"], s["kn"], s["v"], s["g"])
        return self.join(s, ssm.mamba_gated_norm_fwd(y, s["z"], self.w["gate"]), stream)

    def mixer_bwd(self, s, dy):
        t = ssm.mamba_gated_norm_bwd(s["y"], s["z"], self.w["gate"], dy.view_as(s["y"]))
        d = ssm.mamba_linear_attn_bwd(s["qn"], s["kn"], s["v"], s["g"], t["dy"], seq_offsets=s["offsets"])
        da = torch.zeros(dy.shape[0], 16, device=dy.device)
        da[:, :self.hv] = -d["dg"] * torch.sigmoid(s["a"])
        return d["dq"], d["dk"], (d["dv"].flatten(1), t["dz"].flatten(1), da.to(BF)), dict(gate=t["dweight"])


class WindowLayer(Layer):
    """Hq query heads and Hk key and value heads of dim; what generation keeps is a ring of sinks + window keys."""

    def __init__(self, d_model, hq, hk, dim, window, sinks, gen, dev):
        super().__init__([hq * dim, hk * dim, hk * dim], d_model, hq * dim, dim, gen, dev)
        self.hq, self.hk, self.window, self.sinks = hq, hk, window, sinks
        # half of each head turns, with wave lengths up to 10000 tokens
        self.freq = 10000.0 ** -(torch.arange(dim // 4, dtype=torch.float64, device=dev) / (dim // 4))

    def forward(self, x, stream, offsets, positions):
        s, (v,) = self.inputs(x, positions)
        s.update(v=v.unflatten(1, (self.hk, -1)), offsets=offsets)
        s["y"], s["lse"] = ssm.mamba_window_attn_fwd(s["qn"], s["kn"], s["v"], self.window, self.sinks,
                                                     seq_offsets=offsets, return_lse=True)
        cache = [torch.empty(len(offsets) - 1, self.sinks + self.window, self.hk, v.shape[1] // self.hk,
                             device=x.device, dtype=BF) for _ in range(2)]
        ssm.mamba_window_cache_store(*cache, s["kn"], s["v"], self.sinks, seq_offsets=offsets)
        return *self.join(s, s["y"], stream), s, cache

    def step(self, x, stream, positions, cache):
        s, (v,) = self.inputs(x, positions)
        y = ssm.mamba_window_attn_update(*cache, s["qn"], s["kn"], v.unflatten(1, (self.hk, -1)), positions, self.sinks)
        return self.join(s, y, stream)

    def mixer_bwd(self, s, dy):
        d = ssm.mamba_window_attn_bwd(s["qn"], s["kn"], s["v"], s["y"], s["lse"], dy.view_as(s["y"]), self.window,
                                      self.sinks, seq_offsets=s["offsets"])
        return d["dq"], d["dk"], (d["dv"].flatten(1),), {}


class Model:
    def __init__(self, kinds="lw", d_model=256, dim=64, window=48, sinks=2, vocab=64, seed=0, dev="cuda:0"):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.layers = [LinearLayer(d_model, 2, 4, dim, dim, gen, dev) if kind == "l" else
                       WindowLayer(d_model, 4, 2, dim, window, sinks, gen, dev) for kind in kinds]
        self.embed = 0.1 * torch.randn(vocab, d_model, generator=gen, device=dev)
        self.first = torch.ones(d_model, device=dev)

    def start(self, tokens):
        """The stream and its norm, the first layer's input."""
        e = self.embed[tokens].to(BF)
        return ssm.mamba_add_norm_fwd(e, None, self.first, residual_out=torch.empty(e.shape, device=e.device))

    def logits(self, x):
        return project(x, self.embed.to(BF)).float()

    def prefill(self, tokens, offsets):
        """Packed prompts; returns the logits of every token, what generation needs of every layer, and what the
        gradients need."""
        x, stream = self.start(tokens)
        positions = token_positions(offsets, len(tokens))
        memory, saved = [], []
        for layer in self.layers:
            x, stream, s, m = layer.forward(x, stream, offsets, positions)
            memory.append(m)
            saved.append(s)
        return self.logits(x), memory, (saved, x)

    def step(self, tokens, positions, memory):
        """One token for each sequence, `positions` tokens behind its first."""
        x, stream = self.start(tokens)
        for layer, m in zip(self.layers, memory):
            x, stream = layer.step(x, stream, positions, m)
        return self.logits(x)

    def gradients(self, tokens, targets, offsets):
        """The loss and the gradients of every layer's weights."""
        logits, _, (saved, x) = self.prefill(tokens, offsets)
        loss = F.cross_entropy(logits, targets)
        dl = torch.softmax(logits, -1)
        dl[torch.arange(len(targets), device=dl.device), targets] -= 1.0
        dx, _ = project_bwd(x, self.embed.to(BF), (dl / len(targets)).to(BF))
        dstream, grads = None, []
        for layer, s in zip(reversed(self.layers), reversed(saved)):
            dx, dstream, dw = layer.backward(s, dx, dstream)
            grads.insert(0, dw)
        return loss, grads

    def train(self, tokens, targets, offsets, rate):
        """One step of gradient descent on the layers' weights; returns the loss before it."""
        loss, grads = self.gradients(tokens, targets, offsets)
        for layer, dw in zip(self.layers, grads):
            for name, d in dw.items():
                layer.w[name] -= rate * d.float()
        return float(loss)


def sequences(lengths, vocab, seed, dev):
    """Random tokens of which every sequence repeats its first half."""
    gen = torch.Generator().manual_seed(seed)
    rows = []
    for n in lengths:
        half = torch.randint(0, vocab, ((n + 2) // 2,), generator=gen)
        rows.append(torch.cat([half, half])[:n + 1])
    tokens = torch.cat([r[:-1] for r in rows]).to(dev)
    targets = torch.cat([r[1:] for r in rows]).to(dev)
    return tokens, targets, torch.tensor([0] + lengths, device=dev).cumsum(0)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=256)
    a = ap.parse_args(argv)
    dev = "cuda:0"
    model = Model(dev=dev)
    t = a.tokens
    lengths = [t, t // 2, t // 4 + 8, t // 4 - 8]     # multiples of 8 in all: the projections' tokens
    losses = []
    for i in range(a.steps):
        losses.append(model.train(*sequences(lengths, 64, i % 4, dev), rate=0.3))
        if i % 10 == 0 or i == a.steps - 1:
            print(f"step {i}: loss {losses[-1]:.4f}", flush=True)

    # serving: prompts of different lengths in one packed prefill, then 8 tokens each, one at a time
    tokens, _, _ = sequences([t] * 8, 64, 100, dev)
    rows = tokens.view(8, t)
    cut = [t - 8 - 3 * i for i in range(8)]
    cut[-1] -= sum(cut) % 8
    offsets = torch.tensor([0] + cut, device=dev).cumsum(0)
    _, memory, _ = model.prefill(torch.cat([r[:n] for r, n in zip(rows, cut)]), offsets)
    whole = model.prefill(tokens, torch.arange(9, device=dev) * t)[0].view(8, t, -1)
    worst = 0.0
    for i in range(8):
        positions = torch.tensor(cut, device=dev) + i
        got = model.step(torch.stack([r[n + i] for r, n in zip(rows, cut)]), positions, memory)
        want = torch.stack([w[n + i] for w, n in zip(whole, cut)])
        worst = max(worst, float((got - want).norm() / want.norm()))
    print(f"generation against the prefill of the whole sequence: {worst:.2e} (2-norm, relative)", flush=True)
    return losses, worst


if __name__ == "__main__":
    main()
