"""A small recurrent model of gated delta layers, trained, then run as it is served: a packed prefill of
prompts of different lengths, and generation one token at a time from the states it left.

One layer, from the normed residual stream x (tokens, d_model):
    q, k, v, z = projections of x;  a, b = two small ones, a number per head
    q, k       = unit length per head                        (mamba_gated_norm_fwd without a gate)
    y          = gated delta rule(q, k, v, g = -softplus(a), beta = sigmoid(b))   (mamba_delta_fwd)
    y          = norm(y) silu(z) per head                    (mamba_gated_norm_fwd)
    stream, x  = join of the output projection of y          (mamba_add_norm_fwd)
Projections are mamba_gemm_bf16, the residual stream is fp32.  The gradients are the same calls' _bwd and
two products per projection.

    python examples/delta_layer.py [--steps 40] [--tokens 256]

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


class Layer:
    """Weights and passes of one layer; Hk key heads of dk, Hv value heads of dv."""

    def __init__(self, d_model, hk, hv, dk, dv, gen, dev):
        def rand(*shape):
            return torch.randn(*shape, generator=gen, device=dev) * shape[-1] ** -0.5

        self.hk, self.hv, self.dk, self.dv = hk, hv, dk, dv
        self.sizes = [hk * dk, hk * dk, hv * dv, hv * dv, 16, 16]  # q, k, v, z, a, b (16-row pieces)
        self.w = dict(w_in=rand(sum(self.sizes), d_model), w_out=rand(d_model, hv * dv),
                      gate=torch.ones(dv, device=dev), scale=torch.full((d_model,), 0.5, device=dev),
                      norm=torch.ones(d_model, device=dev))
        # a norm of weight 1 / sqrt(dk) gives queries and keys unit length
        self.unit = torch.full((dk,), dk ** -0.5, device=dev)

    def mixer_inputs(self, x):
        self.w_in, self.w_out = (self.w[n].to(BF) for n in ("w_in", "w_out"))
        p = project(x, self.w_in)
        q, k, v, z, a, b = p.split(self.sizes, dim=1)
        heads = lambda t, h: t.unflatten(1, (h, -1))  # noqa: E731
        q, k, v, z = heads(q, self.hk), heads(k, self.hk), heads(v, self.hv), heads(z, self.hv)
        qn = ssm.mamba_gated_norm_fwd(q, None, self.unit)
        kn = ssm.mamba_gated_norm_fwd(k, None, self.unit)
        a, b = (t[:, :self.hv].float() for t in (a, b))
        g, beta = -F.softplus(a), torch.sigmoid(b)
        return q, k, v, z, qn, kn, a, b, g.to(BF), beta.to(BF)

    def finish(self, y, z, stream):
        n = ssm.mamba_gated_norm_fwd(y, z, self.w["gate"])
        o = project(n.flatten(1), self.w_out)
        x, new = ssm.mamba_add_norm_fwd(o, stream, self.w["norm"], scale=self.w["scale"])
        return n, o, x, new

    def forward(self, x, stream, offsets, state=None, keep=None):
        """Packed sequences: x, stream (tokens, d_model).  Returns the next x and stream and the states."""
        q, k, v, z, qn, kn, a, b, g, beta = self.mixer_inputs(x)
        y, last = ssm.mamba_delta_fwd(qn, kn, v, g, beta, seq_offsets=offsets, initial_state=state,
                                      return_last_state=True)
        n, o, out, new = self.finish(y, z, stream)
        if keep is not None:
            keep.update(x=x, q=q, k=k, v=v, z=z, qn=qn, kn=kn, a=a, b=b, g=g, beta=beta, y=y, n=n, o=o,
                        stream=stream, offsets=offsets)
        return out, new, last

    def step(self, x, stream, state):
        """One token for each sequence; the states are updated in place."""
        _, _, v, z, qn, kn, _, _, g, beta = self.mixer_inputs(x)
        y = ssm.mamba_delta_update(state, qn, kn, v, g, beta)
        return self.finish(y, z, stream)[2:]

    def backward(self, s, dx, dstream):
        """Gradients for the next x and stream; returns those of x, of the stream and of the weights."""
        j = ssm.mamba_add_norm_bwd(s["o"], s["stream"], self.w["norm"], dx, dresidual_out=dstream,
                                   scale=self.w["scale"])
        dn, dw_out = project_bwd(s["n"].flatten(1), self.w_out, j["dx"])
        t = ssm.mamba_gated_norm_bwd(s["y"], s["z"], self.w["gate"], dn.view_as(s["n"]))
        d = ssm.mamba_delta_bwd(s["qn"], s["kn"], s["v"], s["g"], s["beta"], t["dy"],
                                seq_offsets=s["offsets"])
        dq = ssm.mamba_gated_norm_bwd(s["q"], None, self.unit, d["dq"])["dy"]
        dk = ssm.mamba_gated_norm_bwd(s["k"], None, self.unit, d["dk"])["dy"]
        sig = torch.sigmoid(s["b"])
        small = torch.zeros(dx.shape[0], 32, device=dx.device)
        small[:, :self.hv] = -d["dg"].float() * torch.sigmoid(s["a"])
        small[:, 16:16 + self.hv] = d["dbeta"].float() * sig * (1 - sig)
        dp = torch.cat([dq.flatten(1), dk.flatten(1), d["dv"].flatten(1), t["dz"].flatten(1),
                        small.to(BF)], dim=1)
        dx, dw_in = project_bwd(s["x"], self.w_in, dp)
        return dx, j["dresidual"], dict(w_in=dw_in, w_out=dw_out, gate=t["dweight"], scale=j["dscale"],
                                        norm=j["dweight"])


class Model:
    def __init__(self, layers=2, d_model=256, hk=2, hv=4, dk=64, dv=64, vocab=64, seed=0, dev="cuda:0"):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.layers = [Layer(d_model, hk, hv, dk, dv, gen, dev) for _ in range(layers)]
        self.embed = 0.1 * torch.randn(vocab, d_model, generator=gen, device=dev)
        self.first = torch.ones(d_model, device=dev)

    def start(self, tokens):
        """The stream and its norm, the first layer's input."""
        e = self.embed[tokens].to(BF)
        return ssm.mamba_add_norm_fwd(e, None, self.first, residual_out=torch.empty(
            e.shape, device=e.device))

    def logits(self, x):
        return project(x, self.embed.to(BF)).float()

    def prefill(self, tokens, offsets, keep=None):
        """Packed prompts; returns the logits of every token and the states of every layer."""
        x, stream = self.start(tokens)
        states = []
        for layer in self.layers:
            saved = None if keep is None else {}
            x, stream, last = layer.forward(x, stream, offsets, keep=saved)
            states.append(last)
            if keep is not None:
                keep.append(saved)
        return self.logits(x), states, x

    def step(self, tokens, states):
        x, stream = self.start(tokens)
        for layer, state in zip(self.layers, states):
            x, stream = layer.step(x, stream, state)
        return self.logits(x)

    def train(self, tokens, targets, offsets, rate):
        """One step of gradient descent on the layers' weights; returns the loss before it."""
        keep = []
        logits, _, x = self.prefill(tokens, offsets, keep)
        loss = F.cross_entropy(logits, targets)
        dl = torch.softmax(logits, -1)
        dl[torch.arange(len(targets), device=dl.device), targets] -= 1.0
        dx, _ = project_bwd(x, self.embed.to(BF), (dl / len(targets)).to(BF))
        dstream = None
        for layer, saved in zip(reversed(self.layers), reversed(keep)):
            dx, dstream, dw = layer.backward(saved, dx, dstream)
            for name, d in dw.items():
                layer.w[name] -= rate * d.float()
        return float(loss)


def sequences(lengths, vocab, seed, dev):
    """Random tokens in which every second token of a sequence repeats: what follows a token that was seen
    before is what followed it then."""
    gen = torch.Generator().manual_seed(seed)
    rows = []
    for n in lengths:
        half = torch.randint(0, vocab, ((n + 2) // 2,), generator=gen)
        rows.append(torch.cat([half, half])[:n + 1])
    tokens = torch.cat([r[:-1] for r in rows]).to(dev)
    targets = torch.cat([r[1:] for r in rows]).to(dev)
    offsets = torch.tensor([0] + lengths, device=dev).cumsum(0)
    return tokens, targets, offsets


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
    cut[-1] -= (sum(cut)) % 8
    offsets = torch.tensor([0] + cut, device=dev).cumsum(0)
    _, states, _ = model.prefill(torch.cat([r[:n] for r, n in zip(rows, cut)]), offsets)
    whole, _, _ = model.prefill(tokens, torch.arange(9, device=dev) * t)
    whole = whole.view(8, t, -1)
    worst = 0.0
    for i in range(8):
        now = torch.stack([r[n + i] for r, n in zip(rows, cut)])
        got = model.step(now, states)
        want = torch.stack([w[n + i] for w, n in zip(whole, cut)])
        worst = max(worst, float((got - want).norm() / want.norm()))
    print(f"generation against the prefill of the whole sequence: {worst:.2e} (2-norm, relative)",
          flush=True)
    return losses, worst


if __name__ == "__main__":
    main()
