"""A small language model of gated delta rule layers, of random weights, on this package's operators: prompts of unequal
lengths in one padded batch, then tokens one by one, with the carried states in slots of a cache.

    python examples/delta_decode.py [--dtype bf16|f32] [--layers N] [--tokens N]

Each layer is  residual = alpha residual + post_norm(out_proj(gatednorm(delta(conv(in_proj(pre_norm(residual)))), z))):
conv_fwd and delta_fwd read their inputs as columns of the projections' rows, gatednorm_fwd normalises each head's
output and applies the gate z, blocknorm_fwd is the norm after a layer, the residual and the norm before the next, and
conv_step and delta_step update the cache in place.

At the end it prefills prompt and generated tokens in one go and prints how far the logits are from
those of the token-by-token run.
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_mamba_gb300 as ssm  # noqa: E402


class DeltaNet:
    def __init__(self, layers=3, d_model=512, heads=8, groups=4, headdim=64, dstate=64, width=4, vocab=1000,
                 dtype=torch.bfloat16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def linear(n_out, n_in):
            return (torch.randn(n_out, n_in, device="cuda", generator=g) / math.sqrt(n_in)).to(dtype)

        def uniform(*shape):
            return torch.rand(shape, device="cuda", generator=g)

        self.dtype, self.width, self.alpha = dtype, width, 0.9
        self.heads, self.groups, self.headdim, self.dstate = heads, groups, headdim, dstate
        self.d_inner, self.d_conv = heads * headdim, 2 * groups * dstate + heads * headdim  # q, k and v side by side
        self.embedding = (0.02 * torch.randn(vocab, d_model, device="cuda", generator=g)).to(dtype)
        self.head = linear(vocab, d_model)
        self.norm = torch.ones(d_model, device="cuda")
        self.layers = []
        for _ in range(layers):
            step = torch.exp(uniform(heads) * math.log(100.0)) * 1e-3  # between 0.001 and 0.1
            self.layers.append({
                # q, k and v; the gate z; dt and beta
                "in": linear(self.d_conv + self.d_inner + 2 * heads, d_model),
                "conv": (2 * uniform(self.d_conv, width) - 1) / math.sqrt(width),
                "A": -torch.exp(uniform(heads) * math.log(16.0)), "dt_bias": step + torch.log(-torch.expm1(-step)),
                "gate_norm": 1 + 0.1 * uniform(headdim), "out": linear(d_model, self.d_inner),
                "post_norm": 1 + 0.1 * uniform(d_model), "next_norm": 1 + 0.1 * uniform(d_model)})

    def new_cache(self, slots):
        """The carried states of `slots` sequences, a pair of each layer."""
        return [(torch.zeros(slots, self.width - 1, self.d_conv, device="cuda", dtype=self.dtype),
                 torch.zeros(slots, self.heads, self.headdim, self.dstate, device="cuda")) for _ in self.layers]

    def _split(self, u, rows):
        """q, k, v of the convolved tokens; dt, beta and z of the projection's rows."""
        n, at = self.groups * self.dstate, self.d_conv + self.d_inner
        q, k = (u[..., i * n : (i + 1) * n].unflatten(-1, (self.groups, self.dstate)) for i in (0, 1))
        v = u[..., 2 * n :].unflatten(-1, (self.heads, self.headdim))
        return (q, k, v, rows[..., at : at + self.heads], rows[..., at + self.heads :]), rows[..., self.d_conv : at]

    def _out(self, p, y, z, residual):
        """The layer's end and the next one's norm: (its input, the residual)."""
        y = ssm.gatednorm_fwd(y.flatten(-2), z, p["gate_norm"], group=self.headdim)
        return ssm.blocknorm_fwd(y @ p["out"].T, p["post_norm"], residual, p["next_norm"], alpha=self.alpha,
                                 residual_out=residual)

    def prefill(self, tokens, lens, cache, slots):
        """tokens [b, L], the first lens[i] of each row; fills the slots and returns the last tokens' logits."""
        residual = self.embedding[tokens].float()
        x, _ = ssm.rmsnorm_fwd(self.embedding[tokens], self.norm)
        at = slots.long()
        for p, (conv_cache, delta_cache) in zip(self.layers, cache):
            rows = x @ p["in"].T
            u, conv_state = ssm.conv_fwd(rows[..., : self.d_conv], p["conv"], lens=lens)
            args, z = self._split(u, rows)
            y, h = ssm.delta_fwd(*args, p["A"], p["dt_bias"], lens=lens)
            conv_cache[at], delta_cache[at] = conv_state, h
            x, residual = self._out(p, y, z, residual)
        last = (lens.long() - 1)[:, None, None].expand(-1, 1, x.shape[-1])
        return (x.gather(1, last)[:, 0] @ self.head.T).float()

    def decode(self, tokens, cache, slots):
        """One token [b] of each sequence; updates its slot and returns the logits."""
        residual = self.embedding[tokens].float()
        x, _ = ssm.rmsnorm_fwd(self.embedding[tokens], self.norm)
        for p, (conv_cache, delta_cache) in zip(self.layers, cache):
            rows = x @ p["in"].T
            u, _ = ssm.conv_step(rows[:, : self.d_conv], p["conv"], None, conv_cache, slots, inplace=True)
            args, z = self._split(u, rows)
            y, _ = ssm.delta_step(*args, p["A"], p["dt_bias"], delta_cache, slots, inplace=True)
            x, residual = self._out(p, y, z, residual)
        return (x @ self.head.T).float()


def run(dtype=torch.bfloat16, layers=3, new_tokens=16, lens=(97, 5, 140, 1), seed=0):
    """Generates greedily; returns the tokens and the distance of its logits from a prefill of everything."""
    model = DeltaNet(layers=layers, dtype=dtype, seed=seed)
    b, L = len(lens), max(lens)
    g = torch.Generator("cuda").manual_seed(seed + 1)
    prompts = torch.randint(0, model.embedding.shape[0], (b, L), device="cuda", generator=g)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    slots = torch.randperm(2 * b, device="cuda", generator=g)[:b].to(torch.int32)
    cache = model.new_cache(2 * b)
    logits = model.prefill(prompts, n, cache, slots)
    generated = []
    for _ in range(new_tokens):
        generated.append(logits.argmax(-1))
        logits = model.decode(generated[-1], cache, slots)
    generated = torch.stack(generated, 1)

    whole = torch.zeros(b, L + new_tokens, dtype=torch.long, device="cuda")
    for i, m in enumerate(lens):
        whole[i, : m + new_tokens] = torch.cat([prompts[i, :m], generated[i]])
    again = model.prefill(whole, n + new_tokens, model.new_cache(2 * b), slots)
    return generated, float((logits - again).norm() / again.norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    ap.add_argument("--layers", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=16)
    args = ap.parse_args()
    out, distance = run(torch.bfloat16 if args.dtype == "bf16" else torch.float32, args.layers, args.tokens)
    for row in out.tolist():
        print(*row)
    print(f"relative distance of the last logits from one prefill: {distance:.2e}")
