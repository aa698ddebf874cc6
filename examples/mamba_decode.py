"""A small Mamba-1 language model of random weights on this package's operators: prompts of unequal
lengths in one padded batch, then tokens one by one, with the carried states in slots of a cache.

    python examples/mamba_decode.py [--dtype bf16|f32] [--fp8] [--group 0|128] [--layers N] [--tokens N]

Each layer is  residual += out_proj(selscan(conv(in_proj(norm(residual)))), gated by z):
rmsnorm_fwd adds the last layer's output to the residual and normalises, conv_fwd and selscan_fwd
read their inputs as columns of the projections' rows, and conv_step and selscan_step update the
cache in place.  With --fp8 the norm's output goes through rmsnorm_fp8_fwd's codes and scales (one a row, or with
--group 128 one for each 128 columns).

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


class Mamba:
    def __init__(self, layers=4, d_model=512, d_inner=1024, d_state=16, width=4, vocab=1000, dtype=torch.bfloat16,
                 fp8=False, seed=0, group=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def linear(n_out, n_in):
            return (torch.randn(n_out, n_in, device="cuda", generator=g) / math.sqrt(n_in)).to(dtype)

        def uniform(*shape):
            return torch.rand(shape, device="cuda", generator=g)

        self.dtype, self.fp8, self.group = dtype, fp8, group
        self.d_inner, self.d_state, self.width, self.rank = d_inner, d_state, width, d_model // 16
        self.embedding = (0.02 * torch.randn(vocab, d_model, device="cuda", generator=g)).to(dtype)
        self.head = linear(vocab, d_model)
        self.norm = torch.ones(d_model, device="cuda")
        self.layers = []
        for _ in range(layers):
            step = torch.exp(uniform(d_inner) * math.log(100.0)) * 1e-3  # between 0.001 and 0.1
            self.layers.append({
                "norm": torch.ones(d_model, device="cuda"), "in": linear(2 * d_inner, d_model),
                "conv": (2 * uniform(d_inner, width) - 1) / math.sqrt(width), "conv_bias": 0.1 * uniform(d_inner),
                "x": linear(self.rank + 2 * d_state, d_inner), "dt": linear(d_inner, self.rank),
                "dt_bias": step + torch.log(-torch.expm1(-step)),
                "A": -torch.arange(1, d_state + 1, device="cuda", dtype=torch.float32).repeat(d_inner, 1),
                "D": torch.ones(d_inner, device="cuda"), "out": linear(d_model, d_inner)})

    def new_cache(self, slots):
        """The carried states of `slots` sequences, a pair of each layer."""
        return [(torch.zeros(slots, self.width - 1, self.d_inner, device="cuda", dtype=self.dtype),
                 torch.zeros(slots, self.d_inner, self.d_state, device="cuda")) for _ in self.layers]

    def _norm(self, x, weight, residual):
        """The norm of x + residual, and that sum (f32, in place of the old one)."""
        if residual is None:  # the first layer: x is the residual
            residual, x = x.float(), torch.zeros_like(x)
        if not self.fp8:
            return ssm.rmsnorm_fwd(x, weight, residual, residual_out=residual)
        q, scale, residual = ssm.rmsnorm_fp8_fwd(x, weight, residual, group=self.group, residual_out=residual)
        scale = scale.repeat_interleave(128, -1)[..., : x.shape[-1]] if self.group else scale[..., None]
        return (q.float() * scale).to(self.dtype), residual

    def _steps(self, p, u):
        """dt, B and C of the convolved tokens."""
        r, n = self.rank, self.d_state
        rows = u @ p["x"].T
        return rows[..., :r] @ p["dt"].T, rows[..., r : r + n].unflatten(-1, (1, n)), rows[..., r + n :].unflatten(-1, (1, n))

    def prefill(self, tokens, lens, cache, slots):
        """tokens [b, L], the first lens[i] of each row; fills the slots and returns the last tokens' logits."""
        x, residual = self.embedding[tokens], None
        at = slots.long()
        for p, (conv_cache, scan_cache) in zip(self.layers, cache):
            x, residual = self._norm(x, p["norm"], residual)
            rows = x @ p["in"].T
            u, conv_state = ssm.conv_fwd(rows[..., : self.d_inner], p["conv"], p["conv_bias"], lens=lens)
            dt, B, C = self._steps(p, u)
            y, h = ssm.selscan_fwd(u, dt, p["A"], B, C, p["D"], rows[..., self.d_inner :], p["dt_bias"], lens=lens)
            conv_cache[at], scan_cache[at] = conv_state, h
            x = y @ p["out"].T
        last = (lens.long() - 1)[:, None, None].expand(-1, 1, x.shape[-1])
        x, _ = self._norm(x.gather(1, last)[:, 0], self.norm, residual.gather(1, last)[:, 0].contiguous())
        return (x @ self.head.T).float()

    def decode(self, tokens, cache, slots):
        """One token [b] of each sequence; updates its slot and returns the logits."""
        x, residual = self.embedding[tokens], None
        for p, (conv_cache, scan_cache) in zip(self.layers, cache):
            x, residual = self._norm(x, p["norm"], residual)
            rows = x @ p["in"].T
            u, _ = ssm.conv_step(rows[:, : self.d_inner], p["conv"], p["conv_bias"], conv_cache, slots, inplace=True)
            dt, B, C = self._steps(p, u)
            y, _ = ssm.selscan_step(u, dt, p["A"], B, C, p["D"], rows[:, self.d_inner :], p["dt_bias"], scan_cache, slots,
                                    inplace=True)
            x = y @ p["out"].T
        x, _ = self._norm(x, self.norm, residual)
        return (x @ self.head.T).float()


def run(dtype=torch.bfloat16, fp8=False, layers=4, new_tokens=16, lens=(37, 5, 64, 1), seed=0, group=0):
    """Generates greedily; returns the tokens and the distance of its logits from a prefill of everything."""
    model = Mamba(layers=layers, dtype=dtype, fp8=fp8, seed=seed, group=group)
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
    ap.add_argument("--fp8", action="store_true")
    ap.add_argument("--group", type=int, choices=(0, 128), default=0)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=16)
    args = ap.parse_args()
    out, distance = run(torch.bfloat16 if args.dtype == "bf16" else torch.float32, args.fp8, args.layers, args.tokens,
                        group=args.group)
    for row in out.tolist():
        print(*row)
    print(f"relative distance of the last logits from one prefill: {distance:.2e}")
