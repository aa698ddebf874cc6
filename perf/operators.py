"""Cases of the operators that stand around a state-space layer's scan, with their plain forms.

Five operators: the short causal convolution for prompts (conv) and single tokens (conv_step), the
selective scan with a decay per channel and state entry for prompts (selscan) and single tokens
(selscan_step), and the root-mean-square norm with the residual's addition (norm), with an output
in 8 bits or in the model's type.

Where `own` is false, run() computes them in elementary torch operations in 32 bits, rounded once
at the end; where it is true, by the calls a user makes of this package.  Widths follow the
package's own workloads: 80, 32 and 24 heads of 64 give 5120, 2048 and 1536 inner channels, and
the convolution also covers B and C of 128 states (5376 and 1792 channels).
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt of one user through the 24-head model's convolution: latency
        {"name": "conv_b1_L17_d1792", "op": "conv", "b": 1, "L": 17, "d": 1792, "W": 4, "dtype": "bf16", "state": False,
         "lens": False, "wide": 0},
        # right-padded prompts of unequal lengths, odd sizes, continued from a state, in f32
        {"name": "conv_b3_L1021_d1001_lens_f32", "op": "conv", "b": 3, "L": 1021, "d": 1001, "W": 3, "dtype": "f32",
         "state": True, "lens": True, "wide": 0},
        # the 80-head model's convolution over long prompts, read from the wide rows of the input projection
        {"name": "conv_b4_L8192_d5376", "op": "conv", "b": 4, "L": 8192, "d": 5376, "W": 4, "dtype": "bf16",
         "state": False, "lens": False, "wide": 5200},
        # one user's next token: latency
        {"name": "conv_step_b1_d1792", "op": "conv_step", "b": 1, "d": 1792, "W": 4, "dtype": "bf16", "slots": 1,
         "wide": 0},
        # continuous batching: 128 sequences whose states lie anywhere in a cache of 192 slots
        {"name": "conv_step_b128_d5376", "op": "conv_step", "b": 128, "d": 5376, "W": 4, "dtype": "bf16",
         "slots": 192, "wide": 5200},
        # a short prompt of one user: latency, too few chains to fill the GPU
        {"name": "selscan_b1_L64_d1536", "op": "selscan", "b": 1, "L": 64, "d": 1536, "N": 16, "G": 1, "dtype": "bf16",
         "h0": False, "lens": False, "z": True},
        # one long document of odd length, few channels, f32: the time axis has to give the parallelism
        {"name": "selscan_b1_L65521_d1536_f32", "op": "selscan", "b": 1, "L": 65521, "d": 1536, "N": 16, "G": 1,
         "dtype": "f32", "h0": True, "lens": False, "z": True},
        # prompts of unequal lengths of the 80-head model's width: the largest
        {"name": "selscan_b4_L8192_d5120_lens", "op": "selscan", "b": 4, "L": 8192, "d": 5120, "N": 16, "G": 1,
         "dtype": "bf16", "h0": False, "lens": True, "z": True},
        # one user's next token: latency
        {"name": "selscan_step_b1_d1536", "op": "selscan_step", "b": 1, "d": 1536, "N": 16, "G": 1, "dtype": "bf16",
         "slots": 1, "z": True},
        # continuous batching: 256 sequences whose states lie anywhere in a cache of 300 slots
        {"name": "selscan_step_b256_d5120", "op": "selscan_step", "b": 256, "d": 5120, "N": 16, "G": 1,
         "dtype": "bf16", "slots": 300, "z": True},
        # the norm in front of a decode step's projection in 8 bits: latency
        {"name": "norm_fp8_1x2560", "op": "norm", "rows": 1, "d": 2560, "dtype": "bf16", "res": "f32", "fp8": True,
         "group": 0},
        # the same over four prompts of 8192 tokens, a scale for each 128 columns
        {"name": "norm_fp8_32768x2560", "op": "norm", "rows": 32768, "d": 2560, "dtype": "bf16", "res": "bf16",
         "fp8": True, "group": 128},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high], odd ones among them."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "selscan", "selscan_step", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "norm":
        d = _spread(rng, 256, 8192)
        d = d if rng.random() < 0.3 else max(256, d // 128 * 128)
        rows = _spread(rng, 1, max(1, min(32768, 32768 * 2560 // d)))
        fp8 = flag()
        return {"op": op, "rows": rows, "d": d, "dtype": dtype, "res": rng.choice(["", "f32", dtype]), "fp8": fp8,
                "group": 128 if fp8 and flag() else 0}
    d = _spread(rng, 768, 5376)
    d = d if rng.random() < 0.3 else max(768, d // 64 * 64)
    if op == "conv":
        b = rng.randint(1, 8)
        L = _spread(rng, 1, max(1, min(65536, 4 * 8192 * 5376 // (b * d * SIZE[dtype] // 2))))
        return {"op": op, "b": b, "L": L, "d": d, "W": rng.randint(2, 4), "dtype": dtype, "state": flag(),
                "lens": flag(), "wide": rng.choice([0, 256])}
    if op == "conv_step":
        b = _spread(rng, 1, 256)
        return {"op": op, "b": b, "d": d, "W": rng.randint(2, 4), "dtype": dtype, "slots": b + rng.randint(0, 64),
                "wide": rng.choice([0, 256])}
    N = rng.choice([8, 16, 16, 32])
    G = rng.choice([1, 1, 2]) if d % 2 == 0 else 1
    if op == "selscan":
        b = rng.randint(1, 8)
        L = _spread(rng, 1, max(1, min(65536, 4 * 8192 * 5120 * 16 // (b * d * N * SIZE[dtype] // 2))))
        return {"op": op, "b": b, "L": L, "d": d, "N": N, "G": G, "dtype": dtype, "h0": flag(), "lens": flag(),
                "z": flag()}
    b = _spread(rng, 1, 256)
    return {"op": op, "b": b, "d": d, "N": N, "G": G, "dtype": dtype, "slots": b + rng.randint(0, 64), "z": flag()}


# ---------------------------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Inputs of one case, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DT[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    def slots():
        return torch.randperm(case["slots"], generator=g, device="cuda")[: case["b"]].to(torch.int32)

    def lens(b, L):  # the longest fills the padded length, the others end anywhere
        n = (rand(b) * (L + 1)).to(torch.int32).clamp(max=L)
        n[0] = L
        return n

    if op == "norm":
        rows, d = case["rows"], case["d"]
        res = randn(rows, d, dtype=DT[case["res"]]) * 4 if case["res"] else None
        return {"x": randn(rows, d, dtype=dtype), "weight": 1 + 0.2 * randn(d), "residual": res, "eps": 1e-5}
    d = case["d"]
    if op in ("conv", "conv_step"):
        W, bound = case["W"], 1 / math.sqrt(case["W"])
        s = {"weight": (2 * rand(d, W) - 1) * bound, "bias": (2 * rand(d) - 1) * bound}
        if op == "conv":  # columns of the projection's rows
            s["x"] = randn(case["b"], case["L"], d + case["wide"], dtype=dtype)[..., :d]
            s["state"] = randn(case["b"], W - 1, d, dtype=dtype) if case["state"] else None
            s["lens"] = lens(case["b"], case["L"]) if case["lens"] else None
        else:
            s["x"] = randn(case["b"], d + case["wide"], dtype=dtype)[..., :d]
            s["state"] = randn(case["slots"], W - 1, d, dtype=dtype)
            s["slots"] = slots()
            s["state_out"] = s["state"].clone()
        return s
    N, G = case["N"], case["G"]
    lead = (case["b"], case["L"]) if op == "selscan" else (case["b"],)
    rank = -(-d // 32) // 8 * 8 + 8  # the rank of the step's projection, beside which B and C lie
    low = torch.exp(rand(d) * math.log(100.0)) * 1e-3  # steps between 0.001 and 0.1 at a zero input
    xproj = randn(*lead, rank + 2 * G * N, dtype=dtype)
    s = {"u": torch.nn.functional.silu(randn(*lead, d)).to(dtype), "dt": (0.5 * randn(*lead, d)).to(dtype),
         "A": -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.2 * randn(d, N)),
         "B": xproj[..., rank : rank + G * N].unflatten(-1, (G, N)),
         "C": xproj[..., rank + G * N :].unflatten(-1, (G, N)),
         "D": 1 + 0.1 * randn(d), "dt_bias": low + torch.log(-torch.expm1(-low)),
         "z": randn(*lead, 2 * d, dtype=dtype)[..., d:] if case["z"] else None}
    if op == "selscan":
        s["h0"] = 0.3 * randn(case["b"], d, N) if case["h0"] else None
        s["lens"] = lens(case["b"], case["L"]) if case["lens"] else None
    else:
        s["state"] = 0.3 * randn(case["slots"], d, N)
        s["slots"] = slots()
        s["state_out"] = s["state"].clone()
    return s


def prepare(case, seed):
    return {"case": case, **_inputs(case, seed)}


# ---------------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import selective_state_space_mamba_gb300 as ssm
    case = s["case"]
    op = case["op"]
    if op == "conv":
        y, state = ssm.conv_fwd(s["x"], s["weight"], s["bias"], s["state"], s["lens"])
        return {"y": y, "state": state}
    if op == "conv_step":
        y, state = ssm.conv_step(s["x"], s["weight"], s["bias"], s["state"], s["slots"], state_out=s["state_out"])
        return {"y": y, "state": state}
    if op == "selscan":
        y, h = ssm.selscan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["h0"], s["lens"])
        return {"y": y, "h": h}
    if op == "selscan_step":
        y, h = ssm.selscan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], s["state"],
                                s["slots"], state_out=s["state_out"])
        return {"y": y, "h": h}
    if case["fp8"]:
        q, scale, res = ssm.rmsnorm_fp8_fwd(s["x"], s["weight"], s["residual"], eps=s["eps"], group=case["group"])
        return {"q": q, "scale": scale, "residual": res}
    y, res = ssm.rmsnorm_fwd(s["x"], s["weight"], s["residual"], eps=s["eps"])
    return {"y": y, "residual": res}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _run_plain(s):
    op = s["case"]["op"]
    if op == "conv":
        return _plain_conv(s["x"], s["weight"], s["bias"], s["state"], s["lens"])
    if op == "conv_step":
        at = s["slots"].long()
        r = _plain_conv(s["x"][:, None], s["weight"], s["bias"], s["state"][at], None)
        s["state_out"][at] = r["state"]
        return {"y": r["y"][:, 0], "state": s["state_out"]}
    if op == "selscan":
        return _plain_selscan(s)
    if op == "selscan_step":
        return _plain_selscan_step(s)
    return _plain_norm(s)


def _plain_conv(x, weight, bias, state, lens):
    b, L, d = x.shape
    W = weight.shape[1]
    if state is None:
        state = x.new_zeros(b, W - 1, d)
    rows = torch.cat([state, x], 1)  # the carried tokens, then the new ones
    wide = rows.float()
    y = _silu(sum(wide[:, k : k + L] * weight[:, k] for k in range(W)) + bias)
    if lens is None:
        return {"y": y.to(x.dtype), "state": rows[:, L:].contiguous()}
    y = y * (torch.arange(L, device=x.device)[None, :] < lens[:, None])[..., None]
    at = lens[:, None].long() + torch.arange(W - 1, device=x.device)
    return {"y": y.to(x.dtype), "state": torch.gather(rows, 1, at[..., None].expand(-1, -1, d))}


def _per_channel(v, d):
    """[..., G, N] -> [..., d or 1, N]: each channel's group."""
    return v if v.shape[-2] == 1 else v.repeat_interleave(d // v.shape[-2], -2)


def _plain_selscan(s):
    u, dt = s["u"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    b, L, d = u.shape
    live = None
    if s["lens"] is not None:  # a padded token leaves the state as it is
        live = (torch.arange(L, device=u.device)[None, :] < s["lens"][:, None])[..., None]
        dt = dt * live
    a = torch.exp(dt[..., None] * s["A"])
    h = (dt * u)[..., None] * _per_channel(s["B"].float(), d)
    if s["h0"] is not None:
        h[:, 0] += a[:, 0] * s["h0"]
    step = 1
    while step < L:  # h[t] covers twice as many tokens after each pass
        h[:, step:] += a[:, step:] * h[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    del a
    last = h[:, -1].clone()
    y = h.mul_(_per_channel(s["C"].float(), d)).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    if live is not None:
        y = y * live
    return {"y": y.to(s["u"].dtype), "h": last}


def _plain_selscan_step(s):
    u, dt = s["u"].float(), _softplus(s["dt"].float() + s["dt_bias"])
    d, at = u.shape[-1], s["slots"].long()
    h = torch.exp(dt[..., None] * s["A"]) * s["state"][at] + (dt * u)[..., None] * _per_channel(s["B"].float(), d)
    y = (h * _per_channel(s["C"].float(), d)).sum(-1) + s["D"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state_out"][at] = h
    return {"y": y.to(s["u"].dtype), "h": s["state_out"]}


def _plain_norm(s):
    case, r = s["case"], s["x"].float()
    res = None
    if s["residual"] is not None:
        r = r + s["residual"].float()
        res = r.to(s["residual"].dtype)
    v = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + s["eps"]) * s["weight"]
    if not case["fp8"]:
        return {"y": v.to(s["x"].dtype), "residual": res}
    rows, d = v.shape
    group = case["group"] or d
    n = -(-d // group)
    blocks = torch.nn.functional.pad(v, (0, n * group - d)).view(rows, n, group)
    scale = torch.clamp(blocks.abs().amax(-1) / 448, min=2.0**-126)
    q = torch.clamp(blocks / scale[..., None], -448, 448).to(torch.float8_e4m3fn).view(rows, n * group)[:, :d]
    return {"q": q.contiguous(), "scale": scale if case["group"] else scale[:, 0], "residual": res}


# ---------------------------------------------------------------------------------- the work of a pass

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "norm":
        n = case["rows"] * case["d"]
        res = 2 * SIZE[case["res"]] if case["res"] else 0
        groups = -(-case["d"] // case["group"]) if case["group"] else 1
        out = n + 4 * case["rows"] * groups if case["fp8"] else n * e
        return {"bytes": n * (e + res) + out + 4 * case["d"], "flops": 6 * n}
    b, d = case["b"], case["d"]
    if op in ("conv", "conv_step"):
        W = case["W"]
        tokens = b * case.get("L", 1)
        states = 2 if op == "conv_step" or case["state"] else 1
        return {"bytes": 2 * tokens * d * e + states * b * (W - 1) * d * e + 4 * d * (W + 1),
                "flops": tokens * d * (2 * W + 5)}
    N, G = case["N"], case["G"]
    tokens = b * case.get("L", 1)
    states = 2 if op == "selscan_step" or case["h0"] else 1
    return {"bytes": tokens * d * e * (4 if case["z"] else 3) + 2 * tokens * G * N * e + 4 * states * b * d * N
            + 4 * d * (N + 2), "flops": tokens * d * (7 * N + 15)}


# ---------------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "norm":
        return _exact_norm(case, s)
    if op in ("conv", "conv_step"):
        return _exact_conv(case, s)
    return _exact_selscan(case, s)


def _exact_conv(case, s):
    """Token by token: a window of the last W tokens moves along each sequence."""
    x = s["x"] if case["op"] == "conv" else s["x"][:, None]
    b, L, d = x.shape
    W = case["W"]
    if case["op"] == "conv_step":
        window = s["state"][s["slots"].long()]
    else:
        window = s["state"] if s["state"] is not None else x.new_zeros(b, W - 1, d)
    lens = [L] * b if s.get("lens") is None else s["lens"].tolist()
    y = torch.zeros(b, L, d, dtype=torch.float64, device=x.device)
    taps = s["weight"].T  # [W, d]
    state = []
    for i, n in enumerate(lens):
        rows = torch.cat([window[i], x[i, :n]])
        v = torch.nn.functional.conv1d(rows.T[None], taps.T[:, None].contiguous(), s["bias"], groups=d)[0].T if n else rows[:0]
        y[i, :n] = v * torch.sigmoid(v)
        state.append(rows[n : n + W - 1])
    state = torch.stack(state)
    if case["op"] == "conv":
        return {"y": y, "state": state}
    out = s["state"].clone()
    out[s["slots"].long()] = state
    return {"y": y[:, 0], "state": out}


def _exact_selscan(case, s):
    """The recurrence, one token after the other."""
    single = case["op"] == "selscan_step"
    u, dt, B, C = (s[k][:, None] if single else s[k] for k in ("u", "dt", "B", "C"))
    z = None if s["z"] is None else s["z"][:, None] if single else s["z"]
    b, L, d = u.shape
    N, G = case["N"], case["G"]
    delta = torch.logaddexp(dt + s["dt_bias"], torch.zeros((), dtype=torch.float64, device=u.device))
    if single:
        h = s["state"][s["slots"].long()]
    else:
        h = s["h0"] if s["h0"] is not None else u.new_zeros(b, d, N)
    h = h.reshape(b, G, d // G, N).clone()
    A = s["A"].view(G, d // G, N)
    lens = s.get("lens")
    y = torch.zeros(b, L, d, dtype=torch.float64, device=u.device)
    for t in range(L):
        step = delta[:, t].view(b, G, d // G, 1)
        new = torch.exp(step * A) * h + step * u[:, t].view(b, G, d // G, 1) * B[:, t, :, None, :]
        out = torch.einsum("bgcn,bgn->bgc", new, C[:, t]).reshape(b, d)
        if lens is None:
            h, y[:, t] = new, out
        else:
            on = (lens > t).view(b, 1)
            h = torch.where(on[..., None, None], new, h)
            y[:, t] = torch.where(on, out + s["D"] * u[:, t], 0.0)
    if lens is None:
        y += s["D"] * u
    if z is not None:
        y *= z * torch.sigmoid(z)
    h = h.reshape(b, d, N)
    if not single:
        return {"y": y, "h": h}
    state = s["state"].clone()
    state[s["slots"].long()] = h
    return {"y": y[:, 0], "h": state}


def _exact_norm(case, s):
    r = s["x"] if s["residual"] is None else s["x"] + s["residual"]
    res = None if s["residual"] is None else r
    v = s["weight"] * r / torch.sqrt(torch.linalg.vector_norm(r, dim=-1, keepdim=True) ** 2 / case["d"] + s["eps"])
    if not case["fp8"]:
        return {"y": v, "residual": res}
    if not case["group"]:
        scale = torch.linalg.vector_norm(v, ord=float("inf"), dim=-1) / 448
        return {"q": v / scale[:, None], "scale": scale, "residual": res}
    parts = v.split(case["group"], -1)
    scale = torch.stack([torch.linalg.vector_norm(p, ord=float("inf"), dim=-1) / 448 for p in parts], -1)
    return {"q": torch.cat([p / scale[:, i, None] for i, p in enumerate(parts)], -1), "scale": scale, "residual": res}
