"""Cases of the gated delta rule and of the norms around it, with their plain forms.

Four operators: the gated delta rule for prompts (delta) and single tokens (delta_step), the norm of
its output with the gate (gatednorm), and the norms after one block and before the next with the
residual between them (blocknorm).

    delta      S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   y_t = scale S_t q_t,
               a state of headdim x dstate a head; a_t = exp(A softplus(dt_t + dt_bias)),
               beta_t = sigmoid of its input, q and k divided by their length
    gatednorm  y = rms(x) w silu(z), or rms(x silu(z)) w, over groups of columns
    blocknorm  r = alpha residual + rms(x) w silu(z),   y = rms(r) w2

Where `own` is false, run() computes them in elementary torch operations in 32 bits (sums of
logarithms of decays in 64), rounded once at the end; where it is true, by the calls a user makes of
this package.  Head counts and sizes follow the package's own workloads (24 and 32 heads of 64, states
of 128, 8 groups, rows of 2560) and the usual square state of 128 x 128.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short prompt of one user: latency, less than one chunk of tokens
        {"name": "delta_b1_L19_nh24", "op": "delta", "b": 1, "L": 19, "nh": 24, "G": 24, "H": 64, "S": 128,
         "dtype": "bf16", "h0": False, "lens": False, "wide": 0},
        # right-padded prompts of unequal lengths, odd sizes, continued from a state, in f32
        {"name": "delta_b3_L517_nh6_f32", "op": "delta", "b": 3, "L": 517, "nh": 6, "G": 3, "H": 96, "S": 64,
         "dtype": "f32", "h0": True, "lens": True, "wide": 3},
        # prompts of unequal lengths, read from the wide rows of a projection and continued from states
        {"name": "delta_b8_L2048_nh24_lens", "op": "delta", "b": 8, "L": 2048, "nh": 24, "G": 24, "H": 64, "S": 128,
         "dtype": "bf16", "h0": True, "lens": True, "wide": 64},
        # one long document of odd length: few chains of many chunks
        {"name": "delta_b1_L65521_nh32_G8", "op": "delta", "b": 1, "L": 65521, "nh": 32, "G": 8, "H": 64, "S": 128,
         "dtype": "bf16", "h0": False, "lens": False, "wide": 0},
        # four long prompts, square states: the largest
        {"name": "delta_b4_L8192_nh32_H128", "op": "delta", "b": 4, "L": 8192, "nh": 32, "G": 16, "H": 128, "S": 128,
         "dtype": "bf16", "h0": False, "lens": False, "wide": 0},
        # one user's next token: latency
        {"name": "delta_step_b1_nh24", "op": "delta_step", "b": 1, "nh": 24, "G": 24, "H": 64, "S": 128,
         "dtype": "bf16", "slots": 1},
        # continuous batching: 128 sequences whose states lie anywhere in a cache of 160 slots
        {"name": "delta_step_b128_nh32_H128", "op": "delta_step", "b": 128, "nh": 32, "G": 16, "H": 128, "S": 128,
         "dtype": "bf16", "slots": 160},
        # the norm behind one token's step, a weight shared by the heads: latency
        {"name": "gatednorm_1x1536", "op": "gatednorm", "rows": 1, "d": 1536, "group": 64, "shared": True,
         "first": False, "dtype": "bf16", "wide": 1536},
        # the same over four prompts of 8192 tokens, heads of 128, the gate read from wider rows
        {"name": "gatednorm_32768x4096", "op": "gatednorm", "rows": 32768, "d": 4096, "group": 128, "shared": True,
         "first": False, "dtype": "bf16", "wide": 4096},
        # the gate before a norm of the whole row, as behind the package's SSD forward, an odd number of rows
        {"name": "gatednorm_8191x5120_first", "op": "gatednorm", "rows": 8191, "d": 5120, "group": 0, "shared": False,
         "first": True, "dtype": "bf16", "wide": 0},
        # between two blocks of one token's pass: latency
        {"name": "blocknorm_1x2560", "op": "blocknorm", "rows": 1, "d": 2560, "dtype": "bf16", "res": "f32",
         "gate": False},
        # between two blocks of four prompts of 8192 tokens, with a gate
        {"name": "blocknorm_32768x2560_gate", "op": "blocknorm", "rows": 32768, "d": 2560, "dtype": "bf16",
         "res": "bf16", "gate": True},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high], odd ones among them."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta_step", "gatednorm", "blocknorm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("gatednorm", "blocknorm"):
        d = _spread(rng, 256, 8192)
        d = d if rng.random() < 0.2 else max(256, d // 128 * 128)
        rows = _spread(rng, 1, max(1, min(32768, 32768 * 2560 // d)))
        if op == "blocknorm":
            return {"op": op, "rows": rows, "d": d, "dtype": dtype, "res": rng.choice(["f32", dtype]), "gate": flag()}
        group = rng.choice([0, 64, 128]) if d % 128 == 0 else 0
        return {"op": op, "rows": rows, "d": d, "group": group, "shared": flag(), "first": flag(), "dtype": dtype,
                "wide": rng.choice([0, 256])}
    G = rng.choice([1, 2, 4, 8, 16])
    nh = G * rng.choice([1, 2, 4])
    nh = nh if nh <= 32 else G
    S, H = rng.choice([64, 128, 128]), rng.choice([64, 96, 128, 128])
    if op == "delta_step":
        b = _spread(rng, 1, max(1, min(256, 128 * 32 * 16384 * 2 // (nh * H * S * 2))))
        return {"op": op, "b": b, "nh": nh, "G": G, "H": H, "S": S, "dtype": dtype, "slots": b + rng.randint(0, 32)}
    b = rng.randint(1, 8)
    most = 4 * 8192 * 32 * 128 * 128 // (b * nh * H * S * (1 if dtype == "bf16" else 8))
    L = _spread(rng, 1, max(1, min(65521, most)))
    return {"op": op, "b": b, "L": L, "nh": nh, "G": G, "H": H, "S": S, "dtype": dtype, "h0": flag(), "lens": flag(),
            "wide": rng.choice([0, 0, 64])}


# ---------------------------------------------------------------------------------- inputs

def _inputs(case, seed):
    """Inputs of one case, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype = case["op"], DT[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    if op == "gatednorm":  # the gate is a part of the projection's wider rows
        rows, d = case["rows"], case["d"]
        group = case["group"] or d
        return {"x": randn(rows, d, dtype=dtype), "z": randn(rows, d + case["wide"], dtype=dtype)[:, case["wide"]:],
                "weight": 1 + 0.2 * randn(group if case["shared"] else d), "eps": 1e-5}
    if op == "blocknorm":
        rows, d = case["rows"], case["d"]
        return {"x": randn(rows, d, dtype=dtype), "weight": 1 + 0.2 * randn(d),
                "residual": randn(rows, d, dtype=DT[case["res"]]) * 4, "next_weight": 1 + 0.2 * randn(d),
                "z": randn(rows, d, dtype=dtype) if case["gate"] else None, "alpha": 0.75, "eps": 1e-5}
    b, nh, G, H, S = (case[k] for k in ("b", "nh", "G", "H", "S"))
    lead = (b, case["L"]) if op == "delta" else (b,)
    # what the short convolution and its SiLU hand on: q, k and v side by side
    conv = torch.nn.functional.silu(randn(*lead, 2 * G * S + nh * H + case.get("wide", 0))).to(dtype)
    low = torch.exp(rand(nh) * math.log(100.0)) * 1e-3  # steps between 0.001 and 0.1 at a zero input
    s = {"q": conv[..., : G * S].unflatten(-1, (G, S)), "k": conv[..., G * S : 2 * G * S].unflatten(-1, (G, S)),
         "v": conv[..., 2 * G * S : 2 * G * S + nh * H].unflatten(-1, (nh, H)),
         "dt": randn(*lead, nh, dtype=dtype), "beta": randn(*lead, nh, dtype=dtype),
         "A": -torch.exp(rand(nh) * math.log(16.0)), "dt_bias": low + torch.log(-torch.expm1(-low))}
    if op == "delta":
        s["h0"] = 0.3 * randn(b, nh, H, S) if case["h0"] else None
        s["lens"] = None
        if case["lens"]:  # the longest fills the padded length, the others end anywhere
            s["lens"] = (rand(b) * (case["L"] + 1)).to(torch.int32).clamp(max=case["L"])
            s["lens"][0] = case["L"]
    else:
        s["state"] = 0.3 * randn(case["slots"], nh, H, S)
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:b].to(torch.int32)
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
    if op == "delta":
        y, h = ssm.delta_fwd(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["dt_bias"], s["h0"], s["lens"])
        return {"y": y, "h": h}
    if op == "delta_step":
        y, h = ssm.delta_step(s["q"], s["k"], s["v"], s["dt"], s["beta"], s["A"], s["dt_bias"], s["state"], s["slots"],
                              state_out=s["state_out"])
        return {"y": y, "h": h}
    if op == "gatednorm":
        return {"y": ssm.gatednorm_fwd(s["x"], s["z"], s["weight"], group=case["group"], gate_first=case["first"],
                                       eps=s["eps"])}
    y, res = ssm.blocknorm_fwd(s["x"], s["weight"], s["residual"], s["next_weight"], s["z"], alpha=s["alpha"],
                               eps=s["eps"])
    return {"y": y, "residual": res}


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _run_plain(s):
    op = s["case"]["op"]
    if op == "delta":
        return _plain_delta(s)
    if op == "delta_step":
        return _plain_delta_step(s)
    if op == "gatednorm":
        return _plain_gatednorm(s)
    return _plain_blocknorm(s)


def _unit(v):
    v = v.float()
    return v * torch.rsqrt((v * v).sum(-1, keepdim=True) + 1e-6)


CHUNK = 64


def _plain_delta(s):
    """In chunks of 64 tokens.  Inside a chunk the tokens' corrections d solve (I + N) d = beta (v - decayed S k), with
    the strictly lower N_ij = beta_i decay_ij k_i.k_j: its inverse by blocks of twice the size in each step."""
    v = s["v"].float()
    b, L, nh, H = v.shape
    S, G = s["q"].shape[-1], s["q"].shape[-2]
    n = -(-L // CHUNK)

    def chunks(x):  # [b, L, nh, ...] -> [b, nh, n, 64, ...]
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * CHUNK - L))
        return x.unflatten(1, (n, CHUNK)).movedim(3, 1)

    def heads(x):
        return chunks(x.repeat_interleave(nh // G, 2))

    q, k = heads(_unit(s["q"]) * S ** -0.5), heads(_unit(s["k"]))
    g = _softplus(s["dt"].float() + s["dt_bias"]) * s["A"]
    beta = 1 / (1 + torch.exp(-s["beta"].float()))
    live = None
    if s["lens"] is not None:  # a padded token leaves the state as it is
        live = torch.arange(L, device=v.device)[None, :, None] < s["lens"][:, None, None]
        g, beta = g * live, beta * live
    g, beta, v = chunks(g[..., None])[..., 0], chunks(beta[..., None]), chunks(v)
    sums = torch.cumsum(g.double(), -1)
    at = torch.arange(CHUNK, device=v.device)
    decay = torch.exp((sums[..., :, None] - sums[..., None, :]).clamp(max=0)).float() * (at[:, None] >= at)
    from_start, to_end = torch.exp(sums).float()[..., None], torch.exp(sums[..., -1:] - sums).float()[..., None]
    N = beta * decay * (k @ k.mT) * (at[:, None] > at)
    P = decay * (q @ k.mT)
    del decay
    inv = torch.eye(CHUNK, device=v.device).expand(b, nh, n, CHUNK, CHUNK)
    for size in (1, 2, 4, 8, 16, 32):
        below = (at[:, None] // size % 2 == 1) & (at[:, None] // size == at // size + 1)
        inv = inv - inv @ ((N * below) @ inv)
    U, W = inv @ (beta * v), inv @ (beta * from_start * k)
    del inv, N
    q, k = q * from_start, k * to_end
    h = s["h0"].mT.clone() if s["h0"] is not None else v.new_zeros(b, nh, S, H)
    y = torch.empty_like(v)
    for c in range(n):
        d = U[:, :, c] - W[:, :, c] @ h
        y[:, :, c] = q[:, :, c] @ h + P[:, :, c] @ d
        h = from_start[:, :, c, -1:] * h + k[:, :, c].mT @ d
    y = y.flatten(2, 3)[:, :, :L].transpose(1, 2)
    if live is not None:
        y = y * live[..., None]
    return {"y": y.to(s["v"].dtype).contiguous(), "h": h.mT.contiguous()}


def _plain_delta_step(s):
    v = s["v"].float()
    nh, G, S, at = v.shape[1], s["q"].shape[1], s["q"].shape[2], s["slots"].long()
    q, k = (_unit(s[n]).repeat_interleave(nh // G, 1)[..., None] for n in ("q", "k"))
    a = torch.exp(_softplus(s["dt"].float() + s["dt_bias"]) * s["A"])[..., None, None]
    beta = 1 / (1 + torch.exp(-s["beta"].float()))
    h = a * s["state"][at]
    h = h + (beta[..., None, None] * (v[..., None] - h @ k)) * k.mT
    y = (h @ q)[..., 0] * S ** -0.5
    s["state_out"][at] = h
    return {"y": y.to(s["v"].dtype), "h": s["state_out"]}


def _rms(v, eps):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)


def _plain_gatednorm(s):
    case, x, gate = s["case"], s["x"].float(), _silu(s["z"].float())
    d = case["d"]
    group = case["group"] or d
    v = x * gate if case["first"] else x
    v = _rms(v.unflatten(-1, (d // group, group)), s["eps"])
    v = v * (s["weight"] if s["weight"].shape[0] == group else s["weight"].unflatten(0, (d // group, group)))
    v = v.flatten(-2)
    return {"y": (v if case["first"] else v * gate).to(s["x"].dtype)}


def _plain_blocknorm(s):
    v = _rms(s["x"].float(), s["eps"]) * s["weight"]
    if s["z"] is not None:
        v = v * _silu(s["z"].float())
    r = s["alpha"] * s["residual"].float() + v
    y = _rms(r, s["eps"]) * s["next_weight"]
    return {"y": y.to(s["x"].dtype), "residual": r.to(s["residual"].dtype)}


# ---------------------------------------------------------------------------------- the work of a pass

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "gatednorm":
        n = case["rows"] * case["d"]
        return {"bytes": 3 * n * e + 4 * case["d"], "flops": 9 * n}
    if op == "blocknorm":
        n = case["rows"] * case["d"]
        return {"bytes": n * ((3 if case["gate"] else 2) * e + 2 * SIZE[case["res"]]) + 8 * case["d"],
                "flops": (16 if case["gate"] else 11) * n}
    b, nh, G, H, S = (case[k] for k in ("b", "nh", "G", "H", "S"))
    tokens = b * case.get("L", 1)
    states = 2 if op == "delta_step" or case["h0"] else 1
    return {"bytes": tokens * e * (2 * G * S + 2 * nh * H + 2 * nh) + 4 * states * b * nh * H * S + 8 * nh,
            "flops": tokens * nh * H * (7 * S + 4)}


# ---------------------------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in _inputs(case, seed).items()}
    if case["op"] == "gatednorm":
        return _exact_gatednorm(case, s)
    if case["op"] == "blocknorm":
        return _exact_blocknorm(s)
    return _exact_delta(case, s)


def _exact_delta(case, s):
    """The recurrence, one token after the other; a head's state as the map that takes a key to a value."""
    single = case["op"] == "delta_step"
    q, k, v, dt, beta = (s[n][:, None] if single else s[n] for n in ("q", "k", "v", "dt", "beta"))
    b, L, nh, H = v.shape
    S, group = q.shape[-1], torch.arange(nh, device=v.device) // (nh // q.shape[-2])
    step = torch.logaddexp(dt + s["dt_bias"], torch.zeros((), dtype=torch.float64, device=v.device))
    keep, rate = torch.exp(s["A"] * step), torch.sigmoid(beta)
    if single:
        h = s["state"][s["slots"].long()]
    else:
        h = s["h0"].clone() if s["h0"] is not None else v.new_zeros(b, nh, H, S)
    lens = s.get("lens")
    y = torch.zeros_like(v)
    for t in range(L):
        kt, qt = k[:, t, group], q[:, t, group]
        kt = kt / torch.sqrt(torch.linalg.vector_norm(kt, dim=-1, keepdim=True) ** 2 + 1e-6)
        qt = qt / torch.sqrt(torch.linalg.vector_norm(qt, dim=-1, keepdim=True) ** 2 + 1e-6)
        old = keep[:, t, :, None, None] * h
        err = v[:, t] - torch.einsum("bhpn,bhn->bhp", old, kt)
        new = old + torch.einsum("bhp,bhn->bhpn", rate[:, t, :, None] * err, kt)
        out = torch.einsum("bhpn,bhn->bhp", new, qt) / math.sqrt(S)
        if lens is None:
            h, y[:, t] = new, out
        else:
            on = (lens > t).view(b, 1, 1)
            h, y[:, t] = torch.where(on[..., None], new, h), torch.where(on, out, 0.0)
    if not single:
        return {"y": y, "h": h}
    state = s["state"].clone()
    state[s["slots"].long()] = h
    return {"y": y[:, 0], "h": state}


def _length(v):
    return torch.linalg.vector_norm(v, dim=-1, keepdim=True)


def _exact_gatednorm(case, s):
    gate = s["z"] * torch.sigmoid(s["z"])
    u = s["x"] * gate if case["first"] else s["x"]
    group = case["group"] or case["d"]
    weight = s["weight"].repeat(case["d"] // s["weight"].shape[0])
    parts = [p / torch.sqrt(_length(p) ** 2 / group + s["eps"]) for p in u.split(group, -1)]
    y = torch.cat(parts, -1) * weight
    return {"y": y if case["first"] else y * gate}


def _exact_blocknorm(s):
    d = s["x"].shape[-1]
    v = s["x"] / torch.sqrt(_length(s["x"]) ** 2 / d + s["eps"]) * s["weight"]
    if s["z"] is not None:
        v = v * s["z"] * torch.sigmoid(s["z"])
    r = s["residual"] * s["alpha"] + v
    return {"y": r / torch.sqrt(_length(r) ** 2 / d + s["eps"]) * s["next_weight"], "residual": r}
