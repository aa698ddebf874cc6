"""GPU parity of the operators around a layer's scan (short convolution, selective scan, norm;
prompts and single tokens) against the float64 definitions in oracle/layer.py.

Every element is held to the bound that oracle/layer.py derives for it from the arithmetic; a bf16
output may be off by 2^-8 of its value besides (its rounding).  NaN stands in every place that a
call must not read: padding, unused slots, columns beside a strided tensor.
"""
import zlib

import numpy as np
import pytest

from oracle import layer as ol

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib(cuda_lib):
    return cuda_lib


def rng_of(*key):
    return np.random.Generator(np.random.PCG64(zlib.crc32(repr(key).encode())))


def dev(a, dtype="f32"):
    import torch
    if a is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def ints(a):
    import torch
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def host(t):
    return t.detach().double().cpu().numpy()


def rounded(a, dtype):
    """The values that a tensor of this type holds."""
    from selective_state_space_mamba_gb300 import synth
    a = np.ascontiguousarray(a, np.float32)
    return synth.round_to_bf16(a) if dtype == "bf16" else a


def strided(a, dtype, pad):
    """A device tensor of a's values whose rows have `pad` columns of NaN on each side."""
    import torch
    if a is None or pad == 0:
        return dev(a, dtype)
    wide = torch.full((*a.shape[:-1], a.shape[-1] + 2 * pad), float("nan"), device="cuda",
                      dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    wide[..., pad:-pad] = dev(a, dtype)
    return wide[..., pad:-pad]


def close(got, ref, err, what, dtype="f32"):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, what
    if not ref.size:
        return
    assert np.isfinite(got).all(), f"{what}: not finite"
    tol = 1.05 * err + 1e-30 + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)
    over = np.abs(got - ref) - tol
    i = np.unravel_index(int(np.argmax(over)), over.shape)
    assert over[i] <= 0, f"{what}: {got[i]!r} for {ref[i]!r} at {i}, off by more than {tol[i]:.3e}"


# ------------------------------------------------------------------------------ convolution

CONV = [  # b, L, d, W, pad, state, lens, bias, silu
    (1, 1, 8, 4, 0, False, None, True, True),
    (1, 1, 5, 2, 0, True, None, False, True),
    (2, 2, 64, 4, 0, True, None, True, True),          # shorter than the window
    (1, 33, 130, 3, 0, False, None, True, False),
    (2, 70, 257, 4, 3, True, [70, 0], True, True),      # odd rows, an empty sequence
    (3, 100, 64, 2, 8, True, [99, 1, 64], False, True),
    (4, 65, 36, 3, 2, True, [2, 1, 0, 65], True, True),  # lengths inside the window
    (1, 300, 1792, 4, 16, False, None, True, True),
    (2, 31, 1026, 4, 1, True, [40, -3], True, True),    # lengths outside 0 .. L are clamped
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv_prompt(case, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, W, pad, has_state, lens, has_bias, silu = case
    r = rng_of("conv", case, dtype)
    x = rounded(r.standard_normal((b, L, d)), dtype)
    w, bias = r.uniform(-0.5, 0.5, (d, W)).astype(np.float32), r.uniform(-0.5, 0.5, d).astype(np.float32)
    state = rounded(r.standard_normal((b, W - 1, d)), dtype) if has_state else None
    bias = bias if has_bias else None
    y_ref, err, s_ref = ol.conv(x, w, bias, state, lens, silu)
    if lens is not None:  # padding may hold anything
        for i, n in enumerate(ol._lens(lens, b, L)):
            x[i, n:] = np.nan
    y, s = ssm.conv_fwd(strided(x, dtype, pad), dev(w), dev(bias), dev(state, dtype), ints(lens), silu=silu)
    close(host(y), y_ref, err, "y", dtype)
    assert np.array_equal(host(s), s_ref), "the carried tokens are copies"
    y2, none = ssm.conv_fwd(strided(x, dtype, pad), dev(w), dev(bias), dev(state, dtype), ints(lens), silu=silu,
                            return_final_state=False)
    assert none is None and np.array_equal(host(y2), host(y))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 8, 4, 0, None, 1), (3, 5, 2, 1, None, 3), (5, 257, 3, 2, [6, -1, 0, 7, 3], 8),
                                  (4, 1792, 4, 8, [2, 9, 1, 1 << 30], 4), (2, 130, 4, 0, [1, 0], 2)], ids=str)
def test_conv_step(case, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, d, W, pad, slots, n = case
    r = rng_of("conv_step", case, dtype)
    x = rounded(r.standard_normal((b, d)), dtype)
    w, bias = r.uniform(-0.5, 0.5, (d, W)).astype(np.float32), r.uniform(-0.5, 0.5, d).astype(np.float32)
    state = rounded(r.standard_normal((n, W - 1, d)), dtype)
    at = np.arange(b) if slots is None else np.asarray(slots)
    used = (at >= 0) & (at < n)
    y_ref, err, s_new = ol.conv(x[used][:, None], w, bias, state[at[used]])
    want, want_s = np.zeros((b, d)), state.astype(np.float64).copy()
    want[used], want_s[at[used]] = y_ref[:, 0], s_new
    e = np.zeros((b, d))
    e[used] = err[:, 0]
    st = dev(state, dtype)
    y, s = ssm.conv_step(strided(x, dtype, pad), dev(w), dev(bias), st, ints(slots))
    close(host(y), want, e, "y", dtype)
    assert np.array_equal(host(s), want_s) and np.array_equal(host(st), state)
    y2, s2 = ssm.conv_step(strided(x, dtype, pad), dev(w), dev(bias), st, ints(slots), inplace=True)
    assert s2.data_ptr() == st.data_ptr() and np.array_equal(host(s2), want_s) and np.array_equal(host(y2), host(y))


def test_conv_step_from_zeros():
    import selective_state_space_mamba_gb300 as ssm
    r = rng_of("conv zeros")
    x, w = r.standard_normal((3, 40)).astype(np.float32), r.standard_normal((40, 4)).astype(np.float32)
    y_ref, err, s_ref = ol.conv(x[:, None], w)
    y, s = ssm.conv_step(dev(x), dev(w))
    close(host(y), y_ref[:, 0], err[:, 0], "y")
    assert np.array_equal(host(s), s_ref)


def test_conv_infinities_stay_where_they_are():
    """An infinite input gives silu(+-inf) and inf - inf in its own W outputs and nowhere else."""
    import selective_state_space_mamba_gb300 as ssm
    r = rng_of("conv inf")
    x, w = r.standard_normal((1, 64, 16)).astype(np.float32), r.uniform(0.1, 0.5, (16, 4)).astype(np.float32)
    clean, _ = ssm.conv_fwd(dev(x), dev(w))
    x[0, 20, 5] = np.inf
    y, _ = ssm.conv_fwd(dev(x), dev(w))
    y, clean = host(y), host(clean)
    assert np.isposinf(y[0, 20:24, 5]).all()
    y[0, 20:24, 5] = clean[0, 20:24, 5]
    assert np.array_equal(y, clean)


# ------------------------------------------------------------------------------ selective scan

def scan_inputs(r, lead, d, N, G, dtype, dt_mean=0.0):
    low = np.exp(r.uniform(np.log(1e-3), np.log(0.1), d))
    return {"u": rounded(r.standard_normal((*lead, d)), dtype), "dt": rounded(dt_mean + 0.5 * r.standard_normal((*lead, d)), dtype),
            "A": (-np.arange(1, N + 1) * np.exp(0.2 * r.standard_normal((d, N)))).astype(np.float32),
            "B": rounded(r.standard_normal((*lead, G, N)), dtype), "C": rounded(r.standard_normal((*lead, G, N)), dtype),
            "D": r.uniform(0.5, 1.5, d).astype(np.float32), "z": rounded(r.standard_normal((*lead, d)), dtype),
            "dt_bias": (low + np.log(-np.expm1(-low))).astype(np.float32)}


def groups_strided(a, dtype, pad):
    """B or C as columns of wider rows."""
    if pad == 0:
        return dev(a, dtype)
    return strided(a.reshape(*a.shape[:-2], -1), dtype, pad).unflatten(-1, a.shape[-2:])


def run_scan(inp, dtype, pad, h0=None, lens=None, softplus=True, **kw):
    import selective_state_space_mamba_gb300 as ssm
    t = {k: strided(inp[k], dtype, pad) for k in ("u", "dt", "z") if inp[k] is not None}
    return ssm.selscan_fwd(t["u"], t["dt"], dev(inp["A"]), groups_strided(inp["B"], dtype, pad),
                           groups_strided(inp["C"], dtype, pad), dev(inp["D"]), t.get("z"), dev(inp["dt_bias"]),
                           dev(h0), ints(lens), softplus=softplus, **kw)


SCAN = [  # b, L, d, N, G, pad, h0, lens, z, bias
    (1, 1, 8, 16, 1, 0, False, None, True, True),
    (1, 1, 1, 8, 1, 0, True, None, False, False),
    (2, 3, 40, 16, 1, 0, True, None, True, True),
    (1, 65, 33, 16, 1, 5, False, None, True, True),           # odd rows
    (2, 64, 64, 8, 2, 8, True, [64, 0], True, True),           # an empty sequence
    (3, 50, 72, 32, 3, 8, True, [50, 1, 33], False, True),
    (2, 97, 30, 64, 2, 1, True, [96, 97], True, True),         # groups of an odd number of channels
    (1, 40, 136, 64, 1, 0, False, None, True, False),
    (1, 300, 48, 16, 1, 8, True, None, True, True),            # the time axis in pieces
    (2, 513, 24, 16, 1, 0, False, [513, 77], True, True),      # pieces that are all padding
    (2, 700, 17, 8, 1, 3, True, [1, 640], True, True),
    (1, 1000, 20, 32, 2, 0, True, None, False, True),
    (1, 2049, 64, 64, 1, 0, True, [2500], True, True),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_selscan_prompt(case, dtype):
    b, L, d, N, G, pad, has_h0, lens, has_z, has_bias = case
    r = rng_of("selscan", case, dtype)
    inp = scan_inputs(r, (b, L), d, N, G, dtype)
    if not has_z:
        inp["z"] = None
    if not has_bias:
        inp["dt_bias"] = inp["D"] = None
    h0 = (0.3 * r.standard_normal((b, d, N))).astype(np.float32) if has_h0 else None
    y_ref, ey, h_ref, eh = ol.selscan(**inp, h0=h0, lens=lens, pieces=L)
    if lens is not None:
        for i, n in enumerate(ol._lens(lens, b, L)):
            for k in ("u", "dt", "B", "C", "z"):
                if inp[k] is not None:
                    inp[k][i, n:] = np.nan
    y, h = run_scan(inp, dtype, pad, h0, lens)
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref, ey, "y", dtype)
    y2, none = run_scan(inp, dtype, pad, h0, lens, return_final_state=False)
    assert none is None and np.array_equal(host(y2), host(y)), "the same from call to call"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_selscan_plain_steps(dtype):
    """Without the softplus; steps of zero leave the state bit for bit."""
    r = rng_of("selscan plain", dtype)
    inp = scan_inputs(r, (2, 70), 40, 16, 1, dtype)
    inp["dt"], inp["dt_bias"] = rounded(r.uniform(0, 0.2, (2, 70, 40)), dtype), None
    h0 = r.standard_normal((2, 40, 16)).astype(np.float32)
    y_ref, ey, h_ref, eh = ol.selscan(**inp, h0=h0, softplus=False, pieces=70)
    y, h = run_scan(inp, dtype, 0, h0, softplus=False)
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref, ey, "y", dtype)
    inp["dt"][:] = 0
    y, h = run_scan(inp, dtype, 0, h0, softplus=False)
    assert np.array_equal(host(h), h0)


@pytest.mark.parametrize("mean", [-40.0, -9.0, 30.0, 120.0])
def test_selscan_extreme_steps(mean):
    """Steps from 4e-18 to over 100: small ones keep their precision, large ones forget the state."""
    r = rng_of("selscan extreme", mean)
    inp = scan_inputs(r, (1, 80), 24, 16, 1, "f32", dt_mean=mean)
    inp["dt_bias"] = None
    h0 = r.standard_normal((1, 24, 16)).astype(np.float32)
    y_ref, ey, h_ref, eh = ol.selscan(**inp, h0=h0, pieces=80)
    y, h = run_scan(inp, "f32", 0, h0)
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref, ey, "y")


@pytest.mark.parametrize("L", [0, 5])
def test_selscan_and_conv_empty(L):
    """No tokens hand the state on; no sequences return nothing."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    b = 2 if L == 0 else 0
    r = rng_of("empty")
    h0, cs = r.standard_normal((b, 8, 16)).astype(np.float32), r.standard_normal((b, 3, 8)).astype(np.float32)
    t = torch.empty(b, L, 8, device="cuda")
    bc = torch.empty(b, L, 1, 16, device="cuda")
    y, h = ssm.selscan_fwd(t, t, -torch.ones(8, 16, device="cuda"), bc, bc, h0=dev(h0))
    assert y.shape == (b, L, 8) and np.array_equal(host(h), h0)
    y, s = ssm.conv_fwd(t, torch.ones(8, 4, device="cuda"), state=dev(cs))
    assert y.shape == (b, L, 8) and np.array_equal(host(s), cs)
    y, s = ssm.conv_fwd(t, torch.ones(8, 4, device="cuda"))
    assert not host(s).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [(1, 8, 16, 1, 0, None, 1), (3, 5, 8, 1, 1, None, 3), (5, 33, 16, 1, 3, [6, -1, 0, 7, 3], 8),
                                  (4, 72, 32, 2, 8, [2, 9, 1, 1 << 30], 4), (2, 30, 64, 3, 0, [1, 0], 2),
                                  (40, 96, 16, 2, 0, None, 40)], ids=str)
def test_selscan_step(case, dtype):
    import selective_state_space_mamba_gb300 as ssm
    b, d, N, G, pad, slots, n = case
    r = rng_of("selscan_step", case, dtype)
    inp = scan_inputs(r, (b,), d, N, G, dtype)
    state = (0.3 * r.standard_normal((n, d, N))).astype(np.float32)
    at = np.arange(b) if slots is None else np.asarray(slots)
    used = (at >= 0) & (at < n)
    one = {k: (v if k in ("A", "D", "dt_bias") else v[used][:, None]) for k, v in inp.items()}
    y1, e1, h1, eh1 = ol.selscan(**one, h0=state[at[used]])
    want, ey, want_h, eh = np.zeros((b, d)), np.zeros((b, d)), state.astype(np.float64).copy(), np.zeros((n, d, N))
    want[used], ey[used], want_h[at[used]], eh[at[used]] = y1[:, 0], e1[:, 0], h1, eh1
    for k in ("u", "dt", "B", "C", "z"):
        inp[k][~used] = np.nan
    t = {k: strided(inp[k], dtype, pad) for k in ("u", "dt", "z")}
    args = (t["u"], t["dt"], dev(inp["A"]), groups_strided(inp["B"], dtype, pad), groups_strided(inp["C"], dtype, pad),
            dev(inp["D"]), t["z"], dev(inp["dt_bias"]))
    st = dev(state)
    y, h = ssm.selscan_step(*args, st, ints(slots))
    close(host(h), want_h, eh, "h")
    close(host(y), want, ey, "y", dtype)
    assert np.array_equal(host(st), state)
    y2, h2 = ssm.selscan_step(*args, st, ints(slots), inplace=True)
    assert h2.data_ptr() == st.data_ptr() and np.array_equal(host(h2), host(h)) and np.array_equal(host(y2), host(y))


def test_selscan_step_bare():
    """From zeros, with neither skip, gate nor bias, and steps as they are given."""
    import selective_state_space_mamba_gb300 as ssm
    r = rng_of("bare")
    inp = scan_inputs(r, (3,), 20, 16, 1, "f32")
    dt = np.abs(inp["dt"])
    y_ref, ey, h_ref, eh = ol.selscan(inp["u"][:, None], dt[:, None], inp["A"], inp["B"][:, None], inp["C"][:, None],
                                      softplus=False)
    y, h = ssm.selscan_step(dev(inp["u"]), dev(dt), dev(inp["A"]), dev(inp["B"]), dev(inp["C"]), softplus=False)
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref[:, 0], ey[:, 0], "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompt_in_two_parts_and_tokens_one_by_one(dtype):
    """The state carried from a prompt to its next part, and then from token to token."""
    import selective_state_space_mamba_gb300 as ssm
    b, L, d, N, W = 2, 120, 40, 16, 4
    r = rng_of("parts", dtype)
    inp = scan_inputs(r, (b, L), d, N, 1, dtype)
    w = r.uniform(-0.5, 0.5, (d, W)).astype(np.float32)
    c_ref, ec, cs_ref = ol.conv(inp["u"], w)
    y_ref, ey, h_ref, eh = ol.selscan(**inp, pieces=L)
    t = {k: dev(inp[k], dtype) for k in ("u", "dt", "B", "C", "z")}
    A, D, bias, w = dev(inp["A"]), dev(inp["D"]), dev(inp["dt_bias"]), dev(w)
    ys, cs, h, conv = [], [], None, None
    for t0, t1 in ((0, 50), (50, 113)):
        p = {k: v[:, t0:t1] for k, v in t.items()}
        c, conv = ssm.conv_fwd(p["u"], w, state=conv)
        y, h = ssm.selscan_fwd(p["u"], p["dt"], A, p["B"], p["C"], D, p["z"], bias, h0=h)
        cs.append(host(c)), ys.append(host(y))
    for i in range(113, L):
        p = {k: v[:, i] for k, v in t.items()}
        c, conv = ssm.conv_step(p["u"], w, state=conv, inplace=True)
        y, h = ssm.selscan_step(p["u"], p["dt"], A, p["B"], p["C"], D, p["z"], bias, h, inplace=True)
        cs.append(host(c)[:, None]), ys.append(host(y)[:, None])
    close(np.concatenate(cs, 1), c_ref, ec, "conv", dtype)
    close(np.concatenate(ys, 1), y_ref, ey, "y", dtype)
    close(host(h), h_ref, eh, "h")
    assert np.array_equal(host(conv), cs_ref)


# ------------------------------------------------------------------------------ norm

NORM = [(1, 1), (1, 7), (3, 8), (2, 257), (5, 1024), (4, 1536), (33, 2560), (2, 5120), (2, 8200), (3, 16391),
        (2, 20000), (1, 65544)]


def norm_inputs(key, rows, d, dtype, res):
    r = rng_of("norm", key, rows, d, dtype, res)
    x = rounded(r.standard_normal((rows, d)), dtype)
    residual = None if res == "none" else rounded(4 * r.standard_normal((rows, d)), res)
    return x, r.uniform(0.5, 1.5, d).astype(np.float32), residual


@pytest.mark.parametrize("dtype,res", [("f32", "none"), ("f32", "f32"), ("bf16", "none"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", NORM, ids=str)
def test_rmsnorm(shape, dtype, res):
    import selective_state_space_mamba_gb300 as ssm
    rows, d = shape
    x, w, residual = norm_inputs("plain", rows, d, dtype, res)
    v, err, r = ol.rmsnorm(x, w, residual)
    pad = 0 if d % 2 else 8
    rd = dev(residual, res)
    y, ro = ssm.rmsnorm_fwd(strided(x, dtype, pad), dev(w), rd)
    close(host(y), v, err, "y", dtype)
    if residual is None:
        assert ro is None
        return
    close(host(ro), r, ol.U * np.abs(r), "residual", res)
    assert np.array_equal(host(rd), residual)
    y2, r2 = ssm.rmsnorm_fwd(strided(x, dtype, pad), dev(w), rd, residual_out=rd)
    assert r2 is rd and np.array_equal(host(r2), host(ro)) and np.array_equal(host(y2), host(y))


def e4m3_close(q, scale, v, err, what):
    """q * scale against v: half a step of e4m3 (2^-4 of the value, 2^-10 of the scale for subnormals)."""
    close(q * scale, v, err + 2.0 ** -4 * np.abs(v) + 2.0 ** -10 * scale + 4 * ol.U * np.abs(v), what)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype,res", [("f32", "none"), ("f32", "f32"), ("bf16", "none"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", NORM, ids=str)
def test_rmsnorm_fp8(shape, dtype, res, group):
    import selective_state_space_mamba_gb300 as ssm
    rows, d = shape
    x, w, residual = norm_inputs("fp8", rows, d, dtype, res)
    v, err, r = ol.rmsnorm(x, w, residual)
    q, scale, ro = ssm.rmsnorm_fp8_fwd(strided(x, dtype, 0 if d % 2 else 8), dev(w), dev(residual, res), group=group)
    q, s = host(q), host(scale)
    n = -(-d // group) if group else 1
    parts = [slice(i * (group or d), min(d, (i + 1) * (group or d))) for i in range(n)]
    assert s.shape == ((rows, n) if group else (rows,))
    s = s.reshape(rows, n)
    for i, p in enumerate(parts):
        amax = np.abs(v[:, p]).max(1)
        assert np.all(np.abs(s[:, i] * 448 - amax) <= err[:, p].max(1) + 2 * ol.U * amax), "scale"
        assert np.abs(q[:, p]).max() <= 448
        e4m3_close(q[:, p], s[:, i : i + 1], v[:, p], err[:, p], f"group {i}")
    if residual is not None:
        close(host(ro), r, ol.U * np.abs(r), "residual", res)


@pytest.mark.parametrize("group", [0, 128])
def test_rmsnorm_fp8_zeros_and_nan(group):
    """A row of zeros has codes of zero and a finite scale; a NaN spoils its own row only."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    x = torch.randn(3, 512, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[1] = 0
    x[2, 300] = float("nan")
    q, s, _ = ssm.rmsnorm_fp8_fwd(x, torch.ones(512, device="cuda"), group=group)
    assert torch.isfinite(q[0].float()).all() and not q[1].float().any() and torch.isnan(q[2].float()).all()
    assert torch.isfinite(s[:2]).all() and (s[:2] > 0).all() and torch.isnan(s[2]).all()
    y, _ = ssm.rmsnorm_fwd(x, torch.ones(512, device="cuda"))
    assert not y[1].any() and torch.isnan(y[2]).all() and torch.isfinite(y[0]).all()


def test_rmsnorm_shapes():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    w = torch.ones(64, device="cuda")
    x = torch.randn(2, 3, 64, device="cuda")
    y, _ = ssm.rmsnorm_fwd(x, w)
    q, s, _ = ssm.rmsnorm_fp8_fwd(x, w, group=128)
    assert y.shape == x.shape and q.shape == x.shape and s.shape == (2, 3, 1)
    assert torch.equal(y.view(6, 64), ssm.rmsnorm_fwd(x.view(6, 64), w)[0])
    e, _ = ssm.rmsnorm_fwd(x[:0], w)
    assert e.shape == (0, 3, 64)


# ------------------------------------------------------------------------------ streams, graphs, refusals

def test_own_stream_and_graph():
    """On a side stream, and captured into a graph that is replayed on new inputs."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    r = rng_of("graph")
    inp = scan_inputs(r, (1, 400), 32, 16, 1, "bf16")
    w = r.uniform(-0.5, 0.5, (32, 4)).astype(np.float32)
    t = {k: dev(inp[k], "bf16") for k in ("u", "dt", "B", "C", "z")}
    A, D, bias, w, g = dev(inp["A"]), dev(inp["D"]), dev(inp["dt_bias"]), dev(w), torch.ones(32, device="cuda")

    def layer():
        v, _ = ssm.rmsnorm_fwd(t["u"], g)
        c, _ = ssm.conv_fwd(v, w)
        return ssm.selscan_fwd(c, t["dt"], A, t["B"], t["C"], D, t["z"], bias)

    want = [host(v) for v in layer()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
    side.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    keep = t["u"].clone()
    t["u"].mul_(0.5)
    want2 = [host(v) for v in layer()]
    graph.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(out, want2))
    t["u"].copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(host(a), b) for a, b in zip(out, want))


def test_kernel_timer_names():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    x = torch.randn(1, 64, 32, device="cuda")
    bc = torch.randn(1, 64, 1, 16, device="cuda")
    A = -torch.ones(32, 16, device="cuda")
    with ssm.KernelTimer() as kt:
        ssm.conv_fwd(x, torch.ones(32, 4, device="cuda"))
        ssm.conv_step(x[:, 0], torch.ones(32, 4, device="cuda"))
        ssm.selscan_fwd(x, x, A, bc, bc)
        ssm.selscan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0])
        ssm.rmsnorm_fwd(x, torch.ones(32, device="cuda"))
    assert all(kt.launches[k] == 1 for k in ("conv", "conv_step", "selscan", "selscan_step", "rmsnorm"))


def test_python_refusals():
    import torch
    import selective_state_space_mamba_gb300 as ssm
    x = torch.randn(2, 5, 16, device="cuda")
    w = torch.randn(16, 4, device="cuda")
    bc, A = torch.randn(2, 5, 1, 16, device="cuda"), -torch.ones(16, 16, device="cuda")
    bad = [
        (TypeError, lambda: ssm.conv_fwd(x.half(), w)),
        (ValueError, lambda: ssm.conv_fwd(x[0], w)),
        (ValueError, lambda: ssm.conv_fwd(x.transpose(1, 2), w)),
        (ValueError, lambda: ssm.conv_fwd(x, w[:8])),
        (ValueError, lambda: ssm.conv_fwd(x, w.bfloat16())),
        (ValueError, lambda: ssm.conv_fwd(x, w, state=torch.zeros(2, 2, 16, device="cuda"))),
        (ValueError, lambda: ssm.conv_fwd(x, w, lens=torch.zeros(2, device="cuda"))),
        (ValueError, lambda: ssm.conv_fwd(x.cpu(), w)),
        (ssm.SsmError, lambda: ssm.conv_fwd(x, torch.ones(16, 5, device="cuda"))),
        (ssm.SsmError, lambda: ssm.conv_fwd(x, w, y=x)),
        (ValueError, lambda: ssm.conv_step(x[:, 0], w, slots=torch.zeros(2, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: ssm.conv_step(x[:, 0], w, inplace=True)),
        (ssm.SsmError, lambda: ssm.conv_step(x[:, 0], w, state=torch.zeros(3, 3, 16, device="cuda"))),
        (ValueError, lambda: ssm.selscan_fwd(x, x[:, :4], A, bc, bc)),
        (ValueError, lambda: ssm.selscan_fwd(x, x, A, bc, bc[..., :8])),
        (ValueError, lambda: ssm.selscan_fwd(x, x, A[:8], bc, bc)),
        (ValueError, lambda: ssm.selscan_fwd(x, x, A, bc, bc, z=x.bfloat16())),
        (ssm.SsmError, lambda: ssm.selscan_fwd(x, x, A[:, :4].contiguous(), bc[..., :4].contiguous(), bc[..., :4].contiguous())),
        (ssm.SsmError, lambda: ssm.selscan_fwd(x, x, A, bc.expand(2, 5, 3, 16).contiguous(), bc.expand(2, 5, 3, 16).contiguous())),
        (ValueError, lambda: ssm.selscan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], state=torch.zeros(2, 16, 8, device="cuda"))),
        (ValueError, lambda: ssm.rmsnorm_fwd(x, w[:, 0].contiguous()[:8])),
        (ValueError, lambda: ssm.rmsnorm_fwd(x, torch.ones(16, device="cuda"), x.half())),
        (ValueError, lambda: ssm.rmsnorm_fwd(x, torch.ones(16, device="cuda"), x[:1])),
        (ValueError, lambda: ssm.rmsnorm_fwd(x, torch.ones(16, device="cuda"), residual_out=x)),
        (ssm.SsmError, lambda: ssm.rmsnorm_fwd(x, torch.ones(16, device="cuda"), y=x)),
        (ssm.SsmError, lambda: ssm.rmsnorm_fp8_fwd(x, torch.ones(16, device="cuda"), group=64, scale=torch.empty(2, 5, 1, device="cuda"))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------ sizes that take the wide variants

@pytest.mark.parametrize("group", [None, 0, 128])
@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "none"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("d", [1032, 1536, 2560, 4104, 10240])
def test_rmsnorm_many_rows(d, dtype, res, group):
    """Rows enough to fill the GPU: several vectors a thread, the last of them partly past the row."""
    import selective_state_space_mamba_gb300 as ssm
    rows = 613
    x, w, residual = norm_inputs("many", rows, d, dtype, res)
    v, err, r = ol.rmsnorm(x, w, residual)
    if group is None:
        y, ro = ssm.rmsnorm_fwd(dev(x, dtype), dev(w), dev(residual, res))
        close(host(y), v, err, "y", dtype)
    else:
        q, scale, ro = ssm.rmsnorm_fp8_fwd(dev(x, dtype), dev(w), dev(residual, res), group=group)
        s = host(scale).reshape(rows, -1)
        each = np.repeat(s, group or d, axis=1)[:, :d]
        pad = np.pad(np.abs(v), ((0, 0), (0, s.shape[1] * (group or d) - d))).reshape(rows, s.shape[1], -1).max(2)
        assert np.all(np.abs(s * 448 - pad) <= err.max(1, keepdims=True) + 2 * ol.U * pad)
        e4m3_close(host(q), each, v, err, "q")
    if residual is not None:
        close(host(ro), r, ol.U * np.abs(r), "residual", res)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,W,b,lens", [(4, 4, 1, None), (6, 3, 2, [4001, 1777]), (5376, 4, 1, None), (999, 2, 1, [3990])])
def test_conv_long(d, W, b, lens, dtype):
    """Several blocks of tokens a run, and a part of one at its end."""
    import selective_state_space_mamba_gb300 as ssm
    L = 4001 if d < 5000 else 301
    r = rng_of("conv long", d, W, b, dtype)
    x = rounded(r.standard_normal((b, L, d)), dtype)
    w, bias = r.uniform(-0.5, 0.5, (d, W)).astype(np.float32), r.uniform(-0.5, 0.5, d).astype(np.float32)
    y_ref, err, s_ref = ol.conv(x, w, bias, None, lens)
    if lens is not None:
        for i, n in enumerate(lens):
            x[i, n:] = np.nan
    y, s = ssm.conv_fwd(dev(x, dtype), dev(w), dev(bias), lens=ints(lens))
    close(host(y), y_ref, err, "y", dtype)
    assert np.array_equal(host(s), s_ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,N,G,pad", [(2048, 16, 1, 0), (4104, 8, 2, 3), (1030, 32, 1, 8), (516, 64, 2, 0)])
def test_selscan_step_many(d, N, G, pad, dtype):
    """Sequences enough that a thread takes four, the last of them fewer; unused places among them."""
    import selective_state_space_mamba_gb300 as ssm
    b, n = 82, 90
    r = rng_of("step many", d, N, G, dtype)
    inp = scan_inputs(r, (b,), d, N, G, dtype)
    state = (0.3 * r.standard_normal((n, d, N))).astype(np.float32)
    at = r.permutation(n)[:b]
    at[[3, 40, 81]] = [-1, n, 1 << 20]
    used = (at >= 0) & (at < n)
    one = {k: (v if k in ("A", "D", "dt_bias") else v[used][:, None]) for k, v in inp.items()}
    y1, e1, h1, eh1 = ol.selscan(**one, h0=state[at[used]])
    want, ey, want_h, eh = np.zeros((b, d)), np.zeros((b, d)), state.astype(np.float64).copy(), np.zeros((n, d, N))
    want[used], ey[used], want_h[at[used]], eh[at[used]] = y1[:, 0], e1[:, 0], h1, eh1
    for k in ("u", "dt", "B", "C", "z"):
        inp[k][~used] = np.nan
    t = {k: strided(inp[k], dtype, pad) for k in ("u", "dt", "z")}
    st = dev(state)
    y, h = ssm.selscan_step(t["u"], t["dt"], dev(inp["A"]), groups_strided(inp["B"], dtype, pad),
                            groups_strided(inp["C"], dtype, pad), dev(inp["D"]), t["z"], dev(inp["dt_bias"]), st, ints(at),
                            inplace=True)
    close(host(h), want_h, eh, "h")
    close(host(y), want, ey, "y", dtype)


QUEUE = (13, 2100, 1544)  # chains enough that the CTAs claim them in items, one after the other


def queue_case(dtype, key):
    """Inputs of a scan that takes the queue, and the sequences and channels that the oracle checks."""
    b, L, d = QUEUE
    r = rng_of("queue", dtype, key)
    inp = scan_inputs(r, (b, L), d, 16, 1, dtype)
    h0 = (0.3 * r.standard_normal((b, d, 16))).astype(np.float32)
    return inp, h0, np.array([0, 5, b - 1]), np.sort(r.choice(d, 40, replace=False))


@pytest.mark.parametrize("dtype,lens", [("bf16", None), ("f32", [2100, 1, 0, 700, 512, 513, 1024, 1040, 2048, 2047, 1536, 31, 1999])])
def test_selscan_queue(dtype, lens):
    """Chains of several items that the CTAs claim one after the other, a state handed on at each:
    against the definition, and bit for bit what the same tokens give in several calls."""
    import selective_state_space_mamba_gb300 as ssm
    inp, h0, bs, cs = queue_case(dtype, lens is None)
    sub = {k: (v[cs] if k in ("A", "D", "dt_bias") else v[bs] if k in ("B", "C") else v[bs][..., cs]) for k, v in inp.items()}
    some = None if lens is None else [lens[i] for i in bs]
    y_ref, ey, h_ref, eh = ol.selscan(**sub, h0=h0[bs][:, cs], lens=some)
    if lens is not None:
        for i, n in enumerate(lens):
            for k in ("u", "dt", "B", "C", "z"):
                inp[k][i, n:] = np.nan
    y, h = run_scan(inp, dtype, 0, h0, lens)
    close(host(h)[bs][:, cs], h_ref, eh, "h")
    close(host(y)[bs][..., cs], y_ref, ey, "y", dtype)
    t = {k: dev(inp[k], dtype) for k in ("u", "dt", "B", "C", "z")}
    A, D, bias, state = dev(inp["A"]), dev(inp["D"]), dev(inp["dt_bias"]), dev(h0)
    for t0 in range(0, QUEUE[1], 512):
        p = {k: v[:, t0 : t0 + 512] for k, v in t.items()}
        n = None if lens is None else ints([min(max(m - t0, 0), 512) for m in lens])
        part, state = ssm.selscan_fwd(p["u"], p["dt"], A, p["B"], p["C"], D, p["z"], bias, state, n)
        assert np.array_equal(host(part), host(y[:, t0 : t0 + 512]))
    assert np.array_equal(host(state), host(h))


def test_selscan_queue_wait_runs_out():
    """An item that never publishes its state: the waits of the chain's later items run out, the call
    reports it, its later outputs are NaN, and the workspace serves the next call."""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    from selective_state_space_mamba_gb300 import _lib
    b, L, d = QUEUE
    g = torch.Generator("cuda").manual_seed(5)
    u, dt = (torch.randn(b, L, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    B, C = (torch.randn(b, L, 1, 16, device="cuda", generator=g).bfloat16() for _ in range(2))
    A = -torch.rand(d, 16, device="cuda", generator=g) - 0.1
    ws = ssm.Workspace("cuda")
    y, h = ssm.selscan_fwd(u, dt, A, B, C, workspace=ws)
    assert ssm.check_device_status(ws) == 0
    assert torch.isfinite(y).all()
    try:
        ssm.debug_set_lookback_fault(3, 2_000_000)
        bad, _ = ssm.selscan_fwd(u, dt, A, B, C, workspace=ws)
        status = ssm.check_device_status(ws)
    finally:
        ssm.debug_set_lookback_fault()
    assert status == _lib.SSM_ERR_TIMEOUT
    assert torch.isnan(bad).any() and torch.equal(bad[:, :256], y[:, :256])
    again, h2 = ssm.selscan_fwd(u, dt, A, B, C, workspace=ws)
    assert ssm.check_device_status(ws) == 0
    assert torch.equal(again, y) and torch.equal(h2, h)


# ------------------------------------------------------------------------------ rows that are not aligned

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [
    (2, 131, 263, 16, 1, 0, True, [131, 113], True, True),
    (3, 64, 197, 8, 1, 1, False, None, True, True),
    (2, 97, 146, 16, 2, 2, True, None, True, False),           # groups of 73 channels
    (2, 80, 101, 32, 1, 3, True, [80, 16], False, True),
    (1, 33, 75, 64, 1, 7, True, None, True, True),
    (2, 48, 132, 16, 1, 4, True, [17, 48], True, True),        # rows on 8 bytes (bf16), on 16 (f32) but d4
    (1, 1500, 65, 16, 1, 0, True, None, True, True),           # and the time axis in pieces
], ids=str)
def test_selscan_ragged_rows(case, dtype):
    """Several channel tiles and tiles of tokens of rows that tensor copies cannot take."""
    test_selscan_prompt(case, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 67, 3])
def test_selscan_rows_on_one_another(d, dtype):
    """Inputs broadcast over sequences (B, C) or tokens (dt, z), or overlapping rows one element apart (u)."""
    import selective_state_space_mamba_gb300 as ssm
    b, L, N = 2, 50, 16
    r = rng_of("broadcast", d, dtype)
    inp = scan_inputs(r, (b, L), d, N, 1, dtype)
    line = rounded(r.standard_normal(b * L + d), dtype)
    inp["u"] = np.lib.stride_tricks.sliding_window_view(line, d)[: b * L].reshape(b, L, d)
    inp["dt"], inp["z"] = (np.broadcast_to(inp[k][:, :1], (b, L, d)) for k in ("dt", "z"))
    inp["B"], inp["C"] = (np.broadcast_to(inp[k][:1], (b, L, 1, N)) for k in ("B", "C"))
    y_ref, ey, h_ref, eh = ol.selscan(**inp)
    t = {k: dev(inp[k][:, :1], dtype).expand(b, L, d) for k in ("dt", "z")}
    g = {k: dev(inp[k][:1], dtype).expand(b, L, 1, N) for k in ("B", "C")}
    u = dev(line, dtype).as_strided((b, L, d), (L, 1, 1))
    y, h = ssm.selscan_fwd(u, t["dt"], dev(inp["A"]), g["B"], g["C"], dev(inp["D"]), t["z"], dev(inp["dt_bias"]))
    close(host(h), h_ref, eh, "h")
    close(host(y), y_ref, ey, "y", dtype)


@pytest.mark.parametrize("b,L,d,dtype,pad", [
    (13, 1100, 1537, "bf16", 0),    # more chains than places, odd rows
    (13, 530, 1541, "f32", 3),
    (7, 1300, 1472, "f32", 0),      # a few more chains than SMs: a CTA an SM
    (7, 1300, 1425, "bf16", 1),
])
def test_selscan_more_queues(b, L, d, dtype, pad):
    """Against the definition, and bit for bit what the same tokens give in several calls."""
    import selective_state_space_mamba_gb300 as ssm
    r = rng_of("more queues", b, L, d, dtype)
    inp = scan_inputs(r, (b, L), d, 16, 1, dtype)
    h0 = (0.3 * r.standard_normal((b, d, 16))).astype(np.float32)
    lens = [L - 37 * i for i in range(b)]
    bs, cs = np.array([0, 3, b - 1]), np.sort(r.choice(d, 24, replace=False))
    sub = {k: (v[cs] if k in ("A", "D", "dt_bias") else v[bs] if k in ("B", "C") else v[bs][..., cs]) for k, v in inp.items()}
    y_ref, ey, h_ref, eh = ol.selscan(**sub, h0=h0[bs][:, cs], lens=[lens[i] for i in bs])
    for i, n in enumerate(lens):
        for k in ("u", "dt", "B", "C", "z"):
            inp[k][i, n:] = np.nan
    y, h = run_scan(inp, dtype, pad, h0, lens)
    close(host(h)[bs][:, cs], h_ref, eh, "h")
    close(host(y)[bs][..., cs], y_ref, ey, "y", dtype)
    state, parts = h0, []
    for t0 in range(0, L, 256):
        p = {k: (v[:, t0 : t0 + 256] if k in ("u", "dt", "B", "C", "z") else v) for k, v in inp.items()}
        part, state = run_scan(p, dtype, pad, state, [min(max(n - t0, 0), 256) for n in lens])
        parts.append(host(part))
        state = host(state)
    assert np.array_equal(np.concatenate(parts, 1), host(y)) and np.array_equal(state, host(h))


@pytest.mark.parametrize("group", [None, 0, 128])
@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "none"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("d", [513, 1031, 1540, 2561, 4099, 10243])
def test_rmsnorm_many_ragged_rows(d, dtype, res, group):
    test_rmsnorm_many_rows(d, dtype, res, group)


@pytest.mark.parametrize("group", [None, 0, 128])
@pytest.mark.parametrize("dtype,res", [("f32", "f32"), ("bf16", "none"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("d", [1, 8, 100, 256, 257, 768, 1000, 1280, 12288])
def test_rmsnorm_many_narrow_rows(d, dtype, res, group):
    """A warp a row, four rows a CTA (613 rows: the last CTA has one); and rows of more than 10240.  With one
    column x + residual is 0 in a row, whose scale is the least."""
    import selective_state_space_mamba_gb300 as ssm
    rows = 613
    x, w, residual = norm_inputs("many", rows, d, dtype, res)
    v, err, r = ol.rmsnorm(x, w, residual)
    if group is None:
        y, ro = ssm.rmsnorm_fwd(dev(x, dtype), dev(w), dev(residual, res))
        close(host(y), v, err, "y", dtype)
    else:
        q, scale, ro = ssm.rmsnorm_fp8_fwd(dev(x, dtype), dev(w), dev(residual, res), group=group)
        s = host(scale).reshape(rows, -1)
        each = np.repeat(s, group or d, axis=1)[:, :d]
        pad = np.pad(np.abs(v), ((0, 0), (0, s.shape[1] * (group or d) - d))).reshape(rows, s.shape[1], -1).max(2)
        least = 448 * 2.0 ** -126
        assert np.all(np.abs(s * 448 - np.maximum(pad, least)) <= err.max(1, keepdims=True) + 2 * ol.U * np.maximum(pad, least))
        e4m3_close(host(q), each, v, err, "q")
    if residual is not None:
        close(host(ro), r, ol.U * np.abs(r), "residual", res)
