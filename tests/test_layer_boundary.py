"""CPU tests of the operators around a layer's scan: the C entry points refuse bad arguments on
the host before anything is enqueued, the split of the time axis covers it, and the float64
definitions agree with closed forms."""
import ctypes

import numpy as np
import pytest

from oracle import layer as ol
from selective_state_space_mamba_gb300 import _lib
from selective_state_space_mamba_gb300._lib import SsmSelscanArgs, SsmTokens

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or enqueues nothing
FAR = 1 << 40   # the outputs' place, away from the inputs'
INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (_lib.SSM_ERR_INVALID_ARG, _lib.SSM_ERR_UNSUPPORTED, _lib.SSM_ERR_ALIGNMENT,
                                              _lib.SSM_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def conv(lib, step=False, **kw):
    a = dict(x=FAKE, bs=1 << 20, ts=64, w=FAKE, bias=None, sin=None, idx=None, y=FAR, sout=2 * FAR, batch=2, L=8, d=64,
             W=4, act=1, dtype=1)
    a.update(kw)
    f = lib.ssm_conv_step if step else lib.ssm_conv_fwd
    return f(SsmTokens(a["x"], a["bs"], a["ts"]), a["w"], a["bias"], a["sin"], a["idx"], a["y"], a["sout"], a["batch"],
             a["L"], a["d"], a["W"], a["act"], a["dtype"], None)


def test_conv_refusals(lib):
    for step, L in ((False, 8), (True, 2)):
        f = lambda **kw: conv(lib, step, **{"L": L, **kw})  # noqa: B023,E731
        assert f(batch=-1) == INVALID
        assert f(L=-1) == INVALID
        assert f(d=0) == INVALID
        assert f(dtype=2) == INVALID
        assert f(act=7) == INVALID
        assert f(W=1) == UNSUPPORTED and f(W=5) == UNSUPPORTED
        assert f(x=None) == INVALID and f(w=None) == INVALID and f(y=None) == INVALID
        assert f(x=FAKE + 1) == ALIGNMENT and f(w=FAKE + 2) == ALIGNMENT and f(y=FAR + 1) == ALIGNMENT
        assert f(bs=-64) == INVALID                       # a row before the pointer
        assert f(bs=1 << 62) == INVALID                   # spans more than an address
        assert f(y=FAKE + 2 * 10) == INVALID              # the output over the input
        assert f(y=2 * FAR + 2) == INVALID                # one output over the other
        assert f(sin=2 * FAR + 2) == INVALID              # partial overlap of the states
        assert f(batch=70000, **({"L": 70000} if step else {})) == UNSUPPORTED
    assert conv(lib, sin=2 * FAR, sout=2 * FAR) == INVALID      # a prompt does not update in place
    assert conv(lib, True, L=3) == INVALID                      # without slots, a state row for each sequence
    assert conv(lib, True, L=2, sout=None) == INVALID
    assert conv(lib, batch=0) == _lib.SSM_OK and conv(lib, True, batch=0, L=0) == _lib.SSM_OK
    assert conv(lib, L=0, sout=None, x=None, y=None) == _lib.SSM_OK


def scan(lib, step=False, ws=(None, 0), slots=None, nslots=None, **kw):
    a = SsmSelscanArgs()
    v = dict(u=FAKE, dt=FAKE, B=FAKE, C=FAKE, z=None, A=FAKE, D=None, dt_bias=None, h0=None, lens=None, y=FAR,
             h_final=2 * FAR, batch=2, seqlen=64, channels=96, dstate=16, ngroups=1, softplus=1, dtype=1, bs=1 << 20, ts=96)
    v.update(kw)
    for k in ("u", "dt", "B", "C", "z"):
        setattr(a, k, SsmTokens(v[k], v["bs"], v["ts"]))
    for k in ("A", "D", "dt_bias", "h0", "lens", "y", "h_final", "batch", "seqlen", "channels", "dstate", "ngroups",
              "softplus", "dtype"):
        setattr(a, k, v[k])
    if step:
        return lib.ssm_selscan_step(a, slots, v["batch"] if nslots is None else nslots, None)
    return lib.ssm_selscan_fwd(a, ws[0], ws[1], None)


def test_selscan_refusals(lib):
    for step in (False, True):
        f = lambda **kw: scan(lib, step, **kw)  # noqa: B023,E731
        assert f(batch=-1) == INVALID and f(channels=0) == INVALID and f(ngroups=0) == INVALID
        assert f(ngroups=5) == INVALID and f(dtype=3) == INVALID
        assert f(dstate=12) == UNSUPPORTED and f(dstate=0) == UNSUPPORTED and f(batch=65536) == UNSUPPORTED
        for k in ("u", "dt", "B", "C", "A", "y"):
            assert f(**{k: None}) == INVALID, k
        for k in ("u", "dt", "B", "C", "z"):
            assert f(**{k: FAKE + 1}) == ALIGNMENT, k
        for k in ("A", "D", "dt_bias", "h0"):
            assert f(**{k: FAKE + 2}) == ALIGNMENT, k
        assert f(bs=-1) == INVALID and f(bs=1 << 62) == INVALID
        assert f(y=FAKE + 96) == INVALID and f(y=2 * FAR + 4) == INVALID
        assert f(h0=2 * FAR + 4) == INVALID
    assert scan(lib, seqlen=-1) == INVALID
    assert scan(lib, h0=2 * FAR) == INVALID           # a prompt does not update in place
    assert scan(lib, ts=-1) == INVALID
    assert scan(lib, True, nslots=3) == INVALID       # without slots, a state row for each sequence
    assert scan(lib, True, h_final=None) == INVALID
    assert scan(lib, batch=0) == _lib.SSM_OK and scan(lib, True, batch=0) == _lib.SSM_OK
    assert scan(lib, seqlen=0, h_final=None) == _lib.SSM_OK
    assert lib.ssm_selscan_fwd(None, None, 0, None) == INVALID
    assert lib.ssm_selscan_step(None, None, 0, None) == INVALID


def test_selscan_workspace(lib):
    f = lib.ssm_selscan_fwd_workspace_bytes
    for bad in ((-1, 8, 8, 16, 1), (1, -1, 8, 16, 1), (1, 8, 0, 16, 1), (1, 8, 8, 12, 1), (1, 8, 8, 16, 3)):
        assert f(*bad) == 0
    assert f(1, 1, 64, 16, 1) == 0                    # one token: nothing to split
    assert f(64, 4096, 5120, 16, 1) == 0              # chains enough
    need = f(1, 4096, 64, 16, 1)
    assert need > 0 and need % 256 == 0
    a = dict(batch=1, seqlen=4096, channels=64, bs=1 << 30, ts=64, y=FAR)
    assert scan(lib, **a) == WORKSPACE
    assert scan(lib, ws=(3 * FAR, need - 1), **a) == WORKSPACE
    assert scan(lib, ws=(3 * FAR + 16, need), **a) == ALIGNMENT


def norm(lib, fp8=False, **kw):
    a = dict(x=FAKE, xs=64, w=FAKE, res=None, rout=None, y=FAR, scale=2 * FAR, rows=4, d=64, group=0, dtype=1, rdtype=1)
    a.update(kw)
    if fp8:
        return lib.ssm_rmsnorm_fp8_fwd(a["x"], a["xs"], a["w"], a["res"], a["rout"], a["y"], a["scale"], a["rows"], a["d"],
                                       a["group"], 1e-5, a["dtype"], a["rdtype"], None)
    return lib.ssm_rmsnorm_fwd(a["x"], a["xs"], a["w"], a["res"], a["rout"], a["y"], a["rows"], a["d"], 1e-5, a["dtype"],
                               a["rdtype"], None)


def test_rmsnorm_refusals(lib):
    for fp8 in (False, True):
        f = lambda **kw: norm(lib, fp8, **kw)  # noqa: B023,E731
        assert f(rows=-1) == INVALID and f(d=0) == INVALID and f(dtype=4) == INVALID
        assert f(x=None) == INVALID and f(w=None) == INVALID and f(y=None) == INVALID
        assert f(res=FAKE, dtype=0, rdtype=1) == INVALID      # a residual of fewer bits than x
        assert f(rout=3 * FAR) == INVALID                     # residual_out without a residual
        assert f(x=FAKE + 1) == ALIGNMENT and f(w=FAKE + 2) == ALIGNMENT
        assert f(res=FAKE + 2, rdtype=0) == ALIGNMENT
        assert f(y=FAKE + 64) == INVALID                      # the output over the input
        assert f(res=3 * FAR, rout=3 * FAR + 2) == INVALID    # partial overlap of the residuals
        assert f(xs=-64) == INVALID and f(xs=1 << 62) == INVALID
        assert f(rows=1 << 31) == UNSUPPORTED
        assert f(rows=0) == _lib.SSM_OK
    assert norm(lib, True, group=64) == UNSUPPORTED and norm(lib, True, group=-1) == INVALID
    assert norm(lib, True, scale=None) == INVALID and norm(lib, True, scale=FAR + 4) == INVALID


def test_size_limits(lib):
    """Sizes whose columns or items no longer fit the kernels' 32-bit indexes are refused."""
    wide = (1 << 30) + 1
    assert conv(lib, d=wide) == UNSUPPORTED and conv(lib, True, L=2, d=wide) == UNSUPPORTED
    for step in (False, True):
        assert scan(lib, step, channels=wide) == UNSUPPORTED
        assert scan(lib, step, channels=(1 << 26) + 1) == UNSUPPORTED      # channels * dstate
    assert lib.ssm_selscan_fwd_workspace_bytes(1, 8, (1 << 26) + 1, 16, 1) == 0
    assert norm(lib, d=wide) == UNSUPPORTED and norm(lib, True, d=wide) == UNSUPPORTED
    # 65535 sequences of 2^20 channel tiles
    far = dict(y=1 << 50, h_final=1 << 58, dstate=64, channels=1 << 24, batch=65535, seqlen=1, bs=0)
    assert scan(lib, **far) == UNSUPPORTED


def test_struct_layout():
    """The ctypes views have the C structs' sizes and offsets (natural alignment, no padding)."""
    assert ctypes.sizeof(SsmTokens) == 24
    assert SsmSelscanArgs.A.offset == 5 * 24
    assert SsmSelscanArgs.batch.offset == 5 * 24 + 7 * 8
    assert ctypes.sizeof(SsmSelscanArgs) == 5 * 24 + 7 * 8 + 16 + 24


# ------------------------------------------------------------------------------ the definitions

def test_oracle_conv_is_a_convolution():
    r = np.random.default_rng(1)
    x, w, bias, state = r.standard_normal((2, 20, 3)), r.standard_normal((3, 4)), r.standard_normal(3), r.standard_normal((2, 3, 3))
    y, err, s = ol.conv(x, w, bias, state, silu=False)
    for i in range(2):
        for c in range(3):
            full = np.convolve(np.concatenate([state[i, :, c], x[i, :, c]]), w[c, ::-1], mode="valid") + bias[c]
            assert np.allclose(y[i, :, c], full, rtol=1e-13)
    assert np.array_equal(s, x[:, -3:]) and (err > 0).all()
    z, _, _ = ol.conv(x, w, bias, state)
    assert np.allclose(z, y * 0.5 * (1 + np.tanh(y / 2)), rtol=1e-12)


def test_oracle_selscan_closed_forms():
    r = np.random.default_rng(2)
    L, d, N = 12, 2, 3
    u, dt, B, C = r.standard_normal((1, L, d)), r.uniform(0.1, 1, (1, L, d)), r.standard_normal((1, L, 1, N)), r.standard_normal((1, L, 1, N))
    A = -r.uniform(0.1, 2, (d, N))
    h0 = r.standard_normal((1, d, N))
    y, ey, h, eh = ol.selscan(u, dt, A, B, C, h0=h0, softplus=False)
    G = np.cumsum(dt[0], 0)  # the sum over all earlier tokens, each with its own decay
    for t in range(L):
        for c in range(d):
            want = np.exp(A[c] * G[t, c]) * h0[0, c] + sum(
                np.exp(A[c] * (G[t, c] - G[j, c])) * dt[0, j, c] * u[0, j, c] * B[0, j, 0] for j in range(t + 1))
            assert np.isclose(y[0, t, c], want @ C[0, t, 0], rtol=1e-12)
    assert np.allclose(h[0, c], want, rtol=1e-12) and (ey > 0).all() and (eh > 0).all()
    # two groups are two scans
    B2 = r.standard_normal((1, L, 2, N))
    y2, _, h2, _ = ol.selscan(u, dt, A, B2, B2)
    for c in range(2):
        y1, _, h1, _ = ol.selscan(u[..., c : c + 1], dt[..., c : c + 1], A[c : c + 1], B2[:, :, c : c + 1], B2[:, :, c : c + 1])
        assert np.allclose(y1, y2[..., c : c + 1]) and np.allclose(h1[0], h2[0, c : c + 1])


@pytest.mark.parametrize("f32", [True, False])
def test_oracle_bounds_hold_and_mistakes_break_them(f32):
    """A plain f32 evaluation stays within the bounds; one with a rounded state does not."""
    r = np.random.default_rng(3)
    L, d, N = 60, 4, 8
    f = np.float32
    u, dt = r.standard_normal((1, L, d)).astype(f), (r.standard_normal((1, L, d)) - 2).astype(f)
    B, C = r.standard_normal((1, L, 1, N)).astype(f), r.standard_normal((1, L, 1, N)).astype(f)
    A = -np.arange(1, N + 1, dtype=f) * np.ones((d, 1), f)
    y_ref, ey, h_ref, eh = ol.selscan(u, dt, A, B, C)
    h = np.zeros((d, N), f)
    worst_h = 0.0
    for t in range(L):
        delta = np.log1p(np.exp(dt[0, t]))
        h = np.exp(delta[:, None] * A) * h + (delta * u[0, t])[:, None] * B[0, t, 0]
        if not f32:
            h = h.astype(np.float16).astype(f)
        y = (h * C[0, t, 0]).sum(-1)
        worst_h = max(worst_h, float((np.abs(y - y_ref[0, t]) / ey[0, t]).max()))
    worst_h = max(worst_h, float((np.abs(h - h_ref[0]) / eh[0]).max()))
    assert (worst_h < 1) == f32


def test_oracle_rmsnorm():
    r = np.random.default_rng(4)
    x, res, w = r.standard_normal((3, 10)), r.standard_normal((3, 10)), r.standard_normal(10)
    v, err, s = ol.rmsnorm(x, w, res, eps=0.0)
    assert np.allclose(s, x + res) and np.allclose((v / w) ** 2 @ np.ones(10), 10) and (err >= 0).all()


# ------------------------------------------------------------------------------ sizes that 32 bits do not hold

WRAPS = (1 << 32) + 256  # 256 in 32 bits


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_python_sizes_that_wrap_are_refused(dtype):
    """Columns, widths, states, groups: refused as any other size beyond the kernels, not taken for the size that
    is left of them in 32 bits.  (Tensors without memory: the sizes are looked at before the device is.)"""
    import torch
    import selective_state_space_mamba_gb300 as ssm
    t = lambda *n: torch.empty(n, device="meta", dtype=getattr(torch, dtype))  # noqa: E731
    f = lambda *n: torch.empty(n, device="meta")  # noqa: E731
    n = WRAPS
    calls = [
        lambda: ssm.conv_fwd(t(1, 1, n), f(n, 4)), lambda: ssm.conv_fwd(t(1, 1, 8), f(8, (1 << 32) + 4)),
        lambda: ssm.conv_step(t(1, n), f(n, 4)), lambda: ssm.conv_step(t(1, 8), f(8, (1 << 32) + 4)),
        lambda: ssm.selscan_fwd(t(1, 1, n), t(1, 1, n), f(n, 16), t(1, 1, 1, 16), t(1, 1, 1, 16)),
        lambda: ssm.selscan_fwd(t(1, 1, 8), t(1, 1, 8), f(8, n), t(1, 1, 1, n), t(1, 1, 1, n)),
        lambda: ssm.selscan_fwd(t(1, 1, 8), t(1, 1, 8), f(8, 16), t(1, 1, n, 16), t(1, 1, n, 16)),
        lambda: ssm.selscan_step(t(1, n), t(1, n), f(n, 16), t(1, 1, 16), t(1, 1, 16)),
        lambda: ssm.selscan_step(t(1, 8), t(1, 8), f(8, n), t(1, 1, n), t(1, 1, n)),
        lambda: ssm.selscan_step(t(1, 8), t(1, 8), f(8, 16), t(1, n, 16), t(1, n, 16)),
        lambda: ssm.rmsnorm_fwd(t(1, n), f(n)), lambda: ssm.rmsnorm_fp8_fwd(t(1, n), f(n)),
        lambda: ssm.rmsnorm_fp8_fwd(t(1, 8), f(8), group=1 << 32),
        lambda: ssm.rmsnorm_fp8_fwd(t(1, 8), f(8), group=(1 << 32) + 128),
        lambda: ssm.rmsnorm_fp8_fwd(t(1, 8), f(8), group=-(1 << 32)),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ssm.SsmError, match="SSM_ERR_UNSUPPORTED"):
            call()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssm.conv_fwd(t(1, 1, 8), f(8, 4))


def test_selscan_workspace_of_sizes_that_are_refused(lib):
    """0 bytes, as for every other invalid size: more sequences than a call takes (their product with the tiles went
    beyond 64 bits)."""
    f = lib.ssm_selscan_fwd_workspace_bytes
    assert f(65535, 4, 8, 16, 1) == 0
    for batch in (65536, 1 << 40, (1 << 62) + 1, (1 << 63) - 1):
        assert f(batch, 1 << 20, 1 << 16, 16, 1) == 0, batch
    for seqlen in ((1 << 40) + 1, 1 << 62, (1 << 63) - 1):
        assert f(1, seqlen, 8, 16, 1) == 0, seqlen
    assert scan(lib, batch=65536) == UNSUPPORTED
    # one channel of 2^41 tokens: the parts of its time axis have too many
    assert scan(lib, batch=1, seqlen=1 << 41, channels=1, ts=0, y=1 << 58, h_final=1 << 60) == UNSUPPORTED


def test_profile_arrays_of_an_older_header(lib):
    """ssm_profile_end writes the nine kernels it wrote before the layer operators came; ssm_profile_end_n as many as it
    is told."""
    foreign = -7

    def run(call, size):
        ms, n = (ctypes.c_double * size)(*[foreign] * size), (ctypes.c_int64 * size)(*[foreign] * size)
        assert call(ctypes.cast(ms, ctypes.c_void_p), ctypes.cast(n, ctypes.c_void_p)) == _lib.SSM_OK
        written = [a != foreign for a in ms]
        assert written == [a != foreign for a in n] and written == sorted(written, reverse=True)
        return sum(written)

    assert run(lib.ssm_profile_end, 20) == 9
    for k in (0, 3, 9, 15, 18):
        assert run(lambda a, b: lib.ssm_profile_end_n(a, b, k), 20) == k  # noqa: B023
    assert lib.ssm_profile_end_n(None, None, 15) == _lib.SSM_OK and lib.ssm_profile_end(None, None) == _lib.SSM_OK
    assert lib.ssm_profile_end_n(None, None, -1) == INVALID
    assert len(_lib.PROFILE_KERNELS) == 15


def test_python_workspace_sizes_that_wrap(lib):
    """0, as for all sizes that are refused, and not the bytes of what is left of them in 32 bits."""
    import selective_state_space_mamba_gb300 as ssm
    f = ssm.selscan_fwd_workspace_bytes
    assert f(1, 4096, 64, 16, 1) > 0
    assert f(1, 4096, (1 << 32) + 64, 16, 1) == 0 and f(1, 4096, 64, (1 << 32) + 16, 1) == 0
    assert f(1, 4096, 64, 16, (1 << 32) + 1) == 0 and f((1 << 64) + 1, 4096, 64, 16, 1) == 0 and f(1, (1 << 64) + 4096, 64, 16) == 0
    assert f(-1, 4096, 64, 16, 1) == 0 and f(1, 4096, -64, 16, 1) == 0
