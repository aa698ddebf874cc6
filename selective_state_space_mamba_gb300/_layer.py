"""Python entry points of the operators around a layer's scan (include/ssm.h, the section of
ssm_tokens): the short causal convolution and the selective scan, for prompts and for single
tokens, and the root-mean-square norm.

They check shapes and types, allocate the outputs on the current stream and enqueue the library's
kernels there.  Token tensors (x, u, dt, z, B, C) may be strided in all but the last dimension,
for example columns of a projection's wider rows.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import SsmSelscanArgs, SsmTokens

_CODE = {torch.float32: _lib.SSM_F32, torch.bfloat16: _lib.SSM_BF16}


def _code(t) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _stream(t) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _fail(name, want):
    raise ValueError(f"{name} must be {want}")


def _tokens(name, t, shape, dtype) -> SsmTokens:
    """A strided token tensor [batch, (seqlen,) channels] or, for B and C, [..., groups, states]."""
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        _fail(name, f"a CUDA tensor {list(shape)} of {dtype}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        _fail(name, "contiguous in its last dimension")
    return SsmTokens(t.data_ptr(), s[0], s[1])


def _groups(name, t, lead, dtype):
    """B or C [*lead, groups, states], a token's groups adjacent; returns (tokens, groups, states)."""
    if t.dim() != len(lead) + 2 or t.shape[:-2] != lead:
        _fail(name, f"[{', '.join(map(str, lead))}, groups, states]")
    G, N = t.shape[-2:]
    if G > 1 and t.stride(-2) != N:
        _fail(name, "contiguous in its last two dimensions")
    return _tokens(name, t, t.shape, dtype), G, N


def _dense(name, t, shape, dtype):
    """Pointer of an optional dense tensor."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        _fail(name, f"a contiguous CUDA tensor {list(shape)} of {dtype}")
    return t.data_ptr()


def conv_fwd(x, weight, bias=None, state=None, lens=None, *, silu: bool = True, y=None, state_out=None,
             return_final_state: bool = True):
    """Short causal convolution over a prompt (ssm_conv_fwd).

    x [b, L, d] (float32 or bfloat16, may be strided), weight [d, W] and bias [d] float32 (W 2 .. 4),
    state [b, W - 1, d] like x: the tokens before the prompt, oldest first (None: zeros), lens [b]
    int32: tokens of each sequence (None: L).  Returns (y, state_out): y [b, L, d], 0 in the
    padding, and the state after the prompt (None when return_final_state is False).
    """
    lib = _lib.load()
    code, dtype = _code(x), x.dtype
    if x.dim() != 3 or weight.dim() != 2:
        _fail("x, weight", "[b, L, d] and [d, W]")
    b, L, d = shape = x.shape
    W = weight.shape[1]
    xt = _tokens("x", x, shape, dtype)
    sshape = (b, W - 1, d)
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=x.device)
    if not return_final_state:
        state_out = None
    elif state_out is None:
        state_out = torch.empty(sshape, dtype=dtype, device=x.device)
    st = lib.ssm_conv_fwd(xt, _dense("weight", weight, (d, W), torch.float32), _dense("bias", bias, (d,), torch.float32),
                          _dense("state", state, sshape, dtype), _dense("lens", lens, (b,), torch.int32),
                          _dense("y", y, shape, dtype), _dense("state_out", state_out, sshape, dtype), b, L, d, W,
                          1 if silu else 0, code, _stream(x))
    if st:
        _lib.check(st, "ssm_conv_fwd")
    return y, state_out


def conv_step(x, weight, bias=None, state=None, slots=None, *, silu: bool = True, y=None, state_out=None,
              inplace: bool = False):
    """Short causal convolution of one new token per sequence (ssm_conv_step).

    x [b, d]; weight, bias as conv_fwd; state [n, W - 1, d] like x (None: zeros, n = b), slots [b]
    int32: each sequence's row of it (None: its own index, n = b; a row outside 0 .. n - 1 marks an unused
    place).  Returns (y, new state): with ``inplace`` the new state overwrites ``state``, else
    only the named rows of state_out are written.
    """
    lib = _lib.load()
    code, dtype = _code(x), x.dtype
    if x.dim() != 2 or weight.dim() != 2:
        _fail("x, weight", "[b, d] and [d, W]")
    b, d = shape = x.shape
    W = weight.shape[1]
    xt = _tokens("x", x, shape, dtype)
    state_out, n = _step_states(state, state_out, inplace, slots, b, (W - 1, d), dtype, x.device)
    sshape = (n, W - 1, d)
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=x.device)
    st = lib.ssm_conv_step(xt, _dense("weight", weight, (d, W), torch.float32),
                           _dense("bias", bias, (d,), torch.float32), _dense("state", state, sshape, dtype),
                           _dense("slots", slots, (b,), torch.int32), _dense("y", y, shape, dtype),
                           _dense("state_out", state_out, sshape, dtype), b, n, d, W, 1 if silu else 0, code, _stream(x))
    if st:
        _lib.check(st, "ssm_conv_step")
    return y, state_out


def _step_states(state, state_out, inplace, slots, b, inner, dtype, device):
    """The state a step writes, and its number of rows."""
    if inplace:
        if state is None or state_out is not None:
            raise ValueError("inplace needs a state and no state_out")
        return state, state.shape[0]
    if state_out is not None:
        return state_out, state_out.shape[0]
    if state is None:
        if slots is not None:
            raise ValueError("slots need a state or a state_out")
        return torch.empty((b, *inner), dtype=dtype, device=device), b
    # rows that no slot names keep what they hold
    return (torch.empty_like(state) if slots is None else state.clone()), state.shape[0]


def selscan_fwd_workspace_bytes(batch, seqlen, channels, dstate, ngroups=1) -> int:
    """Device memory that selscan_fwd needs besides its tensors (0 where the time axis is not split)."""
    return int(_lib.load().ssm_selscan_fwd_workspace_bytes(batch, seqlen, channels, dstate, ngroups))


def _selscan_args(u, dt, A, B, C, D, z, dt_bias, softplus):
    """The arguments that selscan_fwd and selscan_step share."""
    a = SsmSelscanArgs()
    dtype, shape = u.dtype, u.shape
    a.dtype = _code(u)
    d = shape[-1]
    a.u = _tokens("u", u, shape, dtype)
    a.dt = _tokens("dt", dt, shape, dtype)
    a.B, G, N = _groups("B", B, shape[:-1], dtype)
    a.C, GC, NC = _groups("C", C, shape[:-1], dtype)
    if GC != G or NC != N:
        _fail("C", "of B's shape")
    if z is not None:
        a.z = _tokens("z", z, shape, dtype)
    a.A = _dense("A", A, (d, N), torch.float32)
    a.D = _dense("D", D, (d,), torch.float32)
    a.dt_bias = _dense("dt_bias", dt_bias, (d,), torch.float32)
    a.channels, a.dstate, a.ngroups, a.softplus = d, N, G, 1 if softplus else 0
    a.batch = shape[0]
    return a


def selscan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lens=None, *, softplus: bool = True, y=None,
                h_final=None, return_final_state: bool = True, workspace=None):
    """Selective scan over a prompt (ssm_selscan_fwd).

    u, dt, z [b, L, d], B, C [b, L, G, N] (all float32 or all bfloat16, may be strided), A [d, N],
    D, dt_bias [d] float32, h0 [b, d, N] float32 (None: zeros), lens [b] int32: tokens of each
    sequence (None: L); N in {8, 16, 32, 64}; channel c reads group c // (d / G).  Returns (y, h_final): y [b, L, d], 0
    in the padding, and the float32 state after the last token (None when return_final_state is
    False).  Without a workspace (Workspace), one is allocated for the call where it is needed.
    """
    if u.dim() != 3 or A.dim() != 2:
        _fail("u, A", "[b, L, d] and [d, N]")
    lib = _lib.load()
    b, L, d = shape = u.shape
    a = _selscan_args(u, dt, A, B, C, D, z, dt_bias, softplus)
    N = a.dstate
    if y is None:
        y = torch.empty(shape, dtype=u.dtype, device=u.device)
    if not return_final_state:
        h_final = None
    elif h_final is None:
        h_final = torch.empty((b, d, N), dtype=torch.float32, device=u.device)
    a.seqlen = L
    a.h0 = _dense("h0", h0, (b, d, N), torch.float32)
    a.lens = _dense("lens", lens, (b,), torch.int32)
    a.y = _dense("y", y, shape, u.dtype)
    a.h_final = _dense("h_final", h_final, (b, d, N), torch.float32)
    need = lib.ssm_selscan_fwd_workspace_bytes(b, L, d, N, a.ngroups)
    if workspace is not None:
        workspace.ensure(need)
        buf, have = workspace.buf, workspace.nbytes
    else:
        buf, have = torch.empty(need, dtype=torch.uint8, device=u.device) if need else None, need
    st = lib.ssm_selscan_fwd(a, None if buf is None else buf.data_ptr(), have, _stream(u))
    if st:
        _lib.check(st, "ssm_selscan_fwd")
    return y, h_final


def selscan_step(u, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, slots=None, *, softplus: bool = True,
                 y=None, state_out=None, inplace: bool = False):
    """Selective scan of one new token per sequence (ssm_selscan_step).

    u, dt, z [b, d], B, C [b, G, N]; A, D, dt_bias as selscan_fwd; state [n, d, N] float32 (None:
    zeros, n = b), slots [b] int32: each sequence's row of it (None: its own index, n = b; a row
    outside 0 .. n - 1 marks an unused place).  Returns (y, new state): with ``inplace`` the new state
    overwrites ``state``, else only the named rows of state_out are written.
    """
    if u.dim() != 2 or A.dim() != 2:
        _fail("u, A", "[b, d] and [d, N]")
    lib = _lib.load()
    b, d = shape = u.shape
    a = _selscan_args(u, dt, A, B, C, D, z, dt_bias, softplus)
    N = a.dstate
    state_out, n = _step_states(state, state_out, inplace, slots, b, (d, N), torch.float32, u.device)
    if y is None:
        y = torch.empty(shape, dtype=u.dtype, device=u.device)
    a.h0 = _dense("state", state, (n, d, N), torch.float32)
    a.h_final = _dense("state_out", state_out, (n, d, N), torch.float32)
    a.y = _dense("y", y, shape, u.dtype)
    st = lib.ssm_selscan_step(a, _dense("slots", slots, (b,), torch.int32), n, _stream(u))
    if st:
        _lib.check(st, "ssm_selscan_step")
    return y, state_out


def _norm_args(x, weight, residual, residual_out):
    code = _code(x)
    d = x.shape[-1] if x.dim() else 0
    if not x.is_cuda:
        _fail("x", "a CUDA tensor")
    rows = x.numel() // d if d else 0
    if x.is_contiguous():
        stride = d
    elif x.dim() == 2 and (x.stride(1) == 1 or d == 1):
        stride = x.stride(0)
    else:
        stride = x.view(rows, d).stride(0) if x.stride(-1) == 1 or d == 1 else _fail("x", "contiguous in its last dimension")
    w = _dense("weight", weight, (d,), torch.float32)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return code, code, d, rows, stride, w, None, None, None
    if residual.dtype != torch.float32 and residual.dtype != x.dtype:
        _fail("residual", f"of float32 or {x.dtype}")
    if residual_out is None:
        residual_out = torch.empty_like(residual, memory_format=torch.contiguous_format)
    return (code, _CODE[residual.dtype], d, rows, stride, w, _dense("residual", residual, x.shape, residual.dtype),
            _dense("residual_out", residual_out, x.shape, residual.dtype), residual_out)


def rmsnorm_fwd(x, weight, residual=None, *, eps: float = 1e-5, y=None, residual_out=None):
    """Root-mean-square norm after the residual's addition (ssm_rmsnorm_fwd).

    x [..., d] float32 or bfloat16 (rows may be strided), weight [d] float32, residual like x in
    shape, float32 or x's dtype.  Returns (y, residual_out): y like x, residual_out = x + residual of residual's dtype
    (None without a residual; it may be given as ``residual`` itself, to update it in place).
    """
    lib = _lib.load()
    code, rcode, d, rows, stride, w, rp, rop, residual_out = _norm_args(x, weight, residual, residual_out)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    st = lib.ssm_rmsnorm_fwd(x.data_ptr(), stride, w, rp, rop, _dense("y", y, x.shape, x.dtype), rows, d, eps, code, rcode,
                             _stream(x))
    if st:
        _lib.check(st, "ssm_rmsnorm_fwd")
    return y, residual_out


def rmsnorm_fp8_fwd(x, weight, residual=None, *, eps: float = 1e-5, group: int = 0, q=None, scale=None,
                    residual_out=None):
    """rmsnorm_fwd with an output in 8 bits (ssm_rmsnorm_fp8_fwd): returns (q, scale, residual_out).

    q float8_e4m3fn of x's shape; scale float32 [...] (group 0: one a row) or [..., ceil(d / 128)]
    (group 128: one for each 128 columns); q * scale is the norm's value.
    """
    lib = _lib.load()
    code, rcode, d, rows, stride, w, rp, rop, residual_out = _norm_args(x, weight, residual, residual_out)
    sshape = x.shape[:-1] if group == 0 else (*x.shape[:-1], -(-d // 128))
    if q is None:
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if scale is None:
        scale = torch.empty(sshape, dtype=torch.float32, device=x.device)
    st = lib.ssm_rmsnorm_fp8_fwd(x.data_ptr(), stride, w, rp, rop, _dense("q", q, x.shape, torch.float8_e4m3fn),
                                 _dense("scale", scale, sshape, torch.float32), rows, d, group, eps, code, rcode,
                                 _stream(x))
    if st:
        _lib.check(st, "ssm_rmsnorm_fp8_fwd")
    return q, scale, residual_out
