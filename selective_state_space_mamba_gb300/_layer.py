"""Python entry points of the operators around a layer's scan (include/ssm.h, the section of
ssm_tokens): the short causal convolution and the selective scan, for prompts and for single
tokens, and the root-mean-square norm.

They check shapes and types, allocate the outputs on the current stream and enqueue the library's
kernels there.  Token tensors (x, u, dt, z, B, C) may be strided in all but the last dimension,
for example columns of a projection's wider rows.
"""
from __future__ import annotations

import struct

import torch

from . import _lib
from ._lib import SsmSelscanArgs, SsmTokens

_CODE = {torch.float32: _lib.SSM_F32, torch.bfloat16: _lib.SSM_BF16}
_F32, _I32 = torch.float32, torch.int32
_SELSCAN = struct.Struct("@15q7q2q6i")  # ssm_selscan_args, filled in one go: a third of the time of its fields one by one

# A call of one token takes a few microseconds on the GPU, so what stands here is kept short: the
# stream is asked for as a number, and a tensor is checked with the fewest questions.
_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty
_library = None


def _lib_handle():
    global _library
    if _library is None:
        _library = _lib.load()
    return _library


def _code(t) -> int:
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _fail(name, want):
    raise ValueError(f"{name} must be {want}")


def _device(name, t) -> int:
    dev = t.get_device()
    if dev < 0:
        _fail(name, "a CUDA tensor")
    return dev


def _tokens(name, t, shape, dtype, dev):
    """Pointer and strides of a token tensor, strided in all but its last dimension."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _fail(name, f"a CUDA tensor {list(shape)} of {dtype}, on the first one's device")
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        _fail(name, "contiguous in its last dimension")
    return t.data_ptr(), s[0], s[1]


def _groups(name, t, shape, dtype, dev):
    """The same for B or C [..., groups, states], a token's groups adjacent."""
    if shape[-2] > 1 and t.dim() == len(shape) and t.stride(-2) != shape[-1]:
        _fail(name, "contiguous in its last two dimensions")
    return _tokens(name, t, shape, dtype, dev)


def _dense(name, t, shape, dtype, dev):
    """Pointer of a dense tensor."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        _fail(name, f"a contiguous CUDA tensor {list(shape)} of {dtype}, on the first one's device")
    return t.data_ptr()


def _out(name, t, shape, dtype, like, dev):
    """An output, the caller's or a new one, and its pointer."""
    if t is None:
        t = _empty(shape, dtype=dtype, device=like.device)
        return t, t.data_ptr()
    return t, _dense(name, t, shape, dtype, dev)


def _opt(name, t, shape, dtype, dev):
    return 0 if t is None else _dense(name, t, shape, dtype, dev)


def conv_fwd(x, weight, bias=None, state=None, lens=None, *, silu: bool = True, y=None, state_out=None,
             return_final_state: bool = True):
    """Short causal convolution over a prompt (ssm_conv_fwd).

    x [b, L, d] (float32 or bfloat16, may be strided), weight [d, W] and bias [d] float32 (W 2 .. 4),
    state [b, W - 1, d] like x: the tokens before the prompt, oldest first (None: zeros), lens [b]
    int32: tokens of each sequence (None: L).  Returns (y, state_out): y [b, L, d], 0 in the
    padding, and the state after the prompt (None when return_final_state is False).
    """
    code, dtype = _code(x), x.dtype
    if x.dim() != 3 or weight.dim() != 2:
        _fail("x, weight", "[b, L, d] and [d, W]")
    b, L, d = shape = x.shape
    W = weight.shape[1]
    dev = _device("x", x)
    xt = SsmTokens(*_tokens("x", x, shape, dtype, dev))
    sshape = (b, W - 1, d)
    y, yp = _out("y", y, shape, dtype, x, dev)
    state_out, sp = _out("state_out", state_out, sshape, dtype, x, dev) if return_final_state else (None, 0)
    st = _lib_handle().ssm_conv_fwd(
        xt, _dense("weight", weight, (d, W), _F32, dev), _opt("bias", bias, (d,), _F32, dev),
        _opt("state", state, sshape, dtype, dev), _opt("lens", lens, (b,), _I32, dev), yp, sp, b, L, d, W, 1 if silu else 0, code, _stream(dev))
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
    code, dtype = _code(x), x.dtype
    if x.dim() != 2 or weight.dim() != 2:
        _fail("x, weight", "[b, d] and [d, W]")
    b, d = shape = x.shape
    W = weight.shape[1]
    dev = _device("x", x)
    xt = SsmTokens(*_tokens("x", x, shape, dtype, dev))
    state_out, n = _step_states(state, state_out, inplace, slots, b, (W - 1, d), dtype, x.device)
    sshape = (n, W - 1, d)
    y, yp = _out("y", y, shape, dtype, x, dev)
    st = _lib_handle().ssm_conv_step(
        xt, _dense("weight", weight, (d, W), _F32, dev), _opt("bias", bias, (d,), _F32, dev),
        _opt("state", state, sshape, dtype, dev), _opt("slots", slots, (b,), _I32, dev), yp,
        _dense("state_out", state_out, sshape, dtype, dev), b, n, d, W, 1 if silu else 0, code, _stream(dev))
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
        return _empty((b, *inner), dtype=dtype, device=device), b
    # rows that no slot names keep what they hold
    return (torch.empty_like(state) if slots is None else state.clone()), state.shape[0]


def selscan_fwd_workspace_bytes(batch, seqlen, channels, dstate, ngroups=1) -> int:
    """Device memory that selscan_fwd needs besides its tensors (0 where the time axis is not split)."""
    return int(_lib_handle().ssm_selscan_fwd_workspace_bytes(batch, seqlen, channels, dstate, ngroups))


def _selscan_inputs(u, dt, A, B, C, D, z, dt_bias, dev):
    """What selscan_fwd and selscan_step share: the head of ssm_selscan_args, groups and states."""
    dtype, shape = u.dtype, u.shape
    d = shape[-1]
    bshape = B.shape
    if bshape[:-2] != shape[:-1]:
        _fail("B", f"[{', '.join(map(str, shape[:-1]))}, groups, states]")
    G, N = bshape[-2:]
    head = (*_tokens("u", u, shape, dtype, dev), *_tokens("dt", dt, shape, dtype, dev),
            *_groups("B", B, bshape, dtype, dev), *_groups("C", C, bshape, dtype, dev),
            *((0, 0, 0) if z is None else _tokens("z", z, shape, dtype, dev)), _dense("A", A, (d, N), _F32, dev),
            _opt("D", D, (d,), _F32, dev), _opt("dt_bias", dt_bias, (d,), _F32, dev))
    return head, G, N


def selscan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lens=None, *, softplus: bool = True, y=None,
                h_final=None, return_final_state: bool = True, workspace=None):
    """Selective scan over a prompt (ssm_selscan_fwd).

    u, dt, z [b, L, d], B, C [b, L, G, N] (all float32 or all bfloat16, may be strided), A [d, N],
    D, dt_bias [d] float32, h0 [b, d, N] float32 (None: zeros), lens [b] int32: tokens of each
    sequence (None: L); N in {8, 16, 32, 64}; channel c reads group c // (d / G).  Returns (y, h_final): y [b, L, d], 0
    in the padding, and the float32 state after the last token (None when return_final_state is
    False).  Without a workspace (Workspace), one is allocated for the call where it is needed.
    """
    if u.dim() != 3 or B.dim() != 4:
        _fail("u, B", "[b, L, d] and [b, L, G, N]")
    code, dtype, dev = _code(u), u.dtype, _device("u", u)
    b, L, d = shape = u.shape
    head, G, N = _selscan_inputs(u, dt, A, B, C, D, z, dt_bias, dev)
    y, yp = _out("y", y, shape, dtype, u, dev)
    h_final, hp = _out("h_final", h_final, (b, d, N), _F32, u, dev) if return_final_state else (None, 0)
    args = SsmSelscanArgs.from_buffer_copy(_SELSCAN.pack(
        *head, _opt("h0", h0, (b, d, N), _F32, dev), _opt("lens", lens, (b,), _I32, dev), yp, hp, b, L, d, N, G, 1 if softplus else 0, code, 0))
    lib = _lib_handle()
    need = lib.ssm_selscan_fwd_workspace_bytes(b, L, d, N, G)
    if workspace is not None:
        workspace.ensure(need)
        buf, have = workspace.buf, workspace.nbytes
    else:
        buf, have = _empty(need, dtype=torch.uint8, device=u.device) if need else None, need
    st = lib.ssm_selscan_fwd(args, None if buf is None else buf.data_ptr(), have, _stream(dev))
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
    if u.dim() != 2 or B.dim() != 3:
        _fail("u, B", "[b, d] and [b, G, N]")
    code, dtype, dev = _code(u), u.dtype, _device("u", u)
    b, d = shape = u.shape
    head, G, N = _selscan_inputs(u, dt, A, B, C, D, z, dt_bias, dev)
    state_out, n = _step_states(state, state_out, inplace, slots, b, (d, N), _F32, u.device)
    y, yp = _out("y", y, shape, dtype, u, dev)
    args = SsmSelscanArgs.from_buffer_copy(_SELSCAN.pack(
        *head, _opt("state", state, (n, d, N), _F32, dev), 0, yp,
        _dense("state_out", state_out, (n, d, N), _F32, dev), b, 1, d, N, G, 1 if softplus else 0, code, 0))
    st = _lib_handle().ssm_selscan_step(args, _opt("slots", slots, (b,), _I32, dev), n, _stream(dev))
    if st:
        _lib.check(st, "ssm_selscan_step")
    return y, state_out


def _norm_args(x, weight, residual, residual_out):
    code = _code(x)
    dev = _device("x", x)
    shape = x.shape
    d = shape[-1] if shape else 0
    rows = x.numel() // d if d else 0
    if x.is_contiguous():
        stride = d
    elif x.stride(-1) != 1 and d != 1:
        _fail("x", "contiguous in its last dimension")
    else:
        stride = (x if x.dim() == 2 else x.view(rows, d)).stride(0)
    w = _dense("weight", weight, (d,), _F32, dev)
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        return code, code, d, rows, stride, w, 0, 0, None, dev
    rdtype = residual.dtype
    if rdtype is not _F32 and rdtype is not x.dtype:
        _fail("residual", f"of float32 or {x.dtype}")
    rp = _dense("residual", residual, shape, rdtype, dev)
    residual_out, rop = _out("residual_out", residual_out, shape, rdtype, x, dev)
    return code, _CODE[rdtype], d, rows, stride, w, rp, rop, residual_out, dev


def rmsnorm_fwd(x, weight, residual=None, *, eps: float = 1e-5, y=None, residual_out=None):
    """Root-mean-square norm after the residual's addition (ssm_rmsnorm_fwd).

    x [..., d] float32 or bfloat16 (rows may be strided), weight [d] float32, residual like x in
    shape, float32 or x's dtype.  Returns (y, residual_out): y like x, residual_out = x + residual of residual's dtype
    (None without a residual; it may be given as ``residual`` itself, to update it in place).
    """
    code, rcode, d, rows, stride, w, rp, rop, residual_out, dev = _norm_args(x, weight, residual, residual_out)
    y, yp = _out("y", y, x.shape, x.dtype, x, dev)
    st = _lib_handle().ssm_rmsnorm_fwd(x.data_ptr(), stride, w, rp, rop, yp, rows, d, eps, code, rcode, _stream(dev))
    if st:
        _lib.check(st, "ssm_rmsnorm_fwd")
    return y, residual_out


def rmsnorm_fp8_fwd(x, weight, residual=None, *, eps: float = 1e-5, group: int = 0, q=None, scale=None,
                    residual_out=None):
    """rmsnorm_fwd with an output in 8 bits (ssm_rmsnorm_fp8_fwd): returns (q, scale, residual_out).

    q float8_e4m3fn of x's shape; scale float32 [...] (group 0: one a row) or [..., ceil(d / 128)]
    (group 128: one for each 128 columns); q * scale is the norm's value.
    """
    code, rcode, d, rows, stride, w, rp, rop, residual_out, dev = _norm_args(x, weight, residual, residual_out)
    sshape = x.shape[:-1] if group == 0 else (*x.shape[:-1], -(-d // 128))
    q, qp = _out("q", q, x.shape, torch.float8_e4m3fn, x, dev)
    scale, sp = _out("scale", scale, sshape, _F32, x, dev)
    st = _lib_handle().ssm_rmsnorm_fp8_fwd(x.data_ptr(), stride, w, rp, rop, qp, sp, rows, d, group, eps, code, rcode,
                                           _stream(dev))
    if st:
        _lib.check(st, "ssm_rmsnorm_fp8_fwd")
    return q, scale, residual_out
