"""Python entry points of the operators around a layer's scan (include/ssm.h, the section of
ssm_tokens): the short causal convolution and the selective scan, for prompts and for single
tokens, the root-mean-square norm, the gated delta rule and the norms with a gate and a residual.

Token tensors (x, u, dt, z, B, C, q, k, v, beta) may be strided in all but the last dimension, for example
columns of a projection's wider rows.  The checks of shapes and types, the allocation of outputs
and the C calls are in the compiled module _binding (csrc/binding.cpp), because a call for one
token takes less time on the GPU than they take in Python; it is built in-tree beside the
library, and a call fails loudly where it cannot be.
"""
from __future__ import annotations

import ctypes
import importlib

import torch  # noqa: F401 - _binding needs its libraries loaded

from . import _build, _lib

_BOUND = ("ssm_conv_fwd", "ssm_conv_step", "ssm_selscan_fwd_workspace_bytes", "ssm_selscan_fwd", "ssm_selscan_step",
          "ssm_rmsnorm_fwd", "ssm_rmsnorm_fp8_fwd", "ssm_delta_fwd_workspace_bytes", "ssm_delta_fwd", "ssm_delta_step", "ssm_gatednorm_fwd",
          "ssm_blocknorm_fwd")
_native = None


def _load():
    """The compiled module, bound to the library (both built first where they are missing or stale)."""
    global _native
    lib = _lib.load()
    with _lib._lock:
        if _native is None:
            _build.build_binding()
            mod = importlib.import_module("._binding", __package__)
            mod.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _BOUND))
            _native = mod
    return _native


def _checked(r, where):
    if type(r) is int:  # an ssm_status
        _lib.check(r, where)
    return r


def conv_fwd(x, weight, bias=None, state=None, lens=None, *, silu: bool = True, y=None, state_out=None,
             return_final_state: bool = True):
    """Short causal convolution over a prompt (ssm_conv_fwd).

    x [b, L, d] (float32 or bfloat16, may be strided), weight [d, W] and bias [d] float32 (W 2 .. 4),
    state [b, W - 1, d] like x: the tokens before the prompt, oldest first (None: zeros), lens [b]
    int32: tokens of each sequence (None: L).  Returns (y, state_out): y [b, L, d], 0 in the
    padding, and the state after the prompt (None when return_final_state is False).
    """
    r = (_native or _load()).conv_fwd(x, weight, bias, state, lens, silu, y, state_out, return_final_state)
    return _checked(r, "ssm_conv_fwd")


def conv_step(x, weight, bias=None, state=None, slots=None, *, silu: bool = True, y=None, state_out=None,
              inplace: bool = False):
    """Short causal convolution of one new token per sequence (ssm_conv_step).

    x [b, d]; weight, bias as conv_fwd; state [n, W - 1, d] like x (None: zeros, n = b), slots [b]
    int32: each sequence's row of it (None: its own index, n = b; a row outside 0 .. n - 1 marks an unused
    place).  Returns (y, new state): with ``inplace`` the new state overwrites ``state``, else
    only the named rows of state_out are written.
    """
    r = (_native or _load()).conv_step(x, weight, bias, state, slots, silu, y, state_out, inplace)
    return _checked(r, "ssm_conv_step")


def selscan_fwd_workspace_bytes(batch, seqlen, channels, dstate, ngroups=1) -> int:
    """Device memory that selscan_fwd needs besides its tensors (0 where it needs none, or refuses the sizes)."""
    if max(channels, dstate, ngroups) >> 31 or max(batch, seqlen) >> 63:
        return 0  # ctypes would hand on what is left of them in 32 or 64 bits
    return int(_lib.load().ssm_selscan_fwd_workspace_bytes(batch, seqlen, channels, dstate, ngroups))


def kept_workspace(device_index: int, kind: str = "selscan"):
    """The memory that the last selscan_fwd (kind "delta": delta_fwd) without a workspace allocated, or None (for
    check_device_status)."""
    return (_native or _load()).kept_workspace(device_index, kind == "delta")


def selscan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, lens=None, *, softplus: bool = True, y=None,
                h_final=None, return_final_state: bool = True, workspace=None):
    """Selective scan over a prompt (ssm_selscan_fwd).

    u, dt, z [b, L, d], B, C [b, L, G, N] (all float32 or all bfloat16, may be strided), A [d, N],
    D, dt_bias [d] float32, h0 [b, d, N] float32 (None: zeros), lens [b] int32: tokens of each
    sequence (None: L); N in {8, 16, 32, 64}; channel c reads group c // (d / G).  Returns (y, h_final):
    y [b, L, d], 0 in the padding, and the float32 state after the last token (None when
    return_final_state is False).  Without a workspace (Workspace), one is allocated for the call
    where it is needed.  check_device_status(workspace), or check_device_status(kind="selscan") without
    one, tells whether a wait inside the last call that needed one ran out.
    """
    buf = None
    if workspace is not None:
        b, L, d = u.shape
        buf = workspace.ensure(selscan_fwd_workspace_bytes(b, L, d, A.shape[-1], B.shape[-2]))
    r = (_native or _load()).selscan_fwd(u, dt, A, B, C, D, z, dt_bias, h0, lens, softplus, y, h_final, return_final_state,
                                         buf)
    return _checked(r, "ssm_selscan_fwd")


def selscan_step(u, dt, A, B, C, D=None, z=None, dt_bias=None, state=None, slots=None, *, softplus: bool = True,
                 y=None, state_out=None, inplace: bool = False):
    """Selective scan of one new token per sequence (ssm_selscan_step).

    u, dt, z [b, d], B, C [b, G, N]; A, D, dt_bias as selscan_fwd; state [n, d, N] float32 (None:
    zeros, n = b), slots [b] int32: each sequence's row of it (None: its own index, n = b; a row
    outside 0 .. n - 1 marks an unused place).  Returns (y, new state): with ``inplace`` the new state
    overwrites ``state``, else only the named rows of state_out are written.
    """
    r = (_native or _load()).selscan_step(u, dt, A, B, C, D, z, dt_bias, state, slots, softplus, y, state_out, inplace)
    return _checked(r, "ssm_selscan_step")


def rmsnorm_fwd(x, weight, residual=None, *, eps: float = 1e-5, y=None, residual_out=None):
    """Root-mean-square norm after the residual's addition (ssm_rmsnorm_fwd).

    x [..., d] float32 or bfloat16 (rows may be strided), weight [d] float32, residual like x in
    shape, float32 or x's dtype.  Returns (y, residual_out): y like x, residual_out = x + residual of
    residual's dtype (None without a residual; it may be given as ``residual`` itself, to update it
    in place).
    """
    r = (_native or _load()).rmsnorm_fwd(x, weight, residual, eps, y, residual_out)
    return _checked(r, "ssm_rmsnorm_fwd")


def rmsnorm_fp8_fwd(x, weight, residual=None, *, eps: float = 1e-5, group: int = 0, q=None, scale=None,
                    residual_out=None):
    """rmsnorm_fwd with an output in 8 bits (ssm_rmsnorm_fp8_fwd): returns (q, scale, residual_out).

    q float8_e4m3fn of x's shape; scale float32 [...] (group 0: one a row) or [..., ceil(d / 128)]
    (group 128: one for each 128 columns); q * scale is the norm's value.
    """
    r = (_native or _load()).rmsnorm_fp8_fwd(x, weight, residual, eps, group, q, scale, residual_out)
    return _checked(r, "ssm_rmsnorm_fp8_fwd")


def delta_fwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups=1, *, dtype=torch.bfloat16) -> int:
    """Device memory that delta_fwd needs besides its tensors (0 where it needs none, or refuses the sizes)."""
    if max(nheads, headdim, dstate, ngroups) >> 31 or max(batch, seqlen) >> 63:
        return 0  # ctypes would hand on what is left of them in 32 or 64 bits
    code = _lib.SSM_BF16 if dtype == torch.bfloat16 else _lib.SSM_F32
    return int(_lib.load().ssm_delta_fwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups, code))


def delta_fwd(q, k, v, dt, beta, A, dt_bias=None, h0=None, lens=None, *, scale=None, softplus: bool = True,
              sigmoid: bool = True, l2norm: bool = True, y=None, h_final=None, return_final_state: bool = True,
              workspace=None):
    """Gated delta rule over a prompt (ssm_delta_fwd).

    q, k [b, L, G, N], v [b, L, nh, H], dt, beta [b, L, nh] (all float32 or all bfloat16; strided in all but
    the last dimension, heads and groups of a token adjacent), A, dt_bias [nh] float32, h0 [b, nh, H, N] float32
    (None: zeros), lens [b] int32: tokens of each sequence (None: L); N in {32, 64, 128}; head h reads
    group h // (nh / G).  scale: None for N ** -0.5.  Without softplus the decay is exp(A (dt + dt_bias)), without
    sigmoid beta is taken as it is, without l2norm q and k are.  Returns (y, h_final): y [b, L, nh, H], 0 in
    the padding, and the float32 state after the last token (None when return_final_state is False).
    Long bfloat16 prompts go in chunks through the tensor cores, whose operands leave the state off by about 4e-6 of its size and y by
    1.4e-3 besides its rounding; the same tokens as float32 are computed in float32 throughout.
    Without a workspace (Workspace), one is allocated for the call where it is needed, and kept until the next such call (up to
    1 GiB and two states of all heads).  check_device_status(workspace), or check_device_status(kind="delta") without one,
    tells whether a wait inside the last call that needed one ran out.
    """
    buf = None
    if workspace is not None:
        (b, L, nh, H), (G, N) = v.shape, q.shape[-2:]
        buf = workspace.ensure(delta_fwd_workspace_bytes(b, L, nh, H, N, G, dtype=v.dtype))
    r = (_native or _load()).delta_fwd(q, k, v, dt, beta, A, dt_bias, h0, lens, scale, softplus, sigmoid, l2norm, y, h_final,
                                       return_final_state, buf)
    return _checked(r, "ssm_delta_fwd")


def delta_step(q, k, v, dt, beta, A, dt_bias=None, state=None, slots=None, *, scale=None, softplus: bool = True,
               sigmoid: bool = True, l2norm: bool = True, y=None, state_out=None, inplace: bool = False):
    """Gated delta rule of one new token per sequence (ssm_delta_step).

    q, k [b, G, N], v [b, nh, H], dt, beta [b, nh]; the others as delta_fwd; state [n, nh, H, N] float32 (None:
    zeros, n = b), slots [b] int32: each sequence's row of it (None: its own index, n = b; a row outside
    0 .. n - 1 marks an unused place).  Returns (y, new state): with ``inplace`` the new state overwrites
    ``state``, else only the named rows of state_out are written.
    """
    r = (_native or _load()).delta_step(q, k, v, dt, beta, A, dt_bias, state, slots, scale, softplus, sigmoid, l2norm, y,
                                        state_out, inplace)
    return _checked(r, "ssm_delta_step")


def gatednorm_fwd(x, z, weight, *, group: int = 0, gate_first: bool = False, eps: float = 1e-5, y=None):
    """Root-mean-square norm with a gate (ssm_gatednorm_fwd): rms(x) * weight * silu(z), or with gate_first
    rms(x * silu(z)) * weight.

    x, z [..., d] float32 or bfloat16 (rows may be strided), weight float32 [d], or [group] for all groups; the
    mean square is taken over each ``group`` columns (0: the row), which divide d.  Returns y like x, dense.
    """
    r = (_native or _load()).gatednorm_fwd(x, z, weight, group, gate_first, eps, y)
    return _checked(r, "ssm_gatednorm_fwd")


def blocknorm_fwd(x, weight, residual, next_weight, z=None, *, alpha: float = 1.0, eps: float = 1e-5, y=None,
                  residual_out=None):
    """The norm after a block, the residual, and the norm before the next (ssm_blocknorm_fwd):
    r = alpha * residual + rms(x) * weight [* silu(z)], y = rms(r) * next_weight.

    x, z [..., d] float32 or bfloat16 (rows may be strided), weight, next_weight [d] float32, residual like x in
    shape, float32 or x's dtype.  Returns (y, residual_out): y like x, residual_out = r of residual's dtype (it may be
    given as ``residual`` itself, to update it in place).
    """
    r = (_native or _load()).blocknorm_fwd(x, weight, residual, next_weight, z, alpha, eps, y, residual_out)
    return _checked(r, "ssm_blocknorm_fwd")
