"""The other recurrent layers of a hybrid model: the binding of kda_conv_fwd,
kda_ssm_fwd and kda_ssm_step (include/kda.h).

A recurrent layer convolves its projected rows over a few tokens first (KDA's q, k
and v, a state-space layer's x, B and C); a state-space layer then keeps a matrix
state per head with one decay per token.  Both work on the packed rows of the KDA
calls (cu_seqlens) and carry their states from call to call.  Rows may be cut out of
wider ones: x, dt, B and C need to be contiguous but for their first dimension.
"""
from __future__ import annotations

import ctypes

from . import attention as _attention


class _ConvOptions(ctypes.Structure):
    _fields_ = [("x_stride", ctypes.c_int64), ("silu", ctypes.c_int32)]


class _SsmOptions(ctypes.Structure):
    _fields_ = [("x_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("c_stride", ctypes.c_int64),
                ("skip", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("state_dtype", ctypes.c_int32)]


def declare(lib):
    """Argument types of the entry points of this module."""
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    lib.kda_conv_fwd.argtypes = [P, P, P, P, P, P, i64, i32, i32, i32, P, P, P]
    lib.kda_conv_fwd.restype = ctypes.c_int
    lib.kda_ssm_step.argtypes = [P, P, P, P, P, P, P, P, i64, i32, i32, i32, i32, i32, P, P, P]
    lib.kda_ssm_step.restype = ctypes.c_int
    lib.kda_ssm_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.kda_ssm_workspace_size.restype = sz
    lib.kda_ssm_fwd.argtypes = [P, P, P, P, P, P, P, P, i64, i32, i32, i32, i32, i32, P, P, P, sz, P]
    lib.kda_ssm_fwd.restype = ctypes.c_int


def kda_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None, N=None, silu=True,
                 out=None, final_state=None, stream=None, output_final_state=True):
    """Causal convolution of 2 to 4 taps per channel over packed rows: x [T_total, C]
    bf16, C a multiple of 8, weight [C, W] and bias [C] bf16, SiLU after it unless silu is
    False.  initial_state [N, W - 1, C] bf16: the rows before every sequence (None:
    zeros); final_state, the same at its end, may be initial_state itself.  For prompts
    and single tokens.  Returns (out, final_state)."""
    b = _attention._binding or _attention.load_binding()
    return _attention._run(stream, "kda_conv_fwd", b.conv_fwd, x, weight, bias, initial_state, cu_seqlens, N,
                           silu, out, final_state, output_final_state)


def kda_ssm_fwd(x, dt, A, B, C, skip=None, dt_bias=None, initial_state=None, cu_seqlens=None, N=None,
                out=None, final_state=None, workspace=None, stream=None, output_final_state=True):
    """State-space recurrence over packed prompts: x [T_total, H, P], dt [T_total, H], B and
    C [T_total, G, S] bf16, G dividing H, P and S 64 or 128; A, skip, dt_bias fp32 [H], A
    not positive.  Per head, with d = softplus(dt + dt_bias): M = exp(A d) M + d x B^T,
    out = M C + skip x.  States [N, H, P, S] fp32 or bf16 (both the same; the final state is
    allocated with the initial state's dtype, fp32 without one); final_state may be
    initial_state itself.  The weights between tokens and the copy of the state that the outputs
    read are rounded to bf16 once (kda_ssm_step rounds neither); the state and what tokens add to
    it are fp32 whichever state is taken.  Returns (out, final_state)."""
    b = _attention._binding or _attention.load_binding()
    return _attention._run(stream, "kda_ssm_fwd", b.ssm_fwd, x, dt, A, B, C, skip, dt_bias, initial_state,
                           cu_seqlens, N, out, final_state, output_final_state, workspace)


def kda_ssm_step(x, dt, A, B, C, skip=None, dt_bias=None, initial_state=None, cu_seqlens=None, N=None,
                 out=None, final_state=None, stream=None, output_final_state=True):
    """The same token by token with the state in registers, for one or a few tokens
    per sequence.  Returns (out, final_state)."""
    b = _attention._binding or _attention.load_binding()
    return _attention._run(stream, "kda_ssm_step", b.ssm_step, x, dt, A, B, C, skip, dt_bias, initial_state,
                           cu_seqlens, N, out, final_state, output_final_state, None)
