"""The operators around the recurrence (C ABI in ``include/kda_layer.h``): the short causal
convolution, the query/key norm with rotation and the selective state space scan.

Marshalling only, like the rest of the package: a small extension module (``csrc/layer_binding.cpp``)
describes the tensors, allocates what was not given and calls the library.  Every call runs with the
device of its first tensor current, on that device's current stream unless one is given; outputs and
workspaces it allocates are allocated on that stream.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

_activations = {None: 0, "none": 0, "silu": 1}
_norms = {None: 0, "none": 0, "rms": 1, "l2": 2}
_layouts = {"half": 0, "interleaved": 1}
_ext = None


def bind(lib) -> None:
    """Argument types of the functions for callers of the C ABI (descriptor addresses as integers)."""
    V, I = ctypes.c_void_p, ctypes.c_int32
    for name, args in (("kda_conv", [V] * 7 + [I, V]), ("kda_conv_decode", [V] * 7 + [I, I, V]),
                       ("kda_qk_norm", [V] * 10), ("kda_ssm_prefill", [V] * 11),
                       ("kda_ssm_workspace_size", [V] * 11),
                       ("kda_ssm_prefill_ws", [V] * 11 + [ctypes.c_size_t, V]),
                       ("kda_ssm_decode", [V] * 9 + [I, V, V])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def _binding():
    """The extension module, attached to the loaded library."""
    global _ext
    import torch

    from . import KdaError, load_library
    if not torch.cuda.is_available():
        raise RuntimeError("gated_delta_rule_38_amd needs a ROCm GPU (gfx950); none is visible")
    lib = load_library()
    try:
        from . import _layer_binding as ext
    except ImportError as e:
        raise ImportError(f"{e}: build it with `python -m gated_delta_rule_38_amd.build`") from e
    ext.attach(KdaError, torch._C._cuda_getCurrentRawStream,
               *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                 for name in ("kda_conv", "kda_conv_decode", "kda_qk_norm", "kda_ssm_workspace_size",
                              "kda_ssm_prefill_ws", "kda_ssm_decode", "kda_last_error")))
    _ext = ext
    return ext


def _on(stream, x):
    """The context that makes ``stream`` (a torch.cuda.Stream or a raw handle) current."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device)
    elif stream.device != x.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
    return torch.cuda.stream(stream)


def _lookup(table, key, what):
    try:
        return table[key]
    except KeyError:
        raise ValueError(f"{what} must be one of {sorted(str(k) for k in table)}, got {key!r}") from None


def conv(x, weight, bias=None, initial_state=None, cu_seqlens=None, out=None, final_state=None,
         output_final_state: bool = True, activation: Optional[str] = None, stream=None) -> Tuple:
    """Short causal depthwise convolution of prompts.  Returns (out, final_state).

    ``x``: dense [B, T, C], or packed [T, C] with int32 ``cu_seqlens`` [N + 1] on the GPU.
    ``weight`` [C, W] (W in 2..4, the last column meets the current token), ``bias`` [C] or None;
    ``activation``: None or "silu".  States [N, W - 1, C]: the inputs before the first token, oldest
    first; ``final_state`` may be ``initial_state`` itself.  A final state allocated here has
    ``initial_state``'s dtype, or x's.
    """
    args = (x, weight, bias, initial_state, cu_seqlens, out, final_state, output_final_state,
            _lookup(_activations, activation, "activation"))
    if stream is not None:
        with _on(stream, x):
            return (_ext or _binding()).conv(*args)
    return (_ext or _binding()).conv(*args)


def conv_decode(x, weight, state_pool, state_indices, num_tokens=None, bias=None, out=None,
                update_state: bool = True, write_out: bool = True, activation: Optional[str] = None, stream=None):
    """The convolution over 1..8 tokens per request against a pool of states.  Returns out or None.

    ``x`` [R, T, C]; ``state_pool`` [P, W - 1, C]; ``state_indices`` and ``num_tokens`` int32 [R] on
    the GPU, with ``decode``'s meaning (a slot outside [0, P) skips the request).
    ``update_state=False`` only reads the pool (verify); ``write_out=False`` only commits.
    """
    args = (x, weight, bias, state_pool, state_indices, num_tokens, out, write_out, update_state,
            _lookup(_activations, activation, "activation"))
    if stream is not None:
        with _on(stream, x):
            return (_ext or _binding()).conv_decode(*args)
    return (_ext or _binding()).conv_decode(*args)


def qk_norm(q, k=None, q_weight=None, k_weight=None, positions=None, inv_freq=None, norm: Optional[str] = "rms",
            eps: float = 1e-6, layout: str = "half", rotary_offset: int = 0, rotary_scale: float = 1.0, q_out=None,
            k_out=None, stream=None) -> Tuple:
    """Per-head norm of queries and keys and the rotation of their positions, in one pass.
    Returns (q_out, k_out); k_out is None without k.

    ``q`` [T, Hq, D] or [B, T, Hq, D], ``k`` alike with its own head count; ``norm``: "rms", "l2"
    (unit rows, what ``prefill`` and ``decode`` expect) or None; weights fp32 [D] or None.
    ``positions`` int32 [T] / [B, T] and ``inv_freq`` fp32 [rot / 2] (see ``rotary_frequencies``)
    rotate channels [rotary_offset, rotary_offset + rot) in pairs ("half": rot / 2 apart,
    "interleaved": neighbours), cos and sin times ``rotary_scale``; without them nothing rotates.
    ``q_out=q`` and ``k_out=k`` work in place, also on slices of one fused projection.
    """
    if inv_freq is not None and inv_freq.numel() == 0:
        inv_freq = None
    args = (q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out, _lookup(_norms, norm, "norm"), eps,
            _lookup(_layouts, layout, "layout"), rotary_offset, rotary_scale)
    if stream is not None:
        with _on(stream, q):
            return (_ext or _binding()).qk_norm(*args)
    return (_ext or _binding()).qk_norm(*args)


def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original_length: Optional[int] = None, fast: float = 32.0, slow: float = 1.0, device=None):
    """(inv_freq fp32 [rot / 2], rotary_scale) for ``qk_norm``.

    inv_freq_i = base^(-2 i / rot).  ``scaling`` stretches a context of ``original_length`` positions
    by ``factor``:
      * "linear": positions divided by the factor;
      * "base": the base raised to base * factor^(rot / (rot - 2)), so that the slowest pair turns as
        under "linear" and the fastest keeps its speed;
      * "parts": pairs that turn more than ``fast`` times over the original context keep their speed,
        those below ``slow`` turns are divided by the factor, a linear ramp over the pair index in
        between; the scale is 0.1 ln(factor) + 1.
    """
    import torch
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    half = rot // 2
    i = torch.arange(half, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base * factor
    inv = base ** (-2.0 * i / rot)
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "parts":
        if not original_length or not fast > slow > 0:
            raise ValueError("scaling='parts' needs original_length and fast > slow > 0")

        def pair(turns):        # the (fractional) pair that makes `turns` turns over the context
            return rot * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), half - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)      # 0: keep, 1: divide
        inv = inv * (1 - ramp) + inv / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    return inv.float().to(device), scale


def ssm_prefill(x, dt, A, B, C, D=None, dt_bias=None, z=None, initial_state=None, cu_seqlens=None, out=None,
                final_state=None, output_final_state: bool = True, dt_softplus: bool = False, segment: int = 0,
                workspace=None, stream=None) -> Tuple:
    """Selective state space scan of prompts.  Returns (out, final_state).

    ``x`` dense [B, T, H, P] or packed [T, H, P] with int32 ``cu_seqlens``; ``dt`` [.., H] (x's dtype
    or fp32); ``A``, ``D``, ``dt_bias`` fp32 [H]; ``B``, ``C`` [.., G, N]; ``z`` like x.  With
    step = softplus(dt + dt_bias) (``dt_softplus``) or dt + dt_bias:
        S_t = exp(A step_t) S_{t-1} + step_t B_t x_t^T,   out = (S_t^T C_t + D x_t) silu(z_t).
    States [N_seq, H, N, P]; a final state allocated here is fp32.  ``workspace``: an optional uint8
    tensor of at least ``ssm_workspace_size`` + 256 bytes, of one call in flight at a time; by default
    torch allocates one.
    """
    args = (x, dt, A, B, C, initial_state, cu_seqlens, out, final_state, D, dt_bias, z, workspace, output_final_state,
            dt_softplus, segment)
    if stream is not None:
        with _on(stream, x):
            return (_ext or _binding()).ssm_prefill(*args)
    return (_ext or _binding()).ssm_prefill(*args)


def ssm_workspace_size(x, dt, A, B, C, initial_state=None, cu_seqlens=None, segment: int = 0) -> int:
    """Bytes of workspace ``ssm_prefill`` needs for these tensors."""
    return (_ext or _binding()).ssm_workspace_size(x, dt, A, B, C, initial_state, cu_seqlens, segment)


def ssm_decode(x, dt, A, B, C, state_pool, state_indices, num_tokens=None, D=None, dt_bias=None, z=None, out=None,
               update_state: bool = True, write_out: bool = True, dt_softplus: bool = False, stream=None):
    """The scan over 1..8 tokens per request against a pool of states [P, H, N, P].  Returns out or None.

    ``x``, ``z`` [R, T, H, P]; ``dt`` [R, T, H]; ``B``, ``C`` [R, T, G, N]; ``state_indices`` and
    ``num_tokens`` int32 [R] on the GPU with ``decode``'s meaning; ``update_state=False`` only reads
    the pool (verify), ``write_out=False`` only commits.
    """
    args = (x, dt, A, B, C, state_pool, state_indices, num_tokens, out, D, dt_bias, z, write_out, update_state,
            dt_softplus)
    if stream is not None:
        with _on(stream, x):
            return (_ext or _binding()).ssm_decode(*args)
    return (_ext or _binding()).ssm_decode(*args)
