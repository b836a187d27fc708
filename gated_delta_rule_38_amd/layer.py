"""The operators around the recurrence (C ABI in ``include/kda_layer.h``): the short causal
convolution, the query/key norm with rotation and the selective state space scan.

Marshalling only, like the rest of the package, and kept short: these calls run in single-token
steps whose kernels take a few microseconds, so descriptors are packed into one buffer per call.
Every call runs with the device of its first tensor current, on that device's current stream unless
one is given; outputs and workspaces it allocates are allocated on that stream.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

_DESC = struct.Struct("<Qii4q4q")          # kda_tensor_t
_SIZE = _DESC.size
_PAD = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())
_SSM_OPTS = struct.Struct("<QQQii")        # kda_ssm_options_t
_QK_OPTS = struct.Struct("<ifiif")         # kda_qk_norm_options_t
_codes = None
_activations = {None: 0, "none": 0, "silu": 1}
_norms = {None: 0, "none": 0, "rms": 1, "l2": 2}
_layouts = {"half": 0, "interleaved": 1}


def bind(lib) -> None:
    """Argument types of the functions (descriptor addresses are plain integers)."""
    V, I = ctypes.c_void_p, ctypes.c_int32
    for name, args in (("kda_conv", [V] * 7 + [I, V]), ("kda_conv_decode", [V] * 7 + [I, I, V]),
                       ("kda_qk_norm", [V] * 10), ("kda_ssm_prefill", [V] * 11),
                       ("kda_ssm_workspace_size", [V] * 11),
                       ("kda_ssm_prefill_ws", [V] * 11 + [ctypes.c_size_t, V]),
                       ("kda_ssm_decode", [V] * 9 + [I, V, V])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


class _Call:
    """The descriptors of one call's tensors, packed, and where it runs."""
    __slots__ = ("buf", "ptr", "lib", "device", "stream", "guard")

    def __init__(self, tensors, stream, extra=0):
        import torch

        from . import load_library
        global _codes
        if _codes is None:
            _codes = {torch.bfloat16: 0, torch.float32: 1, torch.int32: 2}
        self.lib = load_library()
        device = tensors[0].device
        if not torch.cuda.is_available():
            raise RuntimeError("gated_delta_rule_38_amd needs a ROCm GPU (gfx950); none is visible")
        self.buf = buf = ctypes.create_string_buffer(_SIZE * len(tensors) + extra)
        base = ctypes.addressof(buf)
        self.ptr = ptr = []
        at = 0
        for t in tensors:
            if t is None:
                ptr.append(None)
            else:
                if t.device != device or not t.is_cuda:
                    raise ValueError("all tensors must be on one GPU")
                shape = t.shape
                n = len(shape)
                if n > 4:
                    raise ValueError("at most 4 dimensions")
                pad = _PAD[n]
                _DESC.pack_into(buf, at, t.data_ptr(), _codes.get(t.dtype, -1), n, *shape, *pad, *t.stride(), *pad)
                ptr.append(base + at)
            at += _SIZE
        self.device = device
        self.stream, self.guard = _where(device, stream)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def check(self, status):
        if status:
            from . import KdaError
            raise KdaError(status, self.lib.kda_last_error().decode())


def _where(device, stream):
    """(raw stream, guard): the stream of a call, and the context that makes its device and stream
    current while it runs (None when they already are)."""
    import torch
    index = device.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
        if torch.cuda.current_device() == index:
            return raw, None
        return raw, torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _empty_like(t, device, stream):
    """A contiguous tensor of t's shape and dtype, allocated on the call's stream."""
    return _empty(t.shape, t.dtype, device, stream)


def _empty(shape, dtype, device, stream):
    import torch
    if not device.type == "cuda":
        raise ValueError("all tensors must be on one GPU")
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


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
    act = _lookup(_activations, activation, "activation")
    if out is None:
        out = _empty_like(x, x.device, stream)
    if final_state is None and output_final_state:
        n = cu_seqlens.numel() - 1 if cu_seqlens is not None else x.shape[0]
        dtype = initial_state.dtype if initial_state is not None else x.dtype
        final_state = _empty((n, weight.shape[-1] - 1, x.shape[-1]), dtype, x.device, stream)
    with _Call((x, weight, bias, initial_state, cu_seqlens, out, final_state), stream) as c:
        c.check(c.lib.kda_conv(*c.ptr, act, c.stream))
    return out, final_state


def conv_decode(x, weight, state_pool, state_indices, num_tokens=None, bias=None, out=None,
                update_state: bool = True, write_out: bool = True, activation: Optional[str] = None, stream=None):
    """The convolution over 1..8 tokens per request against a pool of states.  Returns out or None.

    ``x`` [R, T, C]; ``state_pool`` [P, W - 1, C]; ``state_indices`` and ``num_tokens`` int32 [R] on
    the GPU, with ``decode``'s meaning (a slot outside [0, P) skips the request).
    ``update_state=False`` only reads the pool (verify); ``write_out=False`` only commits.
    """
    act = _lookup(_activations, activation, "activation")
    if out is None and write_out:
        out = _empty_like(x, x.device, stream)
    with _Call((x, weight, bias, state_pool, state_indices, num_tokens, out), stream) as c:
        c.check(c.lib.kda_conv_decode(*c.ptr, int(update_state), act, c.stream))
    return out


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
    opts = (_lookup(_norms, norm, "norm"), eps, _lookup(_layouts, layout, "layout"), rotary_offset, rotary_scale)
    if inv_freq is not None and inv_freq.numel() == 0:
        inv_freq = None
    if q_out is None:
        q_out = _empty_like(q, q.device, stream)
    if k_out is None and k is not None:
        k_out = _empty_like(k, q.device, stream)
    with _Call((q, k, q_weight, k_weight, positions, inv_freq, q_out, k_out), stream, _QK_OPTS.size) as c:
        _QK_OPTS.pack_into(c.buf, 8 * _SIZE, *opts)
        c.check(c.lib.kda_qk_norm(*c.ptr, ctypes.addressof(c.buf) + 8 * _SIZE, c.stream))
    return q_out, k_out


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


def _ssm_opts(c, at, ptrs, softplus, segment=0):
    _SSM_OPTS.pack_into(c.buf, at, *(p or 0 for p in ptrs), int(bool(softplus)), segment)
    return ctypes.addressof(c.buf) + at


def ssm_prefill(x, dt, A, B, C, D=None, dt_bias=None, z=None, initial_state=None, cu_seqlens=None, out=None,
                final_state=None, output_final_state: bool = True, dt_softplus: bool = False, segment: int = 0,
                workspace=None, stream=None) -> Tuple:
    """Selective state space scan of prompts.  Returns (out, final_state).

    ``x`` dense [B, T, H, P] or packed [T, H, P] with int32 ``cu_seqlens``; ``dt`` [.., H] (x's dtype
    or fp32); ``A``, ``D``, ``dt_bias`` fp32 [H]; ``B``, ``C`` [.., G, N]; ``z`` like x.  With
    step = softplus(dt + dt_bias) (``dt_softplus``) or dt + dt_bias:
        S_t = exp(A step_t) S_{t-1} + step_t B_t x_t^T,   out = (S_t^T C_t + D x_t) silu(z_t).
    States [N_seq, H, N, P]; a final state allocated here is fp32.  ``workspace``: an optional uint8
    tensor of at least ``ssm_workspace_size`` + 256 bytes; by default torch allocates one.
    """
    if out is None:
        out = _empty_like(x, x.device, stream)
    if final_state is None and output_final_state:
        import torch
        n = cu_seqlens.numel() - 1 if cu_seqlens is not None else x.shape[0]
        final_state = _empty((n, x.shape[-2], B.shape[-1], x.shape[-1]), torch.float32, x.device, stream)
    with _Call((x, dt, A, B, C, initial_state, cu_seqlens, out, final_state, D, dt_bias, z), stream,
               _SSM_OPTS.size + 8) as c:
        opts = _ssm_opts(c, 12 * _SIZE, c.ptr[9:], dt_softplus, segment)
        need = ctypes.c_size_t.from_buffer(c.buf, 12 * _SIZE + _SSM_OPTS.size)
        c.check(c.lib.kda_ssm_workspace_size(*c.ptr[:9], opts, ctypes.addressof(need)))
        base = size = 0
        if need.value:
            if workspace is None:
                import torch
                workspace = _empty((need.value + 256,), torch.uint8, x.device, stream)
            elif workspace.device != x.device or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on the operands' GPU")
            start = workspace.data_ptr()
            base = (start + 255) // 256 * 256
            size = max(0, workspace.numel() * workspace.element_size() - (base - start))
        c.check(c.lib.kda_ssm_prefill_ws(*c.ptr[:9], opts, base, size, c.stream))
    return out, final_state


def ssm_workspace_size(x, dt, A, B, C, initial_state=None, cu_seqlens=None, segment: int = 0) -> int:
    """Bytes of workspace ``ssm_prefill`` needs for these tensors."""
    import torch
    out = torch.empty_like(x)
    with _Call((x, dt, A, B, C, initial_state, cu_seqlens, out, None), None, _SSM_OPTS.size + 8) as c:
        opts = _ssm_opts(c, 9 * _SIZE, (0, 0, 0), False, segment)
        need = ctypes.c_size_t.from_buffer(c.buf, 9 * _SIZE + _SSM_OPTS.size)
        c.check(c.lib.kda_ssm_workspace_size(*c.ptr, opts, ctypes.addressof(need)))
        return need.value


def ssm_decode(x, dt, A, B, C, state_pool, state_indices, num_tokens=None, D=None, dt_bias=None, z=None, out=None,
               update_state: bool = True, write_out: bool = True, dt_softplus: bool = False, stream=None):
    """The scan over 1..8 tokens per request against a pool of states [P, H, N, P].  Returns out or None.

    ``x``, ``z`` [R, T, H, P]; ``dt`` [R, T, H]; ``B``, ``C`` [R, T, G, N]; ``state_indices`` and
    ``num_tokens`` int32 [R] on the GPU with ``decode``'s meaning; ``update_state=False`` only reads
    the pool (verify), ``write_out=False`` only commits.
    """
    if out is None and write_out:
        out = _empty_like(x, x.device, stream)
    with _Call((x, dt, A, B, C, state_pool, state_indices, num_tokens, out, D, dt_bias, z), stream,
               _SSM_OPTS.size) as c:
        opts = _ssm_opts(c, 12 * _SIZE, c.ptr[9:], dt_softplus)
        c.check(c.lib.kda_ssm_decode(*c.ptr[:9], int(update_state), opts, c.stream))
    return out
