"""Host-side checks of the operators of include/kda_layer.h, on any host: every refusal returns its
documented status before anything is launched, and what must be accepted passes validation.

The descriptors point at addresses that are never dereferenced.  A call whose descriptors are valid
would launch, so "accepted" is shown by ``kda_ssm_workspace_size`` (which launches nothing) or by
calls that have no work (no tokens, no requests).
"""
import ctypes
import os
import subprocess
import sys

import pytest

import gated_delta_rule_38_amd as kda
from gated_delta_rule_38_amd import KDA_BF16, KDA_F32, KDA_I32
from test_abi import FAKE, desc, lib  # noqa: F401

NULL, SHAPE, DTYPE, LAYOUT, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5, 6, 7
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def at(i):
    return FAKE + (i << 34)


def ptr(d):
    return ctypes.addressof(d) if d is not None else None


# ------------------------------------------------------------------------------- convolution
def conv_set(T=100, C=64, W=4, N=3, dt=KDA_BF16):
    return dict(x=desc([T, C], dt, at(0)), w=desc([C, W], dt, at(1)), b=desc([C], KDA_F32, at(2)),
                s0=desc([N, W - 1, C], dt, at(3)), cu=desc([N + 1], KDA_I32, at(4)), out=desc([T, C], dt, at(5)),
                sT=desc([N, W - 1, C], dt, at(6)), act=1)


def conv(lib, s):  # noqa: F811
    return lib.kda_conv(*(ptr(s[k]) for k in ("x", "w", "b", "s0", "cu", "out", "sT")), s["act"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(out=None), NULL),
    (dict(w=desc([64, 1], KDA_BF16, at(1))), UNSUPPORTED), (dict(w=desc([64, 5], KDA_BF16, at(1))), UNSUPPORTED),
    (dict(w=desc([63, 4], KDA_BF16, at(1))), SHAPE), (dict(w=desc([64, 4], KDA_BF16, at(1), [8, 1])), LAYOUT),
    (dict(w=desc([64, 4], KDA_I32, at(1))), DTYPE), (dict(b=desc([63], KDA_F32, at(2))), SHAPE),
    (dict(act=2), UNSUPPORTED), (dict(act=-1), UNSUPPORTED),
    (dict(out=desc([100, 64], KDA_F32, at(5))), DTYPE), (dict(out=desc([99, 64], KDA_BF16, at(5))), SHAPE),
    (dict(x=desc([100, 64], KDA_I32, at(0))), DTYPE), (dict(x=desc([100, 64], KDA_BF16, at(0), [128, 2])), LAYOUT),
    (dict(s0=desc([2, 3, 64], KDA_BF16, at(3))), SHAPE), (dict(s0=desc([3, 4, 64], KDA_BF16, at(3))), SHAPE),
    (dict(sT=desc([3, 3, 63], KDA_BF16, at(6))), SHAPE), (dict(cu=desc([4], KDA_F32, at(4))), DTYPE),
    (dict(cu=None), SHAPE),                                          # packed x without offsets
    (dict(out=desc([100, 64], KDA_BF16, at(0))), ALIAS),             # in place: other threads read x
    (dict(out=desc([100, 64], KDA_BF16, at(0) + 128 * 99)), ALIAS),
    (dict(sT=desc([3, 3, 64], KDA_BF16, at(3) + 128)), ALIAS),       # partly over the initial state
    (dict(sT=desc([3, 3, 64], KDA_BF16, at(5))), ALIAS), (dict(sT=desc([3, 3, 64], KDA_BF16, at(1))), ALIAS),
    (dict(out=desc([100, 64], KDA_BF16, at(5), [0, 1])), LAYOUT),    # rows that share memory
    (dict(out=desc([100, 64], KDA_BF16, at(5), [32, 1])), LAYOUT),
    (dict(sT=desc([3, 3, 64], KDA_BF16, at(6), [64, 64, 1])), LAYOUT),
    (dict(x=desc([1 << 31, 64], KDA_BF16, at(0)), out=desc([1 << 31, 64], KDA_BF16, at(50))), SHAPE),
])
def test_conv_refusals(lib, change, status):  # noqa: F811
    s = conv_set()
    s.update(change)
    assert conv(lib, s) == status, kda.load_library().kda_last_error()


def test_conv_without_work(lib):  # noqa: F811
    s = conv_set(T=0, N=0)
    s["sT"] = s["s0"] = None
    assert conv(lib, s) == 0
    # dense, no tokens, no states
    s = dict(x=desc([2, 0, 64], KDA_BF16, 0), w=desc([64, 4], KDA_F32, at(1)), b=None, s0=None, cu=None,
             out=desc([2, 0, 64], KDA_BF16, 0), sT=None, act=0)
    s["x"].data = s["out"].data = None
    assert conv(lib, s) == 0


def conv_decode(lib, s):  # noqa: F811
    return lib.kda_conv_decode(*(ptr(s[k]) for k in ("x", "w", "b", "pool", "idx", "n", "out")), s["update"], s["act"], None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), NULL), (dict(pool=None), NULL), (dict(idx=None), NULL),
    (dict(x=desc([4, 9, 64], KDA_BF16, at(0)), out=desc([4, 9, 64], KDA_BF16, at(5))), UNSUPPORTED),
    (dict(x=desc([4, 0, 64], KDA_BF16, at(0)), out=desc([4, 0, 64], KDA_BF16, at(5))), UNSUPPORTED),
    (dict(x=desc([4, 64], KDA_BF16, at(0))), SHAPE), (dict(out=desc([4, 1, 64], KDA_BF16, at(5))), SHAPE),
    (dict(pool=desc([6, 2, 64], KDA_BF16, at(3))), SHAPE), (dict(pool=desc([6, 3, 64], KDA_I32, at(3))), DTYPE),
    (dict(idx=desc([4], KDA_F32, at(6))), DTYPE), (dict(idx=desc([3], KDA_I32, at(6))), SHAPE),
    (dict(n=desc([5], KDA_I32, at(7))), SHAPE), (dict(out=desc([4, 2, 64], KDA_BF16, at(0))), ALIAS),
    (dict(pool=desc([6, 3, 64], KDA_BF16, at(0))), ALIAS), (dict(pool=desc([6, 3, 64], KDA_BF16, at(5))), ALIAS),
    (dict(pool=desc([6, 3, 64], KDA_BF16, at(3), [0, 64, 1])), LAYOUT), (dict(act=7), UNSUPPORTED),
])
def test_conv_decode_refusals(lib, change, status):  # noqa: F811
    s = dict(x=desc([4, 2, 64], KDA_BF16, at(0)), w=desc([64, 4], KDA_BF16, at(1)), b=None,
             pool=desc([6, 3, 64], KDA_BF16, at(3)), idx=desc([4], KDA_I32, at(6)), n=None,
             out=desc([4, 2, 64], KDA_BF16, at(5)), update=1, act=0)
    s.update(change)
    assert conv_decode(lib, s) == status


# -------------------------------------------------------------------------- norm and rotation
class QkOptions(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("layout", ctypes.c_int32),
                ("offset", ctypes.c_int32), ("scale", ctypes.c_float)]


def qk_set(T=0, Hq=4, Hk=2, D=128, rot=64, dt=KDA_BF16, **o):
    opts = dict(norm=1, eps=1e-6, layout=0, offset=0, scale=1.0)
    opts.update(o)
    return dict(q=desc([T, Hq, D], dt, at(0)), k=desc([T, Hk, D], dt, at(1)), qw=None, kw=None,
                pos=desc([T], KDA_I32, at(2)), freq=desc([rot // 2], KDA_F32, at(3)), qo=desc([T, Hq, D], dt, at(4)),
                ko=desc([T, Hk, D], dt, at(5)), opts=QkOptions(*opts.values()))


def qk(lib, s):  # noqa: F811
    return lib.kda_qk_norm(*(ptr(s[k]) for k in ("q", "k", "qw", "kw", "pos", "freq", "qo", "ko", "opts")), None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(qo=None), NULL), (dict(k=None), NULL), (dict(ko=None), NULL), (dict(opts=None), NULL),
    (dict(pos=None), NULL), (dict(k=None, ko=None, kw=desc([128], KDA_F32, at(6))), NULL),
    (dict(freq=desc([65], KDA_F32, at(3))), SHAPE), (dict(freq=desc([32], KDA_BF16, at(3))), DTYPE),
    (dict(pos=desc([8], KDA_F32, at(2))), DTYPE), (dict(pos=desc([7], KDA_I32, at(2))), SHAPE),
    (dict(qw=desc([64], KDA_F32, at(6))), SHAPE), (dict(qw=desc([128], KDA_BF16, at(6))), DTYPE),
    (dict(qo=desc([8, 4, 128], KDA_F32, at(4))), DTYPE), (dict(ko=desc([8, 3, 128], KDA_BF16, at(5))), SHAPE),
    (dict(k=desc([7, 2, 128], KDA_BF16, at(1))), SHAPE), (dict(k=desc([8, 2, 64], KDA_BF16, at(1))), SHAPE),
    (dict(q=desc([8, 4, 128], KDA_BF16, at(0) + 2)), LAYOUT), (dict(q=desc([8, 4, 128], KDA_BF16, at(0), [514, 128, 1])), LAYOUT),
    (dict(qo=desc([8, 4, 128], KDA_BF16, at(0) + 8)), ALIAS),         # shifted over its input
    (dict(qo=desc([8, 4, 128], KDA_BF16, at(1))), ALIAS), (dict(ko=desc([8, 2, 128], KDA_BF16, at(4))), ALIAS),
    (dict(ko=desc([8, 2, 128], KDA_BF16, at(0))), ALIAS),             # over the other operand
    (dict(qo=desc([8, 4, 128], KDA_BF16, at(4), [0, 128, 1])), LAYOUT),
    (dict(norm=3), UNSUPPORTED), (dict(norm=0, freq=None), UNSUPPORTED), (dict(eps=-1.0), UNSUPPORTED),
    (dict(eps=float("nan")), UNSUPPORTED), (dict(offset=65), SHAPE), (dict(offset=-1), SHAPE),
    (dict(layout=2), UNSUPPORTED), (dict(layout=1, offset=3), UNSUPPORTED), (dict(scale=float("inf")), UNSUPPORTED),
    (dict(norm=0, qw=desc([128], KDA_F32, at(6))), UNSUPPORTED), (dict(D=260), UNSUPPORTED), (dict(D=66, rot=8), UNSUPPORTED),
])
def test_qk_norm_refusals(lib, change, status):  # noqa: F811
    made = {k: v for k, v in change.items() if k in ("norm", "eps", "layout", "offset", "scale", "D", "rot")}
    s = qk_set(T=8, **made)
    s.update({k: v for k, v in change.items() if k not in made})
    assert qk(lib, s) == status


def test_qk_norm_accepts(lib):  # noqa: F811
    """No tokens: the call ends after validation."""
    assert qk(lib, qk_set()) == 0
    assert qk(lib, dict(qk_set(), k=None, ko=None)) == 0
    s = qk_set()
    assert qk(lib, dict(s, qo=s["q"], ko=s["k"])) == 0


def test_qk_norm_slices_of_one_projection(lib):  # noqa: F811
    """q and k as column ranges of one buffer, in place: accepted when the columns are apart, refused
    when they meet.  (A refusal later in the checks, of an overlapping pair of outputs, shows that
    everything before it passed.)"""
    row = 6 * 128 + 8
    q, k = desc([8, 4, 128], KDA_BF16, at(0), [row, 128, 1]), desc([8, 2, 128], KDA_BF16, at(0) + 2 * 512, [row, 128, 1])
    near = desc([8, 2, 128], KDA_BF16, at(0) + 2 * 504, [row, 128, 1])
    s = dict(qk_set(T=8), q=q, qo=q, k=near, ko=near)
    assert qk(lib, s) == ALIAS
    wrap = desc([8, 2, 128], KDA_BF16, at(0) + 2 * (row - 128), [row, 128, 1])     # runs into the next row's q
    assert qk(lib, dict(s, k=wrap, ko=wrap)) == ALIAS
    # apart: the only thing left to refuse is the layout of k_out's rows among themselves
    assert qk(lib, dict(s, k=k, ko=desc([8, 2, 128], KDA_BF16, at(7), [0, 128, 1]))) == LAYOUT


def test_rotary_frequencies():
    import torch
    f, s = kda.rotary_frequencies(8, base=10000.0)
    assert s == 1.0 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001]))
    lin, _ = kda.rotary_frequencies(8, scaling="linear", factor=4.0)
    assert torch.allclose(lin, f / 4)
    b, _ = kda.rotary_frequencies(8, scaling="base", factor=4.0)
    assert torch.allclose(b[0], f[0]) and torch.allclose(b[-1], f[-1] / 4)       # fastest kept, slowest as under linear
    p, s = kda.rotary_frequencies(64, scaling="parts", factor=4.0, original_length=4096)
    g, _ = kda.rotary_frequencies(64)
    r = p / g
    turns = 4096 * g / (2 * torch.pi)
    assert s == pytest.approx(0.1 * 1.3862943611 + 1)
    assert torch.allclose(r[turns > 45], torch.tensor(1.0)) and torch.allclose(r[turns < 0.7], torch.tensor(0.25))
    assert (r[1:] <= r[:-1] + 1e-6).all()
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, factor=0.5), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="parts", factor=2.0)):
        with pytest.raises(ValueError):
            kda.rotary_frequencies(**bad)


# ------------------------------------------------------------------------- state space scan
class SsmOptions(ctypes.Structure):
    _fields_ = [("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p), ("z", ctypes.c_void_p), ("softplus", ctypes.c_int32),
                ("segment", ctypes.c_int32)]


def ssm_set(T=100, H=4, G=2, P=64, N=128, n=3, dt=KDA_BF16):
    return dict(x=desc([T, H, P], dt, at(0)), dt=desc([T, H], KDA_F32, at(1)), A=desc([H], KDA_F32, at(2)),
                B=desc([T, G, N], dt, at(3)), C=desc([T, G, N], dt, at(4)), s0=desc([n, H, N, P], KDA_F32, at(5)),
                cu=desc([n + 1], KDA_I32, at(6)), out=desc([T, H, P], dt, at(7)), sT=desc([n, H, N, P], KDA_F32, at(8)),
                D=desc([H], KDA_F32, at(9)), bias=desc([H], KDA_F32, at(10)), z=desc([T, H, P], dt, at(11)), softplus=1,
                segment=0)


def ssm_args(s):
    o = SsmOptions(ptr(s["D"]), ptr(s["bias"]), ptr(s["z"]), s["softplus"], s["segment"])
    return [ptr(s[k]) for k in ("x", "dt", "A", "B", "C", "s0", "cu", "out", "sT")] + [ctypes.addressof(o)], o


def ssm_size(lib, s):  # noqa: F811
    args, keep = ssm_args(s)
    n = ctypes.c_size_t(0)
    return lib.kda_ssm_workspace_size(*args, ctypes.addressof(n)), n.value


SSM_REFUSALS = [
    (dict(x=None), NULL), (dict(dt=None), NULL), (dict(A=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL),
    (dict(out=None), NULL), (dict(B=desc([100, 3, 128], KDA_BF16, at(3))), SHAPE),
    (dict(C=desc([100, 1, 128], KDA_BF16, at(4))), SHAPE), (dict(C=desc([100, 2, 128], KDA_F32, at(4))), DTYPE),
    (dict(B=desc([100, 2, 96], KDA_BF16, at(3)), C=desc([100, 2, 96], KDA_BF16, at(4))), UNSUPPORTED),
    (dict(x=desc([100, 4, 32], KDA_BF16, at(0))), UNSUPPORTED), (dict(dt=desc([100, 3], KDA_F32, at(1))), SHAPE),
    (dict(dt=desc([100, 4], KDA_I32, at(1))), DTYPE), (dict(A=desc([4], KDA_BF16, at(2))), DTYPE),
    (dict(A=desc([3], KDA_F32, at(2))), SHAPE), (dict(D=desc([3], KDA_F32, at(9))), SHAPE),
    (dict(bias=desc([4], KDA_BF16, at(10))), DTYPE), (dict(z=desc([100, 4, 64], KDA_F32, at(11))), DTYPE),
    (dict(z=desc([99, 4, 64], KDA_BF16, at(11))), SHAPE), (dict(s0=desc([3, 4, 64, 128], KDA_F32, at(5))), SHAPE),
    (dict(sT=desc([2, 4, 128, 64], KDA_F32, at(8))), SHAPE), (dict(sT=desc([3, 4, 128, 64], KDA_I32, at(8))), DTYPE),
    (dict(cu=None), SHAPE), (dict(softplus=2), UNSUPPORTED), (dict(segment=-2), UNSUPPORTED), (dict(segment=33), UNSUPPORTED),
    (dict(x=desc([100, 4, 64], KDA_BF16, at(0) + 2)), LAYOUT), (dict(B=desc([100, 2, 128], KDA_BF16, at(3), [258, 128, 1])), LAYOUT),
    (dict(x=desc([100, 4, 64], KDA_BF16, at(0), [256, 64, 2])), LAYOUT),
    (dict(out=desc([100, 4, 64], KDA_BF16, at(0))), ALIAS), (dict(out=desc([100, 4, 64], KDA_BF16, at(11))), ALIAS),
    (dict(out=desc([100, 4, 64], KDA_BF16, at(7), [0, 64, 1])), LAYOUT),
    (dict(sT=desc([3, 4, 128, 64], KDA_F32, at(5) + 256)), ALIAS), (dict(sT=desc([3, 4, 128, 64], KDA_F32, at(7))), ALIAS),
    (dict(sT=desc([3, 4, 128, 64], KDA_F32, at(8), [0, 8192, 64, 1])), LAYOUT),
    # 32-bit offsets within a chunk
    (dict(x=desc([100, 4, 64], KDA_BF16, 0, [1 << 24, 64, 1])), UNSUPPORTED),
    (dict(B=desc([100, 2, 128], KDA_BF16, 0, [1 << 24, 128, 1])), UNSUPPORTED),
    (dict(x=desc([100, 4, 64], KDA_BF16, 0, [64, 1 << 29, 1])), UNSUPPORTED),
]


@pytest.mark.parametrize("change,status", SSM_REFUSALS)
def test_ssm_refusals(lib, change, status):  # noqa: F811
    s = ssm_set()
    s.update(change)
    for d in change.values():       # views of more than a descriptor's slot lie far from the others
        if hasattr(d, "data") and d.data is None:
            d.data = 1 << 60
    assert ssm_size(lib, s)[0] == status
    args, keep = ssm_args(s)
    assert lib.kda_ssm_prefill(*args, None) == status
    assert lib.kda_ssm_prefill_ws(*args, None, 0, None) == status


def test_ssm_workspace(lib):  # noqa: F811
    """Whole sequences need none; segments one state and one decay per slot and head, sized exactly;
    a workspace too small, misaligned or over a tensor is refused."""
    s = ssm_set()
    s["segment"] = -1
    assert ssm_size(lib, s) == (0, 0)
    assert ssm_size(lib, dict(s, sT=s["s0"])) == (0, 0)              # in place
    s["segment"] = 32
    slots = 100 // 32 + 3
    need = slots * 4 * 128 * 64 * 4 + 256      # (4 bytes of decay a slot and head, to 256)
    assert ssm_size(lib, s) == (0, need)
    args, keep = ssm_args(s)
    assert lib.kda_ssm_prefill_ws(*args, at(20), need - 1, None) == WORKSPACE
    assert lib.kda_ssm_prefill_ws(*args, None, need, None) == WORKSPACE
    assert lib.kda_ssm_prefill_ws(*args, at(20) + 128, need, None) == WORKSPACE
    assert lib.kda_ssm_prefill_ws(*args, at(7) - 256, need, None) == ALIAS
    # dense: segments of every sequence, and none where a sequence fits one
    d = ssm_set()
    for k, shape, i in (("x", [3, 100, 4, 64], 0), ("out", [3, 100, 4, 64], 7), ("z", [3, 100, 4, 64], 11),
                        ("B", [3, 100, 2, 128], 3), ("C", [3, 100, 2, 128], 4)):
        d[k] = desc(shape, KDA_BF16, at(i))
    d["dt"], d["cu"], d["segment"] = desc([3, 100, 4], KDA_BF16, at(1)), None, 64
    assert ssm_size(lib, d) == (0, 6 * 4 * 128 * 64 * 4 + 256)
    d["segment"] = 128
    assert ssm_size(lib, d) == (0, 0)


def test_ssm_decode_refusals(lib):  # noqa: F811
    R, T, H, G, P, N = 4, 2, 4, 2, 64, 128
    base = dict(x=desc([R, T, H, P], KDA_BF16, at(0)), dt=desc([R, T, H], KDA_BF16, at(1)), A=desc([H], KDA_F32, at(2)),
                B=desc([R, T, G, N], KDA_BF16, at(3)), C=desc([R, T, G, N], KDA_BF16, at(4)),
                pool=desc([6, H, N, P], KDA_F32, at(5)), idx=desc([R], KDA_I32, at(6)), n=None,
                out=desc([R, T, H, P], KDA_BF16, at(7)), D=None, bias=None, z=None)

    def call(**change):
        s = dict(base, **change)
        o = SsmOptions(ptr(s["D"]), ptr(s["bias"]), ptr(s["z"]), s.get("softplus", 0), 0)
        return lib.kda_ssm_decode(*(ptr(s[k]) for k in ("x", "dt", "A", "B", "C", "pool", "idx", "n", "out")), 1,
                                  ctypes.addressof(o), None)

    for name in ("x", "dt", "A", "B", "C", "pool", "idx"):
        assert call(**{name: None}) == NULL, name
    assert call(x=desc([R, 9, H, P], KDA_BF16, at(0))) == UNSUPPORTED
    assert call(B=desc([R, T, 3, N], KDA_BF16, at(3))) == SHAPE
    assert call(C=desc([R, 1, G, N], KDA_BF16, at(4))) == SHAPE
    assert call(dt=desc([R, T, G], KDA_BF16, at(1))) == SHAPE
    assert call(pool=desc([6, H, P, N], KDA_F32, at(5))) == SHAPE
    assert call(pool=desc([6, H, N, P], KDA_F32, at(5) + 4)) == LAYOUT
    assert call(pool=desc([6, H, N, P], KDA_F32, at(5), [0, N * P, P, 1])) == LAYOUT
    assert call(pool=desc([6, H, N, P], KDA_F32, at(0))) == ALIAS
    assert call(out=desc([R, T, H, P], KDA_BF16, at(5))) == ALIAS
    assert call(out=desc([R, T, H, P], KDA_BF16, at(0))) == ALIAS
    assert call(idx=desc([R], KDA_F32, at(6))) == DTYPE
    assert call(n=desc([R - 1], KDA_I32, at(8))) == SHAPE
    assert call(z=desc([R, T, H, P], KDA_F32, at(8))) == DTYPE
    assert call(softplus=-1) == UNSUPPORTED
    empty = dict(x=desc([0, T, H, P]), dt=desc([0, T, H]), B=desc([0, T, G, N]), C=desc([0, T, G, N]), idx=desc([0], KDA_I32),
                 out=desc([0, T, H, P]))
    assert call(**empty) == 0


def test_ssm_plan_log(tmp_path):
    """KDA_LOG=1 prints the scan's plan to stderr."""
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import test_layer_abi as t, gated_delta_rule_38_amd as kda\n"
            "s = t.ssm_set(); s['segment'] = 64\n"
            "assert t.ssm_size(kda.load_library(), s)[0] == 0\n" % (ROOT, os.path.join(ROOT, "tests")))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, env=dict(os.environ, KDA_LOG="1"))
    assert r.returncode == 0, r.stderr
    assert "kda: ssm plan" in r.stderr and "segment=64 slots=4" in r.stderr


def test_layer_binding_refuses_without_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    x, w = torch.zeros(4, 64), torch.zeros(64, 4)
    with pytest.raises(RuntimeError):
        kda.conv(x, w)
    with pytest.raises(RuntimeError):
        kda.ssm_workspace_size(x, x, x, x, x)
    with pytest.raises(ValueError):
        kda.conv(x, w, activation="relu")
    with pytest.raises(ValueError):
        kda.qk_norm(x, norm="layer")


def test_ssm_without_sequences_needs_no_workspace(lib):
    """Rows without any sequence: nothing to cut, whatever segment is asked for."""
    s = ssm_set()
    s["cu"] = desc([1], KDA_I32, at(6))
    s["s0"] = s["sT"] = None
    s["segment"] = 32
    assert ssm_size(lib, s) == (0, 0)
