"""GPU tests of the operators around the recurrence (include/kda_layer.h) against plain float64
forms (layer_ref.py).

Bounds, per element, derived from the arithmetic and fixed before the first run.  ``mag`` is the
result's expression with every term by its magnitude; a rounding is off by at most u = eps / 2
relative to the value rounded (bf16 2^-8, fp32 2^-24).
  * convolution, norm and rotation: all sums in fp32, fewer than 64 of its roundings along any path
    (W products and sums; the sum of squares of 256 elements enters under a square root, by a tree
    of at most 8 + 6 levels; exponential, reciprocal, sine and cosine within a few units), then one
    rounding to the output: 64 2^-24 mag + u_out |out|.
  * scan: products of inputs are exact or fp32; along a path at most N + 32 sums, one exponential a
    chunk whose argument is rounded relative to its size (|exponent| <= 64 in these cases for terms
    that matter), T / 32 chunk decays: (512 + T) 2^-24 mag.  On bf16 data out has two more roundings
    to bf16 (the decayed products, the copy of the state), each on part of its terms, before its
    own: 2^-8 mag + 2^-8 |out| on top.
  * decode: the same with T <= 8; bf16 pools add 2^-8 |state|.
"""
import sys

import numpy as np
import pytest

import layer_ref as ref

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def say(*a):
    print("[case]", *a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def kda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_38_amd as k
    k.load_library()
    return k


def dtype_of(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


class Draw:
    def __init__(self, seed):
        import torch
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)

    def randn(self, *shape, dtype="f32"):
        import torch
        return torch.randn(*shape, generator=self.gen, device="cuda").to(dtype_of(dtype))

    def rand(self, *shape):
        import torch
        return torch.rand(*shape, generator=self.gen, device="cuda")


def ints(values):
    import torch
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(int).tolist()


def within(got, want, bound, what):
    got = ref.f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if got.size == 0:
        return
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - want) - bound
    k = int(np.argmax(over))
    assert over.flat[k] <= 0, f"{what}: off by {abs(got - want).flat[k]:.3e} at {k}, bound {np.broadcast_to(bound, want.shape).flat[k]:.3e}"


def bits(t):
    import torch
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def padded(t, pad=8):
    """A view of t's values with longer rows and, before the last two dimensions, spare rows, all of
    the spare room NaN."""
    import torch
    shape = list(t.shape)
    big = shape[:]
    big[-1] += pad
    if len(shape) > 2:
        big[-2] += 1
    b = torch.full(big, float("nan"), dtype=t.dtype, device=t.device)
    v = b[tuple(slice(0, s) for s in shape)]
    v.copy_(t)
    return v, b


# ------------------------------------------------------------------------------ convolution

LENGTHS = {"one": [1], "short": [2, 0, 1, 3, 0], "ragged": [33, 0, 1, 130, 64, 2], "long": [1500, 700]}


def conv_case(lengths, C, W, dtype, state, bias, seed):
    d = Draw(seed)
    T, n = sum(lengths), len(lengths)
    return dict(x=d.randn(T, C, dtype=dtype), weight=d.randn(C, W, dtype=dtype),
                bias=d.randn(C, dtype=dtype) if bias else None,
                initial_state=d.randn(n, W - 1, C, dtype=state) if state else None, cu_seqlens=ints(offsets(lengths)))


def check_conv(c, out, final, activation, dtype):
    want, fin, mag = ref.conv(ref.f64(c["x"]), ref.f64(c["weight"]), ref.f64(c["bias"]), ref.f64(c["initial_state"]),
                              c["cu_seqlens"].cpu(), activation)
    within(out, want, 64 * 2.0 ** -24 * mag + U[dtype] * np.abs(want), "out")
    if final is not None:
        assert np.array_equal(ref.f64(final), fin), "final state: inputs are copied exactly"


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("dtype,state", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", None)])
@pytest.mark.parametrize("C,W", [(64, 4), (515, 3), (2056, 2), (1, 4)])
def test_conv(kda, lengths, dtype, state, C, W):
    say("conv", lengths, dtype, state, C, W)
    act = "silu" if C % 2 == 0 else None
    c = conv_case(LENGTHS[lengths], C, W, dtype, state, C != 64, seed=C + W)
    out, final = kda.conv(**c, activation=act)
    check_conv(c, out, final, act, dtype)


def test_conv_dense_matches_packed_bits_and_views(kda):
    import torch
    d = Draw(5)
    x, w, s0 = d.randn(3, 77, 136, dtype="bf16"), d.randn(136, 4, dtype="f32"), d.randn(3, 3, 136, dtype="bf16")
    out, fin = kda.conv(x, w, initial_state=s0, activation="silu")
    po, pf = kda.conv(x.reshape(-1, 136), w, initial_state=s0, cu_seqlens=ints([0, 77, 154, 231]), activation="silu")
    assert torch.equal(bits(out).view(-1), bits(po).view(-1)) and torch.equal(fin, pf)
    # padded rows for every operand, the padding NaN and left as it was; unaligned rows too
    for pad in (8, 1):
        xv, _ = padded(x, pad)
        sv, _ = padded(s0, pad)
        ov, ob = padded(torch.zeros_like(x), pad)
        fv, fb = padded(torch.zeros_like(s0), pad)
        kda.conv(xv, w, initial_state=sv, activation="silu", out=ov, final_state=fv)
        assert torch.equal(bits(ov), bits(out)) and torch.equal(fv, fin)
        assert torch.isnan(ob[..., 136:]).all() and torch.isnan(ob[:, 77:]).all() and torch.isnan(fb[..., 136:]).all()


@pytest.mark.parametrize("lengths", [[2, 0, 1, 40], [0], [200, 1]])
def test_conv_state_in_place_and_split(kda, lengths):
    """The state written over the initial one; and a batch run in two halves, the second from the
    first's final states, gives the whole run's bits."""
    import torch
    c = conv_case(lengths, 264, 4, "bf16", "bf16", True, seed=9)
    out, fin = kda.conv(**c, activation="silu")
    s = c["initial_state"].clone()
    c2 = dict(c, initial_state=s)
    out2, fin2 = kda.conv(**c2, activation="silu", final_state=s)
    assert fin2 is s and torch.equal(out2, out) and torch.equal(s, fin)
    half = [n // 2 for n in lengths]
    cu = offsets(lengths)
    pick = lambda lo, hi: torch.cat([c["x"][cu[i] + lo[i]:cu[i] + hi[i]] for i in range(len(lengths))])
    zero = [0] * len(lengths)
    a, s1 = kda.conv(pick(zero, half), c["weight"], bias=c["bias"], initial_state=c["initial_state"],
                     cu_seqlens=ints(offsets(half)), activation="silu")
    b, s2 = kda.conv(pick(half, lengths), c["weight"], bias=c["bias"], initial_state=s1,
                     cu_seqlens=ints(offsets([n - h for n, h in zip(lengths, half)])), activation="silu")
    parts, ha, hb = [], offsets(half), offsets([n - h for n, h in zip(lengths, half)])
    for i in range(len(lengths)):
        parts += [a[ha[i]:ha[i + 1]], b[hb[i]:hb[i + 1]]]
    assert torch.equal(torch.cat(parts), out) and torch.equal(s2, fin)


def test_conv_rows_behind_the_last_sequence(kda):
    import torch
    d = Draw(6)
    x, w = d.randn(100, 72, dtype="bf16"), d.randn(72, 4, dtype="bf16")
    x[60:] = float("nan")
    out = torch.full_like(x, -512.0)
    kda.conv(x, w, cu_seqlens=ints([0, 25, 60]), out=out)
    ref_out, _ = kda.conv(x[:60].contiguous(), w, cu_seqlens=ints([0, 25, 60]))
    assert torch.equal(out[:60], ref_out) and (out[60:] == -512.0).all()


@pytest.mark.parametrize("dtype,state", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,C,W", [(1, 2056, 4), (4, 515, 3), (8, 64, 2)])
def test_conv_decode(kda, dtype, state, T, C, W):
    import torch
    say("conv_decode", dtype, state, T, C, W)
    d = Draw(T + C)
    R, P = 6, 9
    x, w, b = d.randn(R, T, C, dtype=dtype), d.randn(C, W, dtype=dtype), d.randn(C, dtype="f32")
    pool = d.randn(P, W - 1, C, dtype=state)
    before = pool.clone()
    slots, counts = [7, 2, -1, 0, 9, 5], [T, 0, T, max(T - 1, 0), T, T + 3]
    out = torch.full_like(x, -512.0)
    verify = kda.conv_decode(x, w, pool, ints(slots), num_tokens=ints(counts), bias=b, activation="silu",
                             update_state=False)
    assert torch.equal(pool, before)
    kda.conv_decode(x, w, pool, ints(slots), num_tokens=ints(counts), bias=b, activation="silu", out=out)
    commit = before.clone()
    assert kda.conv_decode(x, w, commit, ints(slots), num_tokens=ints(counts), bias=b, write_out=False) is None
    assert torch.equal(bits(commit), bits(pool))
    left = set(range(P))
    for r, (s, n) in enumerate(zip(slots, counts)):
        n = min(n, T) if 0 <= s < P else 0
        assert (out[r, n:].float() == -512.0).all()
        if not 0 <= s < P:
            continue
        left.discard(s)
        rows = np.concatenate([ref.f64(before[s]), ref.f64(x[r, :n])])
        y, mag = ref.conv_rows(rows, ref.f64(w), ref.f64(b), "silu")
        within(out[r, :n], y, 64 * 2.0 ** -24 * mag + U[dtype] * np.abs(y), f"request {r}")
        assert torch.equal(bits(verify[r, :n]), bits(out[r, :n]))
        want = torch.tensor(rows[n:n + W - 1] if n else rows[:W - 1]).to(dtype_of(state))
        assert torch.equal(pool[s].cpu(), want)
    for s in left:
        assert torch.equal(bits(pool[s]), bits(before[s]))


def test_conv_prompt_then_decode(kda):
    import torch
    d = Draw(8)
    C, T = 320, 50
    x, w = d.randn(1, T + 5, C, dtype="bf16"), d.randn(C, 4, dtype="bf16")
    whole, _ = kda.conv(x, w, activation="silu")
    a, s = kda.conv(x[:, :T].contiguous(), w, activation="silu")
    pool = torch.zeros(3, 3, C, dtype=torch.bfloat16, device="cuda")
    pool[1] = s[0]
    b = kda.conv_decode(x[:, T:].contiguous(), w, pool, ints([1]), activation="silu")
    assert torch.equal(torch.cat([a, b], 1), whole)


# ------------------------------------------------------------------------ norm and rotation

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", ["rms", "l2", None])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,offset", [(128, 128, 0), (64, 32, 32), (96, 36, 60), (80, 20, 4), (256, 256, 0), (4, 2, 2),
                                          (192, 0, 0), (160, 10, 7)])
def test_qk_norm(kda, dtype, norm, layout, D, rot, offset):
    if layout == "interleaved" and offset % 2:
        offset -= 1
    if norm is None and rot == 0:
        pytest.skip("neither a norm nor a rotation is refused (tested on the CPU)")
    import torch
    say("qk_norm", dtype, norm, layout, D, rot, offset)
    d = Draw(D + rot)
    T, Hq, Hk = 13, 6, 2
    q, k = d.randn(T, Hq, D, dtype=dtype), d.randn(T, Hk, D, dtype=dtype)
    q[3] = 0                                        # a row of zeros stays zeros
    qw, kw = (1 + 0.2 * d.randn(D), d.randn(D)) if norm else (None, None)
    pos = ints([0, 1, 2, 1000, 65535, 1 << 20, (1 << 31) - 1, -5, 7, 7, 123456, 99, 3])
    freq = (1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()
    kw_ = dict(q_weight=qw, k_weight=kw, positions=pos, inv_freq=freq, norm=norm, layout=layout, rotary_offset=offset,
               rotary_scale=1.25, eps=1e-5)
    qo, ko = kda.qk_norm(q, k, **kw_)
    for x, w, o, name in ((q, qw, qo, "q"), (k, kw, ko, "k")):
        want, mag = ref.qk_norm(ref.f64(x), ref.f64(w), norm, 1e-5, pos.cpu().numpy(), ref.f64(freq), layout, offset, 1.25)
        within(o, want, 64 * 2.0 ** -24 * mag + U[dtype] * np.abs(want), name)
    # q alone gives the same bits; in place too, on slices of one projection
    only, none = kda.qk_norm(q, q_weight=qw, **{n: v for n, v in kw_.items() if "weight" not in n})
    assert none is None and torch.equal(bits(only), bits(qo))
    fused = torch.full((T, (Hq + Hk) * D + 8), float("nan"), dtype=q.dtype, device="cuda")
    qv, kv = fused[:, :Hq * D].view(T, Hq, D), fused[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    qv.copy_(q)
    kv.copy_(k)
    kda.qk_norm(qv, kv, q_out=qv, k_out=kv, **kw_)
    assert torch.equal(bits(qv), bits(qo)) and torch.equal(bits(kv), bits(ko))
    assert torch.isnan(fused[:, (Hq + Hk) * D:]).all()


def test_qk_norm_batched_and_many_tokens(kda):
    """[B, T, H, D] with positions [B, T] gives the packed call's bits; one row a token, more tokens
    than one round of workgroups."""
    import torch
    d = Draw(21)
    q, k = d.randn(3, 1700, 5, 128, dtype="bf16"), d.randn(3, 1700, 1, 128, dtype="bf16")
    pos = ints(list(range(1700)) * 3).view(3, 1700)
    freq, scale = kda.rotary_frequencies(64, device="cuda")
    a = kda.qk_norm(q, k, positions=pos, inv_freq=freq, rotary_offset=16)
    b = kda.qk_norm(q.view(-1, 5, 128), k.view(-1, 1, 128), positions=pos.view(-1), inv_freq=freq, rotary_offset=16)
    for x, y in zip(a, b):
        assert torch.equal(bits(x).view(-1), bits(y).view(-1))
    want, mag = ref.qk_norm(ref.f64(q.view(-1, 5, 128)), None, "rms", 1e-6, pos.view(-1).cpu().numpy(), ref.f64(freq),
                            "half", 16, scale)
    within(b[0], want, 64 * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(want), "q")


def test_qk_norm_feeds_the_recurrence(kda):
    """conv -> qk_norm -> prefill as a layer runs them, against the float64 forms chained."""
    import torch

    import oracle
    d = Draw(31)
    H, D, lengths = 2, 128, [70, 0, 33]
    T, cu = sum(lengths), ints(offsets(lengths))
    x = d.randn(T, 3 * H * D, dtype="bf16")
    w = d.randn(3 * H * D, 4, dtype="bf16")
    g, beta = -5 * torch.sigmoid(d.randn(T, H, D)), torch.sigmoid(d.randn(T, H))
    y, _ = kda.conv(x, w, cu_seqlens=cu, activation="silu")
    q, k, v = (y[:, i * H * D:(i + 1) * H * D].view(T, H, D) for i in range(3))
    q, k = kda.qk_norm(q, k, norm="l2")
    out, fin = kda.prefill(q, k, v, g, beta, cu_seqlens=cu)
    yr, _, _ = ref.conv(ref.f64(x), ref.f64(w), None, None, cu.cpu(), "silu")
    yr = torch.tensor(yr).to(torch.bfloat16).double().numpy().reshape(T, 3, H, D)     # rounded where the layer rounds
    qr, kr = (ref.qk_norm(yr[:, i], None, "l2", 1e-6, None, None, "half", 0, 1.0)[0] for i in range(2))
    o_ref, s_ref = oracle.recurrence(qr, kr, yr[:, 2], ref.f64(g), ref.f64(beta), None, offsets(lengths))
    # the recurrence's own tolerance (5e-3) plus the rounding of q and k to bf16 (2^-8 each at most)
    assert oracle.rel_l2(ref.f64(out), o_ref) <= 5e-3 + 2 * 2.0 ** -8
    assert oracle.rel_l2(ref.f64(fin), s_ref) <= 5e-3 + 2 * 2.0 ** -8


@pytest.mark.parametrize("layout,rot,offset,D", [("half", 64, 0, 128), ("half", 64, 32, 128), ("half", 36, 4, 96),
                                                 ("interleaved", 40, 8, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_qk_norm_touches_pairs_alone(kda, layout, rot, offset, D, dtype):
    """Without a norm a NaN or an infinity reaches itself and, where it turns, its partner; other heads
    and tokens, and channels that do not turn, never."""
    import torch
    q = Draw(D + rot).randn(6, 9, D, dtype=dtype)
    freq, _ = kda.rotary_frequencies(rot, device="cuda")
    pos = ints([0, 5, 77, 1000, 3, 8])
    kw = dict(positions=pos, inv_freq=freq, norm=None, layout=layout, rotary_offset=offset)
    clean, _ = kda.qk_norm(q, **kw)
    for c in (0, offset, offset + 1, offset + rot // 2, offset + rot - 1, D - 1):
        for bad in (float("nan"), float("inf")):
            x = q.clone()
            x[2, 4, c] = bad
            out, _ = kda.qk_norm(x, **kw)
            hit = {c}
            if offset <= c < offset + rot:
                i = c - offset
                hit.add(offset + (i ^ 1 if layout == "interleaved" else (i + rot // 2) % rot))
            changed = (bits(out) != bits(clean)).nonzero().tolist()
            assert {(a, b) for a, b, _ in changed} == {(2, 4)} and {e for _, _, e in changed} <= hit
            assert not torch.isfinite(out[2, 4, c])


def test_qk_norm_weights_at_any_address(kda):
    """Weights that start between 16-byte boundaries, and q's and k's own."""
    import torch
    d = Draw(41)
    q, k, w = d.randn(9, 4, 128, dtype="bf16"), d.randn(9, 2, 128, dtype="bf16"), d.randn(300)
    freq, _ = kda.rotary_frequencies(128, device="cuda")
    kw = dict(positions=ints(range(9)), inv_freq=freq)
    want = kda.qk_norm(q, k, q_weight=w[1:129].clone(), k_weight=w[131:259].clone(), **kw)
    got = kda.qk_norm(q, k, q_weight=w[1:129], k_weight=w[131:259], **kw)
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))


def test_conv_nan_stays_in_its_sequence_and_channel(kda):
    """A NaN reaches the W outputs that its input feeds, and the final state where it is one of the last
    inputs."""
    import torch
    c = conv_case([40, 30], 1024, 4, "bf16", "bf16", False, 5)
    clean, cf = kda.conv(**c, activation="silu")
    for t, n in ((20, 4), (38, 2)):
        bad = dict(c, x=c["x"].clone())
        bad["x"][t, 100] = float("nan")
        out, fin = kda.conv(**bad, activation="silu")
        assert torch.isnan(out[t:t + n, 100]).all()
        changed = (bits(out) != bits(clean)).nonzero().tolist()
        assert sorted(changed) == [[t + i, 100] for i in range(n)]
        assert (bits(fin) != bits(cf)).nonzero().tolist() == ([[0, 1, 100]] if t == 38 else [])


# ----------------------------------------------------------------------- state space scan

def ssm_case(lengths, H, G, P, N, dtype, seed, gate=True, full=True, dense=False, softplus=True):
    import torch
    d = Draw(seed)
    lead = (len(lengths), lengths[0]) if dense else (sum(lengths),)
    step = torch.exp(np.log(1e-3) + d.rand(H) * np.log(1e2))
    c = dict(x=d.randn(*lead, H, P, dtype=dtype), B=d.randn(*lead, G, N, dtype=dtype), C=d.randn(*lead, G, N, dtype=dtype),
             A=-(1 + 15 * d.rand(H)), z=d.randn(*lead, H, P, dtype=dtype) if gate else None,
             D=d.randn(H) if full else None, initial_state=0.1 * d.randn(len(lengths), H, N, P) if full else None,
             cu_seqlens=None if dense else ints(offsets(lengths)), dt_softplus=softplus)
    if softplus:
        c.update(dt=d.randn(*lead, H, dtype=dtype), dt_bias=step + torch.log(-torch.expm1(-step)))
    else:
        c.update(dt=0.1 * d.rand(*lead, H), dt_bias=None)
    return c


def ssm_ref(c):
    """Packed float64 reference: out, final, mags."""
    n = {k: ref.f64(v) for k, v in c.items() if k not in ("cu_seqlens", "dt_softplus")}
    parts = []
    for i, (a, b) in enumerate(sequences_of(c)):
        s0 = None if n["initial_state"] is None else n["initial_state"][i]
        parts.append(ref.ssm(n["x"][a:b], n["dt"][a:b], n["A"], n["B"][a:b], n["C"][a:b], n["D"], n["dt_bias"],
                             None if n["z"] is None else n["z"][a:b], s0, c["dt_softplus"]))
    out, fin, mag, fmag = zip(*parts)
    return np.concatenate(out), np.stack(fin), np.concatenate(mag), np.stack(fmag)


def sequences_of(c):
    return ref.sequences(None, c["cu_seqlens"].cpu())


def check_ssm(c, out, final, dtype, state_u=0.0, want=None):
    w, f, mag, fmag = want or ssm_ref(c)
    T = max(b - a for a, b in sequences_of(c))
    acc = (512 + T) * 2.0 ** -24
    bound = acc * mag + U[dtype] * np.abs(w)
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * mag
    within(out, w, bound, "out")
    if final is not None:
        within(final, f, acc * fmag + state_u * np.abs(f), "final state")


@pytest.mark.parametrize("lengths", [[1], [32], [33, 0, 1, 64, 31], [300, 5]])
@pytest.mark.parametrize("H,G,P,N", [(2, 1, 64, 128), (3, 1, 64, 64), (4, 4, 64, 64), (2, 2, 128, 64), (2, 1, 128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prefill(kda, lengths, H, G, P, N, dtype):
    say("ssm", lengths, H, G, P, N, dtype)
    c = ssm_case(lengths, H, G, P, N, dtype, seed=H + P + N + sum(lengths), gate=H != 3, full=H != 4, softplus=G == 1)
    out, fin = kda.ssm_prefill(**c, segment=-1)
    want = ssm_ref(c)
    check_ssm(c, out, fin, dtype, want=want)
    # cut into segments
    for seg in (32, 64):
        o2, f2 = kda.ssm_prefill(**c, segment=seg)
        check_ssm(c, o2, f2, dtype, want=want)


def test_ssm_planned_segments_repeat_bits(kda):
    """The planner's own segments on a batch long enough for them: right, and the same bits twice."""
    import torch
    c = ssm_case([700, 0, 1, 1300], 2, 1, 64, 64, "bf16", seed=77)
    out, fin = kda.ssm_prefill(**c)
    check_ssm(c, out, fin, "bf16")
    o2, f2 = kda.ssm_prefill(**c)
    assert torch.equal(bits(out), bits(o2)) and torch.equal(bits(fin), bits(f2))


@pytest.mark.parametrize("segment", [-1, 64])
def test_ssm_layouts_states_and_views(kda, segment):
    """Dense gives packed's bits; padded views (aligned to 4 elements only) with NaN around them give
    the contiguous call's bits and leave the padding; the state in place; bf16 states; dt in fp32."""
    import torch
    c = ssm_case([100, 100], 4, 2, 64, 128, "bf16", seed=3, dense=True)
    out, fin = kda.ssm_prefill(**c, segment=segment)
    flat = {k: v.reshape((200,) + v.shape[2:]) if k in ("x", "B", "C", "z", "dt") else v for k, v in c.items()}
    flat["cu_seqlens"] = ints([0, 100, 200])
    po, pf = kda.ssm_prefill(**flat, segment=segment)
    if segment == -1:       # (dense and packed segments start at the same tokens here too)
        assert torch.equal(bits(po).view(-1), bits(out).view(-1)) and torch.equal(pf, fin)
    check_ssm(flat, po, pf, "bf16")
    views = {}
    for k in ("x", "B", "C", "z", "initial_state"):
        views[k] = padded(c[k], 4)[0]
    ov, ob = padded(torch.zeros_like(c["x"]), 4)
    fv, fb = padded(torch.zeros_like(fin), 4)
    kda.ssm_prefill(**dict(c, **views), segment=segment, out=ov, final_state=fv)
    assert torch.equal(bits(ov), bits(out)) and torch.equal(fv, fin)
    assert torch.isnan(ob[..., 64:]).all() and torch.isnan(ob[:, :, 4:]).all() and torch.isnan(fb[..., 64:]).all()
    s = c["initial_state"].clone()
    o2, f2 = kda.ssm_prefill(**dict(c, initial_state=s), final_state=s, segment=segment)
    assert f2 is s and torch.equal(s, fin) and torch.equal(bits(o2), bits(out))
    half = flat["initial_state"].to(torch.bfloat16)
    cb = dict(flat, initial_state=half, dt=flat["dt"].float())
    f3 = torch.zeros_like(half)
    o3, _ = kda.ssm_prefill(**cb, final_state=f3, segment=segment)
    check_ssm(cb, o3, f3, "bf16", state_u=2.0 ** -8)


def test_ssm_decay_extremes(kda):
    """Steps of zero (nothing decays, nothing enters), decays that empty the state within a token,
    and both beside slow ones, over chunk and segment borders."""
    import torch
    c = ssm_case([150], 4, 1, 64, 64, "f32", seed=12, softplus=False)
    c["dt"][:, 0] = 0
    c["A"][1] = -4000.0
    c["dt"][40:60, 2] = 20.0
    c["dt"][::7, 3] = 0
    for seg in (-1, 64):
        out, fin = kda.ssm_prefill(**c, segment=seg)
        check_ssm(c, out, fin, "f32")
        assert torch.equal(fin[0, 0], c["initial_state"][0, 0])


def test_ssm_empty_and_behind(kda):
    """Empty sequences keep their state bit for bit; rows behind the last sequence stay."""
    import torch
    c = ssm_case([0, 40, 0], 2, 1, 64, 64, "bf16", seed=13)
    big = {k: torch.cat([c[k], torch.full_like(c[k], float("nan"))]) for k in ("x", "B", "C", "z", "dt")}
    want, wf = kda.ssm_prefill(**c, segment=-1)
    for seg in (-1, 32):
        out = torch.full_like(big["x"], -512.0)
        _, fin = kda.ssm_prefill(**dict(c, **big), out=out, segment=seg)
        assert torch.equal(fin[0], c["initial_state"][0]) and torch.equal(fin[2], c["initial_state"][2])
        assert (out[40:] == -512.0).all()
        if seg == -1:
            assert torch.equal(bits(out[:40]), bits(want)) and torch.equal(fin, wf)
    none = kda.ssm_prefill(**{k: (v[:0] if k in ("x", "B", "C", "z", "dt") else v) for k, v in c.items()
                              if k not in ("cu_seqlens",)}, cu_seqlens=ints([0, 0, 0, 0]))
    assert torch.equal(none[1], c["initial_state"])


@pytest.mark.parametrize("lengths", [[1], [10], [1, 2, 0, 30], [33, 0, 170]])
@pytest.mark.parametrize("H,G,P,N", [(2, 1, 64, 128), (1, 1, 64, 64), (2, 2, 128, 64), (2, 1, 128, 128)])
@pytest.mark.parametrize("gate", [True, False])
def test_ssm_few_tokens_round_once(kda, lengths, H, G, P, N, gate):
    """bf16 batches of few tokens: two bf16 parts (a rest of 2^-16) of the weighted x, of B C^T and of the
    state that feeds the output, so 3 x 2^-16 of the magnitudes beside the output's one rounding.  Some
    heads decay by more than 2^96 a chunk."""
    c = ssm_case(lengths, H, G, P, N, "bf16", seed=sum(lengths) + P + N, gate=gate)
    for strong in (False, True):
        if strong:
            c["A"][0] = -60.0
        out, fin = kda.ssm_prefill(**c)
        w, f, mag, fmag = ssm_ref(c)
        acc = (512 + max(lengths)) * 2.0 ** -24
        within(out, w, (acc + 3 * 2.0 ** -16) * mag + U["bf16"] * np.abs(w), "out")
        within(fin, f, acc * fmag, "final state")


@pytest.mark.parametrize("lengths", [[64, 64, 0, 128, 65, 63, 1], [192, 96, 96], [0, 0, 31, 0], [97, 1, 1, 1, 127]])
@pytest.mark.parametrize("behind", [0, 70])
def test_ssm_segments_of_packed_batches(kda, lengths, behind):
    """Lengths at and around multiples of the segment, empty sequences, rows behind the last one (not
    read: they hold NaN; left as they were)."""
    import torch
    rows = sum(lengths)
    c = ssm_case(lengths, 2, 1, 64, 64, "bf16", seed=rows + behind)
    want = ssm_ref(c)
    for seg in (32, 64, 96):
        call = dict(c)
        for key in ("x", "dt", "B", "C", "z"):
            pad = torch.full((behind, *c[key].shape[1:]), float("nan"), dtype=c[key].dtype, device="cuda")
            call[key] = torch.cat([c[key], pad])
        out = torch.full_like(call["x"], -7.0)
        _, fin = kda.ssm_prefill(**call, out=out, segment=seg)
        check_ssm(c, out[:rows], fin, "bf16", want=want)
        assert (out[rows:] == -7.0).all()


@pytest.mark.parametrize("P,N,dtype", [(64, 128, "bf16"), (128, 128, "bf16"), (128, 64, "f32")])
def test_ssm_start_states_both_ways(kda, P, N, dtype):
    """Final states in place go through the scan's own launch, others mostly not: the same bits."""
    import torch
    c = ssm_case([700, 0, 330, 1, 64], 4, 2, P, N, dtype, seed=P + N)
    for seg in (32, 128, 320):
        out, fin = kda.ssm_prefill(**c, segment=seg)
        s0 = c["initial_state"].clone()
        out2, fin2 = kda.ssm_prefill(**dict(c, initial_state=s0), final_state=s0, segment=seg)
        assert fin2 is s0 and torch.equal(bits(out), bits(out2)) and torch.equal(fin, s0)


def test_layer_without_sequences(kda):
    """cu_seqlens of no sequence: nothing is read or written."""
    import torch
    c = ssm_case([80], 2, 1, 64, 64, "bf16", seed=3, full=False)
    c["cu_seqlens"] = ints([0])
    for seg in (0, -1, 32):
        out = torch.full_like(c["x"], -7.0)
        _, fin = kda.ssm_prefill(**c, out=out, segment=seg)
        assert (out == -7.0).all() and fin.shape == (0, 2, 64, 64)
    x = Draw(1).randn(80, 16, dtype="bf16")
    out = torch.full_like(x, -7.0)
    _, fin = kda.conv(x, Draw(2).randn(16, 4, dtype="bf16"), cu_seqlens=ints([0]), out=out)
    assert (out == -7.0).all() and fin.shape == (0, 3, 16)


def test_ssm_cached_workspace_entry(kda):
    """kda_ssm_prefill (the library's own workspace) gives kda_ssm_prefill_ws's bits, twice in a row,
    the second time with a smaller batch."""
    import ctypes

    import torch

    from test_layer_abi import SsmOptions
    lib = kda.load_library()
    for lengths in ([500, 130], [200]):
        c = ssm_case(lengths, 2, 1, 64, 128, "bf16", seed=len(lengths))
        want, wf = kda.ssm_prefill(**c, segment=64)
        out, fin = torch.full_like(want, float("nan")), torch.full_like(wf, float("nan"))
        ds = {k: kda.describe(v) for k, v in c.items() if isinstance(v, torch.Tensor)}
        ds["out"], ds["final"] = kda.describe(out), kda.describe(fin)
        a = {k: ctypes.addressof(d) for k, d in ds.items()}
        o = SsmOptions(a["D"], a["dt_bias"], a["z"], 1, 64)
        st = lib.kda_ssm_prefill(a["x"], a["dt"], a["A"], a["B"], a["C"], a["initial_state"], a["cu_seqlens"], a["out"],
                                 a["final"], ctypes.addressof(o), torch.cuda.current_stream().cuda_stream)
        assert st == 0, lib.kda_last_error()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want)) and torch.equal(fin, wf)
    kda.release_cached_workspace()


def test_ssm_nan_stays_in_its_sequence_and_head(kda):
    """A NaN in x or dt reaches its own sequence and head alone, later tokens for certain and at most 31
    tokens before; one in C its own token alone."""
    import torch
    c = ssm_case([100, 90], 4, 1, 64, 64, "bf16", seed=15)
    clean, cf = kda.ssm_prefill(**c, segment=-1)
    for key, at in (("x", (50, 1, 7)), ("dt", (50, 1))):
        bad = dict(c, **{key: c[key].clone()})
        bad[key][at] = float("nan")
        for seg in (-1, 32):
            out, fin = kda.ssm_prefill(**bad, segment=seg)
            ref_out, ref_fin = kda.ssm_prefill(**c, segment=seg)
            assert torch.equal(bits(out[100:]), bits(ref_out[100:])) and torch.equal(fin[1], ref_fin[1])
            heads = [0, 2, 3]
            assert torch.equal(bits(out[:, heads]), bits(ref_out[:, heads])) and torch.equal(fin[:, heads], ref_fin[:, heads])
            cols = [7] if key == "x" else list(range(64))
            assert torch.isnan(out[50:100, 1][:, cols]).all() and torch.isnan(fin[0, 1][:, cols]).all()
            assert torch.equal(bits(out[:32]), bits(ref_out[:32]))
    bad = dict(c, C=c["C"].clone())
    bad["C"][50, 0, 3] = float("nan")
    out, fin = kda.ssm_prefill(**bad, segment=-1)
    keep = [t for t in range(190) if t != 50]
    assert torch.isnan(out[50]).all() and torch.equal(bits(out[keep]), bits(clean[keep])) and torch.equal(fin, cf)


def test_ssm_growth_and_long_decay(kda):
    """Heads that grow (A step > 0), and references that move many times: slow decay over 3,000 tokens,
    against the float64 recurrence."""
    c = ssm_case([3000], 3, 1, 64, 64, "f32", seed=19, gate=False, softplus=False)
    c["A"][0], c["A"][1], c["A"][2] = 0.2, -0.5, -30.0
    c["dt"][:, 0] *= 0.1
    for seg in (-1, 512):
        out, fin = kda.ssm_prefill(**c, segment=seg)
        check_ssm(c, out, fin, "f32")


@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("H,G,P,N", [(2, 1, 64, 128), (4, 2, 64, 64), (3, 1, 128, 64), (2, 2, 128, 128)])
@pytest.mark.parametrize("dtype,state", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
def test_ssm_decode(kda, T, H, G, P, N, dtype, state):
    import torch
    say("ssm_decode", T, H, G, P, N, dtype, state)
    R, slots = 5, 7
    c = ssm_case([T] * R, H, G, P, N, dtype, seed=T + H + P, dense=True, gate=H != 3)
    c.pop("cu_seqlens"), c.pop("initial_state")
    pool = 0.1 * Draw(4).randn(slots, H, N, P)
    pool = pool.to(dtype_of(state))
    before = pool.clone()
    idx, counts = [6, -1, 0, 3, 7], [T, T, T + 2, max(T - 1, 0), T]
    verify = kda.ssm_decode(**c, state_pool=pool, state_indices=ints(idx), num_tokens=ints(counts), update_state=False)
    assert torch.equal(bits(pool), bits(before))
    out = torch.full_like(c["x"], -512.0)
    kda.ssm_decode(**c, state_pool=pool, state_indices=ints(idx), num_tokens=ints(counts), out=out)
    commit = before.clone()
    kda.ssm_decode(**c, state_pool=commit, state_indices=ints(idx), num_tokens=ints(counts), write_out=False)
    assert torch.equal(bits(commit), bits(pool))
    n = {k: ref.f64(v) for k, v in c.items() if k != "dt_softplus"}
    left = set(range(slots))
    acc = (512 + T) * 2.0 ** -24
    for r, (s, m) in enumerate(zip(idx, counts)):
        m = min(m, T) if 0 <= s < slots else 0
        assert (out[r, m:].float() == -512.0).all()
        if not 0 <= s < slots:
            continue
        left.discard(s)
        w, f, mag, fmag = ref.ssm(n["x"][r, :m], n["dt"][r, :m], n["A"], n["B"][r, :m], n["C"][r, :m], n["D"], n["dt_bias"],
                                  None if n["z"] is None else n["z"][r, :m], ref.f64(before[s]), True)
        within(out[r, :m], w, acc * mag + U[dtype] * np.abs(w), f"request {r}")
        within(pool[s], f, acc * fmag + (U["bf16"] if state == "bf16" else 0) * np.abs(f), f"slot {s}")
        assert torch.equal(bits(verify[r, :m]), bits(out[r, :m]))
    for s in left:
        assert torch.equal(bits(pool[s]), bits(before[s]))


def test_ssm_prompt_then_decode_and_conv(kda):
    """A layer as it is served: convolution and scan over a prompt, then tokens one by one from the
    pools, against the float64 forms of the whole run."""
    import torch
    d = Draw(41)
    H, P, N, T, more = 2, 64, 64, 45, 6
    width = H * P + 2 * N
    x, w = d.randn(1, T + more, width, dtype="f32"), 0.5 * d.randn(width, 4)
    dt, A, D = d.randn(1, T + more, H), -(1 + d.rand(H)), d.randn(H)

    def split(y):
        return (y[..., :H * P].unflatten(-1, (H, P)), y[..., H * P:H * P + N].unflatten(-1, (1, N)),
                y[..., H * P + N:].unflatten(-1, (1, N)))

    y, cs = kda.conv(x[:, :T].contiguous(), w, activation="silu")
    xs, B, C = split(y)
    out, ss = kda.ssm_prefill(xs, dt[:, :T].contiguous(), A, B, C, D=D, dt_softplus=True)
    outs = [out]
    idx = ints([0])
    for t in range(T, T + more):
        y = kda.conv_decode(x[:, t:t + 1].contiguous(), w, cs, idx, activation="silu")
        xs, B, C = split(y)
        outs.append(kda.ssm_decode(xs, dt[:, t:t + 1].contiguous(), A, B, C, ss, idx, D=D, dt_softplus=True))
    got = torch.cat(outs, 1)[0]
    yr, _, ymag = ref.conv(ref.f64(x[0]), ref.f64(w), None, None, [0, T + more], "silu")
    xr, Br, Cr = yr[:, :H * P].reshape(-1, H, P), yr[:, None, H * P:H * P + N], yr[:, None, H * P + N:]
    want, fin, mag, fmag = ref.ssm(xr, ref.f64(dt[0]), ref.f64(A), Br, Cr, ref.f64(D), None, None, None, True)
    # the convolution's own bound enters through x, B and C: relative to its largest magnitude
    rel = 3 * 64 * 2.0 ** -24 * ymag.max() / np.sqrt((yr * yr).mean())
    within(got, want, (512 + T) * 2.0 ** -24 * mag + rel * mag.max(), "out")
    within(ss[0], fin, (512 + T) * 2.0 ** -24 * fmag + rel * fmag.max(), "state")


# ------------------------------------------------------------------ streams, graphs, shared use

def test_layer_calls_from_two_streams_at_once(kda):
    """The same segmented scan in flight on two streams at once (each with its own workspace): both
    give the lone call's bits."""
    import torch
    c = ssm_case([900, 400], 4, 1, 64, 128, "bf16", seed=71)
    want, wf = kda.ssm_prefill(**c, segment=64)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [kda.ssm_prefill(**c, segment=64, stream=s) for _ in range(5) for s in streams]
    for s in streams:
        s.synchronize()
    for out, fin in got:
        assert torch.equal(bits(out), bits(want)) and torch.equal(fin, wf)


def test_layer_large_offsets(kda):
    """Tensors past 2^31 elements (5 GB of x): the last rows are right."""
    import torch
    rows, C = 17 * 4096, 32768          # 2.28e9 elements
    x = torch.zeros(rows, C, dtype=torch.bfloat16, device="cuda")
    d = Draw(81)
    x[-40:] = d.randn(40, C, dtype="bf16")
    w = d.randn(C, 4, dtype="bf16")
    out = torch.full((rows, C), -512.0, dtype=torch.bfloat16, device="cuda")
    kda.conv(x, w, cu_seqlens=ints([0, rows]), out=out, activation="silu", output_final_state=False)
    want, _ = kda.conv(x[-40:].contiguous(), w, cu_seqlens=ints([0, 40]), activation="silu")
    assert torch.equal(bits(out[-40:]), bits(want)) and (out[:rows - 40] == 0).all()
    q = x.view(rows, C // 128, 128)
    qo, _ = kda.qk_norm(q, norm="l2", q_out=out.view(rows, C // 128, 128))
    small, _ = kda.qk_norm(q[-40:].contiguous(), norm="l2")
    assert torch.equal(bits(qo[-40:]), bits(small))
    H = C // 64 // 2
    xs = x[:, :H * 64].unflatten(1, (H, 64))                # rows 2 x the width apart
    c = dict(dt=torch.zeros(rows, H, device="cuda"), A=-torch.ones(H, device="cuda"), B=d.randn(rows, 1, 64, dtype="bf16"),
             C=d.randn(rows, 1, 64, dtype="bf16"), D=None, dt_bias=None, z=None, initial_state=None, dt_softplus=True)
    ys, fs = kda.ssm_prefill(xs, **c, cu_seqlens=ints([0, rows]))
    # the tokens before the last 40 add nothing, so the last 64 alone have the same result
    tail = {k: (v[-64:].contiguous() if k in ("dt", "B", "C") else v) for k, v in c.items()}
    check_ssm(dict(tail, x=xs[-64:].contiguous(), cu_seqlens=ints([0, 64])), ys[-64:], fs, "bf16")
    assert (ys[:rows - 64] == 0).all()


def test_layer_on_other_stream_and_in_a_graph(kda):
    """The whole step on a stream of its own, then captured and replayed on changed inputs, with
    eager work between the replays: every replay equals the eager result."""
    import torch
    d = Draw(51)
    R, H, P, N = 3, 2, 64, 64
    width = H * P + 2 * N
    x, w, dt, A = d.randn(R, 1, width, dtype="bf16"), d.randn(width, 4, dtype="bf16"), d.randn(R, 1, H), -(1 + d.rand(H))
    conv_pool, state_pool, idx = d.randn(R, 3, width, dtype="bf16"), 0.1 * d.randn(R, H, N, P), ints([2, 0, 1])
    prompt = ssm_case([100, 30], H, 1, P, N, "bf16", seed=52)

    def step(conv_p, state_p):
        y = kda.conv_decode(x, w, conv_p, idx, activation="silu")
        xs = y[..., :H * P].unflatten(-1, (H, P))
        B, C = y[..., H * P:H * P + N].unflatten(-1, (1, N)), y[..., H * P + N:].unflatten(-1, (1, N))
        B, _ = kda.qk_norm(B, norm="l2")
        o = kda.ssm_decode(xs, dt, A, B, C, state_p, idx, dt_softplus=True)
        p, f = kda.ssm_prefill(**prompt, segment=32)
        return o, p, f

    eager = step(conv_pool.clone(), state_pool.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(conv_pool.clone(), state_pool.clone())
    given = kda.conv_decode(x, w, conv_pool.clone(), idx, activation="silu", stream=side)
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(bits(a), bits(b))
    cp, sp = conv_pool.clone(), state_pool.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        captured = step(cp, sp)
    for i in range(4):
        x.copy_(d.randn(R, 1, width, dtype="bf16"))
        prompt["x"].copy_(d.randn(*prompt["x"].shape, dtype="bf16"))
        cp.copy_(conv_pool)
        sp.copy_(state_pool)
        c2, s2 = conv_pool.clone(), state_pool.clone()
        want = step(c2, s2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(bits(a), bits(b)), i
        assert torch.equal(cp, c2) and torch.equal(sp, s2)
    assert given.shape == x.shape


def test_layer_device_checks(kda, monkeypatch):
    """KDA_CHECK=1: bad cu_seqlens and slots named twice are refused before anything runs."""
    import torch
    monkeypatch.setenv("KDA_CHECK", "1")
    d = Draw(91)
    x, w = d.randn(20, 64, dtype="bf16"), d.randn(64, 4, dtype="bf16")
    c = ssm_case([20], 2, 1, 64, 64, "bf16", seed=1, full=False)
    for cu in ([0, 21], [0, 12, 8, 20], [1, 20]):
        out = torch.full_like(x, -7.0)
        with pytest.raises(kda.KdaError):
            kda.conv(x, w, cu_seqlens=ints(cu), out=out)
        y = torch.full_like(c["x"], -7.0)
        with pytest.raises(kda.KdaError):
            kda.ssm_prefill(**dict(c, cu_seqlens=ints(cu)), out=y)
        assert (out == -7.0).all() and (y == -7.0).all()
    assert kda.conv(x, w, cu_seqlens=ints([0, 20]))[0].isfinite().all()
    pool, xs = d.randn(4, 3, 64), d.randn(3, 1, 64, dtype="bf16")
    states, before = d.randn(4, 2, 64, 64), pool.clone()
    s = {k: v for k, v in ssm_case([1] * 3, 2, 1, 64, 64, "bf16", seed=2, dense=True, full=False).items()
         if k not in ("cu_seqlens", "initial_state")}
    with pytest.raises(kda.KdaError):
        kda.conv_decode(xs, w, pool, ints([2, 1, 2]))
    with pytest.raises(kda.KdaError):
        kda.ssm_decode(**s, state_pool=states, state_indices=ints([2, 1, 2]))
    assert torch.equal(pool, before)
    # reading one slot twice is allowed, and gives equal requests equal outputs
    xs[2] = xs[0]
    out = kda.conv_decode(xs, w, pool, ints([2, 1, 2]), update_state=False)
    assert torch.equal(bits(out[0]), bits(out[2])) and torch.equal(pool, before)
    kda.conv_decode(xs, w, pool, ints([2, 1, -1]))


def test_ssm_workspace_misuse(kda):
    import torch
    c = ssm_case([300], 2, 1, 64, 64, "bf16", seed=7)
    need = kda.ssm_workspace_size(*(c[k] for k in ("x", "dt", "A", "B", "C", "initial_state", "cu_seqlens")), segment=64)
    want, wf = kda.ssm_prefill(**c, segment=64)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")       # NaN in every word
    out, fin = kda.ssm_prefill(**c, segment=64, workspace=ws)
    assert torch.equal(bits(out), bits(want)) and torch.equal(fin, wf)
    with pytest.raises(kda.KdaError):
        kda.ssm_prefill(**c, segment=64, workspace=ws[:need // 2])
    for bad in (torch.empty(need + 256, dtype=torch.uint8), ws[::2], 5):
        with pytest.raises(ValueError):
            kda.ssm_prefill(**c, segment=64, workspace=bad)


def test_layer_profile_names(kda):
    c = ssm_case([100], 2, 1, 64, 64, "bf16", seed=61)
    for final, want in ((None, {"kda_ssm_states": 1, "kda_ssm": 1}),
                        (c["initial_state"], {"kda_ssm_states": 1, "kda_ssm_scan": 1, "kda_ssm": 1})):
        kda.profile_enable(True)
        try:
            kda.profile_read()
            kda.ssm_prefill(**c, final_state=final, segment=32)
            names = kda.profile_read_kernels()
        finally:
            kda.profile_enable(False)
        assert {k: v[0] for k, v in names.items()} == want
