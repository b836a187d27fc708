"""The operators around the delta-rule recurrence, as they are timed: the short causal convolution
in front of it, the norm and position rotation of its queries and keys, and the selective state
space scan that stands beside it, for prompts and for single tokens.

``own`` False computes each in plain torch operations in 32 bits (angles and long sums in 64);
``own`` True calls the library.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}

# Eight packed prompts of mixed lengths (the packed workload of this repository's benchmark).
PACKED = "1232,6808,5353,2957,727,5757,2852,7047"


def listed():
    return [
        # the convolution of q, k and v of a 32-head layer in one call, a packed prefill batch
        dict(name="conv prompt packed", op="conv", lengths=PACKED, channels=12288, width=4, silu=True, bias=False,
             dtype="bf16", state="bf16"),
        # a short ragged batch with an empty request, 32-bit data, an odd number of channels
        dict(name="conv prompt small odd", op="conv", lengths="17,0,16", channels=515, width=3, silu=False,
             bias=True, dtype="f32", state="f32"),
        # a decode step of 256 requests
        dict(name="conv decode", op="conv_decode", requests=256, tokens=1, channels=12288, width=4, silu=True,
             bias=False, dtype="bf16", state="bf16", slots=512),
        # a few drafted tokens of a few requests
        dict(name="conv drafts small", op="conv_decode", requests=5, tokens=4, channels=1280, width=4, silu=True,
             bias=True, dtype="bf16", state="f32", slots=8),
        # a packed prefill batch, 64 heads of 64 channels, one B and C for all heads, gated output
        dict(name="scan prompt packed", op="scan", lengths=PACKED, heads=64, groups=1, P=64, N=128, gate=True,
             dtype="bf16"),
        # one very long prompt, few heads
        dict(name="scan prompt long", op="scan", lengths="65536", heads=8, groups=8, P=128, N=128, gate=False,
             dtype="bf16"),
        # an ordinary batch of two prompts
        dict(name="scan prompt pair", op="scan", lengths="4096,4096", heads=16, groups=2, P=64, N=64, gate=True,
             dtype="bf16"),
        # a ragged batch with an empty request in 32 bits: latency
        dict(name="scan prompt small f32", op="scan", lengths="33,0,170", heads=4, groups=2, P=64, N=64, gate=False,
             dtype="f32"),
        # a decode step of 256 requests against a pool of 32-bit states
        dict(name="scan decode", op="scan_decode", requests=256, tokens=1, heads=32, groups=1, P=64, N=128, gate=True,
             dtype="bf16", state="f32", slots=512),
        # a few drafted tokens of a few requests, states in bf16
        dict(name="scan drafts small", op="scan_decode", requests=5, tokens=4, heads=8, groups=2, P=128, N=64,
             gate=False, dtype="bf16", state="bf16", slots=8),
        # queries and keys of a packed prefill batch, RMS norm and the whole head rotated
        dict(name="qk norm prompt", op="qk_norm", tokens=32733, q_heads=32, k_heads=8, D=128, rot=128, offset=0,
             layout="half", norm="rms", weight=True, dtype="bf16"),
        # queries and keys of a decode step: unit length, part of the head rotated, neighbouring pairs
        dict(name="qk norm decode", op="qk_norm", tokens=7, q_heads=16, k_heads=16, D=96, rot=36, offset=60,
             layout="interleaved", norm="l2", weight=False, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ragged(rng, tokens, seqs):
    cuts = sorted(rng.randint(0, tokens) for _ in range(seqs - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [tokens]))


def draw(rng):
    op = rng.choice(["conv", "conv_decode", "scan", "scan", "scan_decode", "qk_norm"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    if op == "conv":
        channels = _spread(rng, 60, 8192)
        if rng.random() < 0.7:
            channels = 8 * max(1, channels // 8)
        return dict(op=op, lengths=_ragged(rng, _spread(rng, 1, 32768), rng.randint(1, 12)), channels=channels,
                    width=rng.randint(2, 4), silu=rng.random() < 0.7, bias=rng.random() < 0.5, dtype=dtype,
                    state=rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32")
    if op == "conv_decode":
        requests = _spread(rng, 1, 384)
        return dict(op=op, requests=requests, tokens=rng.randint(1, 8), channels=8 * _spread(rng, 8, 1024),
                    width=rng.randint(2, 4), silu=rng.random() < 0.7, bias=rng.random() < 0.5, dtype=dtype,
                    state=rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32",
                    slots=requests + rng.randint(0, 128))
    P, N = rng.choice([64, 128]), rng.choice([64, 128])
    groups = rng.choice([1, 2, 4])
    if op == "scan":
        tokens = _spread(rng, 1, 32768 if dtype == "bf16" else 4096)
        heads = groups * _spread(rng, 1, max(1, min(64, 2 ** 20 // tokens) // groups))
        return dict(op=op, lengths=_ragged(rng, tokens, rng.randint(1, 12)), heads=heads, groups=groups, P=P, N=N,
                    gate=rng.random() < 0.5, dtype=dtype)
    if op == "scan_decode":
        requests = _spread(rng, 1, 256)
        return dict(op=op, requests=requests, tokens=rng.randint(1, 8), heads=groups * _spread(rng, 1, 32 // groups),
                    groups=groups, P=P, N=N, gate=rng.random() < 0.5, dtype=dtype,
                    state=rng.choice(["bf16", "f32"]) if dtype == "bf16" else "f32",
                    slots=requests + rng.randint(0, 64))
    D = rng.choice([64, 80, 96, 128, 160, 192, 256])
    norm = rng.choice(["rms", "l2", "none"])
    rot = 2 * rng.randint(1 if norm == "none" else 0, D // 2)
    q_heads = _spread(rng, 1, 32)
    return dict(op=op, tokens=_spread(rng, 1, 16384), q_heads=q_heads, k_heads=rng.randint(1, q_heads), D=D, rot=rot,
                offset=2 * rng.randint(0, (D - rot) // 2), layout=rng.choice(["half", "interleaved"]),
                norm=norm, weight=norm != "none" and rng.random() < 0.5, dtype=dtype)


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    dt = DTYPES[case["dtype"]]
    op = case["op"]
    s = dict(op=op)
    if op in ("conv", "conv_decode"):
        C, W = case["channels"], case["width"]
        s["weight"] = (randn(C, W) / W ** 0.5).to(dt)
        s["bias"] = (0.1 * randn(C)).to(dt) if case["bias"] else None
        s["activation"] = "silu" if case["silu"] else None
    if op in ("scan", "scan_decode"):
        H = case["heads"]
        s["A"] = -(1 + 15 * rand(H))
        # step sizes spread over [0.001, 0.1] as such layers start out
        step = torch.exp(math.log(1e-3) + rand(H) * math.log(1e2))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = randn(H)
    if op in ("conv", "scan"):
        lengths = _lengths(case)
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["longest"] = max(lengths)
        n_seq, lead = len(lengths), (cu[-1],)
    if op in ("conv_decode", "scan_decode"):
        R = case["requests"]
        lead = (R, case["tokens"])
        s["indices"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:R].to(torch.int32)
    if op == "conv":
        s["x"] = randn(*lead, C).to(dt)
        s["initial"] = randn(n_seq, W - 1, C).to(DTYPES[case["state"]])
    elif op == "conv_decode":
        s["x"] = randn(*lead, C).to(dt)
        s["pool"] = randn(case["slots"], W - 1, C).to(DTYPES[case["state"]])
    elif op in ("scan", "scan_decode"):
        P, N, G = case["P"], case["N"], case["groups"]
        s["x"] = randn(*lead, H, P).to(dt)
        s["B"], s["C"] = randn(*lead, G, N).to(dt), randn(*lead, G, N).to(dt)
        s["dt"] = randn(*lead, H).to(dt)
        s["z"] = randn(*lead, H, P).to(dt) if case["gate"] else None
        if op == "scan":
            s["initial"] = 0.1 * randn(n_seq, H, N, P)
        else:
            s["pool"] = (0.1 * randn(case["slots"], H, N, P)).to(DTYPES[case["state"]])
    else:
        T, D, rot = case["tokens"], case["D"], case["rot"]
        s["q"], s["k"] = randn(T, case["q_heads"], D).to(dt), randn(T, case["k_heads"], D).to(dt)
        s["q_weight"] = 1 + 0.1 * randn(D) if case["weight"] else None
        s["k_weight"] = 1 + 0.1 * randn(D) if case["weight"] else None
        # tokens anywhere in a context of 2^20
        s["positions"] = torch.randint(0, 1 << 20, (T,), generator=gen, device="cuda", dtype=torch.int32)
        s["inv_freq"] = (1e6 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(1, rot))).float()
        s["norm"] = None if case["norm"] == "none" else case["norm"]
        s["layout"], s["offset"] = case["layout"], case["offset"]
    return s


# ------------------------------------------------------------------------------ plain forms

def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(x, weight, bias, initial, cu, activation):
    T, C = x.shape
    W = weight.shape[1]
    N = cu.numel() - 1
    cu = cu.long()
    rows = torch.cat([initial.float().reshape(N * (W - 1), C), x.float()])  # states, then tokens
    taps = torch.arange(W, device=x.device) - (W - 1)
    t = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)

    def source(pos, n):     # row of position pos of sequence n, in its state where pos < 0
        return torch.where(pos >= 0, N * (W - 1) + cu[n] + pos, n * (W - 1) + W - 1 + pos)

    src = source((t - cu[seq])[:, None] + taps, seq[:, None])
    y = (rows[src] * weight.float().t()).sum(1)
    if bias is not None:
        y = y + bias.float()
    if activation == "silu":
        y = _silu(y)
    n = torch.arange(N, device=x.device)
    final = rows[source((cu[1:] - cu[:-1])[:, None] + taps[:-1], n[:, None])]
    return y.to(x.dtype), final.to(initial.dtype)


def _plain_conv_decode(x, weight, bias, pool, indices, activation):
    R, T, C = x.shape
    W = weight.shape[1]
    idx = indices.long()
    rows = torch.cat([pool[idx].float(), x.float()], 1)                 # [R, W - 1 + T, C]
    y = (rows.unfold(1, W, 1) * weight.float()).sum(-1)
    if bias is not None:
        y = y + bias.float()
    if activation == "silu":
        y = _silu(y)
    pool[idx] = rows[:, T:].to(pool.dtype)
    return y.to(x.dtype), pool


def _steps(dt, dt_bias):
    """softplus(dt + bias) in 32 bits."""
    v = dt.float() + dt_bias
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _heads(x, H):
    """[..., G, N] to [..., H, N]: head h reads group h / (H / G)."""
    return x.repeat_interleave(H // x.shape[-2], -2)


def _plain_scan(x, step, A, B, C, initial):
    """The scan of [n, T] tokens in chunks, every chunk at once: within a chunk by its matrix of
    decays, between chunks by theirs.  Tokens with step 0 change nothing."""
    n, T, H, P = x.shape
    G, N = B.shape[-2:]
    L = min(64, T)
    c = -(-T // L)
    pad = c * L - T
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, pad)).view(n, c, L, H, P).transpose(2, 3)
    step = torch.nn.functional.pad(step, (0, 0, 0, pad)).view(n, c, L, H).transpose(2, 3)
    B = torch.nn.functional.pad(B.float(), (0, 0, 0, 0, 0, pad)).view(n, c, L, G, N).transpose(2, 3).contiguous()
    C = torch.nn.functional.pad(C.float(), (0, 0, 0, 0, 0, pad)).view(n, c, L, G, N).transpose(2, 3).contiguous()
    cum = torch.cumsum((step * A[:, None]).double(), -1)                # [n, c, H, L]
    low = torch.ones(L, L, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).float().masked_fill(~low, -math.inf))
    pair = torch.matmul(C, B.transpose(-1, -2).contiguous()).repeat_interleave(H // G, 2) * decay
    y = torch.matmul(pair * step[..., None, :], x)
    left = torch.exp((cum[..., -1:] - cum).float()) * step              # what a token leaves at the chunk's end
    Bh = B.repeat_interleave(H // G, 2)
    add = torch.matmul(Bh.transpose(-1, -2).contiguous(), left[..., None] * x)  # [n, c, H, N, P]
    total = torch.nn.functional.pad(torch.cumsum(cum[..., -1], 1).transpose(1, 2), (1, 0))  # [n, H, c + 1]
    low = torch.ones(c + 1, c + 1, dtype=torch.bool, device=x.device).tril()
    carry = torch.exp((total[..., :, None] - total[..., None, :]).float().masked_fill(~low, -math.inf))
    states = torch.cat([initial.float()[:, None], add], 1).transpose(1, 2).reshape(n, H, c + 1, N * P)
    states = torch.matmul(carry, states).view(n, H, c + 1, N, P)
    start = states[:, :, :-1].transpose(1, 2)                           # [n, c, H, N, P]
    Ch = C.repeat_interleave(H // G, 2) * torch.exp(cum.float())[..., None]
    y = y + torch.matmul(Ch, start)
    return y.transpose(2, 3).reshape(n, c * L, H, P)[:, :T], states[:, :, -1]


def _plain_scan_prompt(s):
    x, cu, H = s["x"], s["cu"].long(), s["x"].shape[1]
    N = cu.numel() - 1
    T = max(1, s["longest"])
    t = torch.arange(T, device=x.device)
    valid = t < (cu[1:] - cu[:-1])[:, None]                             # [N, T]
    src = torch.where(valid, cu[:-1, None] + t, 0)
    step = _steps(s["dt"], s["dt_bias"])[src].masked_fill(~valid[..., None], 0.0)
    y, final = _plain_scan(x[src], step, s["A"], s["B"][src], s["C"][src], s["initial"])
    y = y[valid] + s["D"][:, None] * x.float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    return y.to(x.dtype), final


def _plain_scan_decode(s):
    x, idx = s["x"], s["indices"].long()
    y, final = _plain_scan(x, _steps(s["dt"], s["dt_bias"]), s["A"], s["B"], s["C"], s["pool"][idx])
    y = y + s["D"][:, None] * x.float()
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["pool"][idx] = final.to(s["pool"].dtype)
    return y.to(x.dtype), s["pool"]


EPS = 1e-6


def _plain_norm(x, weight, norm):
    y = x.float()
    if norm is None:
        return y
    sq = y.square().sum(-1, keepdim=True)
    y = y / torch.sqrt((sq / x.shape[-1] if norm == "rms" else sq) + EPS)
    return y if weight is None else y * weight


def _plain_rotate(x, cos, sin, offset, layout):
    rot = 2 * cos.shape[-1]
    part = x[..., offset:offset + rot]
    if layout == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([x[..., :offset], turned, x[..., offset + rot:]], -1)


def _plain_qk_norm(s):
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return tuple(_plain_rotate(_plain_norm(s[x], s[x + "_weight"], s["norm"]), cos, sin, s["offset"],
                               s["layout"]).to(s[x].dtype) for x in ("q", "k"))


def _own_run(s):
    import gated_delta_rule_38_amd as kda
    op = s["op"]
    if op == "conv":
        return kda.conv(s["x"], s["weight"], bias=s["bias"], initial_state=s["initial"], cu_seqlens=s["cu"],
                        final_state=None, activation=s["activation"])
    if op == "conv_decode":
        out = kda.conv_decode(s["x"], s["weight"], s["pool"], s["indices"], bias=s["bias"],
                              activation=s["activation"])
        return out, s["pool"]
    if op == "scan":
        return kda.ssm_prefill(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], dt_bias=s["dt_bias"], z=s["z"],
                               initial_state=s["initial"], cu_seqlens=s["cu"], dt_softplus=True)
    if op == "scan_decode":
        out = kda.ssm_decode(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], s["indices"], D=s["D"],
                             dt_bias=s["dt_bias"], z=s["z"], dt_softplus=True)
        return out, s["pool"]
    return kda.qk_norm(s["q"], s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"], positions=s["positions"],
                       inv_freq=s["inv_freq"], norm=s["norm"], eps=EPS, layout=s["layout"],
                       rotary_offset=s["offset"])


def run(state):
    if own:
        return _own_run(state)
    op = state["op"]
    if op == "conv":
        return _plain_conv(state["x"], state["weight"], state["bias"], state["initial"], state["cu"],
                           state["activation"])
    if op == "conv_decode":
        return _plain_conv_decode(state["x"], state["weight"], state["bias"], state["pool"], state["indices"],
                                  state["activation"])
    if op == "scan":
        return _plain_scan_prompt(state)
    if op == "scan_decode":
        return _plain_scan_decode(state)
    return _plain_qk_norm(state)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op == "qk_norm":
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["D"]
        return {"bytes": 2 * n * es + 4 * case["tokens"] + 2 * case["rot"], "flops": 4 * n + 3 * n * case["rot"] / case["D"]}
    if op in ("conv", "conv_decode"):
        C, W = case["channels"], case["width"]
        ss = 2 if case["state"] == "bf16" else 4
        seqs, tokens = (case["requests"], case["requests"] * case["tokens"]) if op == "conv_decode" else \
            (len(_lengths(case)), sum(_lengths(case)))
        return {"bytes": 2 * tokens * C * es + 2 * seqs * (W - 1) * C * ss + C * (W + 1) * es,
                "flops": tokens * C * (2 * W + (4 if case["silu"] else 0))}
    H, G, P, N = case["heads"], case["groups"], case["P"], case["N"]
    ss = 4
    if op == "scan_decode":
        seqs, tokens = case["requests"], case["requests"] * case["tokens"]
        ss = 2 if case["state"] == "bf16" else 4
    else:
        seqs, tokens = len(_lengths(case)), sum(_lengths(case))
    token = H * P * es * (3 if case["gate"] else 2) + H * es + 2 * G * N * es
    # the recurrence itself: one update and one read of the state for each token
    return {"bytes": tokens * token + 2 * seqs * H * N * P * ss + 12 * H, "flops": tokens * H * N * P * 4}


# --------------------------------------------------------------- the definitions, in 64 bits

def _exact_conv_rows(rows, weight, bias, silu):
    """rows [n, W - 1 + T, C] of consecutive inputs."""
    W = weight.shape[1]
    T = rows.shape[1] - (W - 1)
    y = torch.zeros_like(rows[:, :T])
    for w in range(W):
        y += rows[:, w:w + T] * weight[:, w].double()
    if bias is not None:
        y += bias.double()
    return y * torch.sigmoid(y) if silu else y


def _exact_recurrence(S, x, step, A, B, C):
    """One sequence after the other in time: S [n, H, N, P], x [n, T, H, P]; token t of a sequence
    with step 0 leaves its state as it is."""
    ys = []
    for t in range(x.shape[1]):
        d = step[:, t]
        S = S * torch.exp(d * A)[..., None, None]
        S += (d[..., None] * B[:, t])[..., None] * x[:, t, :, None, :]
        ys.append((S * C[:, t, :, :, None]).sum(-2))
    return torch.stack(ys, 1), S


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "conv":
        ys, fs = [], []
        cu = s["cu"].tolist()
        for n in range(len(cu) - 1):
            rows = torch.cat([s["initial"][n].double(), s["x"][cu[n]:cu[n + 1]].double()])
            ys.append(_exact_conv_rows(rows[None], s["weight"], s["bias"], case["silu"])[0])
            fs.append(rows[rows.shape[0] - (case["width"] - 1):])
        return torch.cat(ys), torch.stack(fs)
    if op == "conv_decode":
        rows = torch.cat([s["pool"][s["indices"].long()].double(), s["x"].double()], 1)
        pool = s["pool"].double()
        pool[s["indices"].long()] = rows[:, case["tokens"]:]
        return _exact_conv_rows(rows, s["weight"], s["bias"], case["silu"]), pool
    if op == "qk_norm":
        out = []
        for name in ("q", "k"):
            y = s[name].double()
            sq = (y * y).sum(-1, keepdim=True)
            if case["norm"] != "none":
                y = y * torch.rsqrt((sq / case["D"] if case["norm"] == "rms" else sq) + EPS)
            if s[name + "_weight"] is not None:
                y = y * s[name + "_weight"].double()
            rot, o = case["rot"], case["offset"]
            phase = torch.polar(torch.ones((), dtype=torch.float64, device=y.device),
                                s["positions"].double()[:, None] * s["inv_freq"].double())[:, None]
            if case["layout"] == "half":
                i = o + torch.arange(rot // 2, device=y.device)
                j = i + rot // 2
            else:
                i = o + 2 * torch.arange(rot // 2, device=y.device)
                j = i + 1
            z = torch.complex(y[..., i], y[..., j]) * phase
            y[..., i], y[..., j] = z.real, z.imag
            out.append(y)
        return tuple(out)
    H = case["heads"]
    v = s["dt"].double() + s["dt_bias"].double()
    step = torch.logaddexp(v, torch.zeros_like(v))
    A = s["A"].double()
    if op == "scan":
        lengths = _lengths(case)
        n, T = len(lengths), max(1, max(lengths))
        cu = s["cu"].tolist()

        def padded(t):
            r = torch.zeros((n, T) + t.shape[1:], dtype=t.dtype, device=t.device)
            for i, m in enumerate(lengths):
                r[i, :m] = t[cu[i]:cu[i + 1]]
            return r

        y, S = _exact_recurrence(s["initial"].double(), padded(s["x"]).double(), padded(step), A,
                                 _heads(padded(s["B"]), H).double(), _heads(padded(s["C"]), H).double())
        y = torch.cat([y[i, :m] for i, m in enumerate(lengths)])
    else:
        idx = s["indices"].long()
        y, S = _exact_recurrence(s["pool"][idx].double(), s["x"].double(), step, A, _heads(s["B"], H).double(),
                                 _heads(s["C"], H).double())
        pool = s["pool"].double()
        pool[idx] = S
        S = pool
    y = y + s["D"].double()[:, None] * s["x"].double()
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    return y, S
