"""Plain float64 forms of the operators of include/kda_layer.h, token by token and on the CPU, for
their tests, with the sums of magnitudes that error bounds are taken from.

Each returns its result and ``mag``, the same expression with every product and state taken by its
absolute value: k roundings of relative size u anywhere along the sums that form a result are off by
at most k u mag.
"""
import numpy as np


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def sequences(x, cu):
    """[(first, last)) token ranges] of a packed (cu given) batch."""
    c = [int(v) for v in cu]
    return list(zip(c[:-1], c[1:]))


def silu(y):
    with np.errstate(over="ignore"):
        return y / (1 + np.exp(-y))


def conv_rows(rows, weight, bias, activation):
    """rows [W - 1 + T, C]: consecutive inputs.  (out [T, C], mag)"""
    W = weight.shape[1]
    T = rows.shape[0] - (W - 1)
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for w in range(W):
        y += rows[w:w + T] * weight[:, w]
        mag += np.abs(rows[w:w + T] * weight[:, w])
    if bias is not None:
        y += bias
        mag += np.abs(bias)
    if activation == "silu":
        # |d silu| <= 1.1 |d y|, and silu's own rounding is relative to its value
        return silu(y), 1.1 * mag + np.abs(silu(y))
    return y, mag


def conv(x, weight, bias, initial, cu, activation):
    """Packed.  (out, final, mag)"""
    W = weight.shape[1]
    outs, fins, mags = [], [], []
    for n, (a, b) in enumerate(sequences(x, cu)):
        first = initial[n] if initial is not None else np.zeros((W - 1, x.shape[1]))
        rows = np.concatenate([first, x[a:b]])
        y, m = conv_rows(rows, weight, bias, activation)
        outs.append(y)
        mags.append(m)
        fins.append(rows[rows.shape[0] - (W - 1):])
    return np.concatenate(outs), np.stack(fins), np.concatenate(mags)


def step_size(dt, dt_bias, softplus):
    v = dt + (0 if dt_bias is None else dt_bias)
    return np.logaddexp(v, 0.0) if softplus else v


def ssm(x, dt, A, B, C, D, dt_bias, z, initial, softplus):
    """One sequence: x [T, H, P], B, C [T, G, N], initial [H, N, P] or None.
    (out, final, mag of out, mag of final)"""
    T, H, P = x.shape
    G, N = B.shape[1:]
    S = np.zeros((H, N, P)) if initial is None else initial.copy()
    M = np.abs(S)
    out, mag = np.zeros((T, H, P)), np.zeros((T, H, P))
    step = step_size(dt, dt_bias, softplus)
    for t in range(T):
        d = step[t]                                             # [H]
        e = np.exp(A * d)[:, None, None]
        Bt, Ct = (np.repeat(v[t], H // G, axis=0) for v in (B, C))    # [H, N]
        add = (d[:, None] * Bt)[:, :, None] * x[t][:, None, :]
        S = e * S + add
        M = e * M + np.abs(add)
        out[t] = np.einsum("hnp,hn->hp", S, Ct)
        mag[t] = np.einsum("hnp,hn->hp", M, np.abs(Ct))
        if D is not None:
            out[t] += D[:, None] * x[t]
            mag[t] += np.abs(D[:, None] * x[t])
    if z is not None:
        out, mag = out * silu(z), mag * np.abs(silu(z))
    return out, S, mag, M


def qk_norm(x, weight, norm, eps, positions, inv_freq, layout, offset, scale):
    """x [T, H, D].  (out, mag)"""
    y = x.copy()
    if norm:
        sq = (x * x).mean(-1, keepdims=True) if norm == "rms" else (x * x).sum(-1, keepdims=True)
        y = y / np.sqrt(sq + eps)
        if weight is not None:
            y = y * weight
    mag = np.abs(y)
    if inv_freq is None or len(inv_freq) == 0:
        return y, mag
    half = len(inv_freq)
    angle = positions.astype(np.float64)[:, None] * inv_freq[None, :]
    i = offset + np.arange(half) * (1 if layout == "half" else 2)
    j = i + (half if layout == "half" else 1)
    c, s = (scale * f(angle)[:, None, :] for f in (np.cos, np.sin))
    out = y.copy()
    out[..., i] = y[..., i] * c - y[..., j] * s
    out[..., j] = y[..., j] * c + y[..., i] * s
    m = abs(scale) * (mag[..., i] + mag[..., j])
    mag[..., i], mag[..., j] = m, m
    return out, mag
