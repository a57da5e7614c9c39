"""Float64 statements of the sublayer operators around the block-local tail (numpy, CPU).

Shares no code with the GPU path. Arrays are float64 holding exactly the stored (bf16) inputs.
"""
from __future__ import annotations

import numpy as np

GROUP = 64


def bf16(x):
    """float64 -> the nearest bf16 value (ties to even), as float64."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)  # |m| in [0.5, 1): 8 significant bits
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.where(np.isfinite(x) & (x != 0), np.rint(x / step) * step, x)


def kv4_quantise(x):
    """Codes, scales and biases of rows [..., D]: one group per 64 channels (affine, 0..15)."""
    f = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    lo, hi = f.min(-1), f.max(-1)
    scale, bias = bf16((hi - lo) / 15.0), bf16(lo)
    s = scale[..., None]
    code = np.where(s > 0, np.clip(np.rint((f - bias[..., None]) / np.where(s > 0, s, 1.0)), 0, 15), 0.0)
    return code, scale, bias


def kv4_values(x):
    """What the codes of rows [..., D] stand for."""
    code, scale, bias = kv4_quantise(x)
    return (code * scale[..., None] + bias[..., None]).reshape(x.shape)


def seen(G, L, N, causal, window):
    """[G, L + N] which keys each row sees; row t stands at L + N - G + t."""
    pos = L + N - G + np.arange(G)[:, None]
    key = np.arange(L + N)[None, :]
    s = np.ones((G, L + N), bool)
    if causal:
        s &= key <= pos
    if window > 0:
        s &= key > pos - window
    return s


def attention(q, K, V, see, scale):
    """One sequence: q [G, Hq, D], K / V [n, Hkv, D], see [G, n]. Returns out [G, Hq, D] and the
    standard deviation of its rounding errors when the probabilities, the values and the keys are
    each rounded to bf16 and the result once more (independent, uniform within half a step: a
    relative 2^-8 / sqrt(3) each; a key's error reaches the output through its score)."""
    G, Hq, D = q.shape
    R = Hq // K.shape[1]
    out, var = np.zeros((G, Hq, D)), np.zeros((G, Hq, D))
    u2 = 2.0 ** -16 / 3
    for t in range(G):
        i = np.nonzero(see[t])[0]
        if i.size == 0:
            continue
        for h in range(Hq):
            k, v = K[i, h // R], V[i, h // R]
            qk = k * q[t, h]
            s = qk.sum(-1) * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            o = p @ v
            ds2 = scale ** 2 * (qk ** 2).sum(-1)
            out[t, h] = o
            var[t, h] = u2 * (o ** 2 + 2 * (p ** 2) @ (v ** 2) + (p ** 2 * ds2) @ ((v - o) ** 2))
    return out, np.sqrt(var)


def act(g, kind):
    """act(g), act'(g)."""
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = np.sqrt(2.0 / np.pi)
    t = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def gated_ffn(x, wg, wu, kind):
    """h, g, u."""
    g, u = x @ wg.T, x @ wu.T
    return act(g, kind)[0] * u, g, u


def gated_ffn_backward(dh, g, u, x, wg, wu, kind):
    """dx, dwg, dwu and the gradients dg, du at the pre-activations."""
    a, d = act(g, kind)
    dg, du = dh * u * d, dh * a
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du
