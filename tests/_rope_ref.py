"""Plain fp64 forms of the rotating append and of the shared-prefix attention,
and the inputs their tests share.

Error bounds of the fp32 kernels, in units of u = 2^-24:
* a row's norm: the mean of D squares is off by at most (D + 2) u relative, the
  root halves it, and root, quotient and the two products add 4 u; so a normed
  value is off by at most ((D + 2) / 2 + 6) u relative.
* a rotation: the phase reaches the kernel as a fraction of half a turn in
  fp32, off by 2^-25 half-turns (pi / 2 u radians) at most; cos and sin are off by
  2 ulp (4 u) more, their product with the factor by u, the two products and
  the sum by 3 u: at most 10 u of m (|y_a| + |y_b|).
"""
import numpy as np
import torch

U = 2.0 ** -24
BF16 = 2.0 ** -8  # half a step of bf16, relative


def bf16_f64(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16_bits(x):
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16)


def bf16_tensor(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16).copy()).view(torch.bfloat16)


def inv_freq(rot, base=1e4):
    return base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))


def fixed_point(inv):
    """Turns per position as fractions of 2^64."""
    out = np.zeros(len(inv), np.uint64)
    for i, f in enumerate(inv):
        out[i] = round(float(f) / (2 * np.pi) * 2.0 ** 64) & (2 ** 64 - 1)
    return out


def norm_rotate(bits, weight, eps, pos, freqs, rot, interleaved, factor):
    """(y, bound): the exact rows [n][h][d] of bf16 bits at positions pos [n], and
    how far an fp32 evaluation may be off."""
    x = bf16_f64(bits)
    d = x.shape[-1]
    bound = np.zeros_like(x)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * bf16_f64(weight)
        bound = np.abs(x) * (((d + 2) / 2 + 6) * U)
    # the exact phase: an integer product modulo 2^64
    turn = np.array([[(int(p) * int(f)) % 2 ** 64 / 2.0 ** 64 for f in freqs] for p in pos],
                    np.float64).reshape(len(pos), len(freqs))
    c, s = np.cos(2 * np.pi * turn)[:, None] * factor, np.sin(2 * np.pi * turn)[:, None] * factor
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    y, e = x.copy(), bound.copy()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    m = abs(factor)
    spread = m * (np.abs(a) + np.abs(b)) * 10 * U + m * (bound[..., ia] + bound[..., ib])
    e[..., ia] = spread
    e[..., ib] = spread
    return y, e


def attend(q_bits, k, v, scale):
    """fp64 attention of query rows [r][d] over rows k, v [n][d]; no row: zeros."""
    q = bf16_f64(q_bits)
    if k.shape[0] == 0:
        return np.zeros_like(q)
    z = scale * q @ k.T
    w = np.exp(z - z.max(-1, keepdims=True))
    return (w @ v) / w.sum(-1, keepdims=True)
