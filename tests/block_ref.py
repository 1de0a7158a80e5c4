"""Plain 64-bit NumPy implementations of the decoder-layer operators, for the tests.

Written from the formulas, with loops where they are the plainest; nothing is shared with
the library.  U is half an ulp of 1 in fp32."""

import numpy as np

U = 2.0 ** -24


def bf16(a):
    """Rounds to the nearest bfloat16 value (ties to even), returned as float64."""
    import torch
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(torch.bfloat16).to(torch.float64).numpy()


def bf16_gap(a):
    """Half the distance between neighbouring bfloat16 numbers at a (and at least the smallest normal's)."""
    e = np.floor(np.log2(np.maximum(np.abs(a), 2.0 ** -126)))
    return 2.0 ** (e - 8)


def hadamard256():
    """Closed form: entry (i, j) is the product over the four base-4 digits of -1 where the digits add to 3."""
    h = np.ones((256, 256))
    for i in range(256):
        for j in range(256):
            for d in range(4):
                if (i >> 2 * d & 3) + (j >> 2 * d & 3) == 3:
                    h[i, j] = -h[i, j]
    return h / 16


H256 = hadamard256()


def rotate(y):
    m, k = y.shape
    return (y.reshape(-1, 256) @ H256).reshape(m, k)


def norm(h, weight, eps):
    rstd = 1 / np.sqrt((h ** 2).mean(1) + eps)
    y = h * rstd[:, None] * weight
    return rstd, y, rotate(y)


def norm_grad(g, h, weight, eps, rotated):
    """Gradients of sum(g * v) (rotated) or sum(g * y)."""
    m, k = h.shape
    rstd = 1 / np.sqrt((h ** 2).mean(1) + eps)
    gy = rotate(g) if rotated else g
    u = gy * weight
    dh = rstd[:, None] * u - h * (rstd ** 3 * (u * h).mean(1))[:, None]
    return dh, (gy * h * rstd[:, None]).sum(0), gy


def rope(x, pos, inv_freq, sections, interleaved=False, inverse=False):
    """x [T, heads, D]; pos [axes, T]."""
    out = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    for p in range(n):
        angle = pos[axis[p]].astype(np.float64) * float(inv_freq[p])
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        s = -s if inverse else s
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + n)
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    return out


def attention(q, k, v, first_pos, scale, causal, window):
    """One head: q [n, D] at positions first_pos + i over k, v [L, D].  Returns out, lse and the weights' mean of |v|."""
    n, length = q.shape[0], k.shape[0]
    out, lse, size = np.zeros((n, v.shape[1])), np.full(n, -np.inf), np.zeros((n, v.shape[1]))
    j = np.arange(length)
    for i in range(n):
        p = first_pos + i
        seen = np.ones(length, bool)
        if causal:
            seen &= j <= p
        if window:
            seen &= j > p - window
        if not seen.any():
            continue
        s = scale * (k[seen] @ q[i])
        top = s.max()
        w = np.exp(s - top)
        out[i] = w @ v[seen] / w.sum()
        size[i] = w @ np.abs(v[seen]) / w.sum()
        lse[i] = top + np.log(w.sum())
    return out, lse, size
