"""Plain 64-bit forms of the operators of a prompt's layer, with how far a kernel may be from them.

A rounding to a type is off by at most eps / 2 of the value: binary16 2^-11 (or 2^-25 near zero), fp32 2^-24.
"""
import math

import numpy as np
import torch

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
SLOPE = 1.13       # the steepest of the activations (GELU near 1.41; SiLU has 1.10)


def q4_bytes(n, k, seed, scales=None):
    """Q4_0 rows [n][k/32][18] with every code, and scales of both signs around 1 / sqrt(k) (or the given ones, one per block)."""
    rng = np.random.default_rng(seed)
    blocks = np.empty((n, k // 32, 18), dtype=np.uint8)
    d = rng.normal(size=(n, k // 32)) / (4 * math.sqrt(k)) if scales is None else np.broadcast_to(scales, (n, k // 32))
    blocks[..., :2] = d.astype(np.float16)[..., None].view(np.uint8)
    blocks[..., 2:] = rng.integers(0, 256, size=(n, k // 32, 16))
    return blocks


def weights(blocks):
    """float64 [n][k]: f16((q - 8) * d).  (The product is exact in fp32: 4 bits times 11.)"""
    d = blocks[..., :2].copy().view(np.float16).astype(np.float32)
    q = np.concatenate([blocks[..., 2:] & 15, blocks[..., 2:] >> 4], axis=-1).astype(np.float32) - 8
    with np.errstate(over="ignore", invalid="ignore"):
        return (q * d).astype(np.float16).astype(np.float64).reshape(blocks.shape[0], -1)


def act(t, name):
    if name == "relu":
        return np.where(t > 0, t, 0.0)
    if name == "silu":
        return t / (1 + np.exp(-t))
    if name == "gelu":
        return t * 0.5 * (1 + np.vectorize(math.erf, otypes=[float])(t / math.sqrt(2)))
    if name == "gelu_tanh":
        return t * 0.5 * (1 + np.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def product(w, x, bias=None):
    """(W x + bias, how far an fp32 sum of it may be): w [n][k], x [rows][k] float64.  A sum of k products loses at most k 2^-23 of
    sum |w x| (each step may cut off a last bit of what is summed so far), the bias one more rounding."""
    t, s = x @ w.T, np.abs(x) @ np.abs(w).T
    b = 0.0 if bias is None else bias.astype(np.float64)
    return t + b, w.shape[1] * 2.0 ** -23 * s + 2.0 ** -23 * np.abs(t + b)


def rounded(y, off):
    """How far binary16 values may be when the value before the rounding is off by `off`."""
    return off + 2.0 ** -11 * (np.abs(y) + off) + 2.0 ** -25


def gemm(w, x, bias=None, act_name="none", scale=1.0, residual=None):
    t, off = product(w, x, bias)
    a = act(t, act_name)
    # an activation is within 2^-20 of its value plus 2^-22 of its argument (erff, tanhf, expf and a division: a few last bits each)
    off = SLOPE * off + 2.0 ** -20 * np.abs(a) + 2.0 ** -22 * np.abs(t)
    y = a * np.float32(scale).astype(np.float64)
    off = off * abs(scale) + 2.0 ** -23 * np.abs(y)
    if residual is not None:
        y = y + residual
        off = off + 2.0 ** -23 * (np.abs(y) + np.abs(residual))
    return y, rounded(y, off)


def gated(wg, wu, x, bg=None, bu=None, act_name="silu"):
    (g, dg), (u, du) = product(wg, x, bg), product(wu, x, bu)
    a = act(g, act_name)
    da = SLOPE * dg + 2.0 ** -20 * np.abs(a) + 2.0 ** -22 * np.abs(g)
    y = a * u
    return y, rounded(y, np.abs(a) * du + da * np.abs(u) + da * du + 2.0 ** -23 * np.abs(y))


def norm(v, off, kind, eps, weight=None, bias=None):
    """(norm(v) * weight + bias, how far fp32 may be) for rows v that are themselves off by `off`."""
    n = v.shape[-1]
    if kind == "layer":
        mean = v.mean(-1, keepdims=True)
        # a sum of n values by threads and a tree: at most 64 additions deep, 2^-24 of the sum of magnitudes each
        off = off + off.mean(-1, keepdims=True) + 64 * 2.0 ** -24 * np.abs(v).mean(-1, keepdims=True) + 2.0 ** -23 * (np.abs(v) + np.abs(mean))
        v = v - mean
    rms = np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    # the mean of squares: 64 roundings deep and what the values are off, relative to itself; then the root and the division
    rel = 66 * 2.0 ** -24 + 4 * 2.0 ** -23 + np.sqrt((off * off).mean(-1, keepdims=True)) / rms
    z = v / rms
    dz = off / rms + rel * np.abs(z) * 1.01
    if weight is not None:
        w = weight.astype(np.float64)
        z, dz = z * w, dz * np.abs(w) + 2.0 ** -23 * np.abs(z * w)
    if bias is not None:
        b = bias.astype(np.float64)
        z, dz = z + b, dz + 2.0 ** -23 * (np.abs(z + b) + np.abs(z))
    return z, dz


def block_norm(block, residual, kind="rms", eps=1e-5, post=False, post_weight=None, post_bias=None, scale=1.0, gate=None, weight=None, bias=None):
    """((t, off), (z, off)) in fp32, before they are rounded to what they are stored as; gate [rows or 1][n]."""
    if block is None:
        t, off = residual, np.zeros_like(residual)
    else:
        u, off = (norm(block, np.zeros_like(block), kind, eps, post_weight, post_bias)) if post else (block, np.zeros_like(block))
        s = np.float32(scale).astype(np.float64) * (1.0 if gate is None else gate.astype(np.float64))
        u, off = u * s, off * np.abs(s) + 2.0 ** -23 * np.abs(u * s)
        t = u if residual is None else u + residual
        off = off + 2.0 ** -23 * np.abs(t)
    return (t, off), norm(t, off, kind, eps, weight, bias)


def rope(x, places, freqs, axes, head_dim, halves, inverse=False):
    """(y, off before a rounding to binary16): x [rows][heads * head_dim] float64, places [axes][rows] whole numbers."""
    rows, pairs = x.shape[0], len(freqs)
    h = x.reshape(rows, -1, head_dim)
    y = h.copy()
    first = np.arange(pairs) if halves else 2 * np.arange(pairs)
    second = first + (pairs if halves else 1)
    angle = np.asarray(places, dtype=np.float64)[np.asarray(axes)].T * np.asarray(freqs)       # [rows][pairs]
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None] * (-1 if inverse else 1)
    a, b = h[..., first], h[..., second]
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    off = np.zeros_like(h)
    # cosines and sines within 2^-22; the 64-bit angle itself within 2^-52 of it; two products and a sum
    far = 2.0 ** -22 + np.abs(angle)[:, None] * 2.0 ** -51
    off[..., first] = off[..., second] = (np.abs(a) + np.abs(b)) * (far + 2.0 ** -23)
    return y.reshape(rows, -1), off.reshape(rows, -1)


def assert_near(got, want, off, what=""):
    got = np.asarray(got, dtype=np.float64)
    bad = ~(np.abs(got - want) <= off)
    if bad.any():
        at = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / np.maximum(off, 1e-300), 0)), got.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.size} values too far off; worst at {at}: {got[at]} for {want[at]} +- {off[at]}")


def host(t):
    return t.detach().cpu().to(torch.float64).numpy()
