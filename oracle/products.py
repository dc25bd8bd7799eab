"""The experts' products outside the layer, in float64: the matrix product
grouped by expert with its gradients, 4-bit weights (int4 with group scales and
zero points, MXFP4), and the layer's forward on them.

Pins: tests/test_oracle_products.py (brute force, closed forms, differences,
``oracle.moe.forward``)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def grouped(x, w, offsets):
    """y[r] = w[e] x[r] for offsets[e] <= r < offsets[e + 1]; zeros in the other rows."""
    y = np.zeros((x.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        y[offsets[e]:offsets[e + 1]] = x[offsets[e]:offsets[e + 1]] @ w[e].T
    return y


def grouped_backward(dy, x, w, offsets):
    """(dx, dw) of ``grouped``."""
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    for e in range(w.shape[0]):
        rows = slice(offsets[e], offsets[e + 1])
        dx[rows] = dy[rows] @ w[e]
        dw[e] = dy[rows].T @ x[rows]
    return dx, dw


def bf16(v):
    """v rounded to bf16 (nearest, ties to even); finite values."""
    u = np.asarray(v, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32).astype(np.float64)


def quantize(w, form, group, zero_point=False):
    """w [..., k] (values exact in fp32) -> (codes 0..15 [..., k], scale, zero or None): scale the bf16 value, or the
    E8M0 byte. Divisions are rounded to fp32 as the library's are, then to whole numbers."""
    b = np.asarray(w, np.float32).reshape(*w.shape[:-1], -1, group)
    if form == "mxfp4":
        amax = np.abs(b).max(-1).astype(np.float64)
        x = np.where(amax > 0, np.frexp(amax)[1] - 3, -127).clip(-127, 127)
        v = np.abs(b.astype(np.float64)) * 2.0 ** -x[..., None].astype(np.float64)
        far = np.abs(v[..., None] - E2M1)
        best = far.min(-1, keepdims=True)
        # ties to the even code: of two equally near ones, the one with an even number
        near = far == best
        low = near.argmax(-1)
        code = np.where((near.sum(-1) == 2) & (low % 2 == 1), low + 1, low)
        return (code + 8 * np.signbit(b)).reshape(w.shape), (x + 127).astype(np.uint8), None
    f32 = np.float32
    with np.errstate(divide="ignore", invalid="ignore"):
        if zero_point:
            lo, hi = np.minimum(b.min(-1), 0), np.maximum(b.max(-1), 0)
            scale = bf16((hi - lo).astype(f32) / f32(15)).astype(f32)
            zero = np.where(scale > 0, np.rint(-lo / scale).clip(0, 15), 0)
            code = np.where(scale[..., None] > 0, (np.rint(b / scale[..., None]) + zero[..., None]).clip(0, 15), 0)
            return code.astype(int).reshape(w.shape), scale.astype(np.float64), zero.astype(int)
        scale = bf16(np.abs(b).max(-1) / f32(7)).astype(f32)
        code = np.where(scale[..., None] > 0, np.rint(b / scale[..., None]).clip(-8, 7), 0) + 8
    return code.astype(int).reshape(w.shape), scale.astype(np.float64), None


def values(codes, scale, zero=None, mxfp4=False):
    """What codes [..., k] stand for; scale as ``quantize`` gives it."""
    c = codes.reshape(*scale.shape, -1)
    if mxfp4:
        v = np.where(c > 7, -1.0, 1.0) * E2M1[c & 7] * np.exp2(scale.astype(np.float64) - 127)[..., None]
    else:
        v = (c - (8 if zero is None else zero[..., None])) * scale[..., None]
    return v.reshape(codes.shape)


def pack(codes):
    """Two codes to a byte, the even column in the low half."""
    return (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)


def unpack(packed):
    p = np.asarray(packed).astype(int)
    return np.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], -1)


def mlp(x, gate, up, down, limit=0.0):
    """(y, h) of one expert."""
    g, u = x @ gate.T, x @ up.T
    if limit:
        g, u = np.minimum(g, limit), np.clip(u, -limit, limit)
    h = g / (1 + np.exp(-g)) * u
    return h @ down.T, h


def layer(x, router_w, ids, gate, up, down, shared=None, limit=0.0):
    """out[t] = sum over the choices of expert e = ids[t, j] in [0, E), plus the shared expert's."""
    y = np.zeros(x.shape) if shared is None else mlp(x, *shared, limit)[0]
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if 0 <= e < gate.shape[0]:
                y[t] += router_w[t, j] * mlp(x[t:t + 1], gate[e], up[e], down[e], limit)[0][0]
    return y
