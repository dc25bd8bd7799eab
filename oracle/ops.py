"""Float64 NumPy reference of the operators around the layer: RMS norm, top-k
router and AdamW step. Test infrastructure; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def rms_norm(x, w, residual=None, eps=1e-6):
    s = np.asarray(x, np.float64)
    if residual is not None:
        s = s + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=-1) + eps)
    return s * rstd[..., None] * w, s, rstd


def rms_norm_backward(dy, s, rstd, w, d_sum=None):
    xh = s * rstd[..., None]
    g = dy * w
    ds = rstd[..., None] * (g - xh * np.mean(g * xh, axis=-1, keepdims=True))
    if d_sum is not None:
        ds = ds + d_sum
    return ds, np.sum(dy * xh, axis=tuple(range(dy.ndim - 1)))


# ---------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------

def _keys(logits32, bias, mask):
    key = logits32.astype(np.float32)
    with np.errstate(invalid="ignore"):
        if bias is not None:
            key = key + bias.astype(np.float32)  # the definition: one fp32 addition
    T = key.shape[0]
    keep = np.ones(T, bool) if mask is None else mask.astype(bool)
    broken = keep & (np.isnan(key).any(1) | (key == np.inf).any(1))
    live = keep & (broken | (key > -np.inf).any(1))
    return key, keep, broken, live


def _scores(l, scoring):
    l = l.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return np.where(l == -np.inf, 0.0, 1.0 / (1.0 + np.exp(-l)))
        top = l.max(1, keepdims=True)
        e = np.where(l == -np.inf, 0.0, np.exp(l - top))
        return e / e.sum(1, keepdims=True)


def router(logits32, k, scoring="softmax", renormalize=True, scale=1.0, bias=None, mask=None):
    """(weights, ids, counts, losses) from float32 logits."""
    T, E = logits32.shape
    key, keep, broken, live = _keys(logits32, bias, mask)
    ids = np.full((T, k), -1, np.int64)
    weights = np.zeros((T, k))
    psum, zsum = np.zeros(E), 0.0
    for t in range(T):
        if not live[t]:
            continue
        if broken[t]:
            weights[t] = psum[:] = zsum = np.nan
            continue
        order = sorted((e for e in range(E) if key[t, e] > -np.inf), key=lambda e: (-key[t, e], e))[:k]
        ids[t, :len(order)] = order
        l = logits32[t].astype(np.float64)
        s = _scores(l[None], scoring)[0]
        c = s[order]
        if renormalize:
            # by the logits, so that scores that underflow keep their ratio
            if scoring == "sigmoid":
                ls = np.minimum(l[order], 0) - np.log1p(np.exp(-np.abs(l[order])))
            else:
                ls = l[order]
            c = np.exp(ls - ls.max())
            c = c / c.sum()
        weights[t, :len(order)] = c * scale
        if scoring == "sigmoid":
            with np.errstate(invalid="ignore"):
                ls = np.where(l == -np.inf, -np.inf, np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l))))
            s = np.exp(ls - ls.max())
        psum += s / s.sum()
        top = l.max()
        zsum += (top + np.log(np.exp(l - top).sum())) ** 2
    counts = np.concatenate([np.bincount(ids[ids >= 0], minlength=E), [live.sum()]])
    n = max(int(live.sum()), 1)
    balance = (counts[:E] * psum).sum() * E / k / n / n
    return weights, ids, counts, np.array([balance, zsum / n if scoring == "softmax" else 0.0])


def router_backward(dw, logits32, ids, scoring="softmax", renormalize=True, scale=1.0, bias=None, mask=None,
                    counts=None, d_losses=None):
    """d_logits of sum(dw * weights) + sum(d_losses * losses), row by row."""
    T, E = logits32.shape
    _, _, broken, live = _keys(logits32, bias, mask)
    out = np.zeros((T, E))
    for t in range(T):
        if not live[t]:
            continue
        l = logits32[t].astype(np.float64)
        # gradient to the log scores (ratios of scores by their logs: no underflow), then to the logits
        with np.errstate(invalid="ignore", over="ignore"):
            ls = np.where(l == -np.inf, -np.inf, np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))) \
                if scoring == "sigmoid" else l - l.max() - np.log(np.exp(l - l.max()).sum())
        s = np.exp(ls)
        dlog = np.zeros(E)
        sel = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < E]
        if sel:
            g = np.array([dw[t, j] * scale for j, _ in sel])
            c = np.array([ls[e] for _, e in sel])
            if renormalize:
                q = np.exp(c - c.max())
                q = q / q.sum()
                g = q * (g - (q * g).sum())
            else:
                g = np.exp(c) * g
            for (_, e), v in zip(sel, g):
                dlog[e] += v
        if counts is not None:
            n = max(int(counts[E]), 1)
            a = d_losses[0] * E / ids.shape[1] / n / n * counts[:E]
            p = np.exp(ls - ls.max())
            p = p / p.sum()
            dlog += p * (a - (p * a).sum())
        d = dlog - s * dlog.sum() if scoring == "softmax" else dlog * (1 - s)
        if counts is not None and scoring == "softmax":
            d += d_losses[1] * 2 / n * (l.max() + np.log(np.exp(l - l.max()).sum())) * s
        out[t] = np.nan if broken[t] else d
    return out


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def decode8(codes, scale):
    """Values of E4M3 codes with one E8M0 byte per 32."""
    c = np.asarray(codes, np.uint8).reshape(-1)
    v = np.where(c & 0x80, -1.0, 1.0) * E4M3[np.minimum(c & 0x7F, 126)]
    x = np.asarray(scale, np.uint8).reshape(-1)
    f = np.where(x == 255, np.nan, np.exp2(x.astype(np.float64) - 127))
    return v * np.repeat(f, 32)[:c.size]


def adamw(p, g, m, v, step, lr, b1, b2, eps, wd):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p * (1 - lr * wd) - lr / (1 - b1 ** step) * m / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return p, m, v


def state_exponent(values):
    """Per block of 32: the smallest x with max |value| <= 448 * 2^x."""
    a = np.abs(np.asarray(values, np.float64).reshape(-1))
    a = np.concatenate([a, np.zeros(-a.size % 32)]).reshape(-1, 32).max(1)
    with np.errstate(divide="ignore"):
        x = np.ceil(np.log2(a / 448.0))
    x = np.where(448.0 * np.exp2(x - 1) >= a, x - 1, x)
    x = np.where(448.0 * np.exp2(x) < a, x + 1, x)
    return np.where(a > 0, np.clip(x, -127, 127), -127)


def uniforms(n, seed, first=0):
    """The random numbers of elements first .. first + n of a call."""
    i = np.arange(first, first + n, dtype=np.uint64)
    M = np.uint64(0xFFFFFFFF)
    x = ((i >> np.uint64(1)) * np.uint64(0x9E3779B1) + np.uint64(seed)) & M
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x85157AF5)) & M
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0x2C1B3C6D)) & M
    x ^= x >> np.uint64(16)
    half = np.where(i & np.uint64(1), x >> np.uint64(16), x & np.uint64(0xFFFF))
    return (half.astype(np.float64) + 0.5) / 65536.0
