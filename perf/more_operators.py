"""The experts' products outside the fused layer, as cases to be measured.

Ragged products for training and prompts, 4-bit weights for decoding: the
matrix product grouped by expert and its backward pass, the 4-bit weights
themselves (quantized and read back), the product of a few rows with such
weights, and the layer's forward on 4-bit experts for a few tokens. Each case
is one call of one of them (the quantizer's: one call and its inverse).

With ``own`` false, ``run`` computes the plain form from elementary torch
operations in 32 bits, rounded once at the end. With ``own`` true it makes the
package's calls.

Formulas
  grouped      y[r] = W_e x[r] for rows r in [offsets[e], offsets[e + 1]); rows of no
               expert get zeros
  grouped bwd  dx[r] = W_e^T dy[r];  dW_e = sum over e's rows of dy[r] x[r]^T
  int4         groups of 32, 64 or 128 along K, codes 0..15, value (code - zero) * scale.
               symmetric: scale = bf16(amax / 7), zero = 8, code = clamp(rint(w / scale), -8, 7) + 8
               zero point: lo = min(0, min w), hi = max(0, max w), scale = bf16((hi - lo) / 15),
               zero = clamp(rint(-lo / scale), 0, 15), code = clamp(rint(w / scale) + zero, 0, 15)
               (scale 0: the code is the zero point, which is then 8, or 0)
  mxfp4        groups of 32, scale = 2^X with X = floor(log2 amax) - 2 (at least -127; -127 for
               zeros), codes E2M1 to nearest even of w / scale, at most 6
  w4 product   y[t] = sum over k of x[t, k] * value[n, k]
  w4 layer     y[t] = sum over j of w[t, j] * Wd_e (silu(g) * u) + the shared expert's with weight 1,
               e = ids[t, j] (none if negative), g = Wg_e x[t], u = Wu_e x[t]; with a limit L
               g = min(g, L), u = clamp(u, -L, L)
"""
import math

import torch

own = False


def listed():
    return [
        # one decoded token's eight experts, up projection of the 128-expert layer: weights read for one row each
        dict(name="grouped_decode", op="grouped", rows=8, experts=128, n=768, k=2048, tail=False),
        # a training step: 8192 tokens, top-8, up projection of the 128-expert layer
        dict(name="grouped_train", op="grouped", rows=65536, experts=128, n=768, k=2048, tail=False),
        # experts of an odd width on a ragged batch with padding rows behind the last expert
        dict(name="grouped_odd", op="grouped", rows=4099, experts=37, n=1001, k=1037, tail=True),
        # the backward pass of the 128-expert layer's down projection
        dict(name="grouped_backward", op="grouped_bwd", rows=65536, experts=128, n=2048, k=768, tail=False,
             dw="bf16"),
        # the backward pass of wide experts, weight gradients kept in fp32
        dict(name="grouped_backward_wide", op="grouped_bwd", rows=32768, experts=32, n=2048, k=7168, tail=True,
             dw="fp32"),
        # the gate projections of a layer brought to 4 bits and back
        dict(name="w4_weights", op="w4_weights", experts=128, n=768, k=2048, format="int4", group=128, zero=False),
        # one projection with a zero point per group, rows that fill no round number of workgroups
        dict(name="w4_weights_zero", op="w4_weights", experts=1, n=1001, k=1568, format="int4", group=32, zero=True),
        # one token through a dense projection of the 4096-column layer
        dict(name="w4_product_decode", op="w4_product", tokens=1, n=1536, k=4096, format="int4", group=128, zero=True),
        # a batch of decoded tokens through a wide projection
        dict(name="w4_product_batch", op="w4_product", tokens=48, n=7168, k=2048, format="mxfp4", group=32,
             zero=False),
        # one token through the 128-expert layer with its shared expert
        dict(name="w4_layer_decode", op="w4_layer", tokens=1, hidden=2048, inter=768, experts=128, topk=8, shared=768,
             format="int4", group=128, zero=False, mask=False, limit=0.0),
        # 64 tokens decoded together: nearly every expert is read
        dict(name="w4_layer_batch", op="w4_layer", tokens=64, hidden=2048, inter=768, experts=128, topk=8, shared=768,
             format="mxfp4", group=32, zero=False, mask=False, limit=0.0),
        # a padded batch through wide experts with zero points
        dict(name="w4_layer_wide", op="w4_layer", tokens=17, hidden=7168, inter=2048, experts=32, topk=8, shared=0,
             format="int4", group=64, zero=True, mask=True, limit=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 64, else of 8, else any."""
    step = rng.choice([64, 64, 64, 8, 1])
    return max(step, _log(rng, lo, hi) // step * step)


def _format(rng):
    if rng.random() < 0.35:
        return dict(format="mxfp4", group=32, zero=False)
    return dict(format="int4", group=rng.choice([32, 64, 128, 128]), zero=rng.random() < 0.5)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "grouped_bwd", "grouped_bwd", "w4_weights", "w4_product", "w4_product",
                     "w4_layer", "w4_layer"])
    if op in ("grouped", "grouped_bwd"):
        n, k = _width(rng, 48, 7168), _width(rng, 48, 7168)
        experts = _log(rng, 1, max(1, min(256, 480_000_000 // (n * k))))
        odd = n % 8 or k % 8
        most = min(65536, (1 << 38 if odd else 1 << 39) // (n * k), 480_000_000 // max(n, k))
        case = dict(op=op, rows=_log(rng, 1, most), experts=experts, n=n, k=k, tail=rng.random() < 0.3)
        if op == "grouped_bwd":
            case["dw"] = rng.choice(["bf16", "fp32"])
        return case
    how = _format(rng)
    wide = 128 if rng.random() < 0.7 else how["group"]

    def cut(lo, hi):
        return max(1, _log(rng, lo, hi) // wide) * wide

    if op == "w4_weights":
        n, k = _log(rng, 1, 7168), cut(128, 7168)
        return dict(op=op, experts=_log(rng, 1, max(1, min(128, 200_000_000 // (n * k)))), n=n, k=k, **how)
    if op == "w4_product":
        return dict(op=op, tokens=_log(rng, 1, 256), n=_log(rng, 16, 16384), k=cut(128, 8192), **how)
    hidden, inter = cut(256, 7168), cut(128, 2048)
    experts = _log(rng, 2, max(2, min(128, 470_000_000 // (hidden * inter))))
    topk = rng.randint(1, min(8, experts))
    return dict(op=op, tokens=_log(rng, 1, 128), hidden=hidden, inter=inter, experts=experts, topk=topk,
                shared=cut(128, 2048) if rng.random() < 0.5 else 0, mask=rng.random() < 0.3,
                limit=rng.choice([0.0, 0.0, 2.0]), **how)


def _w4_bytes(case, elements):
    if case["format"] == "mxfp4":
        return elements * (1 / 2 + 1 / 32)
    return elements * (1 / 2 + (3 if case["zero"] else 2) / case["group"])


def work(case):
    op = case["op"]
    if op in ("grouped", "grouped_bwd"):
        r, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        touched = e * (1 - (1 - 1 / e) ** r)  # experts with rows, about
        if op == "grouped":
            return {"bytes": 2 * (r * k + touched * n * k + r * n), "flops": 2 * r * n * k}
        dw = 2 if case["dw"] == "bf16" else 4
        return {"bytes": 2 * r * n + 4 * r * k + 2 * touched * n * k + dw * e * n * k, "flops": 4 * r * n * k}
    if op == "w4_weights":
        m = case["experts"] * case["n"] * case["k"]
        return {"bytes": 4 * m + 2 * (_w4_bytes(case, m) - m / 2), "flops": 6 * m}
    if op == "w4_product":
        t, n, k = case["tokens"], case["n"], case["k"]
        return {"bytes": _w4_bytes(case, n * k) + 2 * t * (n + k), "flops": 2 * t * n * k}
    t, h, i, e, k = (case[x] for x in ("tokens", "hidden", "inter", "experts", "topk"))
    touched = e * (1 - (1 - k / e) ** t)
    return {"bytes": _w4_bytes(case, 3 * h * (touched * i + case["shared"])) + 4 * t * h + 12 * t * k,
            "flops": 6 * t * h * (k * i + case["shared"])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _prepare_grouped(case, normal, gen):
    s, r, e, n, k = dict(case), case["rows"], case["experts"], case["n"], case["k"]
    # a router's choice: experts more and less in demand
    demand = torch.softmax(normal(e, std=0.5), 0)
    used = r - r // 20 if case["tail"] else r
    sizes = torch.bincount(torch.multinomial(demand, used, replacement=True, generator=gen), minlength=e)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), sizes.cumsum(0)]).int()
    s["longest"] = int(sizes.max())
    s["x"] = normal(r, k, dtype=torch.bfloat16)
    s["w"] = normal(e, n, k, std=k ** -0.5, dtype=torch.bfloat16)
    if case["op"] == "grouped_bwd":
        s["dy"] = normal(r, n, dtype=torch.bfloat16)
        s["dw_type"] = torch.bfloat16 if case["dw"] == "bf16" else torch.float32
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 31)

    def normal(*shape, std=1.0, dtype=torch.float32):
        if len(shape) == 3:  # a large weight, expert by expert
            out = torch.empty(shape, dtype=dtype, device="cuda")
            for part in out:
                part.copy_(torch.randn(*part.shape, generator=gen, device="cuda") * std)
            return out
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op = case["op"]
    if op in ("grouped", "grouped_bwd"):
        return _prepare_grouped(case, normal, gen)
    s, how = dict(case), (case["format"], case["group"], case["zero"])
    if op == "w4_weights":
        s["w"] = normal(case["experts"], case["n"], case["k"], std=0.02, dtype=torch.bfloat16)
        return s
    if op == "w4_product":
        s["x"] = normal(case["tokens"], case["k"], dtype=torch.bfloat16)
        s["codes"], s["scale"], s["zeros"] = _quantize(normal(case["n"], case["k"], std=0.02), *how)
        return s
    t, h, i, e, k = (case[x] for x in ("tokens", "hidden", "inter", "experts", "topk"))
    s["x"] = normal(t, h, dtype=torch.bfloat16)
    logits = normal(t, e) + normal(e, std=0.5)
    top, s["ids"] = torch.topk(torch.softmax(logits, 1), k, dim=1)
    s["rw"] = top / top.sum(1, keepdim=True)
    if case["mask"]:  # padding tokens, as the router marks them
        gone = torch.rand(t, generator=gen, device="cuda") < 0.2
        s["ids"] = torch.where(gone[:, None], -1, s["ids"])
        s["rw"] = torch.where(gone[:, None], 0.0, s["rw"])
    s["weights"] = {}
    shapes = {"routed_gate": (e, i, h), "routed_up": (e, i, h), "routed_down": (e, h, i)}
    if case["shared"]:
        shapes |= {"shared_gate": (case["shared"], h), "shared_up": (case["shared"], h),
                   "shared_down": (h, case["shared"])}
    for name, shape in shapes.items():
        codes, scale, zeros = _quantize(normal(*shape, std=0.02, dtype=torch.bfloat16), *how)
        s["weights"] |= {name: codes, name + "_scale": scale}
        if zeros is not None:
            s["weights"][name + "_zero"] = zeros
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _quantize(w, form, group, zero):
    """(codes two to a byte, the even column in the low half; scales; zero points or None)."""
    b = w.float().unflatten(-1, (-1, group))
    if form == "mxfp4":
        amax = b.abs().amax(-1)
        x = torch.where(amax > 0, (torch.frexp(amax)[1] - 3).clamp(-127, 127), -127)
        scale = (x + 127).to(torch.uint8)
        v = b / scale.view(torch.float8_e8m0fnu).float()[..., None]
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
        q = (torch.round(v / step) * step).abs().clamp(max=6.0)
        # the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 in order
        c = torch.where(q <= 2, q * 2, torch.where(q <= 4, q + 2, q / 2 + 4)).to(torch.uint8)
        c = c + torch.where(torch.signbit(b), 8, 0).to(torch.uint8)
        zeros = None
    else:
        if zero:
            lo, hi = b.amin(-1).clamp(max=0.0), b.amax(-1).clamp(min=0.0)
            scale = ((hi - lo) / 15).to(torch.bfloat16)
            div = scale.float().where(scale > 0, 1.0)
            zeros = torch.round(-lo / div).clamp(0, 15).where(scale > 0, 0.0)
            c = (torch.round(b / div[..., None]) + zeros[..., None]).clamp(0, 15)
            c = c.where((scale > 0)[..., None], 0.0).to(torch.uint8)
            zeros = zeros.to(torch.uint8)
        else:
            scale = (b.abs().amax(-1) / 7).to(torch.bfloat16)
            div = scale.float().where(scale > 0, 1.0)
            c = torch.round(b / div[..., None]).clamp(-8, 7).where((scale > 0)[..., None], 0.0)
            c, zeros = (c + 8).to(torch.uint8), None
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), scale, zeros


def _values(codes, scale, zeros):
    """What 4-bit weights stand for, in 32 bits."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (scale.shape[-1], -1))
    if scale.dtype == torch.uint8:
        m = (c & 7).float()
        v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))
        v = torch.where(c > 7, -v, v) * scale.view(torch.float8_e8m0fnu).float()[..., None]
    else:
        z = 8.0 if zeros is None else zeros.float()[..., None]
        v = (c.float() - z) * scale.float()[..., None]
    return v.flatten(-2)


def _padded(s):
    """Row numbers of every expert's rows, [experts, longest], and which of them are its own."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["longest"], device="cuda")
    mine = at < off[1:, None]
    return torch.where(mine, at, 0), mine


def _rows_back(t, at, mine, rows):
    """[experts, longest, columns] back to [rows, columns], zeros where no expert has the row."""
    out = torch.zeros(rows + 1, t.shape[2], device="cuda")
    out.index_copy_(0, torch.where(mine, at, rows).flatten(), t.flatten(0, 1))
    return out[:rows].to(torch.bfloat16)


def _grouped(s):
    at, mine = _padded(s)
    x = s["x"].float()[at] * mine[..., None]
    return _rows_back(torch.bmm(x, s["w"].float().transpose(1, 2)), at, mine, s["rows"])


def _grouped_bwd(s):
    at, mine = _padded(s)
    dy = s["dy"].float()[at] * mine[..., None]
    dx = _rows_back(torch.bmm(dy, s["w"].float()), at, mine, s["rows"])
    x = s["x"].float()[at] * mine[..., None]
    return dx, torch.bmm(dy.transpose(1, 2), x).to(s["dw_type"])


def _w4_weights(s):
    codes, scale, zeros = _quantize(s["w"], s["format"], s["group"], s["zero"])
    return _seen(_values(codes, scale, zeros).to(torch.bfloat16), scale, zeros)


def _seen(values, scale, zeros):
    scale = scale.view(torch.float8_e8m0fnu) if scale.dtype == torch.uint8 else scale
    return (values, scale) if zeros is None else (values, scale, zeros)


def _w4_product(s):
    return (s["x"].float() @ _values(s["codes"], s["scale"], s["zeros"]).t()).to(torch.bfloat16)


def _swiglu(g, u, limit):
    if limit:
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1 + torch.exp(-g)) * u


def _w4_layer(s):
    w, x, ids = s["weights"], s["x"].float(), s["ids"].clamp(min=0)
    kept = torch.where(s["ids"] >= 0, s["rw"], 0.0)

    def values(name, chosen=None):
        part = [w[name], w[name + "_scale"], w.get(name + "_zero")]
        return _values(*[None if p is None else p if chosen is None else p[chosen] for p in part])

    if ids.numel() <= s["experts"]:  # few choices: each with its own expert's weights
        pick = ids.flatten()
        rows = x.repeat_interleave(s["topk"], 0)[..., None]
        h = _swiglu(values("routed_gate", pick) @ rows, values("routed_up", pick) @ rows, s["limit"])
        y = (values("routed_down", pick) @ h)[..., 0].unflatten(0, ids.shape)
        y = (y * kept[..., None]).sum(1)
    else:  # every expert on every token
        g = x @ values("routed_gate").flatten(0, 1).t()
        h = _swiglu(g, x @ values("routed_up").flatten(0, 1).t(), s["limit"]).unflatten(1, (s["experts"], -1))
        each = torch.zeros(x.shape[0], s["experts"], device="cuda").scatter_add_(1, ids, kept)
        h = (h * each[..., None]).transpose(0, 1).contiguous()
        y = torch.bmm(h, values("routed_down").transpose(1, 2)).sum(0)
    if s["shared"]:
        h = _swiglu(x @ values("shared_gate").t(), x @ values("shared_up").t(), s["limit"])
        y = y + h @ values("shared_down").t()
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(s):
    import mixture_experts_layer_build_amd as mok
    op = s["op"]
    if op == "grouped":
        return mok.grouped_matmul(s["x"], s["w"], s["offsets"])
    if op == "grouped_bwd":
        return mok.grouped_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"], dw_dtype=s["dw_type"])
    if op == "w4_weights":
        codes, scale, zeros = mok.w4_quantize(s["w"], format=s["format"], group=s["group"], zero_point=s["zero"])
        return _seen(mok.w4_dequantize(codes, scale, zeros), scale, zeros)
    if op == "w4_product":
        return mok.w4_matmul(s["x"], s["codes"], s["scale"], s["zeros"])
    return mok.forward_w4(s["x"], s["rw"], s["ids"], s["weights"], swiglu_limit=s["limit"])


def run(state):
    if own:
        return _run_own(state)
    return {"grouped": _grouped, "grouped_bwd": _grouped_bwd, "w4_weights": _w4_weights, "w4_product": _w4_product,
            "w4_layer": _w4_layer}[state["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values64(codes, scale, zeros):
    """[n, k/2] codes to [n, k] doubles."""
    n, groups = scale.shape
    c = torch.empty(n, codes.shape[1] * 2, dtype=torch.int64, device="cuda")
    c[:, 0::2], c[:, 1::2] = codes.long() % 16, codes.long() // 16
    per = c.shape[1] // groups
    if scale.dtype == torch.uint8:
        table = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device="cuda")
        return table[c] * torch.exp2(scale.double() - 127).repeat_interleave(per, 1)
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(per, 1)
    return (c.double() - z) * scale.double().repeat_interleave(per, 1)


def _weights64(s):
    w = s["w"].double().reshape(s["experts"] * s["n"], -1, s["group"])
    if s["format"] == "mxfp4":
        e = torch.frexp(w.abs().amax(2))[1].double() - 1
        scale = torch.exp2((e - 2).where(w.abs().amax(2) > 0, -127.0).clamp(-127, 127))
        v = w / scale[..., None]
        grid = torch.tensor(_E2M1, dtype=torch.float64, device="cuda")
        half = (grid[1:] + grid[:-1]) / 2
        a = v.abs()
        below = torch.bucketize(a, half)  # the number of half ways below a: its place, but for a tie
        tie = (below < 7) & (half[below.clamp(max=6)] == a)
        q = grid[torch.where(tie & (below % 2 == 1), below + 1, below)]
        out = torch.copysign(q, v) * scale[..., None]
        zeros = None
    elif s["zero"]:
        lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
        scale = ((hi - lo) / 15).to(torch.bfloat16).double()
        d = torch.where(scale > 0, scale, 1.0)
        z = torch.round(-lo / d).clamp(0, 15) * (scale > 0)
        out = ((torch.round(w / d[..., None]) + z[..., None]).clamp(0, 15) - z[..., None]) * scale[..., None]
        zeros = z.reshape(s["experts"], s["n"], -1)
    else:
        scale = (w.abs().amax(2) / 7).to(torch.bfloat16).double()
        d = torch.where(scale > 0, scale, 1.0)
        out = torch.round(w / d[..., None]).clamp(-8, 7) * scale[..., None]
        zeros = None
    out = (out.reshape(s["w"].shape), scale.reshape(s["experts"], s["n"], -1))
    return out if zeros is None else out + (zeros,)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("grouped", "grouped_bwd"):
        off = s["offsets"].tolist()
        r, n, k = case["rows"], case["n"], case["k"]
        a = torch.zeros(r, n if op == "grouped" else k, dtype=torch.float64, device="cuda")
        dw = torch.zeros(case["experts"], n, k, dtype=torch.float64, device="cuda") if op == "grouped_bwd" else None
        for e in range(case["experts"]):
            rows = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            x, w = s["x"][rows].double(), s["w"][e].double()
            if op == "grouped":
                a[rows] = x @ w.T
            else:
                dy = s["dy"][rows].double()
                a[rows] = dy @ w
                dw[e] = dy.T @ x
        return a if dw is None else (a, dw)
    if op == "w4_weights":
        return _weights64(s)
    x = s["x"].double()
    if op == "w4_product":
        return x @ _values64(s["codes"], s["scale"], s["zeros"]).T

    def mlp(rows, kind, e=None):
        def product(v, name):
            part = [s["weights"].get(kind + name + end) for end in ("", "_scale", "_zero")]
            return v @ _values64(*[p if p is None or e is None else p[e] for p in part]).T
        g, u = product(rows, "gate"), product(rows, "up")
        if case["limit"]:
            g, u = torch.minimum(g, torch.full_like(g, case["limit"])), u.clamp(-case["limit"], case["limit"])
        return product(g * torch.sigmoid(g) * u, "down")

    y = mlp(x, "shared_") if case["shared"] else torch.zeros_like(x)
    for e in range(case["experts"]):
        w = (s["rw"].double() * (s["ids"] == e)).sum(1)
        rows = (s["ids"] == e).any(1).nonzero()[:, 0]
        if len(rows):
            y[rows] += w[rows, None] * mlp(x[rows], "routed_", e)
    return y
