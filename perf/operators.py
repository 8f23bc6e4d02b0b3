"""The routed feed-forward's operators and 4-bit group-scaled weights, as measured workloads.

A case is a dict of plain values; prepare() makes its inputs on the GPU, run() makes one pass: the
operators in plain torch, or, with `own` set, through the package's entry points.  exact() gives
the same outputs from the definitions in 64 bits.

    route     router logits [T, E] -> expert ids and weights (train: and the logits' gradient)
    sort      tokens sorted by expert, with the index tables (train: and the gradient of x)
    unsort    expert outputs back in token order, weighted and summed (train: and both gradients)
    gemv      y = x W^T with W in 4-bit codes and one scale (and zero point) per group
    experts   the same over sorted rows and stacked experts, optionally with the SwiGLU epilogue
    quant     16-bit weights to 4-bit codes with group scales, and the values they stand for
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's router: eight sequences, one token each
        {"name": "route_decode", "op": "route", "T": 8, "E": 512, "k": 10, "dtype": "f32", "score": "softmax",
         "renorm": True, "train": False, "pad": False},
        # a training step's router over a full batch of tokens, forward and backward
        {"name": "route_train", "op": "route", "T": 4096, "E": 512, "k": 10, "dtype": "f32", "score": "softmax",
         "renorm": True, "train": True, "pad": False},
        # the same decode step's tokens brought into expert order
        {"name": "sort_decode", "op": "sort", "T": 8, "E": 512, "k": 10, "H": 2048, "dtype": "bf16", "train": False,
         "pad": False},
        # a training batch into expert order, and the gradient back to the tokens
        {"name": "sort_train", "op": "sort", "T": 4096, "E": 512, "k": 10, "H": 2048, "dtype": "bf16", "train": True,
         "pad": False},
        # the decode step's expert outputs (fp32, as the products leave them) combined per token
        {"name": "unsort_decode", "op": "unsort", "T": 8, "E": 512, "k": 10, "H": 2048, "dtype": "f32", "out": "bf16",
         "train": False, "pad": False},
        # a training batch combined, and the gradients of the expert outputs and the router weights
        {"name": "unsort_train", "op": "unsort", "T": 4096, "E": 512, "k": 10, "H": 2048, "dtype": "bf16",
         "out": "bf16", "train": True, "pad": False},
        # one token through a hidden-width projection
        {"name": "gemv_token", "op": "gemv", "M": 1, "N": 5120, "K": 5120, "G": 128, "zeros": False, "dtype": "bf16"},
        # eight sequences, small groups with zero points, an odd number of rows and a ragged K
        {"name": "gemv_batch", "op": "gemv", "M": 8, "N": 5119, "K": 5152, "G": 32, "zeros": True, "dtype": "f16"},
        # one token through an output head
        {"name": "gemv_head", "op": "gemv", "M": 1, "N": 151936, "K": 4096, "G": 128, "zeros": False, "dtype": "bf16"},
        # a decode step through the routed experts' gate / up projections
        {"name": "experts_decode", "op": "experts", "T": 8, "E": 512, "k": 10, "N": 1024, "K": 2048, "G": 128,
         "zeros": False, "dtype": "bf16", "swiglu": True},
        # a small projection with odd sizes, zero points and groups of 32
        {"name": "quant_small", "op": "quant", "N": 1027, "K": 2080, "G": 32, "zeros": True, "dtype": "f16"},
        # a wide projection weight, symmetric
        {"name": "quant_wide", "op": "quant", "N": 12288, "K": 5120, "G": 128, "zeros": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "sort", "unsort", "gemv", "experts", "quant"])
    if op == "route":
        E = _log(rng, 2, 512)
        k = rng.randint(1, min(E, 10))
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": k, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "score": rng.choice(["softmax", "sigmoid"]),
                "renorm": k > 1 and rng.random() < 0.5,  # a single weight renormalised is always one
                "train": rng.random() < 0.6, "pad": rng.random() < 0.5}
    if op in ("sort", "unsort"):
        E = _log(rng, 2, 512)
        k, H = rng.randint(1, min(E, 10)), _log(rng, 16, 8192)
        if rng.random() < 0.7:
            H = (H + 7) // 8 * 8  # model widths are even; the others are odd sizes
        T = _log(rng, 1, max(1, min(16384, 75_000_000 // ((k + 2) * H))))
        c = {"op": op, "T": T, "E": E, "k": k, "H": H, "dtype": rng.choice(["f32", "bf16", "f16"] if op == "unsort" else ["bf16", "bf16", "f16", "f32"]),
             "train": rng.random() < 0.5, "pad": rng.random() < 0.5}
        if c["dtype"] == "f32":
            c["T"] = max(1, T // 2)
        if op == "unsort":
            c["out"] = rng.choice(["f32", c["dtype"]]) if c["dtype"] != "f32" else rng.choice(["f32", "bf16", "f16"])
        return c
    G = rng.choice([32, 64, 128])
    if op == "quant":
        K = G * max(1, _log(rng, 64, 16384) // G)
        return {"op": op, "N": _log(rng, 1, max(2, min(32768, 60_000_000 // K))), "K": K, "G": G,
                "zeros": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16"])}
    if op == "gemv":
        K = G * max(1, _log(rng, 256, 16384) // G)
        return {"op": op, "M": _log(rng, 1, 16), "N": _log(rng, 32, max(33, min(160000, 300_000_000 // K))), "K": K, "G": G,
                "zeros": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16"])}
    E, swiglu = _log(rng, 4, 256), rng.random() < 0.5
    K = G * max(1, _log(rng, 256, 4096) // G)
    T, k = _log(rng, 1, 12), rng.randint(1, min(E, 10))
    F = _log(rng, 32, min(2048, 400_000_000 // (K * min(T * k, E)), 8_000_000_000 // (K * T * k)))
    return {"op": op, "T": T, "E": E, "k": k, "N": 2 * (F // 2) if swiglu else F, "K": K, "G": G,
            "zeros": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16"]), "swiglu": swiglu}


# ------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, sigma=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).to(dtype)


def _live(c):
    """Tokens that are not padding: the last tenth of a padded batch is."""
    return c["T"] - (c["T"] // 10 if c["pad"] else 0)


def _logits(g, T, E):
    """Router logits: some experts are liked more than others."""
    return _randn(g, T, E) + 0.5 * _randn(g, 1, E)


def _routing(g, c):
    r = _logits(g, c["T"], c["E"]).topk(c["k"], dim=1).indices.int()
    if c.get("pad"):
        r[_live(c):] = -1
    return r


def _weights4(g, rows, K, G, zeros, dtype):
    """Codes as a normal weight's are: a bell over the 16 codes; two codes per byte, the even one low."""
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        q = (torch.randn(min(step, rows - r), K, generator=g, device="cuda") * 2.6 + 8).round_().clamp_(0, 15).to(torch.uint8)
        codes[r:r + step] = q[:, 0::2] | (q[:, 1::2] << 4)
    scales = ((torch.rand(rows, K // G, generator=g, device="cuda") * 0.4 + 0.8) * (0.02 / 2.6)).to(dtype)
    z = torch.randint(5, 11, (rows, K // G), generator=g, device="cuda").to(torch.uint8) if zeros else None
    return codes, scales, z


def _plan(routing, E):
    """The stable order of the (token, slot) entries by expert; empty ones (-1) come last."""
    ids = routing.reshape(-1).long()
    ok = (ids >= 0) & (ids < E)
    key = torch.where(ok, ids, torch.full_like(ids, E))
    rows = torch.arange(ids.numel(), device=ids.device)
    sorted_key, order = torch.sort(key, stable=True)
    pos = torch.empty_like(ids)
    pos[order] = rows
    held = sorted_key < E
    offsets = torch.searchsorted(sorted_key, torch.arange(E + 1, device=ids.device))
    return (torch.where(ok, pos, torch.full_like(pos, -1)).int().reshape(routing.shape),
            torch.where(held, order, torch.full_like(order, -1)).int(),
            torch.where(held, sorted_key, torch.full_like(sorted_key, -1)).int(), offsets.int())


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        logits = _logits(g, T, E)
        if c["pad"]:
            logits[_live(c):] = -math.inf  # padding tokens have no expert
            logits[:, E - E // 8:] = -math.inf  # and some experts are switched off
        s["logits"], s["dw"] = logits.to(dt), _randn(g, T, k)
        s["outs"] = (torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda"))
        s["dlogits"] = torch.zeros(T, E, dtype=dt, device="cuda")
    elif c["op"] == "sort":
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        n = T * k
        s["routing"], s["x"] = _routing(g, c), _randn(g, T, H, dtype=dt)
        if c["train"]:
            s["dxs"], s["dx"] = _randn(g, n, H, dtype=dt), torch.zeros(T, H, dtype=dt, device="cuda")
        # rows behind the last expert's are not written: they stay the zeros they are here
        s["outs"] = (torch.zeros(n, H, dtype=dt, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"),
                     torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"),
                     torch.zeros(E + 1, dtype=torch.int32, device="cuda"))
    elif c["op"] == "unsort":
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        n, odt = T * k, TYPES[c["out"]]
        s["pos"] = _plan(_routing(g, c), E)[0]
        s["ys"] = _randn(g, n, H, dtype=dt)
        s["w"] = torch.rand(T, k, generator=g, device="cuda")
        s["w"] /= s["w"].sum(1, keepdim=True)
        s["y"] = torch.zeros(T, H, dtype=odt, device="cuda")
        if c["train"]:
            s["dy"] = _randn(g, T, H, dtype=odt)
            s["outs"] = (torch.zeros(n, H, dtype=dt, device="cuda"), torch.zeros(T, k, device="cuda"))
    elif c["op"] == "gemv":
        s["x"] = _randn(g, c["M"], c["K"], dtype=dt)
        s["w"] = _weights4(g, c["N"], c["K"], c["G"], c["zeros"], dt)
        s["y"] = torch.zeros(c["M"], c["N"], device="cuda")
    elif c["op"] == "experts":
        n = c["T"] * c["k"]
        _, _, s["row_expert"], s["offsets"] = _plan(_routing(g, c), c["E"])
        s["x"] = _randn(g, n, c["K"], dtype=dt)
        s["w"] = _weights4(g, c["E"] * c["N"], c["K"], c["G"], c["zeros"], dt)
        s["y"] = torch.zeros(n, c["N"] // 2, dtype=dt, device="cuda") if c["swiglu"] else torch.zeros(n, c["N"], device="cuda")
    else:
        N, K, G = c["N"], c["K"], c["G"]
        s["x"] = _randn(g, N, K, sigma=0.02, dtype=dt)
        s["w"] = (torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.zeros(N, K // G, dtype=dt, device="cuda"),
                  torch.zeros(N, K // G, dtype=torch.uint8, device="cuda") if c["zeros"] else None)
        s["values"] = torch.zeros(N, K, dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------------------------ plain forms

def _route(l, k, score, renorm):
    v, idx = torch.sort(l, dim=1, descending=True, stable=True)
    v, idx = v[:, :k], idx[:, :k]
    ok = v > -math.inf
    if score == "softmax":
        e = torch.exp(v - v[:, :1])
        total = e.masked_fill(~ok, 0).sum(1, keepdim=True) if renorm else torch.exp(l - v[:, :1]).sum(1, keepdim=True)
    else:
        e = 1 / (1 + torch.exp(-v))
        total = e.masked_fill(~ok, 0).sum(1, keepdim=True) if renorm else 1
    w = torch.where(ok, e / total, torch.zeros_like(e))
    return torch.where(ok, idx, torch.full_like(idx, -1)).int(), w


def _route_backward(l, routing, w, dw, score, renorm):
    ok = routing >= 0
    at = routing.clamp(min=0).long()
    g = dw.to(l.dtype).masked_fill(~ok, 0)
    v = torch.gather(l, 1, at).masked_fill(~ok, 0)
    dot = (w * g).sum(1, keepdim=True)
    d = torch.zeros_like(l)
    if score == "softmax":
        d.scatter_add_(1, at, (w * (g - dot if renorm else g)).masked_fill(~ok, 0))
        if not renorm:
            e = torch.exp(l - l.amax(1, keepdim=True))
            d -= torch.where(ok.any(1, keepdim=True), e / e.sum(1, keepdim=True), torch.zeros_like(e)) * dot
        return d
    up, down = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
    if renorm:
        total = up.masked_fill(~ok, 0).sum(1, keepdim=True)
        g = (g - dot) / torch.where(total > 0, total, torch.ones_like(total))
    return d.scatter_add_(1, at, (g * up * down).masked_fill(~ok, 0))


def _gather(rows, pos, w=None):
    """sum_s w[t, s] rows[pos[t, s]], in the type of `rows`."""
    v = rows[pos.clamp(min=0).long()]
    v = v.masked_fill((pos < 0)[..., None], 0)
    return (v if w is None else v * w[..., None]).sum(1)


def _values4(codes, scales, zeros, G):
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1, G).to(scales.dtype)
    z = 8 if zeros is None else (zeros & 15).to(scales.dtype)[..., None]
    return ((q - z) * scales[..., None]).flatten(-2)


def _swiglu(y):
    g, u = y.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def _plain(s):
    c = s["case"]
    f = torch.float32
    if c["op"] == "route":
        l = s["logits"].to(f)
        routing, w = _route(l, c["k"], c["score"], c["renorm"])
        if not c["train"]:
            return routing, w
        return routing, w, _route_backward(l, routing, w, s["dw"], c["score"], c["renorm"]).to(s["logits"].dtype)
    if c["op"] == "sort":
        pos, src, row_expert, offsets = _plan(s["routing"], c["E"])
        xs = s["x"][src.clamp(min=0).long() // c["k"]].masked_fill((src < 0)[:, None], 0)
        if not c["train"]:
            return xs, pos, src, row_expert, offsets
        return xs, pos, src, row_expert, offsets, _gather(s["dxs"].to(f), pos).to(xs.dtype)
    if c["op"] == "unsort":
        pos, ys, w = s["pos"], s["ys"].to(f), s["w"]
        y = _gather(ys, pos, w).to(s["y"].dtype)
        if not c["train"]:
            return y
        dy, held = s["dy"].to(f), pos >= 0
        at = pos.clamp(min=0).long()
        dw = (dy[:, None] * ys[at]).sum(2).masked_fill(~held, 0)
        dys = torch.zeros_like(ys)
        dys[at[held]] = (dy[:, None] * w[..., None])[held]
        return y, dys.to(s["ys"].dtype), dw
    if c["op"] == "gemv":
        codes, scales, zeros = s["w"]
        return s["x"].to(f) @ _values4(codes, scales.to(f), zeros, c["G"]).t()
    if c["op"] == "experts":
        codes, scales, zeros = (None if t is None else t.view(c["E"], c["N"], -1)[s["row_expert"].long()] for t in s["w"])
        y = torch.bmm(_values4(codes, scales.to(f), zeros, c["G"]), s["x"].to(f)[..., None])[..., 0]
        return _swiglu(y).to(s["x"].dtype) if c["swiglu"] else y
    # quant: the scale is held in w's type, so the quotients below are those of 16-bit numbers, and
    # 32 bits keep every one of them on its side of a rounding border
    w = s["x"].to(f).reshape(c["N"], -1, c["G"])
    if c["zeros"]:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scales = ((hi - lo) / 15).to(s["x"].dtype)
    else:
        scales = (w.abs().amax(2) / 7).to(s["x"].dtype)
    sf = scales.to(f)
    sf = torch.where(sf < 2.0 ** -126, torch.zeros_like(sf), sf)
    d = torch.where(sf > 0, sf, torch.ones_like(sf))
    z = torch.floor(-lo / d + 0.5).clamp(0, 15) if c["zeros"] else torch.full_like(sf, 8)
    q = (torch.floor(w / d[..., None] + 0.5) + z[..., None]).clamp(0, 15)
    q = torch.where(sf[..., None] > 0, q, z[..., None])
    values = ((q - z[..., None]) * sf[..., None]).to(s["x"].dtype).reshape(c["N"], -1)
    return sf.to(s["x"].dtype), z.to(torch.uint8) if c["zeros"] else None, values


# ------------------------------------------------------------------------------------ the package's calls

def _own(s):
    import fp16_gemm_b200 as sp
    c = s["case"]
    if c["op"] == "route":
        score = sp.ROUTE_SOFTMAX if c["score"] == "softmax" else sp.ROUTE_SIGMOID
        routing, w = sp.moe_route(s["logits"], c["k"], score, c["renorm"], out=s["outs"])
        if not c["train"]:
            return routing, w
        return routing, w, sp.moe_route_backward(s["dw"], s["logits"], routing, score, c["renorm"], out=s["dlogits"])
    if c["op"] == "sort":
        r = sp.moe_sort(s["x"], s["routing"], c["E"], out=s["outs"])
        if not c["train"]:
            return tuple(r)
        return (*r, sp.moe_sort_backward(s["dxs"], r[1], out=s["dx"]))
    if c["op"] == "unsort":
        y = sp.moe_unsort(s["ys"], s["pos"], s["w"], out=s["y"])
        if not c["train"]:
            return y
        return (y, *sp.moe_unsort_backward(s["dy"], s["ys"], s["pos"], s["w"], out=s["outs"]))
    if c["op"] == "gemv":
        return sp.gemv_w4(s["x"], sp.W4Tensor(*s["w"]), out=s["y"])
    if c["op"] == "experts":
        return sp.gemv_w4_grouped(s["x"], sp.W4Tensor(*s["w"]), s["offsets"],
                                  act=sp.ACT_SWIGLU if c["swiglu"] else sp.ACT_NONE, out=s["y"])
    q = sp.quantize_w4(s["x"], c["G"], zeros=c["zeros"], out=sp.W4Tensor(*s["w"]))
    return q.scales, q.zeros, sp.dequantize_w4(q, s["x"].dtype, out=s["values"])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    b = BYTES[c["dtype"]]
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * b + 8 * T * k + (T * E * b + 4 * T * k if c["train"] else 0),
                "flops": T * (4 * E + 4 * k) * (2 if c["train"] else 1)}
    if c["op"] in ("sort", "unsort"):
        T, k, H = c["T"], c["k"], c["H"]
        n = T * k
        live = _live(c) * k
        if c["op"] == "sort":
            fwd = _live(c) * H * b + live * H * b + 4 * n + 12 * n + 4 * (c["E"] + 1)
            return {"bytes": fwd + (live * H * b + T * H * b if c["train"] else 0), "flops": live * H if c["train"] else 0}
        ob = BYTES[c["out"]]
        fwd = live * H * b + 8 * n + T * H * ob
        return {"bytes": fwd + (_live(c) * H * ob + live * H * b + 4 * n if c["train"] else 0),
                "flops": 2 * live * H * (3 if c["train"] else 1)}
    per = lambda rows: rows * c["K"] // 2 + rows * (c["K"] // c["G"]) * (b + (1 if c["zeros"] else 0))  # noqa: E731
    if c["op"] == "gemv":
        return {"bytes": per(c["N"]) + c["M"] * c["K"] * b + 4 * c["M"] * c["N"], "flops": 2 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "experts":
        n = c["T"] * c["k"]
        met = min(n, c["E"], max(1, round(c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"]))))  # experts met, on average
        out = c["N"] // 2 * b if c["swiglu"] else c["N"] * 4
        return {"bytes": per(met * c["N"]) + n * c["K"] * b + n * out + 4 * (c["E"] + 1), "flops": 2 * n * c["N"] * c["K"]}
    return {"bytes": 2 * c["N"] * c["K"] * b + per(c["N"]), "flops": 4 * c["N"] * c["K"]}


# ------------------------------------------------------------------------------------ 64 bits

def _exact_route(s, c):
    l = s["logits"].double()
    T, E, k = c["T"], c["E"], c["k"]
    left, ids, w, sel = l.clone(), [], [], []
    number = torch.arange(E, device=l.device).expand(T, E)
    for _ in range(k):  # the largest one left, the lowest of equals
        top = left.amax(1, keepdim=True)
        at = torch.where(left == top, number, torch.full_like(number, E)).amin(1, keepdim=True)
        ids.append(torch.where(top > -math.inf, at, torch.full_like(at, -1)))
        sel.append(top)
        left.scatter_(1, at, -math.inf)
    ids, v = torch.cat(ids, 1), torch.cat(sel, 1)
    ok = ids >= 0
    if c["score"] == "softmax":
        logw = v - (torch.logsumexp(v, 1, keepdim=True) if c["renorm"] else torch.logsumexp(l, 1, keepdim=True))
        w = torch.where(ok, logw.exp(), torch.zeros_like(v))
    else:
        w = torch.sigmoid(v)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        w = torch.where(ok, w, torch.zeros_like(v))
    out = [ids.int(), w]
    if c["train"]:
        g = torch.where(ok, s["dw"].double(), torch.zeros_like(w))
        dot = (w * g).sum(1, keepdim=True)
        if c["score"] == "softmax":
            part = w * (g - dot) if c["renorm"] else w * g
        else:
            slope = torch.sigmoid(v) * torch.sigmoid(-v)
            part = slope * ((g - dot) / torch.sigmoid(v).sum(1, keepdim=True) if c["renorm"] else g)
        part = torch.where(ok, part, torch.zeros_like(part))
        d = torch.zeros(T, E + 1, dtype=torch.float64, device=l.device)
        d.scatter_(1, torch.where(ok, ids, torch.full_like(ids, E)), part)
        d = d[:, :E]
        if c["score"] == "softmax" and not c["renorm"]:
            d = d - torch.nan_to_num(torch.softmax(l, 1)) * dot
        out.append(d)
    return out


def _exact_values(codes, scales, zeros, G):
    q = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    q[:, 0::2] = (codes % 16).double()
    q[:, 1::2] = (codes // 16).double()
    z = torch.full(scales.shape, 8.0, dtype=torch.float64, device=codes.device) if zeros is None else zeros.double()
    return (q - z.repeat_interleave(G, 1)) * scales.double().repeat_interleave(G, 1)


def _exact_product(x, w, G):
    codes, scales, zeros = w
    step = max(1, (1 << 26) // x.shape[1])
    parts = [x.double() @ _exact_values(codes[r:r + step], scales[r:r + step], None if zeros is None else zeros[r:r + step], G).t()
             for r in range(0, codes.shape[0], step)]
    return torch.cat(parts, 1)


def _exact_quant(s, c):
    # the definition's own roundings: the scale to fp32 and then to w's type
    w = s["x"].double().view(c["N"], c["K"] // c["G"], c["G"])
    lo, hi = torch.clamp(w.amin(2), max=0), torch.clamp(w.amax(2), min=0)
    span = (hi - lo).float().double() / 15 if c["zeros"] else torch.maximum(hi, -lo) / 7
    scale = span.float().to(s["x"].dtype).double()
    scale[scale < 2.0 ** -126] = 0
    z = torch.floor(-lo / scale + 0.5).clamp(0, 15) if c["zeros"] else torch.full_like(scale, 8)
    z = torch.where(scale > 0, z, torch.zeros_like(z) if c["zeros"] else z)
    n = torch.floor(w / scale[..., None] + 0.5)
    n = torch.where(scale[..., None] > 0, torch.minimum(torch.maximum(n, -z[..., None]), 15 - z[..., None]), torch.zeros_like(n))
    return [scale, z.to(torch.uint8) if c["zeros"] else None, (n * scale[..., None]).view(c["N"], c["K"])]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return tuple(_exact_route(s, c))
    if c["op"] == "sort":
        E, k = c["E"], c["k"]
        ids = s["routing"].reshape(-1)
        n = ids.numel()
        number = torch.arange(n, device="cuda")
        place = torch.where(ids >= 0, ids.long(), torch.full_like(number, E)) * n + number  # expert first, then order
        order = torch.argsort(place)
        held = ids[order] >= 0
        pos = torch.empty_like(number)
        pos[order] = number
        pos[ids < 0] = -1
        src = torch.where(held, order, torch.full_like(order, -1))
        offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"),
                             torch.bincount(ids[ids >= 0].long(), minlength=E).cumsum(0)))
        xs = torch.zeros(n, c["H"], dtype=torch.float64, device="cuda")
        xs[held] = s["x"].double()[order[held] // k]
        out = [xs, pos.view(c["T"], k).int(), src.int(), ids[order].int(), offsets.int()]
        if c["train"]:
            d = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
            d.index_add_(0, number[ids >= 0] // k, s["dxs"].double()[pos[ids >= 0]])
            out.append(d)
        return tuple(out)
    if c["op"] == "unsort":
        k, pos = c["k"], s["pos"].reshape(-1).long()
        live = (pos >= 0).nonzero()[:, 0]
        ys, w = s["ys"].double(), s["w"].double().reshape(-1)
        y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        y.index_add_(0, live // k, ys[pos[live]] * w[live, None])
        if not c["train"]:
            return y
        dy = s["dy"].double()[live // k]
        dw, dys = torch.zeros_like(w), torch.zeros_like(ys)
        dw[live] = torch.linalg.vecdot(dy, ys[pos[live]])
        dys[pos[live]] = dy * w[live, None]
        return y, dys, dw.view(c["T"], k)
    if c["op"] == "gemv":
        return _exact_product(s["x"], s["w"], c["G"])
    if c["op"] == "experts":
        at, n = s["offsets"].tolist(), c["N"]
        y = torch.zeros(s["x"].shape[0], n, dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            if at[e] < at[e + 1]:
                part = tuple(None if t is None else t[e * n:(e + 1) * n] for t in s["w"])
                y[at[e]:at[e + 1]] = _exact_product(s["x"][at[e]:at[e + 1]], part, c["G"])
        return y[:, :n // 2] * torch.sigmoid(y[:, :n // 2]) * y[:, n // 2:] if c["swiglu"] else y
    return tuple(_exact_quant(s, c))
