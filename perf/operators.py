"""Timed cases of the operators around the expert layer, with their plain forms.

  norm         h = x + residual, y = rmsnorm(h) in bf16, and y in MXFP8 (codes and tiled scales)
  norm_bwd     its gradient: dx (with the residual stream's own gradient added) and dw
  route        top-k choice over router logits, routing weights, per-expert counts, balance loss
  route_bwd    the gradient of the weights and of the balance loss with respect to the logits
  dprob        the gradient of the routing weights from the expert outputs
  gather       MXFP8 rows (codes and tiled scales) into the expert-ordered layout

`run` computes each in elementary torch operations in 32 bits, or, where `own` is true, by the
framework's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
#: logits at or below bf16's lowest finite value (and NaN) mark an expert out of reach
LOWEST = -3.3895313892515355e38
FLT_MAX = 3.4028234663852886e38


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step of the 671B-shaped layer: latency only
        {"name": "norm_T1_K7168", "op": "norm", "T": 1, "K": 7168, "pad": 0, "residual": True, "quant": True, "w32": False},
        # the 30B-shaped layer's forward, 16384 tokens
        {"name": "norm_T16384_K2048", "op": "norm", "T": 16384, "K": 2048, "pad": 0, "residual": True, "quant": True, "w32": False},
        # the 671B-shaped layer's forward, 32768 tokens, fp32 norm weights: the largest
        {"name": "norm_T32768_K7168", "op": "norm", "T": 32768, "K": 7168, "pad": 0, "residual": True, "quant": True, "w32": True},
        # a training step of the 30B-shaped layer: both readers of y send a gradient, and the residual stream its own
        {"name": "norm_bwd_T8192_K2048", "op": "norm_bwd", "T": 8192, "K": 2048, "pad": 0, "two": True, "dh": True, "w32": True},
        # ragged: an odd number of tokens, a width that is no multiple of 32, rows inside a wider buffer
        {"name": "norm_bwd_T4093_K1544", "op": "norm_bwd", "T": 4093, "K": 1544, "pad": 24, "two": False, "dh": True, "w32": False},
        # a decode batch of 64 tokens over 256 experts, sigmoid scores with a choice bias
        {"name": "route_T64_E256", "op": "route", "T": 64, "E": 256, "k": 8, "score": "sigmoid", "norm": True, "bf16": False, "masked": 0.0, "dead": 0.0, "skew": 0.0},
        # the 671B-shaped layer's 32768 tokens, Zipf-skewed expert load
        {"name": "route_T32768_E256", "op": "route", "T": 32768, "E": 256, "k": 8, "score": "softmax", "norm": True, "bf16": False, "masked": 0.0, "dead": 0.0, "skew": 1.1},
        # training on ragged batches: padding tokens, experts masked out, bf16 logits (many ties)
        {"name": "route_bwd_T8191_E128", "op": "route_bwd", "T": 8191, "E": 128, "k": 8, "score": "softmax", "norm": True, "bf16": True, "masked": 0.1, "dead": 0.05, "skew": 0.0},
        # the routing weights' gradient of the 30B-shaped training step
        {"name": "dprob_T8192_H2048", "op": "dprob", "T": 8192, "H": 2048, "E": 128, "k": 8, "dropped": 0.0},
        # a small ragged batch of wide rows, some slots dropped
        {"name": "dprob_T257_H7168", "op": "dprob", "T": 257, "H": 7168, "E": 256, "k": 6, "dropped": 0.02},
        # a decode batch's rows into 16-row segments: mostly padding rows
        {"name": "gather_T64_K7168", "op": "gather", "T": 64, "K": 7168, "E": 256, "k": 8, "pad_rows": 16},
        # the 30B-shaped layer's rows into 256-row segments
        {"name": "gather_T8192_K2048", "op": "gather", "T": 8192, "K": 2048, "E": 128, "k": 8, "pad_rows": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "route", "route_bwd", "dprob", "gather"])
    if op == "norm":
        quant = rng.random() < 0.6
        K = 32 * _log(rng, 2, 256) if quant else _log(rng, 33, 8192)
        T = _log(rng, 1, max(1, min(32768, (1 << 27) // K)))
        return {"op": op, "T": T, "K": K, "pad": rng.choice([0, 0, 8, 40]), "residual": rng.random() < 0.7, "quant": quant, "w32": rng.random() < 0.5}
    if op == "norm_bwd":
        K = 8 * _log(rng, 8, 1024) if rng.random() < 0.7 else _log(rng, 33, 8192)
        T = _log(rng, 1, max(1, min(32768, (1 << 27) // K)))
        return {"op": op, "T": T, "K": K, "pad": rng.choice([0, 0, 8, 40]), "two": rng.random() < 0.5, "dh": rng.random() < 0.7, "w32": rng.random() < 0.5}
    if op in ("route", "route_bwd"):
        E = _log(rng, 8, 512)
        return {"op": op, "T": _log(rng, 1, 32768), "E": E, "k": _log(rng, 1, min(E, 16)), "score": rng.choice(["softmax", "sigmoid"]), "norm": rng.random() < 0.6, "bf16": rng.random() < 0.5, "masked": rng.choice([0.0, 0.1]), "dead": rng.choice([0.0, 0.05]), "skew": rng.choice([0.0, 1.1])}
    E, k = _log(rng, 8, 256), rng.choice([1, 2, 4, 6, 8])
    if op == "dprob":
        H = 8 * _log(rng, 16, 896)
        return {"op": op, "T": _log(rng, 1, max(1, min(16384, (1 << 28) // (H * k)))), "H": H, "E": E, "k": k, "dropped": rng.choice([0.0, 0.02])}
    K = 64 * _log(rng, 2, 112)
    return {"op": op, "T": _log(rng, 1, max(1, min(16384, (1 << 28) // (K * k)))), "K": K, "E": E, "k": k, "pad_rows": rng.choice([16, 128, 256])}


# ---------------------------------------------------------------- inputs

def _pad(n, m):
    return (n + m - 1) // m * m


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, device="cuda", generator=g) * std).to(dtype)


def _rows(g, T, K, pad, std=1.0):
    """bf16 [T, K] inside rows of K + pad elements; a few large entries, as residual streams have."""
    v = torch.randn(T, K + pad, device="cuda", generator=g) * std
    v *= torch.where(torch.rand(T, K + pad, device="cuda", generator=g) < 1e-3, 30.0, 1.0)
    return v.to(torch.bfloat16)[:, :K]


def _segments(g, T, E, k, pad_rows):
    """(seg [E+1], perm [cap], inv [T*k], prob [T, k]) of k distinct random experts a token."""
    z = torch.randn(T, E, device="cuda", generator=g)
    prob, ids = torch.sort(torch.softmax(z, 1), dim=1, descending=True, stable=True)
    k = min(k, E)
    prob, ids = prob[:, :k], ids[:, :k]
    prob = (prob / prob.sum(1, keepdim=True)).contiguous()
    flat = ids.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    padded = (counts + pad_rows - 1) // pad_rows * pad_rows
    seg = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    seg[1:] = torch.cumsum(padded, 0)
    order = torch.sort(flat, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    row = seg[:-1][flat[order]] + torch.arange(flat.numel(), device="cuda") - first[flat[order]]
    cap = _pad(T * k, pad_rows) + pad_rows * E
    perm = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    perm[row] = order.to(torch.int32)
    inv = torch.empty(T * k, dtype=torch.int32, device="cuda")
    inv[order] = row.to(torch.int32)
    return seg.to(torch.int32), perm, inv, prob, cap


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, T = case["op"], case["T"]
    if op == "norm":
        K = case["K"]
        s["x"] = _rows(g, T, K, case["pad"])
        s["r"] = _rows(g, T, K, case["pad"], 2.0) if case["residual"] else None
        s["w"] = 1.0 + 0.1 * torch.randn(K, device="cuda", generator=g)
        s["w"] = s["w"] if case["w32"] else s["w"].to(torch.bfloat16)
    elif op == "norm_bwd":
        K = case["K"]
        s["h"] = _rows(g, T, K, case["pad"], 2.0)
        s["w"] = 1.0 + 0.1 * torch.randn(K, device="cuda", generator=g)
        s["w"] = s["w"] if case["w32"] else s["w"].to(torch.bfloat16)
        s["dy"] = _rows(g, T, K, case["pad"], 1e-3)
        s["dy2"] = _rows(g, T, K, case["pad"], 1e-3) if case["two"] else None
        s["dh"] = _rows(g, T, K, case["pad"], 1e-3) if case["dh"] else None
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
    elif op in ("route", "route_bwd"):
        E, k = case["E"], min(case["k"], case["E"])
        s["k"] = k
        z = torch.randn(T, E, device="cuda", generator=g)
        if case["skew"]:
            # Gumbel noise on Zipf log-probabilities: skewed expert load
            u = torch.rand(T, E, device="cuda", generator=g).clamp(1e-7, 1 - 1e-7)
            z = -case["skew"] * torch.log(torch.arange(E, device="cuda") + 1.0) - torch.log(-torch.log(u))
        if case["dead"]:
            out = torch.rand(T, E, device="cuda", generator=g) < case["dead"]
            z = torch.where(out, torch.full_like(z, -math.inf), z)
            z[:: max(3, T // 7)] = -math.inf          # rows whose mask leaves no expert
        s["logits"] = z.to(torch.bfloat16) if case["bf16"] else z
        s["bias"] = 0.05 * torch.randn(E, device="cuda", generator=g) if case["score"] == "sigmoid" else None
        s["mask"] = (torch.rand(T, device="cuda", generator=g) >= case["masked"]) if case["masked"] else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        if op == "route_bwd":
            ids, _, _, live = _choose(s, s["logits"])
            m = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device="cuda")
            picked = torch.gather(live, 1, ids) & m[:, None]
            s["ids"] = ids.to(torch.int32)
            s["counts"] = torch.bincount(ids[picked], minlength=E).to(torch.int32)
            s["n_tokens"] = m.sum().to(torch.int32).reshape(1)
            s["dprob"] = 1e-2 * torch.randn(T, k, device="cuda", generator=g)
            s["dloss"] = torch.full((1,), 0.01, device="cuda")
    elif op == "dprob":
        k = s["k"] = min(case["k"], case["E"])
        _, _, inv, prob, cap = _segments(g, T, case["E"], k, 256)
        if case["dropped"]:
            inv = torch.where(torch.rand(T * k, device="cuda", generator=g) < case["dropped"], torch.full_like(inv, -1), inv)
        s["inv"], s["prob"] = inv, prob
        s["y"] = torch.empty(cap, case["H"], dtype=torch.bfloat16, device="cuda")
        for at in range(0, cap, 65536):
            s["y"][at:at + 65536] = _normal(g, min(65536, cap - at), case["H"], std=0.1)
        s["dout"] = _normal(g, T, case["H"], std=1e-3)
    elif op == "gather":
        K, E = case["K"], case["E"]
        k = s["k"] = min(case["k"], E)
        s["seg"], s["perm"], _, _, s["cap"] = _segments(g, T, E, k, case["pad_rows"])
        q = torch.randint(0, 254, (T, K), device="cuda", generator=g)
        s["q"] = (q + (q >= 127)).to(torch.uint8)      # every E4M3 code but the two NaNs
        sc = torch.randint(119, 135, (T, K // 32), device="cuda", generator=g).to(torch.uint8)
        s["s"] = _tile(sc)
        # the layer's own buffers, kept from call to call; rows past the last segment are never written
        s["out"] = (torch.zeros(s["cap"], K, dtype=torch.uint8, device="cuda"),
                    torch.zeros(_pad(s["cap"], 128) * _pad(K // 32, 4), dtype=torch.uint8, device="cuda"))
    return s


# ---------------------------------------------------------------- plain forms

def _tile(sc):
    """Scale matrix [rows, cols] -> flat 128x4 tiles, zero padded: entry (r, c) of a tile at
    (r % 32) * 16 + (r / 32) * 4 + c."""
    rows, cols = sc.shape
    p = torch.zeros(_pad(rows, 128), _pad(cols, 4), dtype=sc.dtype, device=sc.device)
    p[:rows, :cols] = sc
    return p.view(p.shape[0] // 128, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _untile(flat, rows, cols):
    rt, ct = _pad(rows, 128) // 128, _pad(cols, 4) // 4
    return flat.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:rows, :cols]


def _f8(codes):
    return codes.view(torch.float8_e4m3fn)


def _e8(scales):
    return scales.view(torch.float8_e8m0fnu)


def _choose(s, logits):
    """(ids, scores, exp sums or None, live) of the k chosen experts, ties to the lower id."""
    l = logits.float()
    live = l > LOWEST
    if s["bias"] is not None:
        live = live & (s["bias"] > LOWEST)[None, :]
    l = torch.where(live, l.clamp(max=FLT_MAX), torch.full_like(l, -math.inf))
    if s["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        e = torch.where(live, torch.exp(l - m), torch.zeros_like(l))
        total = e.sum(1, keepdim=True)
        sc = e / torch.where(total > 0, total, torch.ones_like(total))
        key = l
    else:
        sc = torch.where(live, 1.0 / (1.0 + torch.exp(-l)), torch.zeros_like(l))
        key = torch.where(live, sc + s["bias"] if s["bias"] is not None else sc, torch.full_like(l, -math.inf))
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    return ids, sc, l, live


def _shares(s, sc):
    """Scores as shares of one per token: what the balance loss averages."""
    if s["score"] == "softmax":
        return sc
    total = sc.sum(1, keepdim=True)
    return sc / torch.where(total > 0, total, torch.ones_like(total))


def _plain_norm(s):
    h = s["x"].float()
    o = {}
    if s["r"] is not None:
        h = h + s["r"].float()
        o["h"] = h.to(torch.bfloat16)
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    y = (h * rstd[:, None] * s["w"].float()).to(torch.bfloat16)
    o["y"], o["rstd"] = y, rstd
    if s["quant"]:
        b = y.float().view(y.shape[0], -1, 32)
        bits = b.abs().amax(2).view(torch.int32)
        e = ((bits >> 23) - 127) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
        e = torch.where((bits >> 23) == 0, torch.full_like(e, -127), e).clamp(-127, 127)
        o["row_q"] = (b * torch.exp2(-e.float())[:, :, None]).to(torch.float8_e4m3fn).view(y.shape)
        o["row_s"] = _e8(_tile((e + 127).to(torch.uint8)))
    return o


def _plain_norm_bwd(s):
    h, w = s["h"].float(), s["w"].float()
    dy = s["dy"].float()
    if s["dy2"] is not None:
        dy = dy + s["dy2"].float()
    xh = h * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * xh).sum(0)}


def _plain_route(s):
    T, E = s["logits"].shape
    k = s["k"]
    ids, sc, _, live = _choose(s, s["logits"])
    w = torch.gather(sc, 1, ids)
    if s["norm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    w = w * s["scale"]
    m = s["mask"] if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=w.device)
    prob = torch.where(m[:, None], w, torch.zeros_like(w))
    picked = torch.gather(live, 1, ids) & m[:, None]
    counts = torch.zeros(E, dtype=torch.int32, device=w.device)
    counts.index_add_(0, ids.reshape(-1), picked.reshape(-1).to(torch.int32))
    n = m.sum().to(torch.int32)
    share = torch.where(m[:, None], _shares(s, sc), torch.zeros_like(sc))
    load = share.sum(0) / n.clamp(min=1)
    loss = (counts * load).sum() * E / (k * n.clamp(min=1))
    return {"ids": ids.to(torch.int32), "prob": prob, "counts": counts, "n_tokens": n.reshape(1), "load": load, "loss": loss.reshape(1)}


def _plain_route_bwd(s):
    T, E = s["logits"].shape
    k = s["k"]
    l = s["logits"].float()
    live = l > LOWEST
    if s["bias"] is not None:
        live = live & (s["bias"] > LOWEST)[None, :]
    l = torch.where(live, l.clamp(max=FLT_MAX), torch.full_like(l, -math.inf))
    n = s["n_tokens"].float().clamp(min=1.0)
    c = s["dloss"] * E * s["counts"].float() / (k * n * n)
    ids = s["ids"].long()
    d = s["dprob"] * s["scale"]
    zero = torch.zeros_like(l)
    if s["score"] == "softmax":
        e = torch.where(live, torch.exp(l - l.amax(1, keepdim=True)), zero)
        total = e.sum(1, keepdim=True)
        sc = e / torch.where(total > 0, total, torch.ones_like(total))
        local = 1.0
    else:
        sc = torch.where(live, 1.0 / (1.0 + torch.exp(-l)), zero)
        local = sc * (1.0 - sc)
    w = torch.gather(sc, 1, ids)
    if s["norm"]:
        total = w.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        q = w / total
        d = (d - (d * q).sum(1, keepdim=True)) / total
    ds = zero.scatter_add(1, ids, d)
    if s["score"] == "softmax":
        ds = ds + c
        dl = sc * (ds - (sc * ds).sum(1, keepdim=True))
    else:
        total = sc.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        ds = ds + (c - (sc / total * c).sum(1, keepdim=True)) / total
        dl = ds * local
    dl = torch.where(live, dl, zero)
    if s["mask"] is not None:
        dl = torch.where(s["mask"][:, None], dl, zero)
    return dl.to(s["logits"].dtype)


def _plain_dprob(s):
    T, k = s["prob"].shape
    inv = s["inv"].long()
    rows = s["y"][inv.clamp(min=0)].view(T, k, -1)
    dot = (rows.float() * s["dout"].float()[:, None, :]).sum(2)
    ok = (inv.view(T, k) >= 0) & (s["prob"] != 0)
    return torch.where(ok, dot / torch.where(ok, s["prob"], torch.ones_like(dot)), torch.zeros_like(dot))


def _plain_gather(s):
    T, K = s["q"].shape
    tok = s["perm"].long()
    rows = torch.where((tok >= 0)[:, None], s["q"][tok.clamp(min=0) // s["k"]], torch.zeros_like(s["q"][:1]))
    sc = _untile(s["s"], T, K // 32)
    sc = torch.where((tok >= 0)[:, None], sc[tok.clamp(min=0) // s["k"]], torch.zeros_like(sc[:1]))
    return {"row_q": _f8(rows), "row_s": _e8(_tile(sc))}


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["op"]
    if not own:
        plain = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "route": _plain_route,
                 "route_bwd": _plain_route_bwd, "dprob": _plain_dprob, "gather": _plain_gather}
        return plain[op](s)
    from microscaled_precision_moe_gb300 import ops
    if op == "norm":
        o = ops.add_rmsnorm(s["x"], s["w"], residual=s["r"], eps=EPS, quantize=s["quant"])
        if s["quant"]:
            o["row_q"], o["row_s"] = _f8(o["row_q"]), _e8(o["row_s"])
        return o
    if op == "norm_bwd":
        dx, dw = ops.add_rmsnorm_backward(s["dy"], s["h"], s["rstd"], s["w"], dy2=s["dy2"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "route":
        return ops.moe_route(s["logits"], s["k"], score=s["score"], normalize=s["norm"], scale=s["scale"],
                             bias=s["bias"], token_mask=s["mask"])
    if op == "route_bwd":
        return ops.moe_route_backward(s["logits"], s["ids"], s["counts"], s["n_tokens"], dprob=s["dprob"],
                                      dloss=s["dloss"], score=s["score"], normalize=s["norm"],
                                      scale=s["scale"], bias=s["bias"], token_mask=s["mask"])
    if op == "dprob":
        return ops.moe_combine_dprob(s["dout"], s["y"], s["inv"], s["prob"])
    q, sc = ops.moe_gather_mxfp8(s["q"], s["s"], s["perm"], s["seg"], s["E"], s["k"], s["cap"], out=s["out"])
    return {"row_q": _f8(q), "row_s": _e8(sc)}


def work(case):
    op, T = case["op"], case["T"]
    if op == "norm":
        n = T * case["K"]
        b = 4 * n + (4 * n if case["residual"] else 0) + (n + n // 32 if case["quant"] else 0)
        return {"bytes": b + 4 * T + case["K"] * (4 if case["w32"] else 2), "flops": 6 * n}
    if op == "norm_bwd":
        n = T * case["K"]
        return {"bytes": n * (6 + 2 * case["two"] + 2 * case["dh"]) + 4 * T + case["K"] * (8 if case["w32"] else 6), "flops": 12 * n}
    if op in ("route", "route_bwd"):
        k = min(case["k"], case["E"])
        n = T * case["E"] * (2 if case["bf16"] else 4)
        mask = T if case["masked"] else 0
        return {"bytes": n * (1 if op == "route" else 2) + 8 * T * k + mask + 8 * case["E"], "flops": 10 * T * case["E"]}
    k = min(case["k"], case["E"])
    if op == "dprob":
        return {"bytes": 2 * T * case["H"] * (1 + k) + 12 * T * k, "flops": 2 * T * k * case["H"]}
    # each token's row is read once; each routed row and each padding row of a segment is written once.  The
    # segments' lengths depend on the routing: the expected number of experts hit, each padded by half a
    # pad on average, or to one pad where an expert has few rows
    n, pad = case["K"] + case["K"] // 32, case["pad_rows"]
    hit = case["E"] * (1.0 - (1.0 - k / case["E"]) ** T)
    rows = hit * max(pad, T * k / hit + pad / 2)
    return {"bytes": T * n + rows * (n + 4), "flops": 0}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_bwd":
        return _exact_norm_bwd(s)
    if op == "route":
        return _exact_route(s)
    if op == "route_bwd":
        return _exact_route_bwd(s)
    if op == "dprob":
        T, k = s["prob"].shape
        out = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        for at in range(0, T, 512):
            d = s["dout"][at:at + 512].double().repeat_interleave(k, 0)
            i = s["inv"][at * k:at * k + d.shape[0]].long()
            v = torch.einsum("nh,nh->n", d, s["y"].index_select(0, i.clamp(min=0)).double())
            p = s["prob"].reshape(-1)[at * k:at * k + d.shape[0]].double()
            out[at * k:at * k + d.shape[0]] = torch.where((i >= 0) & (p != 0), v / p, torch.zeros_like(v))
        return out.view(T, k)
    T, K = s["q"].shape
    token = torch.div(s["perm"].long(), s["k"], rounding_mode="floor")
    value = _f8(torch.arange(256, device="cuda").to(torch.uint8)).double()
    codes = torch.zeros(s["cap"], K, dtype=torch.float64, device="cuda")
    at = (s["perm"] >= 0).nonzero().reshape(-1)
    codes[at] = value[s["q"][token[at]].long()]
    r = torch.arange(_pad(s["cap"], 128), device="cuda")
    words = _pad(K // 32, 4) // 4
    scales = torch.zeros(r.numel() * words * 4, dtype=torch.float64, device="cuda") + 2.0 ** -127
    for c in range(K // 32):
        place = lambda row: (row // 128 * words + c // 4) * 512 + row % 32 * 16 + row // 32 % 4 * 4 + c % 4  # noqa: E731
        scales[place(at)] = torch.exp2(s["s"][place(token[at])].double() - 127)
    return {"row_q": codes, "row_s": scales}


def _exact_norm(s):
    x = s["x"].double() if s["r"] is None else s["x"].double().add_(s["r"].double())
    T, K = x.shape
    inv = 1.0 / torch.sqrt(torch.einsum("tk,tk->t", x, x) / K + EPS)
    o = {"rstd": inv}
    if s["r"] is not None:
        o["h"] = x
    y = torch.einsum("tk,t,k->tk", x, inv, s["w"].double())
    o["y"] = y
    if s["quant"]:
        # the 8-bit output is the quantisation of the bf16 output: 32 values share 2^e, the smallest with max <= 448 * 2^e
        b = y.to(torch.bfloat16).double().reshape(T, K // 32, 32)
        top = b.abs().amax(2)
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).clamp(-127, 127)
        o["row_q"] = (b * torch.exp2(-e)[..., None]).float().to(torch.float8_e4m3fn).double().reshape(T, K)
        cols = _pad(K // 32, 4)
        full = torch.full((_pad(T, 128), cols), -127.0, dtype=torch.float64, device="cuda")
        full[:T, :K // 32] = e
        r, c = torch.meshgrid(torch.arange(full.shape[0], device="cuda"), torch.arange(cols, device="cuda"), indexing="ij")
        o["row_s"] = torch.zeros(full.numel(), dtype=torch.float64, device="cuda")
        o["row_s"][(r // 128 * (cols // 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4] = torch.exp2(full)
    return o


def _exact_norm_bwd(s):
    h, w, r = s["h"].double(), s["w"].double(), s["rstd"].double()
    dy = s["dy"].double()
    if s["dy2"] is not None:
        dy = dy + s["dy2"].double()
    K = h.shape[1]
    # y = h r w with r = (mean h^2 + eps)^(-1/2), so dr/dh = -r^3 h / K
    dw = torch.einsum("tk,tk,t->k", dy, h, r)
    through = torch.einsum("tk,k,tk->t", dy, w, h)
    dx = dy * w * r[:, None] - h * (through * r ** 3 / K)[:, None]
    return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": dw}


def _exact_scores(s):
    l = s["logits"].double()
    out = torch.isnan(l) | (l <= LOWEST)
    if s["bias"] is not None:
        out |= torch.isnan(s["bias"])[None] | (s["bias"].double() <= LOWEST)[None]
    l = torch.where(out, torch.full_like(l, -math.inf), l.clamp(max=FLT_MAX))
    if s["score"] == "softmax":
        sc = torch.softmax(l, 1).nan_to_num(0.0)
        key = l
    else:
        sc = torch.sigmoid(l)
        key = sc if s["bias"] is None else torch.where(out, torch.full_like(l, -math.inf), sc + s["bias"].double())
        key = torch.where(out, torch.full_like(l, -math.inf), key)
    return sc, key, out


def _exact_route(s):
    sc, key, out = _exact_scores(s)
    T, E = sc.shape
    k = s["k"]
    order = torch.argsort(-key, dim=1, stable=True)[:, :k]
    hot = torch.zeros_like(sc).scatter_(1, order, 1.0)
    w = torch.gather(sc, 1, order)
    if s["norm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    keep = torch.ones(T, 1, dtype=torch.float64, device="cuda") if s["mask"] is None else s["mask"].double()[:, None]
    n = max(float(keep.sum()), 1.0)
    share = (sc / sc.sum(1, keepdim=True)).nan_to_num(0.0)
    load = (share * keep).sum(0) / n
    counts = (hot * keep * (~out)).sum(0)
    return {"ids": None, "prob": w * s["scale"] * keep, "counts": None, "n_tokens": None, "load": load,
            "loss": (torch.dot(counts, load) * E / (k * n)).reshape(1)}


def _exact_route_bwd(s):
    sc, _, out = _exact_scores(s)
    T, E = sc.shape
    k, ids = s["k"], s["ids"].long()
    n = max(float(s["n_tokens"]), 1.0)
    keep = torch.ones(T, 1, dtype=torch.float64, device="cuda") if s["mask"] is None else s["mask"].double()[:, None]
    with torch.enable_grad():
        x = torch.where(out, torch.full_like(sc, -1e30), s["logits"].double().clamp(max=FLT_MAX)).requires_grad_(True)
        if s["score"] == "softmax":
            p = torch.softmax(x, 1) * (~out)
        else:
            p = torch.sigmoid(x) * (~out)
        w = torch.gather(p, 1, ids)
        if s["norm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        share = p if s["score"] == "softmax" else p / p.sum(1, keepdim=True).clamp(min=1e-300)
        load = (share * keep).sum(0) / n
        total = (w * s["scale"] * keep * s["dprob"].double()).sum() + float(s["dloss"]) * E / (k * n) * (s["counts"].double() * load).sum()
        (dl,) = torch.autograd.grad(total, x)
    return torch.where(out, torch.zeros_like(dl), dl)
