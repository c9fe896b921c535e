"""Timed cases of the operators of a rollout and of its scoring, with their plain forms.

  few          a whole expert layer for a few tokens (decode): quantise x, FC1, SwiGLU, quantise D, FC2,
               weighted sum over each token's experts, on NVFP4 or MXFP8 weights
  logprob      log probabilities of given tokens over the vocabulary, with the log-sum-exp, the entropy
               and the most likely alternatives
  logprob_bwd  the gradient of log probabilities and entropies with respect to the logits

`run` computes each in elementary torch operations in 32 bits, or, where `own` is true, by the
framework's entry points.
"""
import math

import torch

own = False

#: logits at or below bf16's lowest finite value mark a token out of reach
LOWEST = -3.3895313892515355e38
FLT_MAX = 3.4028234663852886e38
FLOOR = 2.0 ** -116


# ---------------------------------------------------------------- cases

def listed():
    few = {"op": "few", "E": 256, "H": 7168, "I": 2048, "k": 8, "dead": 0.0, "skew": 0.0}
    small = {"op": "few", "E": 128, "H": 2048, "I": 768, "k": 8, "dead": 0.0, "skew": 0.0}
    return [
        # one token of a decode step of the 671B-shaped layer: eight experts' weights, read once
        {"name": "few_nvfp4_T1_H7168", "kind": "nvfp4", "T": 1, **few},
        # a small decode batch of it, an odd number of tokens
        {"name": "few_nvfp4_T7_H7168", "kind": "nvfp4", "T": 7, **few},
        # the rollout batch of the decode benchmark: about 220 of 256 experts active, Zipf-skewed load
        {"name": "few_nvfp4_T64_H7168", "kind": "nvfp4", "T": 64, **few, "skew": 1.1},
        # one token of the 30B-shaped layer: latency counts
        {"name": "few_mxfp8_T1_H2048", "kind": "mxfp8", "T": 1, **small},
        # a ragged batch of it, a third of the tokens finished already (weights 0)
        {"name": "few_mxfp8_T33_H2048", "kind": "mxfp8", "T": 33, **small, "dead": 0.33},
        # one sampled token: log probability, entropy and 20 alternatives out of a large vocabulary
        {"name": "logprob_T1_V131072", "op": "logprob", "T": 1, "V": 131072, "bf16": False, "pad": 0, "top": 20, "entropy": True, "masked": 0.0, "unscored": 0.0, "temperature": 1.0},
        # a decode batch with 8 alternatives a token, bf16 logits (many ties), sampling temperature
        {"name": "logprob_T64_V131072", "op": "logprob", "T": 64, "V": 131072, "bf16": True, "pad": 0, "top": 8, "entropy": True, "masked": 0.0, "unscored": 0.0, "temperature": 0.7},
        # scoring the rollout's tokens before a training step: every position, no alternatives
        {"name": "logprob_T8192_V32768", "op": "logprob", "T": 8192, "V": 32768, "bf16": True, "pad": 0, "top": 0, "entropy": True, "masked": 0.0, "unscored": 0.0, "temperature": 1.0},
        # ragged: an odd vocabulary (rows start off 16 bytes), prompt positions not scored, tokens masked out
        {"name": "logprob_T2047_V50001", "op": "logprob", "T": 2047, "V": 50001, "bf16": False, "pad": 0, "top": 4, "entropy": True, "masked": 0.1, "unscored": 0.3, "temperature": 1.0},
        # the policy gradient of that scoring, with an entropy bonus
        {"name": "logprob_bwd_T8192_V32768", "op": "logprob_bwd", "T": 8192, "V": 32768, "bf16": True, "pad": 0, "entropy": True, "masked": 0.0, "unscored": 0.0, "temperature": 1.0},
        # ragged: an odd vocabulary in fp32, prompt positions not scored, no entropy
        {"name": "logprob_bwd_T1021_V50001", "op": "logprob_bwd", "T": 1021, "V": 50001, "bf16": False, "pad": 0, "entropy": False, "masked": 0.1, "unscored": 0.3, "temperature": 0.7},
        # a micro-batch of short answers over a byte-sized vocabulary: latency counts
        {"name": "logprob_bwd_T96_V1000", "op": "logprob_bwd", "T": 96, "V": 1000, "bf16": True, "pad": 24, "entropy": True, "masked": 0.0, "unscored": 0.1, "temperature": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "logprob", "logprob", "logprob_bwd"])
    if op == "few":
        H, I = 256 * _log(rng, 1, 28), 256 * _log(rng, 1, 8)
        E = _log(rng, 4, max(4, min(256, (1 << 32) // (3 * H * I))))
        return {"op": op, "kind": rng.choice(["nvfp4", "mxfp8"]), "T": _log(rng, 1, 64), "E": E, "H": H, "I": I,
                "k": rng.randint(1, min(E, 8)), "dead": rng.choice([0.0, 0.0, 0.4]), "skew": rng.choice([0.0, 1.1])}
    V = _log(rng, 40, 262144)
    T = _log(rng, 1, max(1, min(8192, (1 << 27) // V)))
    c = {"op": op, "T": T, "V": V, "bf16": rng.random() < 0.6, "pad": rng.choice([0, 0, 8, 13]),
         "entropy": rng.random() < 0.7, "masked": rng.choice([0.0, 0.1]), "unscored": rng.choice([0.0, 0.3]),
         "temperature": rng.choice([1.0, 0.7, 1.3])}
    if op == "logprob":
        c["top"] = rng.choice([0, 0, 1, 5, 20, 32])
    return c


# ---------------------------------------------------------------- inputs

def _pad(n, m):
    return (n + m - 1) // m * m


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


def _weights_nvfp4(g, E, R, K):
    """Gaussian expert weights in NVFP4: (codes [E, R, K/2], scales of each expert in tiles, outer scale [E])."""
    q = torch.empty(E, R, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, _pad(R, 128) * _pad(K // 16, 4), dtype=torch.uint8, device="cuda")
    ts = torch.empty(E, dtype=torch.float32, device="cuda")
    for e in range(E):
        w = 0.02 * torch.randn(R, K // 16, 16, device="cuda", generator=g)
        ts[e] = w.abs().max() / 2688.0
        sb = (w.abs().amax(2) / (6.0 * ts[e])).to(torch.float8_e4m3fn)
        m = (w / (sb.float() * ts[e]).clamp(min=1e-30)[:, :, None]).abs()
        code = ((m > 0.25).to(torch.uint8) + (m > 0.75) + (m > 1.25) + (m > 1.75) + (m > 2.5) + (m > 3.5) + (m > 5.0) + 8 * (w < 0)).view(R, K // 2, 2)
        q[e] = code[:, :, 0] | (code[:, :, 1] << 4)
        s[e] = _tile(sb.view(torch.uint8))
    return q, s.view(-1), ts


def _weights_mxfp8(g, rows, K):
    """Gaussian expert weights in MXFP8: (codes [rows, K], scales in tiles)."""
    w = 0.02 * torch.randn(rows, K // 32, 32, device="cuda", generator=g)
    e = torch.ceil(torch.log2(w.abs().amax(2).clamp(min=1e-30) / 448.0))
    q = (w * torch.exp2(-e)[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, K)
    return q, _tile((e + 127).to(torch.uint8))


def _prepare_few(s, g):
    T, E, H, I, k = (s[n] for n in ("T", "E", "H", "I", "k"))
    x = torch.randn(T, H, device="cuda", generator=g)
    x *= torch.where(torch.rand(T, H, device="cuda", generator=g) < 1e-3, 10.0, 1.0)
    s["x"] = x.to(torch.bfloat16)
    z = torch.randn(T, E, device="cuda", generator=g)
    if s["skew"]:
        # Gumbel noise on Zipf log-probabilities: skewed expert load
        u = torch.rand(T, E, device="cuda", generator=g).clamp(1e-7, 1 - 1e-7)
        z = -s["skew"] * torch.log(torch.arange(E, device="cuda") + 1.0) - torch.log(-torch.log(u))
    z, ids = torch.sort(z, dim=1, descending=True)
    s["ids"] = ids[:, :k].to(torch.int32).contiguous()
    s["prob"] = torch.softmax(z[:, :k], 1)
    if s["dead"]:
        alive = torch.rand(T, 1, device="cuda", generator=g) >= s["dead"]
        alive[0] = True
        s["prob"] = s["prob"] * alive
    s["prob"] = s["prob"].contiguous()
    if s["kind"] == "nvfp4":
        s["w1"], s["w2"] = _weights_nvfp4(g, E, 2 * I, H), _weights_nvfp4(g, E, H, I)
    else:
        s["w1"], s["w2"] = _weights_mxfp8(g, E * 2 * I, H), _weights_mxfp8(g, E * H, I)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "few":
        _prepare_few(s, g)
        return s
    T, V = case["T"], case["V"]
    z = torch.randn(T, V + case["pad"], device="cuda", generator=g) * 2.0
    likely = torch.randint(0, V, (T, 1), device="cuda", generator=g)
    z.scatter_add_(1, likely, 18.0 * torch.rand(T, 1, device="cuda", generator=g))
    if case["masked"]:
        z.masked_fill_(torch.rand(z.shape, device="cuda", generator=g) < case["masked"], -math.inf)
        if T > 2:
            z[T // 2] = -math.inf                   # a row whose mask leaves nothing
    z = (z.to(torch.bfloat16) if case["bf16"] else z)[:, :V]
    other = torch.randint(0, V, (T, 1), device="cuda", generator=g)
    t = torch.where(torch.rand(T, 1, device="cuda", generator=g) < 0.7, likely, other)[:, 0]
    if case["unscored"]:
        out = torch.rand(T, device="cuda", generator=g) < case["unscored"]
        out[0] = False
        t = torch.where(out, torch.full_like(t, -100), t)
    s["logits"], s["targets"] = z, t
    if case["op"] == "logprob_bwd":
        f = _plain_logprob({**s, "entropy": True, "top": 0})
        s["lse"], s["H"] = f["lse"], f["entropy"]
        s["dlogp"] = torch.randn(T, device="cuda", generator=g) / T
        s["dH"] = torch.full((T,), 0.01 / T, device="cuda") if case["entropy"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _round_e2m1(y):
    """To the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), with the sign."""
    m = y.abs()
    q = 0.5 * ((m > 0.25).float() + (m >= 0.75) + (m > 1.25) + (m >= 1.75)) + (m > 2.5) + (m >= 3.5) + 2.0 * (m > 5.0)
    return torch.copysign(q, y)


def _quant_nvfp4(x):
    """(values without the outer scale, outer scale of each row): the scale is the quotient rounded once, since a
    bit of it moves values across the border between two codes"""
    b = x.view(*x.shape[:-1], -1, 16)
    a = x.abs().amax(-1)
    sg = torch.where(a > 0, (a.double() / 2688.0).float().clamp(min=FLOOR), torch.zeros_like(a))
    safe = torch.where(sg > 0, sg, torch.ones_like(sg))[..., None]
    sb = (b.abs().amax(-1) / (6.0 * safe)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = torch.where(sb > 0, 1.0 / (torch.where(sb > 0, sb, torch.ones_like(sb)) * safe), torch.zeros_like(sb))
    return (_round_e2m1(b * r[..., None]) * sb[..., None]).view(x.shape), sg


def _quant_mxfp8(x):
    b = x.view(*x.shape[:-1], -1, 32)
    bits = b.abs().amax(-1).view(torch.int32)
    e = ((bits >> 23) - 127) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    e = torch.where((bits >> 23) == 0, torch.full_like(e, -127), e).clamp(-127, 127).float()
    return ((b * torch.exp2(-e)[..., None]).to(torch.float8_e4m3fn).float() * torch.exp2(e)[..., None]).view(x.shape)


def _values(s, w, rows, K, experts):
    """fp32 weights [experts, rows, K] of these experts, without an outer scale."""
    n, block = experts.numel(), 16 if s["kind"] == "nvfp4" else 32
    tiles = w[1].view(s["E"], -1)[experts].reshape(-1)
    sc = _untile(tiles, n * rows, K // block)
    if s["kind"] == "nvfp4":
        pair = torch.arange(256, device="cuda")
        half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        table = torch.stack((half[pair & 7] * (1 - (pair >> 2 & 2)), half[pair >> 4 & 7] * (1 - (pair >> 6 & 2))), 1)
        v = table[w[0][experts].int()].view(n, rows, K // 16, 16)
        return (v * sc.view(torch.float8_e4m3fn).float().view(n, rows, K // 16, 1)).view(n, rows, K)
    v = w[0].view(s["E"], rows, K)[experts].view(torch.float8_e4m3fn).float().view(n, rows, K // 32, 32)
    return (v * torch.exp2(sc.float() - 127.0).view(n, rows, K // 32, 1)).view(n, rows, K)


def _plain_few(s):
    T, E, H, I, k = (s[n] for n in ("T", "E", "H", "I", "k"))
    nv = s["kind"] == "nvfp4"
    weight = torch.zeros(E, T, device="cuda")
    weight[s["ids"].long(), torch.arange(T, device="cuda")[:, None]] = s["prob"]
    # the experts that tokens go to come first; there are at most T k of them
    order = torch.sort((weight != 0).any(1), descending=True, stable=True).indices[:min(E, T * k)]
    x = s["x"].float()
    x, xs = _quant_nvfp4(x) if nv else (_quant_mxfp8(x), None)
    out = torch.zeros(T, H, device="cuda")
    for at in range(0, order.numel(), 16):           # the fp32 weights of 16 experts fit in memory
        ex = order[at:at + 16]
        c = torch.matmul(x, _values(s, s["w1"], 2 * I, H, ex).transpose(1, 2))
        if nv:
            c = c * (xs[None, :] * s["w1"][2][ex][:, None])[..., None]
        gate, up = c[..., :I], c[..., I:]
        d = (gate / (1.0 + torch.exp(-gate)) * up * weight[ex][..., None]).to(torch.bfloat16).float()
        d, ds = _quant_nvfp4(d) if nv else (_quant_mxfp8(d), None)
        y = torch.matmul(d, _values(s, s["w2"], H, I, ex).transpose(1, 2))
        if nv:
            y = y * (ds * s["w2"][2][ex][:, None])[..., None]
        out += y.sum(0)
    return {"out": out.to(torch.bfloat16)}


def _scaled(s):
    """(scaled logits with -inf for tokens out of reach, that mask, scored rows)"""
    l = s["logits"].float()
    live = l > LOWEST
    z = torch.where(live, (l.clamp(max=FLT_MAX) / s["temperature"]).clamp(max=FLT_MAX), torch.full_like(l, -math.inf))
    return z, live, s["targets"] >= 0


def _plain_logprob(s):
    z, live, scored = _scaled(s)
    m, first = z.max(1, keepdim=True)
    m = m.clamp(min=-FLT_MAX)
    some = live.any(1)
    # the sum without one of its largest terms, which is 1: where that token is nearly certain the others are what counts
    e = torch.exp(z - m).scatter(1, first, 0.0)
    rest = e.sum(1)
    zt = torch.gather(z, 1, s["targets"].clamp(min=0)[:, None])[:, 0]
    zero, low = torch.zeros_like(rest), torch.full_like(rest, -math.inf)
    lse = torch.where(some, m[:, 0] + torch.log1p(rest), low)
    o = {"logp": torch.where(scored, torch.where(some, zt - m[:, 0] - torch.log1p(rest), low), zero),
         "lse": torch.where(scored, lse, zero)}
    if s["entropy"]:
        h = torch.log1p(rest) - torch.where(live, e * (z - m), torch.zeros_like(e)).sum(1) / (1.0 + rest)
        o["entropy"] = torch.where(scored & some, h, zero)
    if s["top"]:
        v, i = torch.sort(z, dim=1, descending=True, stable=True)
        v, i = v[:, :s["top"]], i[:, :s["top"]]
        has = (v > -math.inf) & scored[:, None]
        o["top_ids"] = torch.where(has, i, torch.full_like(i, -1)).to(torch.int32)
        o["top_logp"] = torch.where(has, v - m - torch.log1p(rest)[:, None], torch.full_like(v, -math.inf))
    return o


def _plain_logprob_bwd(s):
    z, live, scored = _scaled(s)
    logp = z - s["lse"][:, None]
    ok = live & scored[:, None]
    p = torch.where(ok, torch.exp(logp), torch.zeros_like(z))
    d = -s["dlogp"][:, None] * p
    if s["dH"] is not None:
        d = d - s["dH"][:, None] * torch.where(ok, p * (logp + s["H"][:, None]), torch.zeros_like(p))
    # the given token's own 1 - p, without the difference where it is nearly certain
    at = s["targets"].clamp(min=0)[:, None]
    d.scatter_add_(1, at, s["dlogp"][:, None] * torch.gather(p, 1, at))
    d.scatter_add_(1, at, -s["dlogp"][:, None] * torch.expm1(torch.gather(logp, 1, at)))
    return {"dlogits": torch.where(ok, d / s["temperature"], torch.zeros_like(d)).to(s["logits"].dtype)}


# ---------------------------------------------------------------- one pass

def run(s):
    if not own:
        return {"few": _plain_few, "logprob": _plain_logprob, "logprob_bwd": _plain_logprob_bwd}[s["op"]](s)
    from microscaled_precision_moe_gb300 import _lib as L, ops
    if s["op"] == "few":
        kind = L.KIND_NVFP4 if s["kind"] == "nvfp4" else L.KIND_MXFP8
        return {"out": ops.moe_few_tokens(kind, s["x"], s["ids"], s["prob"], s["w1"], s["w2"], s["E"], s["I"])}
    if s["op"] == "logprob":
        return ops.token_logprob(s["logits"], s["targets"], temperature=s["temperature"], entropy=s["entropy"], top=s["top"])
    return {"dlogits": ops.token_logprob_backward(s["logits"], s["targets"], s["lse"], dlogp=s["dlogp"],
                                                  entropy=None if s["dH"] is None else s["H"], dentropy=s["dH"],
                                                  temperature=s["temperature"])}


def work(case):
    T = case["T"]
    if case["op"] == "few":
        E, H, I, k = (case[n] for n in ("E", "H", "I", "k"))
        alive = T * (1.0 - case["dead"])
        if case["skew"]:
            # k draws without replacement from Zipf shares, about as many distinct experts as T k independent draws
            share = [(i + 1.0) ** -case["skew"] for i in range(E)]
            hit = sum(1.0 - (1.0 - v / sum(share)) ** (alive * k) for v in share)
        else:
            hit = E * (1.0 - (1.0 - k / E) ** alive)
        per = 0.5 + 1.0 / 16 if case["kind"] == "nvfp4" else 1.0 + 1.0 / 32
        return {"bytes": hit * 3 * H * I * per + 4 * T * H + 8 * T * k, "flops": 2 * alive * k * 3 * H * I}
    n = T * case["V"] * (2 if case["bf16"] else 4) * (1.0 - case["unscored"])
    if case["op"] == "logprob":
        return {"bytes": n + T * (16 + 4 * case["entropy"] + 8 * case["top"]), "flops": 6 * T * case["V"]}
    whole = T * case["V"] * (2 if case["bf16"] else 4)          # rows that are not scored are written, not read
    return {"bytes": n + whole + T * (16 + 8 * case["entropy"]), "flops": 8 * T * case["V"]}


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "few":
        return _exact_few(s)
    l = s["logits"].double()
    out = ~(l > LOWEST)
    x = torch.minimum(l, torch.full((), FLT_MAX, dtype=torch.float64, device="cuda")) / s["temperature"]
    x = torch.minimum(x, torch.full((), FLT_MAX, dtype=torch.float64, device="cuda")).masked_fill(out, -math.inf)
    t = s["targets"]
    rows = torch.nonzero(t >= 0)[:, 0]
    T = t.numel()
    if case["op"] == "logprob":
        res = {"logp": torch.zeros(T, dtype=torch.float64, device="cuda")}
        res["lse"] = torch.zeros_like(res["logp"])
        norm = torch.logsumexp(x[rows], 1)
        res["lse"][rows] = norm
        own_logp = x[rows, t[rows]] - norm
        res["logp"][rows] = torch.where(torch.isnan(own_logp), torch.full_like(norm, -math.inf), own_logp)
        p = torch.softmax(x[rows], 1).nan_to_num(0.0)
        if s["entropy"]:
            res["entropy"] = torch.zeros_like(res["logp"])
            res["entropy"][rows] = -torch.special.xlogy(p, p).sum(1)
        if s["top"]:
            value = torch.topk(x[rows], min(s["top"], x.shape[1]), dim=1).values - norm[:, None]
            res["top_ids"] = None
            res["top_logp"] = torch.full((T, value.shape[1]), -math.inf, dtype=torch.float64, device="cuda")
            res["top_logp"][rows] = torch.where(torch.isnan(value), torch.full_like(value, -math.inf), value)
        return res
    d = torch.zeros_like(x)
    for at in range(0, rows.numel(), 512):
        r = rows[at:at + 512]
        keep = ~out[r]
        p = torch.exp(x[r] - s["lse"][r].double()[:, None]).masked_fill(~keep, 0.0)
        hot = torch.zeros_like(p).scatter_(1, t[r][:, None], 1.0)
        v = s["dlogp"][r].double()[:, None] * (hot - p)
        if s["dH"] is not None:
            v -= s["dH"][r].double()[:, None] * (torch.special.xlogy(p, p) + p * s["H"][r].double()[:, None])
        d[r] = (v / s["temperature"]).masked_fill(~keep, 0.0)
    return {"dlogits": d}


def _exact_grid(v):
    """The nearest E2M1 value of each, ties to the even code."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    odd = torch.arange(8, device="cuda") % 2
    near = torch.argmin((v.abs()[..., None] - grid).abs() + 1e-9 * odd, dim=-1)
    return grid[near] * torch.sign(v)


def _exact_rows_nvfp4(v):
    """Per-token NVFP4 of [n, K], decoded: its scales are 32-bit numbers by definition."""
    n, K = v.shape
    a = v.abs().amax(1)
    sg = (a / 2688.0).clamp(min=FLOOR).float().double() * (a > 0)
    blocks = v.reshape(n, K // 16, 16)
    six = (6.0 * sg).float().double()[:, None]
    ratio = (blocks.abs().amax(2) / six).nan_to_num(0.0).float()
    sb = ratio.clamp(max=448.0).to(torch.float8_e4m3fn).double()
    inv = (1.0 / (sb * sg[:, None]).float().double()).float().double()
    y = (blocks * torch.where(sb > 0, inv, torch.zeros_like(inv))[..., None]).float().double()
    return (_exact_grid(y) * (sb * sg[:, None])[..., None]).reshape(n, K)


def _exact_rows_mxfp8(v):
    n, K = v.shape
    blocks = v.reshape(n, K // 32, 32)
    # 32 values share 2^e, the smallest with max <= 448 * 2^e
    e = torch.ceil(torch.log2(blocks.abs().amax(2).clamp(min=2.0 ** -140) / 448.0)).clamp(-127, 127)
    q = (blocks * torch.exp2(-e)[..., None]).float().to(torch.float8_e4m3fn).double()
    return (q * torch.exp2(e)[..., None]).reshape(n, K)


def _exact_weight(s, w, e, R, K):
    """One expert's [R, K] weights in 64 bits."""
    b = 16 if s["kind"] == "nvfp4" else 32
    tiles = w[1].view(s["E"], -1)[e]
    r, c = torch.meshgrid(torch.arange(R, device="cuda"), torch.arange(K // b, device="cuda"), indexing="ij")
    sc = tiles[(r // 128 * (_pad(K // b, 4) // 4) + c // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + c % 4]
    if s["kind"] == "nvfp4":
        code = w[0][e].to(torch.int16)
        v = torch.stack((code % 16, code // 16), dim=2).reshape(R, K).long()
        grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
        v = torch.cat((grid, -grid))[v] * sc.view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        return v * float(w[2][e])
    v = w[0].view(s["E"], R, K)[e].view(torch.float8_e4m3fn).double()
    return v * torch.exp2(sc.double() - 127.0).repeat_interleave(32, 1)


def _exact_few(s):
    T, E, H, I = (s[n] for n in ("T", "E", "H", "I"))
    rows = _exact_rows_nvfp4 if s["kind"] == "nvfp4" else _exact_rows_mxfp8
    x = rows(s["x"].double())
    ids, prob = s["ids"].tolist(), s["prob"].double()
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    mine = {}
    for t in range(T):
        for j, e in enumerate(ids[t]):
            mine.setdefault(e, []).append((t, j))
    for e, slots in mine.items():
        t, j = torch.tensor(slots, device="cuda").unbind(1)
        c = x[t] @ _exact_weight(s, s["w1"], e, 2 * I, H).T
        d = torch.nn.functional.silu(c[:, :I]) * c[:, I:] * prob[t, j][:, None]
        out.index_add_(0, t, rows(d.to(torch.bfloat16).double()) @ _exact_weight(s, s["w2"], e, H, I).T)
    return {"out": out}
