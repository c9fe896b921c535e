"""Log probabilities of tokens, their entropy and alternatives, and the
gradient, in fp64 numpy.

    z = logits / temperature, over the tokens in reach (logit above bf16's lowest finite value)
    lse = log sum e^z,  logp = z[target] - lse,  H = -sum p log p
    dz_i = g_l ([i = target] - p_i) - g_h p_i (log p_i + H)

A negative target leaves its row out.  A row with NaN or +inf is NaN.
"""
import numpy as np

LOW = -(2.0 - 2.0 ** -7) * 2.0 ** 127          # bf16's lowest finite value


def _row(l, temperature):
    """(z, in reach, M, rest, w): rest = sum of e^(z - M) without one largest
    term, w = sum of e^(z - M) |z - M|."""
    live = l > LOW
    z = np.where(live, l, 0.0) / temperature
    if not live.any():
        return z, live, -np.inf, 0.0, 0.0
    M = z[live].max()
    e = np.where(live, np.exp(np.where(live, z - M, 0.0)), 0.0)
    first = np.flatnonzero(live & (z == M))[0]
    w = float((e * np.where(live, M - z, 0.0)).sum())
    e[first] = 0.0
    return z, live, float(M), float(e.sum()), w


def token_logprob(logits, targets=None, temperature=1.0, top=0):
    """A dict of logp, lse, entropy [T] and top_ids, top_logp [T, top], and of
    what rounding errors scale with: M, rest, w [T]."""
    l = np.asarray(logits, np.float64)
    T = l.shape[0]
    o = {n: np.zeros(T) for n in ("logp", "lse", "entropy", "M", "rest", "w")}
    o["top_ids"], o["top_logp"] = np.full((T, top), -1, np.int64), np.full((T, top), -np.inf)
    for t in range(T):
        if targets is not None and targets[t] < 0:
            continue
        if np.isnan(l[t]).any() or (l[t] == np.inf).any():
            for n in ("logp", "lse", "entropy"):
                o[n][t] = np.nan
            continue
        z, live, M, rest, w = _row(l[t], temperature)
        if M == -np.inf:
            o["lse"][t] = o["logp"][t] = -np.inf
            continue
        lr = np.log1p(rest)
        o["M"][t], o["rest"][t], o["w"][t] = M, rest, w
        o["lse"][t] = M + lr
        o["entropy"][t] = lr + w / (1.0 + rest)
        if targets is not None:
            o["logp"][t] = (z[targets[t]] - M) - lr if live[targets[t]] else -np.inf
        order = np.argsort(-np.where(live, l[t], -np.inf), kind="stable")[:top]
        order = order[live[order]]
        o["top_ids"][t, :order.size] = order
        o["top_logp"][t, :order.size] = (z[order] - M) - lr
    return o


def token_logprob_backward(logits, targets, lse, dlogp=None, entropy=None, dentropy=None, temperature=1.0, logp=None):
    """(dlogits, mag): the gradient from the given lse (and entropy; and log p of the
    targets where it is given), and the sum of the magnitudes of the terms each
    element is made of."""
    l = np.asarray(logits, np.float64)
    T, V = l.shape
    d, mag = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if (targets is not None and targets[t] < 0) or lse[t] == -np.inf:
            continue
        live = l[t] > LOW
        lp = np.where(live, l[t], 0.0) / temperature - lse[t]
        if logp is not None and live[targets[t]]:
            lp[targets[t]] = logp[t]
        p = np.where(live, np.exp(np.where(live, lp, -np.inf)), 0.0)
        g = 0.0 if dlogp is None else float(dlogp[t])
        gh = 0.0 if dentropy is None else float(dentropy[t])
        H = 0.0 if dentropy is None else float(entropy[t])
        hot = np.zeros(V)
        if targets is not None and live[targets[t]]:
            hot[targets[t]] = 1.0
        one_minus = np.where(hot > 0, -np.expm1(np.where(live, lp, 0.0)), -p)
        d[t] = np.where(live, g * one_minus - gh * p * (lp + H), 0.0) / temperature
        mag[t] = np.where(live, abs(g) * np.abs(one_minus) + abs(gh) * p * (np.abs(lp) + abs(H)), 0.0) / temperature
    return d, mag
