"""The router in fp64 numpy: top-k choice, routing weights, expert counts and
balance loss, their gradient, and the gradient of the routing weights through
the combine.

Out of reach: a logit (or bias) that is NaN or at most bf16's lowest finite
value.  Choice: within reach before out of reach, larger key first, lower
expert first; the key is the logit (softmax) or score + bias (sigmoid).
"""
import numpy as np

LOWEST = -3.3895313892515355e38
FLT_MAX = 3.4028234663852886e38


def _within(logits, bias):
    with np.errstate(invalid="ignore"):
        live = logits > LOWEST
        if bias is not None:
            live = live & (np.asarray(bias, np.float64) > LOWEST)[None, :]
    return live, np.where(live, np.minimum(logits, FLT_MAX), -np.inf)


def scores(logits, score, bias=None):
    """(scores, within reach, capped logits)"""
    live, l = _within(np.asarray(logits, np.float64), bias)
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            s = np.where(live, 1.0 / (1.0 + np.exp(-l)), 0.0)
        else:
            m = np.where(live.any(1, keepdims=True), l.max(1, keepdims=True), 0.0)
            e = np.where(live, np.exp(l - m), 0.0)
            t = e.sum(1, keepdims=True)
            s = e / np.where(t > 0, t, 1.0)
    return s, live, l


def _shares(s):
    t = s.sum(1, keepdims=True)
    return s / np.where(t > 0, t, 1.0)


def _loss(s, counts, keep, k):
    n = max(float(keep.sum()), 1.0)
    load = (_shares(s) * keep[:, None]).sum(0) / n
    return load, s.shape[1] / (k * n) * float(np.dot(counts, load))


def weights(s, ids, normalize, scale):
    w = np.take_along_axis(s, ids, 1)
    if normalize:
        t = w.sum(1, keepdims=True)
        w = w / np.where(t > 0, t, 1.0)
    return w * scale


def route(logits, k, score="softmax", normalize=True, scale=1.0, bias=None, mask=None):
    s, live, l = scores(logits, score, bias)
    T, E = s.shape
    key = l if score == "softmax" else s + (0.0 if bias is None else np.asarray(bias, np.float64)[None, :])
    key = np.where(live, key, -np.inf)
    ids = np.argsort(np.where(live, -key, np.inf), axis=1, kind="stable")[:, :k]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    prob = weights(s, ids, normalize, scale) * keep[:, None]
    picked = np.take_along_axis(live, ids, 1) & keep[:, None]
    counts = np.bincount(ids[picked], minlength=E)
    load, loss = _loss(s, counts, keep, k)
    return {"ids": ids, "prob": prob, "counts": counts, "n_tokens": int(keep.sum()), "load": load,
            "loss": loss, "key": key}


def objective(logits, ids, counts, dprob, dloss, score, normalize, scale, bias=None, mask=None):
    """What moe_route_backward differentiates, for a fixed choice and fixed
    counts: <dprob, prob> + dloss * loss."""
    s, _, _ = scores(logits, score, bias)
    keep = np.ones(s.shape[0], bool) if mask is None else np.asarray(mask).astype(bool)
    prob = weights(s, ids, normalize, scale) * keep[:, None]
    return float((np.asarray(dprob, np.float64) * prob).sum()
                 + dloss * _loss(s, counts, keep, ids.shape[1])[1])


def route_backward(logits, ids, counts, dprob, dloss, score, normalize, scale, bias=None, mask=None):
    """(dlogits, mag): the gradient and the magnitude its terms add up to."""
    s, live, l = scores(logits, score, bias)
    T, E = s.shape
    k = ids.shape[1]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    n = max(float(keep.sum()), 1.0)
    dp = dloss * E / (k * n * n) * np.asarray(counts, np.float64) * np.ones((T, 1))
    d = np.asarray(dprob, np.float64) * scale
    da = np.abs(d)
    w = np.take_along_axis(s, ids, 1)
    if normalize:
        t = w.sum(1, keepdims=True)
        t = np.where(t > 0, t, 1.0)
        q = w / t
        d, da = (d - (d * q).sum(1, keepdims=True)) / t, (da + (da * q).sum(1, keepdims=True)) / t
    ds, dsa = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(ds, ids, d, 1)
    np.put_along_axis(dsa, ids, da, 1)
    if score == "softmax":
        ds, dsa = ds + dp, dsa + np.abs(dp)
        dl = s * (ds - (s * ds).sum(1, keepdims=True))
        mag = s * (dsa + (s * dsa).sum(1, keepdims=True))
    else:
        t = s.sum(1, keepdims=True)
        t = np.where(t > 0, t, 1.0)
        sh = s / t
        ds = ds + (dp - (sh * dp).sum(1, keepdims=True)) / t
        dsa = dsa + (np.abs(dp) + (sh * np.abs(dp)).sum(1, keepdims=True)) / t
        z = np.exp(-np.abs(l))
        local = z / (1.0 + z) ** 2
        dl, mag = local * ds, local * dsa
    on = live & keep[:, None]
    return np.where(on, dl, 0.0), np.where(on, mag, 0.0)


def combine_dprob(dout, y_perm, inv, prob):
    """(dprob, mag): <dout[t], y[inv[t, j]]> / prob[t, j], 0 where the slot
    has no row or its weight is 0."""
    prob = np.asarray(prob, np.float64)
    T, k = prob.shape
    inv = np.asarray(inv).reshape(T, k)
    out, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if inv[t, j] >= 0 and prob[t, j] != 0:
                v = np.asarray(dout[t], np.float64) * np.asarray(y_perm[inv[t, j]], np.float64)
                out[t, j], mag[t, j] = v.sum() / prob[t, j], np.abs(v).sum() / abs(prob[t, j])
    return out, mag
