"""The whole expert layer on few tokens, in fp64 numpy.

    xq = Q(x);  c = xq W1_e^T;  D = bf16(silu(gate) up prob);  dq = Q(D)
    out_t = sum_j dq_tj W2_e^T

Q is the NVFP4 per-token or the MXFP8 row-wise quantisation of oracle.quant; W1 and
W2 are given decoded.  Slots of weight 0 and expert ids out of range are left out.
"""
import numpy as np

from . import formats as F
from . import quant as Q

UNIT = 2.0 ** -24


def quantise(x, kind):
    """x [M, K] bf16 values -> what its codes and scales stand for."""
    if kind == "nvfp4":
        q, s, ts = Q.nvfp4_quantize_per_token(x)
        return Q.nvfp4_dequantize(q, s, ts)
    q, s = Q.mxfp8_quantize_rowwise(x)
    return Q.mxfp8_dequantize(q, s)


def forward(x, ids, prob, w1, w2, kind):
    """(out [T, H], tol [T, H]).

    tol bounds what fp32 arithmetic may differ by before the last rounding.  A sum
    of n terms is taken in steps of 64 (NVFP4) or 32 (MXFP8), each rounding to 2^-23 of the
    sum of their magnitudes at most.  g and u carry that, silu a few ulps and 1 + |g|
    times g's error; where such an error takes an element of D across a rounding
    border, its code moves with it: D is rounded and quantised at both ends of its
    interval, and the differences go through |W2|."""
    E, H, I = w2.shape
    step = 64 if kind == "nvfp4" else 32
    xq = quantise(np.asarray(x, np.float64), kind)
    ids, prob = np.asarray(ids), np.asarray(prob, np.float64)
    k = ids.shape[1]
    out, tol = np.zeros((len(ids), H)), np.zeros((len(ids), H))
    live = (prob != 0) & (ids >= 0) & (ids < E)
    for e in np.unique(ids[live]):
        t, j = np.nonzero(live & (ids == e))
        p = prob[t, j][:, None]
        c = xq[t] @ w1[e].T
        err = (H / step + 2) * 2 * UNIT * (np.abs(xq[t]) @ np.abs(w1[e]).T) + 2 * UNIT * np.abs(c)
        g, u, dg, du = c[:, :I], c[:, I:], err[:, :I], err[:, I:]
        with np.errstate(over="ignore"):
            sig = 1.0 / (1.0 + np.exp(-g))
        d = g * sig * u * p
        dd = np.abs(p) * (np.abs(u) * sig * (1 + np.abs(g) * (1 - sig)) * dg + np.abs(g * sig) * du) \
            + np.abs(d) * UNIT * (16 + 4 * np.abs(g))
        mid, lo, hi = (quantise(F.bf16_round(v), kind) for v in (d, d - dd, d + dd))
        moved = np.abs(lo - mid) + np.abs(hi - mid)
        w = np.abs(w2[e])
        np.add.at(out, t, mid @ w2[e].T)
        np.add.at(tol, t, moved @ w.T + ((I / step + 2 + k) * 2 * UNIT) * (np.abs(mid) @ w.T))
    return out, tol
