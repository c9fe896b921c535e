"""Token log probabilities and their gradient at the ends of what they take: masks of most of a large vocabulary at
the lowest temperature, against values known in closed form.

u = 2^-24; an exponential is off by 4 u, a logarithm by 4 u of its result at most.
"""
import math

import numpy as np
import pytest
import torch

from oracle import logprob as O
from tests.gpu_util import need_gpu
from tests.test_gpu_logprob import _close

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _ops():
    from microscaled_precision_moe_gb300 import ops
    return ops


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,temperature", [(1, 2_000_000, 1e-3), (100, 400_000, 1e-3), (160, 1_600_000, 1e-3), (400, 7000, 1e-3),
                                             (400, 900, 1e-3), (1, 1 << 20, 0.0025)])
def test_entropy_beside_a_mask_of_most_of_the_row(bf16, T, V, temperature):
    """Two equal tokens in reach among masked ones, which a part of the row (a block, a warp) holds alone: ln 2.
    Terms that are 0 add 0, however many and however far they are."""
    l = torch.full((T, V), -torch.inf, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    l[:, :2] = 1.5
    t = torch.zeros(T, dtype=torch.int64, device="cuda")
    o = _ops().token_logprob(l, t, temperature=temperature, entropy=True, top=3)
    tol = 8 * UNIT
    assert (o["entropy"] - math.log(2)).abs().max() <= tol
    assert (o["logp"] + math.log(2)).abs().max() <= tol
    assert (o["top_ids"] == torch.tensor([0, 1, -1], device="cuda")).all()
    # and with the tokens in reach at the row's end
    l[:, :2] = torch.finfo(l.dtype).min
    l[:, V - 2:] = 1.5
    t += V - 1
    o = _ops().token_logprob(l, t, temperature=temperature, entropy=True)
    assert (o["entropy"] - math.log(2)).abs().max() <= tol and (o["logp"] + math.log(2)).abs().max() <= tol
    assert _ops().get_device_status() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(4, 300), (4, 40000), (2000, 300)])
def test_gradient_of_a_row_with_nan_and_a_masked_target(bf16, T, V):
    l = torch.randn(T, V, device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
    t = torch.full((T,), 3, device="cuda")
    l[1:3, 3] = -torch.inf
    l[1, 5], l[2, 6] = torch.nan, torch.inf
    o = _ops().token_logprob(l, t, entropy=True)
    one = torch.ones(T, device="cuda")
    for a, b in ((one, None), (None, one), (one, one)):
        got = _ops().token_logprob_backward(l, t, o["lse"], dlogp=a, entropy=o["entropy"] if b is not None else None, dentropy=b)
        assert got[1:3].isnan().all() and got[0].isfinite().all() and got[3:].isfinite().all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(6, 300), (6, 50001), (400, 300), (400, 4000), (400, 7000), (400, 15000)])
def test_alternatives_of_a_row_with_nan(bf16, T, V):
    """Every log probability of such a row is NaN, those of places that no token takes among them."""
    l = torch.randn(6, V, device="cuda").to(torch.bfloat16 if bf16 else torch.float32)
    l[1] = torch.nan
    l[2] = -torch.inf
    l[2, 7] = torch.nan
    l[3, 1::2] = torch.nan
    l[3, ::2] = -torch.inf
    l[4, 5] = torch.inf
    l[5, V - 1] = torch.nan
    l = l.repeat((T + 5) // 6, 1)[:T].contiguous()
    o = _ops().token_logprob(l, None, top=4)
    row = torch.arange(T, device="cuda") % 6
    assert (o["lse"].isnan() == (row > 0)).all()
    assert (o["top_logp"].isnan() == (row > 0)[:, None]).all()
    assert ((o["top_ids"] >= -1) & (o["top_ids"] < V)).all()


def _in_range(v, what):
    """Log probabilities past fp32's numbers are -inf."""
    return v if what == "lse" else np.where(v < -float(np.finfo(np.float32).max), -np.inf, v)


def _forward(l, targets, temperature, top, distinct):
    """token_logprob of rows that repeat the first `distinct` ones, each against fp64.  What moves a result: a term
    e^(z - M) by 4 u of the exponential and by its argument's five roundings (1 / temperature, its product with
    log2 e and that constant, the difference, the product with it), 5 u |z - M|; the sum of V terms by (40 + V / 1024) u; w's
    terms by theirs times |z - M|."""
    ops = _ops()
    V = l.shape[1]
    n, nt = l[:distinct].float().cpu().numpy().astype(np.float64), targets[:distinct].cpu().numpy()
    want = O.token_logprob(n, nt, temperature, top)
    o = ops.token_logprob(l, targets, temperature=temperature, entropy=True, top=top)
    live = n > O.LOW
    d = np.where(live, (want["M"][:, None] - np.where(live, n, 0) / temperature), np.inf)
    e = np.exp(-d)
    far = np.where(d < 1e3, d, 0)                  # e is 0 beyond
    some = live.any(1)
    near = lambda f: np.where(some, (e * f).sum(1), 0)
    rest, w, s2 = want["rest"], near(far), near(far * far)
    rel = (44 + V / 1024) * UNIT
    d_rest = rel * rest + 5 * UNIT * w
    lr = np.log1p(rest)
    d_lr = d_rest / (1 + rest) + 4 * UNIT * lr
    w1 = w / (1 + rest)
    tol = {"lse": d_lr + 4 * UNIT * (np.abs(want["M"]) + lr),
           "entropy": d_lr + (rel * w + 5 * UNIT * s2) / (1 + rest) + w1 * (d_rest / (1 + rest) + 6 * UNIT) + 2 * UNIT * (lr + w1)}
    gap = lambda x, r: np.where(np.isfinite(x), np.abs(np.where(np.isfinite(x), x, 0) + r), 0)
    tol["logp"] = d_lr + 4 * UNIT * (gap(want["logp"], lr) + lr)
    tol["top_logp"] = d_lr[:, None] + 4 * UNIT * (gap(want["top_logp"], lr[:, None]) + lr[:, None])
    T = l.shape[0]
    of = np.arange(T) % distinct
    for k in tol:
        if k in o:
            _close(o[k].cpu().numpy(), _in_range(want[k], k)[of], tol[k][of], k)
    if top:
        assert np.array_equal(o["top_ids"].cpu().numpy(), want["top_ids"][of]), "alternatives"
    assert ops.get_device_status() == 0
    return o


def _odd_rows(T, V, dtype, temperature, seed=0):
    """Rows whose logits reach the ends of the type's range, repeated; (logits, targets)."""
    rng = np.random.default_rng(seed)
    low = float(torch.finfo(torch.bfloat16).min)
    r = rng.normal(size=(8, V)) * 2
    t = np.zeros(8, np.int64)
    hit = rng.permutation(V)
    r[0, hit[:V // 3]] = -1e35                     # far down, in reach all the same: no weight, but a log probability
    t[0] = hit[0]
    r[1] = -1e31 * (1 + rng.integers(0, 8, V) / 8)  # nothing above -2^100
    t[1] = r[1].argmax()
    r[2] = -np.inf                                 # alternatives from both ends
    r[2, hit[:5]] = 1.0, 0.5, -2e30, -1e33, -3e38
    t[2] = hit[3]
    r[3, hit[:3]] = 1e31                           # three equal ones above 2^100
    t[3] = hit[1]
    r[4] = np.where(rng.random(V) < 0.5, -2e38, -np.inf)
    r[4, hit[0]] = 2e38
    t[4] = hit[0]
    r[5] = low                                     # the lowest value is a mask, the next one is not (its quotient in range)
    r[5, hit[0]] = -2e38 if temperature < 1 else np.nextafter(np.float32(low), np.float32(0)) if dtype == torch.float32 else -3.3762318e38
    t[5] = hit[0]
    r[6, hit[0]] = 2.3e38
    t[6] = hit[2]
    t[7] = r[7].argmax()
    l = torch.from_numpy(r.astype(np.float32)).to(dtype)
    n = (T + 7) // 8
    return l.repeat(n, 1)[:T].contiguous().cuda(), torch.from_numpy(t).repeat(n)[:T].cuda()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,top", [(8, 300, 5), (8, 50001, 20), (40, 131072, 32), (700, 777, 0), (400, 4000, 5), (400, 7000, 1), (400, 15000, 8)])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 1.3])
def test_every_finite_logit_above_the_lowest_is_in_reach(bf16, T, V, top, temperature):
    l, t = _odd_rows(T, V, torch.bfloat16 if bf16 else torch.float32, temperature)
    o = _forward(l, t, temperature, top, 8)
    assert o["logp"].isfinite().all() and o["lse"].isfinite().all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(8, 300), (8, 50001), (2000, 300), (1400, 1500)])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 1.3])
def test_gradient_of_logits_at_the_ends_of_the_range(bf16, T, V, temperature):
    """Where lse is huge p is 1 at the largest logits and 0 elsewhere; a target far below the others gets its dlogp."""
    dtype = torch.bfloat16 if bf16 else torch.float32
    l, t = _odd_rows(T, V, dtype, temperature)
    o = _ops().token_logprob(l, t, temperature=temperature, entropy=True)
    g = torch.Generator(device="cuda").manual_seed(V)
    dl, dh = (torch.randn(8, device="cuda", generator=g).repeat((T + 7) // 8)[:T].contiguous() for _ in range(2))
    n, nt = l[:8].float().cpu().numpy().astype(np.float64), t[:8].cpu().numpy()
    lse, H = o["lse"][:8].cpu().numpy().astype(np.float64), o["entropy"][:8].cpu().numpy().astype(np.float64)
    assert abs(H[3] - math.log(3)) <= 8 * UNIT and np.abs(H[[4, 5, 6]]).max() == 0
    for a, b in ((dl, dh), (dl, None), (None, dh)):
        na, nb = (np.zeros(8) if x is None else x[:8].cpu().numpy().astype(np.float64) for x in (a, b))
        want, mag = O.token_logprob_backward(n[[0, 2, 7]], nt[[0, 2, 7]], lse[[0, 2, 7]], na[[0, 2, 7]], H[[0, 2, 7]], nb[[0, 2, 7]], temperature)
        full, size = np.zeros((8, V)), np.zeros((8, V))
        full[[0, 2, 7]], size[[0, 2, 7]] = want, mag
        for r in (1, 3, 4, 5, 6):
            top = n[r] == n[r].max()
            full[r] = np.where(top, -(na[r] + nb[r] * H[r]), 0.0) / temperature
            full[r, nt[r]] = (-nb[r] * H[r] if top[nt[r]] else na[r]) / temperature
            size[r] = np.where(top, np.abs(na[r]) + np.abs(nb[r]) * H[r], 0.0) / temperature
        live = np.where(n > -2.0 ** 100, n, 0.0)
        arg = np.where((np.abs(lse) < 1e20)[:, None], np.abs(live) / temperature + np.abs(lse)[:, None], 0.0)
        # a p below fp32's normal numbers is 0; a result of one product, dlogp / temperature, is off by the roundings of 1 /
        # temperature and of itself
        tol = 2 * UNIT * np.abs(full) + size * (16 * UNIT + 8 * UNIT * arg) + 8 * UNIT * arg * (np.abs(na) + np.abs(nb))[:, None] / temperature + 2.0 ** -120
        for out in (None, torch.full((T, V), 7.0, dtype=torch.float32, device="cuda"), l.clone()):
            src = out if out is not None and out.dtype == dtype and out.shape == l.shape and torch.equal(out, l) else l
            got = _ops().token_logprob_backward(src, t, o["lse"], dlogp=a, entropy=None if b is None else o["entropy"],
                                                dentropy=b, temperature=temperature, out=out)
            extra = 2.0 ** -8 * np.abs(full) if got.dtype == torch.bfloat16 else 0.0
            of = np.arange(T) % 8
            _close(got.float().cpu().numpy(), full[of], (tol + extra)[of], "dlogits")
    assert _ops().get_device_status() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(4, 300), (4, 50001), (400, 300), (400, 4000), (400, 15000)])
def test_quotients_past_the_range(bf16, T, V):
    """Where no fp32 number holds the largest quotient by the temperature, lse is NaN and the gradient of the row with it; what is
    taken of differences is not.  Logits far below the largest may have such a quotient."""
    l = torch.randn(4, V, device="cuda")
    l[1, 5] = 3e38
    l[2] = -3e38
    l[3, ::3] = -3e38
    l = l.to(torch.bfloat16 if bf16 else torch.float32).repeat((T + 3) // 4, 1)[:T].contiguous()
    t = torch.full((T,), 5, device="cuda")
    o = _ops().token_logprob(l, t, temperature=0.5, entropy=True, top=2)
    row = torch.arange(T, device="cuda") % 4
    bad = (row == 1) | (row == 2)
    assert torch.equal(o["lse"].isnan(), bad)
    assert o["logp"].isfinite().all() and o["entropy"].isfinite().all() and not o["top_logp"].isnan().any()
    assert (o["logp"][row == 1] == 0).all() and (o["entropy"][row == 1] == 0).all()
    for k, v in (("logp", -math.log(V)), ("entropy", math.log(V))):
        assert ((o[k][row == 2] - v).abs() <= 8 * UNIT * math.log(V) + 2 * (44 + V / 1024) * UNIT).all()
    one = torch.ones(T, device="cuda")
    for a, b in ((one, None), (None, one)):
        d = _ops().token_logprob_backward(l, t, o["lse"], dlogp=a, entropy=None if b is None else o["entropy"], dentropy=b, temperature=0.5)
        assert d[bad].isnan().all() and d[~bad].isfinite().all()


def _certain_rows(T, V, dtype):
    """Rows with one token far above the others, by 14 to 26, shifted so that lse is about 0, 20 and 40."""
    gap = torch.arange(T) % 13 + 14.0
    l = torch.zeros(T, V)
    top = (torch.arange(T) * 613) % V
    l[torch.arange(T), top] = gap
    return (l + (torch.arange(T) % 3 * 20.0)[:, None]).to(dtype).cuda(), top.cuda(), gap.double().numpy()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(39, 4096), (39, 50001), (1300, 1000)])
def test_gradient_of_nearly_certain_targets(bf16, T, V):
    """With the forward's logp the target's 1 - p is relatively exact, and the terms of a row cancel: against the closed
    form, p = 1 / (1 + (V - 1) e^-gap).  logp is off by its own bound, (44 + V / 1024) u of it and 5 u gap of its argument's
    rounding, and by 4 u; expm1, the products and the entropy's two terms add 16 u of the terms' magnitudes."""
    ops = _ops()
    l, t, gap = _certain_rows(T, V, torch.bfloat16 if bf16 else torch.float32)
    o = ops.token_logprob(l, t, entropy=True)
    rest = (V - 1) * np.exp(-gap)
    p, lr = 1 / (1 + rest), np.log1p(rest)
    H = lr + rest * gap / (1 + rest)
    f32 = torch.zeros(T, V, device="cuda")
    ones = torch.ones(T, device="cuda")
    rel = (44 + V / 1024 + 5 * gap + 4) * UNIT
    at = t.cpu().numpy()
    # dlogp: the target's 1 - p
    d = ops.token_logprob_backward(l, t, o["lse"], dlogp=ones, out=f32, logp=o["logp"]).cpu().numpy().astype(np.float64)
    want = -np.expm1(-lr)
    assert np.all(np.abs(d[np.arange(T), at] - want) <= want * (rel + 16 * UNIT))
    # the rest of the row is -p of each other token, off by lse's rounding, which is 2^-24 of it, and as much of the scaled logit
    lse = l.float().cpu().numpy().max(1) + lr
    assert np.all(np.abs(d.sum(1)) <= want * (rel + (32 + 4 * lse) * UNIT))
    # dentropy at the target: -p (log p + H), whose terms are lr and H
    d = ops.token_logprob_backward(l, t, o["lse"], entropy=o["entropy"], dentropy=ones, out=f32, logp=o["logp"]).cpu().numpy()
    want = -p * (H - lr)
    s2 = rest * gap * gap / (1 + rest)
    tol = (rel + 16 * UNIT) * (lr + H) + 5 * UNIT * s2
    assert np.all(np.abs(d[np.arange(T), at] - want) <= tol)
    assert ops.get_device_status() == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_gradient_with_logp_is_the_same_elsewhere(bf16):
    """Ordinary targets, unscored rows, masked targets, rows with nothing in reach, NaN: with logp within the rounding of
    lse at the target, and the same bits everywhere else; in place and captured too."""
    ops = _ops()
    T, V = 61, 3001
    l = torch.randn(T, V + 3, device="cuda").mul_(2).to(torch.bfloat16 if bf16 else torch.float32)[:, :V]
    t = torch.randint(0, V, (T,), device="cuda")
    l[3, ::2] = -torch.inf
    l[4] = -torch.inf
    l[5, t[5]] = -torch.inf
    l[6, 9] = torch.nan
    t[7:9] = -1
    o = ops.token_logprob(l, t, entropy=True)
    dl, dh = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    kw = dict(dlogp=dl, entropy=o["entropy"], dentropy=dh)
    base = ops.token_logprob_backward(l, t, o["lse"], **kw)
    got = ops.token_logprob_backward(l, t, o["lse"], logp=o["logp"], **kw)
    hot = torch.zeros(T, V, dtype=torch.bool, device="cuda")
    hot[t >= 0, t[t >= 0]] = True
    same = lambda a, b: torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
    assert same(torch.where(hot, 0, got), torch.where(hot, 0, base))
    live = (t >= 0) & o["logp"].isfinite()
    # log p by either way: off by 4 u of |z| + |lse| (below 30 here); the derivative of both terms by it is below |dl| + 3 |dh|
    diff = (got.float() - base.float()).abs()[live, t[live]]
    assert (diff <= 4 * UNIT * 30 * (dl.abs() + 16 * dh.abs())[live] + (2.0 ** -7 * base.float().abs()[live, t[live]] if bf16 else 1e-30)).all()
    assert not got[4].any() and got[5, t[5]] == 0 and got[6].isnan().all() and not got[7:9].any()
    want = got.clone()
    torch.cuda.synchronize()
    buf = l.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.token_logprob_backward(buf, t, o["lse"], out=buf, logp=o["logp"], **kw)
    g.replay()
    torch.cuda.synchronize()
    assert same(buf, want)
    for bad in (dict(logp=o["logp"][:5]), dict(logp=o["logp"][:, None])):
        with pytest.raises(ValueError):
            ops.token_logprob_backward(l, t, o["lse"], dlogp=dl, **bad)
    with pytest.raises(TypeError):
        ops.token_logprob_backward(l, t, o["lse"], dlogp=dl, logp=o["logp"].double())
    with pytest.raises(ValueError):
        ops.token_logprob_backward(l, None, o["lse"], entropy=o["entropy"], dentropy=dh, logp=o["logp"])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(9, 50001), (9, 900), (400, 4000), (400, 7000), (400, 15000), (3, 131072)])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 3.0])
def test_entropy_within_its_own_rounding(bf16, T, V, temperature):
    """Near certainty, near uniformity and between: no more than what the terms' roundings give."""
    rng = np.random.default_rng(V)
    r = rng.normal(size=(9, V)) * np.array([0.01, 0.3, 1, 2, 4, 8, 1, 2, 0])[:, None]
    r[6:9, V // 3] += [30, 12, 25]
    l = torch.from_numpy(r.astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32)
    t = l.float().argmax(1)
    n = (T + 8) // 9
    _forward(l.repeat(n, 1)[:T].contiguous().cuda(), t.repeat(n)[:T].cuda(), temperature, 0, min(T, 9))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V", [(3, 300), (2000, 300), (3, 40000)])
def test_gradient_of_a_target_without_probability(bf16, T, V):
    """Far below the others its log p weighs nothing, however large dentropy is: its gradient is dlogp / temperature."""
    ops = _ops()
    l = torch.randn(T, V, device="cuda")
    l[:, 5] = -1e9
    l[1, 5] = -1e33
    l = l.to(torch.bfloat16 if bf16 else torch.float32)
    t = torch.full((T,), 5, device="cuda")
    o = ops.token_logprob(l, t, temperature=1e-3, entropy=True)
    dl, dh = torch.full((T,), 0.5, device="cuda"), torch.full((T,), 1e30, device="cuda")
    out = torch.zeros(T, V, device="cuda")
    for logp in (None, o["logp"]):
        d = ops.token_logprob_backward(l, t, o["lse"], dlogp=dl, entropy=o["entropy"], dentropy=dh, temperature=1e-3, out=out, logp=logp)
        assert d.isfinite().all() and ((d[:, 5] - 500).abs() <= 500 * 4 * UNIT).all()
