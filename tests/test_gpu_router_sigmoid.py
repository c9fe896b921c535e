"""Sigmoid routing on the GPU where scores vanish, saturate or are swayed by a
bias, in every type and width of the kernels.

The choice is by the scores and sums rounded to fp32, which elementary torch
operations give; weights, loads, loss and gradient are those of the choice, in
fp64.  A score is an fp32 number: the sigmoid of a logit below about -88.7 is 0.

Bounds as for the router's other tests: weights within 1e-5 of themselves (a
score that is an fp32 subnormal is off by at most 2^-150 / 2^-128 = 2.4e-7
more), loads within 2e-5, gradients within 2e-5 of the sum of their terms'
magnitudes, a bf16 result by 2^-8 of itself more.
"""
import numpy as np
import pytest
import torch

from oracle import router as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

PROB, LOAD, GRAD, BF16 = 1e-5, 2e-5, 2e-5, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _close(got, want, tol, what):
    got = got.float().cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {np.broadcast_to(want, got.shape)[bad][0]}"


def _route(l, k, normalize, scale, bias, mask):
    """The call, and its outputs checked: (outputs, logits in fp64 with -inf
    where the score is 0, ids)."""
    from microscaled_precision_moe_gb300 import ops
    T, E = l.shape
    o = ops.moe_route(l, k, score="sigmoid", normalize=normalize, scale=scale, bias=bias, token_mask=mask)
    f = l.float()
    live = f > R.LOWEST
    if bias is not None:
        live &= (bias > R.LOWEST)[None]
    s32 = 1.0 / (1.0 + torch.exp(-f.clamp(max=R.FLT_MAX)))
    key = torch.where(live, s32 if bias is None else s32 + bias, torch.full_like(f, -torch.inf))
    ids = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    assert torch.equal(o["ids"].long(), ids)
    keep = np.ones(T, bool) if mask is None else mask.cpu().numpy()
    picked = torch.gather(live, 1, ids).cpu().numpy() & keep[:, None]
    ids = ids.cpu().numpy()
    counts = np.bincount(ids[picked], minlength=E)
    assert np.array_equal(o["counts"].cpu().numpy(), counts) and int(o["n_tokens"]) == keep.sum()
    ref = torch.where(live & (s32 > 0), f.double(), torch.full_like(f, -torch.inf).double()).cpu().numpy()
    s, _, _ = R.scores(ref, "sigmoid")
    prob = R.weights(s, ids, normalize, scale) * keep[:, None]
    total = s.sum(1, keepdims=True)
    load = (s / np.where(total > 0, total, 1.0) * keep[:, None]).sum(0) / max(keep.sum(), 1)
    loss = E / (k * max(keep.sum(), 1)) * np.dot(counts, load)
    _close(o["prob"], prob, PROB * np.abs(prob) + 1e-30, "prob")
    _close(o["load"], load, LOAD * load + 1e-12, "load")
    _close(o["loss"], loss, LOAD * loss + 1e-12, "loss")
    assert ops.get_device_status() == 0
    return o, ref, ids


def _bias(E, g):
    """Distinct sways, one infinite, some experts out of reach."""
    b = 0.3 * torch.randn(E, device="cuda", generator=g)
    b[E // 3], b[E // 2], b[-1] = float("-inf"), float("nan"), torch.finfo(torch.bfloat16).min
    return b


def _logits(T, E, std, shift, bf16, g):
    l = torch.randn(T, E, device="cuda", generator=g) * std + shift
    return l.to(torch.bfloat16) if bf16 else l


CASES = [(40, 33, 5, 1.0, 0.0), (300, 60, 4, 12.0, -40.0), (130, 128, 8, 30.0, -70.0), (257, 256, 8, 1.0, -15.0),
         (70, 300, 16, 1.0, 9.0), (150, 700, 20, 4.0, -87.0), (9, 1024, 40, 2.0, 0.0)]


@pytest.mark.parametrize("T,E,k,std,shift", CASES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("normalize", [True, False])
def test_forward(T, E, k, std, shift, bf16, biased, normalize):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = _logits(T, E, std, shift, bf16, g)
    mask = torch.arange(T, device="cuda") % 6 != 4
    _route(l, k, normalize, 2.5, _bias(E, g) if biased else None, mask)


@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("E,equal", [(8, False), (64, False), (64, True), (256, True)])
@pytest.mark.parametrize("biased", [True, False])
def test_weights_of_subnormal_scores(k, E, equal, biased):
    """Every score of a row below fp32's normal range (logits of -88.7 to -85):
    normalised weights are finite shares of one.  With masses of equal keys the
    choice is made one expert after the other."""
    g = torch.Generator(device="cuda").manual_seed(k + E)
    l = -88.7 + 3.7 * torch.rand(200, E, device="cuda", generator=g)
    if equal:
        l = l[:, :1].expand(200, E).contiguous()
    b = 0.01 * torch.randn(E, device="cuda", generator=g) if biased and not equal else None
    if biased and equal:
        b = torch.zeros(E, device="cuda")
    o, _, _ = _route(l, k, True, 2.5, b, None)
    total = o["prob"].double().sum(1)
    assert (total - 2.5).abs().max() < 2.5 * PROB
    # the shares of a token whose scores are all that small count as any other's
    assert abs(float(o["load"].double().sum()) - 1.0) < LOAD


def _gradient(l, k, normalize, scale, bias, mask, size, seed):
    """The gradient of weights and loss, apart and together, where a score of 0
    passes nothing on."""
    from microscaled_precision_moe_gb300 import ops
    o, ref, ids = _route(l, k, normalize, scale, bias, mask)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dprob = torch.randn(ids.shape, device="cuda", generator=g) * size
    dloss = torch.full((1,), size, device="cuda")
    for dp, dl in ((dprob, dloss), (dprob, None), (None, dloss)):
        got = ops.moe_route_backward(l, o["ids"], o["counts"], o["n_tokens"], dprob=dp, dloss=dl, score="sigmoid",
                                     normalize=normalize, scale=scale, bias=bias, token_mask=mask)
        want, mag = R.route_backward(ref, ids, o["counts"].cpu().numpy(),
                                     np.zeros(ids.shape) if dp is None else dp.cpu().numpy(),
                                     0.0 if dl is None else size, "sigmoid", normalize, scale, None,
                                     None if mask is None else mask.cpu().numpy())
        _close(got, want, GRAD * mag + 1e-30 * max(size, 1.0) + (BF16 * np.abs(want) if l.dtype == torch.bfloat16 else 0),
               "dlogits")
    assert ops.get_device_status() == 0


@pytest.mark.parametrize("T,E,k,std,shift", CASES)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient(T, E, k, std, shift, bf16, biased, normalize):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = _logits(T, E, std, shift, bf16, g)
    mask = torch.arange(T, device="cuda") % 6 != 4
    _gradient(l, k, normalize, 2.5, _bias(E, g) if biased else None, mask, 1.0, E)


@pytest.mark.parametrize("k", [1, 2, 4])
@pytest.mark.parametrize("lo,hi", [(-88.7, -85.0), (-87.3, -86.5), (-88.7, -20.0), (-110.0, -80.0)])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("size", [0.01, 30.0, 1e4])
def test_gradient_of_subnormal_scores(k, lo, hi, biased, size):
    """Normalised weights of scores near and below fp32's normal range: their
    gradient is of the order of dprob, and so is the kernel's, whatever the sum
    of the scores."""
    g = torch.Generator(device="cuda").manual_seed(k)
    l = lo + (hi - lo) * torch.rand(120, 64, device="cuda", generator=g)
    b = 0.01 * torch.randn(64, device="cuda", generator=g) if biased else None
    _gradient(l, k, True, 2.5, b, None, size, 7)


def test_extreme_rows_have_finite_gradients():
    """Saturated, vanishing and huge logits, every row of the gradient."""
    from microscaled_precision_moe_gb300 import ops
    g = torch.Generator(device="cuda").manual_seed(10)
    l = torch.randn(30, 24, device="cuda", generator=g) * 2
    l[1] *= 1e4
    l[2] = -90.0 - torch.arange(24, device="cuda")      # sigmoids that are 0 in fp32
    l[3] = 3e38
    l[3, :4] = -3e38
    l[4] = -88.0
    l[5] = -87.3
    for normalize in (True, False):
        o = ops.moe_route(l, 4, score="sigmoid", normalize=normalize)
        d = ops.moe_route_backward(l, o["ids"], o["counts"], o["n_tokens"], score="sigmoid", normalize=normalize,
                                   dprob=30.0 * torch.randn(30, 4, device="cuda", generator=g),
                                   dloss=torch.full((1,), 30.0, device="cuda"))
        assert torch.isfinite(o["prob"]).all() and torch.isfinite(o["loss"]).all() and torch.isfinite(d).all()
        assert not d[2].any() and not o["prob"][2].any()


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("scale", [1e-3, 1e6])
def test_gradient_of_swayed_choices_among_large_scores(normalize, scale):
    """A bias that picks vanishing scores among ordinary ones: the gradient that
    the others get through the load is as small, and the weights' gradient times
    a large scale stays finite."""
    g = torch.Generator(device="cuda").manual_seed(3)
    l = torch.randn(200, 96, device="cuda", generator=g) * 3
    l[:, :8] = -40.0 - 45.0 * torch.rand(200, 8, device="cuda", generator=g)
    b = torch.zeros(96, device="cuda")
    b[:8] = 5.0 + torch.arange(8, device="cuda")
    _gradient(l, 3, normalize, scale, b, None, 1e3, 5)
