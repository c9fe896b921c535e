"""The router, the routing weights' gradient and the MXFP8 gather on the GPU
against their fp64 definitions.

Choices, counts and copied bytes are exact.  Bounds: an fp32 exponential is
within 2 ulp and its argument, a difference of two logits below 40, within
2^-24 * 40 (5e-6 together with the sums over at most 1024 experts); gradients
are off by 2e-5 of the sum of their terms' magnitudes, a bf16 result by 2^-8 of
itself more.
"""
import numpy as np
import pytest
import torch

from oracle import router as R
from microscaled_precision_moe_gb300 import synth
from tests.gpu_util import need_gpu, np_bf16, u8

pytestmark = pytest.mark.gpu

PROB, LOAD, GRAD, BF16 = 1e-5, 2e-5, 2e-5, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _ops():
    from microscaled_precision_moe_gb300 import ops
    return ops


def _logits(seed, T, E, bf16=False, pad=0, ties=False, dead=0.0):
    rng = np.random.default_rng(seed)
    l = rng.normal(size=(T, E + pad)) * 2
    if ties:
        l = np.round(l * 4) / 4
    if dead:
        l[rng.random(l.shape) < dead] = -np.inf
    return torch.from_numpy(l.astype(np.float32)).to(torch.bfloat16 if bf16 else torch.float32).cuda()[:, :E]


def _np(l):
    return l.float().cpu().numpy().astype(np.float64)


def _close(got, want, tol, what):
    got = np.asarray(got, np.float64)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {np.broadcast_to(want, got.shape)[bad][0]}"


def _distinct(key, ties_ok):
    """Sigmoid keys are rounded to fp32: no two that differ may be within 1e-6."""
    s = np.sort(np.where(np.isfinite(key), key, -1e9), axis=1)
    gap = np.diff(s, axis=1)
    gap = gap[gap > (1e-14 if ties_ok else -1)]
    return gap[s[:, 1:][np.diff(s, axis=1) > (1e-14 if ties_ok else -1)] > -1e8].min(initial=1) > 1e-6


def _check(l, k, score="softmax", normalize=True, scale=1.0, bias=None, mask=None):
    ops = _ops()
    T, E = l.shape
    kw = dict(score=score, normalize=normalize, scale=scale, bias=bias, token_mask=mask)
    o = ops.moe_route(l, k, **kw)
    torch.cuda.synchronize()
    nb = None if bias is None else bias.cpu().numpy()
    nm = None if mask is None else mask.cpu().numpy()
    r = R.route(_np(l), k, score, normalize, scale, nb, nm)
    if score == "sigmoid":
        assert _distinct(r["key"], bias is None), "the test's own inputs: keys too close for fp32"
    assert np.array_equal(o["ids"].cpu().numpy(), r["ids"])
    assert np.array_equal(o["counts"].cpu().numpy(), r["counts"])
    assert int(o["n_tokens"]) == r["n_tokens"]
    _close(o["prob"].cpu().numpy(), r["prob"], PROB * np.abs(r["prob"]) + 1e-30, "prob")
    _close(o["load"].cpu().numpy(), r["load"], LOAD * r["load"] + 1e-12, "load")
    _close(float(o["loss"]), r["loss"], LOAD * r["loss"], "loss")
    again = ops.moe_route(l, k, **kw)
    assert all(torch.equal(again[n], o[n]) for n in o)

    g = torch.Generator(device="cuda").manual_seed(T + E)
    dprob = torch.randn(T, k, device="cuda", generator=g)
    dloss = torch.full((1,), 0.7, device="cuda")
    for dp, dl in ((dprob, dloss), (dprob, None), (None, dloss)):
        got = ops.moe_route_backward(l, o["ids"], o["counts"], o["n_tokens"], dprob=dp, dloss=dl, **kw)
        want, mag = R.route_backward(_np(l), r["ids"], r["counts"],
                                     np.zeros((T, k)) if dp is None else dp.cpu().numpy(),
                                     0.0 if dl is None else 0.7, score, normalize, scale, nb, nm)
        tol = GRAD * mag + 1e-30 + (BF16 * np.abs(want) if l.dtype == torch.bfloat16 else 0)
        _close(got.float().cpu().numpy(), want, tol, "dlogits")
    assert ops.get_device_status() == 0
    return o


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 2, 1), (7, 31, 3), (64, 32, 4), (65, 33, 5),
                                   (130, 60, 6), (257, 128, 8), (100, 129, 9), (512, 256, 8), (33, 300, 16),
                                   (40, 512, 33), (20, 1024, 64), (4000, 64, 2), (9001, 128, 8)])
@pytest.mark.parametrize("bf16", [False, True])
def test_softmax(T, E, k, bf16):
    _check(_logits(T + E, T, E, bf16), k, normalize=k > 1)


@pytest.mark.parametrize("normalize,scale", [(True, 1.0), (False, 2.5)])
def test_softmax_pitch_ties_masks(normalize, scale):
    l = _logits(1, 203, 96, True, pad=5, ties=True, dead=0.3)
    l[7] = float("-inf")
    l[8] = float("nan")
    l[9, 3] = float("nan")
    l[10] = torch.finfo(torch.bfloat16).min
    l[11, 4:] = torch.finfo(torch.bfloat16).min
    l[12, 20] = float("inf")
    l[13, 20:22] = float("inf")
    l[14] = 3.0                                    # all equal
    mask = (torch.arange(203, device="cuda") % 7) != 2
    o = _check(l, 6, normalize=normalize, scale=scale, mask=mask)
    assert o["ids"][14].tolist() == [0, 1, 2, 3, 4, 5]
    assert o["ids"][7].tolist() == [0, 1, 2, 3, 4, 5] and not o["prob"][7].any()


@pytest.mark.parametrize("T,E,k", [(300, 256, 8), (700, 60, 4), (90, 700, 20), (40, 40, 40)])
@pytest.mark.parametrize("std,shift", [(1.0, 0.0), (0.01, 0.0), (12.0, 0.0), (1.0, -15.0), (1.0, 9.0), (30.0, -70.0)])
@pytest.mark.parametrize("bias", [None, 0.1, 300.0, float("inf")])
def test_sigmoid_choice_is_by_the_fp32_keys(T, E, k, std, shift, bias):
    """Saturated, vanishing and nearly equal scores: the choice is that of the
    scores and sums rounded to fp32, ties to the lower expert."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    l = torch.randn(T, E, device="cuda", generator=g) * std + shift
    b = None
    if bias is not None:
        b = torch.randn(E, device="cuda", generator=g) * (bias if bias < 1e3 else 1.0)
        if bias > 1e3:
            b[::7] = bias
    key = 1.0 / (1.0 + torch.exp(-l))
    if b is not None:
        key = key + b
    want = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :k]
    o = _ops().moe_route(l, k, score="sigmoid", bias=b)
    assert torch.equal(o["ids"].long(), want)


def test_lowest_fp32_value_is_a_mask_too():
    l = _logits(2, 40, 16)
    l[:, 5] = torch.finfo(torch.float32).min
    l[3] = torch.finfo(torch.float32).min
    o = _check(l, 4)
    assert int(o["counts"][5]) == 0


@pytest.mark.parametrize("T,E,k", [(1, 16, 2), (64, 256, 8), (300, 60, 6), (2000, 40, 4)])
@pytest.mark.parametrize("normalize", [True, False])
def test_sigmoid(T, E, k, normalize):
    # logits on a grid: keys that differ do so by far more than fp32's rounding
    _check(_logits(5 + T, T, E, ties=True, dead=0.1), k, "sigmoid", normalize, 2.5,
           mask=torch.arange(T, device="cuda") % 5 != 1 if T > 1 else None)


def test_sigmoid_bias_sways_the_choice_only():
    T, E, k = 120, 48, 6
    # grid logits (steps of 1/4) and biases of distinct multiples of 1e-3 + 1e-5: no accidental near-ties
    l = _logits(8, T, E, ties=True)
    bias = torch.arange(E, device="cuda", dtype=torch.float32) * 1.01e-3
    bias[3] = float("-inf")
    bias[4] = float("nan")
    ops = _ops()
    o = ops.moe_route(l, k, score="sigmoid", bias=bias)
    r = R.route(_np(l), k, "sigmoid", True, 1.0, bias.cpu().numpy())
    same = o["ids"].cpu().numpy() == r["ids"]
    key = r["key"]
    for t, j in np.argwhere(~same):                # only keys fp32 cannot tell apart may swap
        a, b = key[t, o["ids"][t, j].item()], key[t, r["ids"][t, j]]
        assert abs(a - b) < 2.0 ** -22, (t, j)
    assert not ((o["ids"] == 3) | (o["ids"] == 4)).any()
    s, _, _ = R.scores(_np(l), "sigmoid", bias.cpu().numpy())
    w = R.weights(s, o["ids"].cpu().numpy(), True, 1.0)
    _close(o["prob"].cpu().numpy(), w, PROB * w, "prob")


def test_no_counted_tokens():
    l = _logits(9, 12, 16)
    o = _check(l, 2, mask=torch.zeros(12, dtype=torch.bool, device="cuda"))
    assert float(o["loss"]) == 0 and not o["prob"].any() and not o["counts"].any()


def test_extreme_logits():
    l = _logits(10, 30, 24)
    l[1] *= 1e4
    l[2] = -90.0 - torch.arange(24, device="cuda")      # sigmoids that underflow
    l[3] = 3e38
    l[3, :4] = -3e38
    _check(l, 4)
    ops = _ops()
    o = ops.moe_route(l, 4, score="sigmoid")
    d = ops.moe_route_backward(l, o["ids"], o["counts"], o["n_tokens"], score="sigmoid",
                               dprob=torch.ones(30, 4, device="cuda"), dloss=torch.ones(1, device="cuda"))
    assert torch.isfinite(o["prob"]).all() and torch.isfinite(o["loss"]).all()
    assert torch.isfinite(d[3:]).all() and torch.isfinite(d[:2]).all()


def test_outputs_feed_the_segment_build():
    ops = _ops()
    shape = synth.scaled(synth.MOE_30B, T=500, E=24, k=4)
    ids, prob = synth.routing(shape)
    key = synth.stream_key(0, synth.TID_LOGITS)
    l = synth.normal_f64(key, 0, 500 * 24).view(500, 24).float().cuda()
    o = ops.moe_route(l, 4)
    assert torch.equal(o["ids"].cpu(), ids)
    assert (o["prob"].cpu() - prob).abs().max() < 1e-6
    seg = ops.moe_build_segments(o["ids"], o["prob"], 24)
    ref = ops.moe_build_segments(ids.cuda(), prob.cuda(), 24)
    assert torch.equal(seg[0], ref[0]) and torch.equal(seg[1], ref[1])
    assert int(o["counts"].sum()) == 2000


def test_in_place_gradient_stream_and_graph():
    ops = _ops()
    l = _logits(11, 300, 128)
    kw = dict(token_mask=torch.arange(300, device="cuda") % 3 != 0)
    ref = ops.moe_route(l, 8, **kw)
    dprob, dloss = torch.randn(300, 8, device="cuda"), torch.ones(1, device="cuda")
    back = lambda z, r, out=None: ops.moe_route_backward(z, r["ids"], r["counts"], r["n_tokens"],  # noqa: E731
                                                         dprob=dprob, dloss=dloss, out=out, **kw)
    dref = back(l, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o = ops.moe_route(l, 8, **kw)
        d = back(l, o)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o2 = ops.moe_route(l, 8, **kw)
        d2 = back(l, o2)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a in (o, o2):
        assert all(torch.equal(a[n], ref[n]) for n in ref)
    z = l.clone()
    for a in (d, d2, back(z, ref, z)):
        assert torch.equal(a, dref)


@pytest.mark.parametrize("T,E,pad", [(100, 128, 0), (77, 33, 0), (64, 160, 96), (50, 61, 3)])
def test_gradient_type_of_its_own(T, E, pad):
    """bf16 gradients of fp32 logits are the fp32 ones rounded once, and the
    other way round the fp32 gradients of bf16 logits round to the bf16 ones."""
    ops = _ops()
    for bf16 in (False, True):
        l = _logits(20 + T, T, E, bf16)
        o = ops.moe_route(l, 4)
        g = torch.Generator(device="cuda").manual_seed(T)
        kw = dict(dprob=torch.randn(T, 4, device="cuda", generator=g), dloss=torch.ones(1, device="cuda"))
        a = (l, o["ids"], o["counts"], o["n_tokens"])
        full = ops.moe_route_backward(*a, out=torch.empty(T, E, device="cuda"), **kw)
        buf = torch.full((T, E + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        ops.moe_route_backward(*a, out=buf[:, :E], **kw)
        assert torch.equal(buf[:, :E], full.to(torch.bfloat16)) and (buf[:, E:] == 7).all()
        assert torch.equal(ops.moe_route_backward(*a, **kw), full.to(l.dtype))


def test_nothing_outside_the_gradient_is_written_and_bad_ids():
    ops = _ops()
    buf = torch.full((12, 40), 7.0, device="cuda")
    l = _logits(12, 10, 33)
    o = ops.moe_route(l, 2)
    ops.moe_route_backward(l, o["ids"], o["counts"], o["n_tokens"], dprob=torch.ones(10, 2, device="cuda"),
                           out=buf[1:11, :33])
    assert (buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, 33:] == 7).all()
    assert ops.get_device_status() == 0
    bad = o["ids"].clone()
    bad[4, 1], bad[5, 0] = 33, -1
    d = ops.moe_route_backward(l, bad, o["counts"], o["n_tokens"], dprob=torch.ones(10, 2, device="cuda"))
    torch.cuda.synchronize()
    assert ops.get_device_status() == 7 and torch.isfinite(d).all()


# ---------------------------------------------------------------- the routing weights' gradient

@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (5, 64, 2), (33, 2048, 8), (17, 7168, 6), (9, 264, 3), (3, 136, 64),
                                   (4, 16392, 2)])
def test_combine_dprob(T, H, k):
    ops = _ops()
    rng = np.random.default_rng(T + H)
    cap = 2 * T * k + 5
    g = torch.Generator(device="cuda").manual_seed(H)
    y = torch.randn(cap, H, device="cuda", generator=g).to(torch.bfloat16)
    dout = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    inv = rng.permutation(cap)[:T * k].astype(np.int32)
    unused = np.setdiff1d(np.arange(cap), inv)
    y[torch.from_numpy(unused).cuda()] = float("nan")      # rows no slot names
    prob = rng.uniform(0.01, 1, size=(T, k)).astype(np.float32)
    if T * k > 3:
        inv[1] = -1
        prob.reshape(-1)[2] = 0.0
        y[int(inv[2])] = float("nan")
    got = ops.moe_combine_dprob(dout, y, torch.from_numpy(inv).cuda(), torch.from_numpy(prob).cuda())
    want, mag = R.combine_dprob(np_bf16(dout), np_bf16(y), inv, prob)
    # fp32 products are exact to 2^-24; chains of at most H / 32 + 40 additions
    _close(got.cpu().numpy(), want, (H / 32 + 40) * 2.0 ** -24 * mag + 1e-30, "dprob")
    assert ops.get_device_status() == 0
    again = ops.moe_combine_dprob(dout, y, torch.from_numpy(inv).cuda(), torch.from_numpy(prob).cuda())
    assert torch.equal(got, again)


def test_combine_dprob_bad_row_sets_status():
    ops = _ops()
    y, dout = torch.ones(10, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.tensor([0, 1, 2, 10, 4, 5], dtype=torch.int32, device="cuda")
    d = ops.moe_combine_dprob(dout, y, inv, torch.ones(3, 2, device="cuda"))
    torch.cuda.synchronize()
    assert ops.get_device_status() == 7
    assert d.view(-1).tolist() == [64, 64, 64, 0, 64, 64]


# ---------------------------------------------------------------- MXFP8 gather

@pytest.mark.parametrize("T,K,E,k,pad", [(1, 32, 4, 1, 128), (64, 7168, 40, 8, 16), (700, 544, 12, 4, 128),
                                         (300, 2080, 16, 8, 256), (130, 96, 20, 6, 64), (2000, 2048, 9, 2, 32)])
def test_gather_mxfp8_gives_the_bytes_of_quantise_gather(T, K, E, k, pad):
    ops = _ops()
    shape = synth.scaled(synth.MOE_30B, T=T, H=K, E=E, k=k)
    ids, prob = synth.routing(shape)
    seg, perm, inv, rp, cap = ops.moe_build_segments(ids.cuda(), prob.cuda(), E, pad=pad)
    x = synth.normal_bf16(3, 77, (T, K), "cuda", std=2.0, outlier_p=0.01, outlier_mul=50.0)
    R_ = int(seg[-1])

    def bufs():
        return (torch.full((cap, K), 0xA5, dtype=torch.uint8, device="cuda"),
                torch.full((ops.scale_bytes(cap, K // 32),), 0x5A, dtype=torch.uint8, device="cuda"))
    q = ops.mxfp8_quantize(x, colwise=False)
    got = bufs()
    ops.moe_gather_mxfp8(q["row_q"], q["row_s"], perm, seg, E, k, cap, out=got)
    ref = bufs()
    ops.mxfp8_quantize_gather(x, perm, seg, E, k, cap, colwise=False, out={"row_q": ref[0], "row_s": ref[1]})
    torch.cuda.synchronize()
    assert ops.get_device_status() == 0
    assert torch.equal(got[0][:R_], ref[0][:R_]) and (got[0][R_:] == 0xA5).all()
    from oracle import quant as Q
    a, b = (Q.unswizzle_scales(u8(t[1]), cap, K // 32)[:R_] for t in (got, ref))
    live = perm[:R_].cpu().numpy() >= 0
    assert np.array_equal(a[live], b[live]) and not a[~live].any()


def test_gather_mxfp8_bad_token_sets_status():
    ops = _ops()
    shape = synth.scaled(synth.MOE_30B, T=64, H=256, E=4, k=2)
    ids, prob = synth.routing(shape)
    seg, perm, inv, rp, cap = ops.moe_build_segments(ids.cuda(), prob.cuda(), 4)
    q = ops.mxfp8_quantize(synth.moe_activations(shape, device="cuda"), colwise=False)
    bad = perm.clone()
    row = int(inv[9])
    bad[row] = 64 * 2
    dq, ds = ops.moe_gather_mxfp8(q["row_q"], q["row_s"], bad, seg, 4, 2, cap)
    torch.cuda.synchronize()
    assert ops.get_device_status() == 7
    assert not dq[row].any() and torch.equal(dq[int(inv[8])], q["row_q"][4])


@pytest.mark.parametrize("T,H,I,E,k,kw", [(256, 512, 256, 8, 4, {}), (100, 256, 256, 12, 3, {"tile_m": 128}),
                                          (256, 512, 256, 8, 2, {"fc2": "online"})])
def test_nvfp4_layer_prob_grad(T, H, I, E, k, kw):
    """The NVFP4 layer's gradient of the routing weights is that of its own
    combined rows, and doubling a weight moves the output by that much."""
    from microscaled_precision_moe_gb300.moe import NVFP4MoE, NVFP4Weights
    ops = _ops()
    shape = synth.scaled(synth.MOE_30B, T=T, H=H, I=I, E=E, k=k)
    ids, prob = (t.cuda() for t in synth.routing(shape))
    w = NVFP4Weights.quantize(*synth.moe_weights(shape, device="cuda"))
    x = synth.moe_activations(shape, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(T)
    dout = torch.randn(T, H, device="cuda", generator=g).to(torch.bfloat16)
    prob[3, 1] = 0.0
    layer = NVFP4MoE(T, H, I, E, k, **kw)
    out = layer.forward(x, ids, prob, w).float().clone()
    y, inv = layer.y.clone(), layer.seg[2].clone()
    got = layer.prob_grad(dout, prob)
    want, mag = R.combine_dprob(np_bf16(dout), np_bf16(y), inv.cpu().numpy(), prob.cpu().numpy())
    _close(got.cpu().numpy(), want, (H / 32 + 40) * 2.0 ** -24 * mag + 1e-30, "dprob")
    assert float(got[3, 1]) == 0.0
    # D and so its scales double with the weight, exactly; out is rounded to bf16 twice
    twice = prob.clone()
    twice[:, 0] *= 2
    moved = layer.forward(x, ids, twice, w).float() - out
    change = (moved.double() * dout.double()).sum(1)
    size = (out.abs().double() + moved.abs().double()) * dout.double().abs()
    assert ((change - (got[:, 0] * prob[:, 0]).double()).abs() <= 2 * BF16 * size.sum(1)).all()
    assert ops.get_device_status() == 0
