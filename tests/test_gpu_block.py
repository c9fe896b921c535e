"""MoEBlock: the norm, the router and the expert layer run together, and their
gradients joined, checked piece by piece against the fp64 definitions on the
block's own intermediate values."""
import numpy as np
import pytest
import torch

from oracle import norm as N
from oracle import router as R
from microscaled_precision_moe_gb300 import synth
from tests.gpu_util import need_gpu, np_bf16

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _block(T=256, H=512, I=256, E=24, k=4, **kw):
    from microscaled_precision_moe_gb300.block import MoEBlock
    shape = synth.scaled(synth.MOE_30B, T=T, H=H, I=I, E=E, k=k)
    w1, w2 = synth.moe_weights(shape, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    wr = (torch.randn(E, H, device="cuda", generator=g) * H ** -0.5).to(torch.bfloat16)
    wn = 1.0 + 0.1 * torch.randn(H, device="cuda", generator=g)
    x = synth.moe_activations(shape, device="cuda")
    res = synth.moe_activations(shape, seed=2, device="cuda")
    return MoEBlock(T, H, I, E, k, wn, wr, w1, w2, **kw), x, res, wr, wn, w1, w2


def _rel(a, b):
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("score,with_res", [("softmax", True), ("sigmoid", False)])
def test_forward_and_gradients(score, with_res):
    from microscaled_precision_moe_gb300 import ops
    from microscaled_precision_moe_gb300.moe import MXFP8MoE
    scale = 2.5 if score == "sigmoid" else 1.0
    b, x, res, wr, wn, w1, w2 = _block(score=score, scale=scale)
    T, H, I, E, k = b.T, b.H, b.I, b.E, b.k
    res = res if with_res else None
    mask = torch.arange(T, device="cuda") % 11 != 3
    keep_x = x.clone()
    out, h = b.forward(x, res, mask)
    out, h = out.clone(), h.clone()
    # norm
    rh, ry, _ = N.add_rmsnorm(np_bf16(x), wn.cpu().numpy(), None if res is None else np_bf16(res))
    y = b.norm["y"].clone()
    assert np.all(np.abs(np_bf16(y) - ry) <= (BF16 + 1e-5) * np.abs(ry) + 1e-38)
    assert np.all(np.abs(np_bf16(h) - rh) <= (BF16 + 1e-6) * np.abs(rh) + 1e-38)
    # logits: fp32 sums of H exact bf16 products
    l = np_bf16(y).astype(np.float64) @ np_bf16(wr).astype(np.float64).T
    mag = np.abs(np_bf16(y)).astype(np.float64) @ np.abs(np_bf16(wr)).astype(np.float64).T
    logits = b.logits.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(logits - l) <= H * 2.0 ** -24 * mag)
    # router, on the block's own logits; routing and experts as the layer alone runs them
    r = R.route(logits, k, score, True, scale, None, mask.cpu().numpy())
    assert np.array_equal(b.route["counts"].cpu().numpy(), r["counts"])
    assert abs(float(b.route["loss"]) - r["loss"]) <= 2e-5 * r["loss"]
    layer = MXFP8MoE(T, H, I, E, k)
    layer.quantize_weights(w1, w2)
    assert torch.equal(layer.forward(y, b.route["ids"], b.route["prob"]), out)
    assert not out[3::11].any()                       # masked tokens weigh nothing

    dout = synth.moe_grad_out(synth.scaled(synth.MOE_30B, T=T, H=H), device="cuda")
    dh = synth.moe_activations(synth.scaled(synth.MOE_30B, T=T, H=H), seed=5, device="cuda") * 1e-3
    dloss = torch.full((1,), 0.01, device="cuda")
    prob = b.route["prob"].clone()
    g = b.backward(dout, dh=dh, dloss=dloss)
    dy, dw1, dw2 = layer.backward(dout)
    assert torch.equal(g["dw1"], dw1) and torch.equal(g["dw2"], dw2)
    # the weights' gradient and the logits'
    inv = layer.seg[2].cpu().numpy()
    dprob, dmag = R.combine_dprob(np_bf16(dout), np_bf16(layer.y), inv, prob.cpu().numpy())
    assert np.all(np.abs(b.dprob.cpu().numpy() - dprob) <= (H / 32 + 40) * 2.0 ** -24 * dmag + 1e-30)
    ids = b.route["ids"].cpu().numpy().astype(np.int64)
    dl, lmag = R.route_backward(logits, ids, r["counts"], b.dprob.cpu().numpy(), 0.01, score, True, scale,
                                None, mask.cpu().numpy())
    got_dl = np_bf16(b.dlogits_p[:, :E])
    assert np.all(np.abs(got_dl - dl) <= 2e-5 * lmag + BF16 * np.abs(dl) + 1e-30)
    assert not b.dlogits_p[:, E:].any()
    # router weight: fp32 sums over tokens of exact bf16 products
    want = got_dl.astype(np.float64).T @ np_bf16(y).astype(np.float64)
    wmag = np.abs(got_dl).astype(np.float64).T @ np.abs(np_bf16(y)).astype(np.float64)
    assert np.all(np.abs(g["dw_router"].cpu().numpy() - want) <= T * 2.0 ** -24 * wmag + 1e-30)
    # the norm's gradient of both readers and the residual stream
    dy_r = got_dl.astype(np.float64) @ np_bf16(wr).astype(np.float64)
    assert _rel(np_bf16(b.dy_router), dy_r) < BF16
    total = np_bf16(dy).astype(np.float64) + np_bf16(b.dy_router)
    dx, dw, mx, mw = N.add_rmsnorm_backward(total, np_bf16(h), b.norm["rstd"].cpu().numpy(), wn.cpu().numpy(),
                                            np_bf16(dh))
    assert np.all(np.abs(np_bf16(g["dx"]) - dx) <= BF16 * np.abs(dx) + 1e-5 * mx + 1e-38)
    assert np.all(np.abs(g["dw_norm"].cpu().numpy() - dw) <= 2e-5 * mw + 1e-38)
    assert torch.equal(x, keep_x)
    torch.cuda.synchronize()
    assert ops.get_device_status() == 0


def test_rollout_gives_the_training_forward_bytes():
    b, x, res, *_ = _block()
    out, h = b.forward(x, res)
    out, h = out.clone(), h.clone()
    d = b.experts.d.clone()
    got, gh = b.infer(x, res)
    R_ = int(b.experts.seg[0][-1])
    assert torch.equal(got, out) and torch.equal(gh, h)
    assert torch.equal(b.experts.d[:R_], d[:R_])


def test_a_few_steps_lower_the_loss():
    """Plain gradient steps on the router and the norm weight of a regression
    to the block's own output under another router: the loss must fall."""
    b, x, res, wr, wn, *_ = _block(T=128, H=256, I=256, E=8, k=2)
    target = b.forward(x, res)[0].float().clone()
    g = torch.Generator(device="cuda").manual_seed(9)
    master = wr.float() + 0.5 * 256 ** -0.5 * torch.randn(8, 256, device="cuda", generator=g)
    losses = []
    for _ in range(12):
        b.set_weights(router_weight=master.to(torch.bfloat16))
        err = b.forward(x, res)[0].float() - target
        losses.append(float(err.square().sum()))
        grads = b.backward(err.to(torch.bfloat16))
        master -= 0.5 / grads["dw_router"].norm() * grads["dw_router"]
    assert min(losses[6:]) < 0.9 * losses[0], losses


def test_refusals():
    from microscaled_precision_moe_gb300.block import MoEBlock
    w = torch.ones(256, device="cuda")
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="multiple"):
        MoEBlock(100, 256, 128, 8, 2, w, z(8, 256), z(8, 256, 256), z(8, 256, 128))
    with pytest.raises(ValueError, match="router_weight"):
        MoEBlock(128, 256, 256, 8, 2, w, z(4, 256), z(8, 512, 256), z(8, 256, 256))
    with pytest.raises(ValueError, match="multiple"):
        MoEBlock(128, 256, 128, 8, 2, w, z(8, 256), z(8, 256, 256), z(8, 256, 128))


def test_backward_needs_the_forward_it_belongs_to():
    """A rollout overwrites what the forward kept: no gradient of a mixture."""
    b, x, res, *_ = _block(T=128, H=256, I=256, E=8, k=2)
    dout = synth.moe_grad_out(synth.scaled(synth.MOE_30B, T=128, H=256), device="cuda")
    b.infer(x, res)
    with pytest.raises(RuntimeError, match="forward"):
        b.backward(dout)
    b.forward(x, res)
    want = {n: t.clone() for n, t in b.backward(dout).items()}
    b.forward(x, res)
    b.infer(res, x)
    with pytest.raises(RuntimeError, match="forward"):
        b.backward(dout)
    b.forward(x, res)
    assert all(torch.equal(t, want[n]) for n, t in b.backward(dout).items())
    # a rollout that is refused halfway has overwritten the norm's rows
    with pytest.raises((TypeError, ValueError)):
        b.infer(res, x, token_mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(RuntimeError, match="forward"):
        b.backward(dout)


@pytest.mark.parametrize("mode", ["mxfp8", "high_precision", "dequantized"])
def test_expert_layer_backward_after_a_quantised_forward(mode):
    from microscaled_precision_moe_gb300 import ops
    from microscaled_precision_moe_gb300.moe import MXFP8MoE
    shape = synth.scaled(synth.MOE_30B, T=128, H=256, I=256, E=8, k=2)
    w1, w2 = synth.moe_weights(shape, device="cuda")
    ids, prob = (t.cuda() for t in synth.routing(shape))
    x, dout = synth.moe_activations(shape, device="cuda"), synth.moe_grad_out(shape, device="cuda")
    layer = MXFP8MoE(128, 256, 256, 8, 2)
    layer.quantize_weights(w1, w2)
    if mode != "mxfp8":
        layer.prepare_backward_weights(mode, w1, w2)
    back = (lambda: layer.backward(dout)) if mode == "mxfp8" else (lambda: layer.backward_bf16(dout, mode))
    layer.forward(x, ids, prob)
    back()
    q = ops.mxfp8_quantize(x, colwise=False)
    layer.forward_quantized(q["row_q"], q["row_s"], ids, prob)
    with pytest.raises(RuntimeError, match="forward"):
        back()


def test_set_weights_takes_both_experts_weights_and_the_routers_shape():
    b, x, res, wr, wn, w1, w2 = _block(T=128, H=256, I=256, E=8, k=2)
    out = b.forward(x, res)[0].clone()
    for kw in (dict(w2=w2), dict(w1=w1), dict(router_weight=wr[:1]), dict(router_weight=wr[0]),
               dict(router_weight=wr.t())):
        with pytest.raises(ValueError, match="router_weight|together"):
            b.set_weights(**kw)
    b.set_weights(w1=w1, w2=2 * w2)
    assert torch.equal(b.forward(x, res)[0], 2 * out)


def test_quantised_rows_of_another_shape_are_refused():
    from microscaled_precision_moe_gb300 import ops
    b, x, *_ = _block(T=128, H=512, I=256, E=8, k=2)
    ids = torch.arange(256, dtype=torch.int32, device="cuda").view(128, 2) % 8
    prob = torch.full((128, 2), 0.5, device="cuda")
    for rows in (x[:, :256].contiguous(), x[:64]):
        q = ops.mxfp8_quantize(rows, colwise=False)
        with pytest.raises(ValueError, match="x_q"):
            b.experts.forward_quantized(q["row_q"], q["row_s"], ids, prob)
