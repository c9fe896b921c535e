"""The fp64 norm and router definitions: gradients against central
differences, the choice against its definition one token at a time, and the
cases a mask makes (CPU only)."""
import numpy as np
import pytest

from oracle import norm as N
from oracle import router as R


def _differences(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = eps
        g[i] = (f(x + d) - f(x - d)) / (2 * eps)
    return g


@pytest.mark.parametrize("K", [1, 5, 32])
def test_norm_gradient_against_differences(K):
    rng = np.random.default_rng(K)
    h, w = rng.normal(size=(3, K)), rng.normal(size=K)
    dy, dh = rng.normal(size=(3, K)), rng.normal(size=(3, K))
    eps = 1e-2

    def obj(h_, w_):
        return float((N.add_rmsnorm(h_, w_, eps=eps)[1] * dy).sum() + (dh * h_).sum())

    rstd = N.add_rmsnorm(h, w, eps=eps)[2]
    dx, dw, _, _ = N.add_rmsnorm_backward(dy, h, rstd, w, dh)
    # central differences of a smooth O(1) function: error about eps^2 + 1e-16 / eps
    assert np.allclose(dx, _differences(lambda v: obj(v, w), h), atol=1e-7)
    assert np.allclose(dw, _differences(lambda v: obj(h, v), w), atol=1e-7)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_router_gradient_against_differences(score, normalize):
    rng = np.random.default_rng(3)
    T, E, k = 4, 9, 3
    l = rng.normal(size=(T, E))
    bias = 0.1 * rng.normal(size=E) if score == "sigmoid" else None
    mask = np.array([1, 1, 0, 1], bool)
    r = R.route(l, k, score, normalize, 1.7, bias, mask)
    dprob, dloss = rng.normal(size=(T, k)), 0.8
    args = (r["ids"], r["counts"], dprob, dloss, score, normalize, 1.7, bias, mask)
    dl, mag = R.route_backward(l, *args)
    assert np.allclose(dl, _differences(lambda v: R.objective(v, *args), l), atol=1e-7)
    assert np.all(np.abs(dl) <= mag + 1e-15)
    assert not dl[2].any()                           # the masked token


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_is_the_definition(score):
    rng = np.random.default_rng(5)
    T, E, k = 40, 12, 4
    l = np.round(rng.normal(size=(T, E)) * 2) / 2     # many ties
    l[3, :10] = -np.inf                               # fewer than k left
    l[4] = np.nan
    l[5, 2] = np.inf
    r = R.route(l, k, score)
    for t in range(T):
        left = [e for e in range(E) if l[t, e] > R.LOWEST]
        want = sorted(left, key=lambda e: (-l[t, e], e))
        want += [e for e in range(E) if e not in left]
        assert list(r["ids"][t]) == want[:k], t
    assert not r["prob"][4].any() and np.allclose(np.delete(r["prob"], 4, 0).sum(1), 1.0)
    assert r["prob"][3, 2] == 0 and r["prob"][3, 3] == 0
    assert r["counts"].sum() == T * k - k - 2


def test_balanced_loss_is_one_and_no_tokens_is_zero():
    E, k = 8, 2
    l = np.full((E, E), -20.0)
    for t in range(E):
        l[t, t] = l[t, (t + 1) % E] = 5.0
    assert abs(R.route(l, k)["loss"] - 1.0) < 1e-9
    r = R.route(l, k, mask=np.zeros(E))
    assert r["loss"] == 0 and r["n_tokens"] == 0 and not r["counts"].any()


def test_combine_dprob_is_the_derivative():
    """out[t] = sum_j p_j u_j with y = p u: the derivative by p_j is <dout, u_j>."""
    rng = np.random.default_rng(7)
    u, dout = rng.normal(size=(6, 4)), rng.normal(size=(2, 4))
    p = rng.uniform(0.1, 1, size=(2, 3))
    inv = np.array([[0, 2, 4], [1, 3, -1]])
    y = u.copy()
    for t in range(2):
        for j in range(3):
            if inv[t, j] >= 0:
                y[inv[t, j]] = u[inv[t, j]] * p[t, j]
    p[0, 1] = 0.0
    got, _ = R.combine_dprob(dout, y, inv, p)
    want = np.einsum("th,tjh->tj", dout, u[np.maximum(inv, 0)])
    want[1, 2] = want[0, 1] = 0.0
    assert np.allclose(got, want)


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def lib():
    from microscaled_precision_moe_gb300 import build, _lib
    build.build()
    return _lib.load()


NULL, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4
P, Q = 0x10000, 0x10002          # never dereferenced: validation fails first


def test_norm_refusals(lib):
    def f(x=P, M=4, K=64, ldx=64, r=None, ldr=64, w=P, wd=0, eps=1e-6, h=None, ldh=64, y=P, ldy=64,
          rstd=None, q=None, s=None):
        return lib.mpm_add_rmsnorm(x, M, K, ldx, r, ldr, w, wd, eps, h, ldh, y, ldy, rstd, q, s, None)

    assert f(x=None) == NULL and f(w=None) == NULL and f(y=None) == NULL
    assert f(q=P) == NULL and f(s=P) == NULL
    assert f(wd=2) == UNSUP
    assert f(M=0) == SHAPE and f(K=0) == SHAPE and f(K=16385, ldx=16385, ldy=16385) == SHAPE
    assert f(M=1 << 31) == SHAPE
    assert f(ldx=63) == SHAPE and f(ldy=63) == SHAPE
    assert f(r=P, ldr=63) == SHAPE and f(h=P, ldh=63) == SHAPE
    assert f(K=48, q=P, s=P) == SHAPE
    for eps in (0.0, -1.0, float("inf"), float("nan")):
        assert f(eps=eps) == SHAPE
    assert f(x=P + 1) == ALIGN and f(w=Q, wd=1) == ALIGN and f(rstd=Q) == ALIGN
    assert f(q=P + 8, s=P) == ALIGN

    def b(dy=P, lddy=64, dy2=None, h=P, ldh=64, rstd=P, w=P, wd=0, dh=None, lddh=64, M=4, K=64, dx=P,
          lddx=64, dw=P, ws=P, wsb=1 << 20):
        return lib.mpm_add_rmsnorm_backward(dy, lddy, dy2, 63, h, ldh, rstd, w, wd, dh, lddh, M, K, dx,
                                            lddx, dw, ws, wsb, None)

    for a in ("dy", "h", "rstd", "w", "dx", "ws"):
        assert b(**{a: None}) == NULL, a
    assert b(wd=3) == UNSUP
    assert b(M=0) == SHAPE and b(K=0) == SHAPE and b(lddy=63) == SHAPE and b(ldh=63) == SHAPE
    assert b(dy2=P) == SHAPE and b(dh=P, lddh=63) == SHAPE and b(lddx=63) == SHAPE
    need = lib.mpm_add_rmsnorm_backward_workspace_bytes(4, 64)
    assert need > 0 and b(wsb=need - 1) == SHAPE
    assert lib.mpm_add_rmsnorm_backward_workspace_bytes(0, 64) == 0
    assert b(ws=Q) == ALIGN and b(dw=Q) == ALIGN and b(dx=P + 1) == ALIGN


def test_router_refusals(lib):
    def f(l=P, dt=1, T=4, E=16, ld=16, k=2, sc=0, nm=1, scale=1.0, bias=None, ids=P, loss=P, ws=P, wsb=1 << 20):
        return lib.mpm_moe_route(l, dt, T, E, ld, k, sc, nm, scale, bias, None, ids, P, P, P, P, loss, ws,
                                 wsb, None)

    assert f(l=None) == NULL and f(ids=None) == NULL and f(loss=None) == NULL
    assert f(dt=2) == UNSUP and f(sc=2) == UNSUP and f(bias=P, sc=0) == UNSUP
    assert f(T=0) == SHAPE and f(E=0, ld=16) == SHAPE and f(E=1025, ld=1025) == SHAPE
    assert f(k=0) == SHAPE and f(k=17) == SHAPE and f(E=128, ld=128, k=65) == SHAPE
    assert f(ld=15) == SHAPE and f(T=(1 << 30)) == SHAPE and f(scale=float("nan")) == SHAPE
    need = lib.mpm_moe_route_workspace_bytes(4096, 16)
    assert need > 0 and f(T=4096, wsb=need - 1) == SHAPE and f(T=4096, ws=None) == NULL
    assert lib.mpm_moe_route_workspace_bytes(0, 16) == 0
    assert f(l=Q) == ALIGN and f(bias=Q, sc=1) == ALIGN and f(ws=Q) == ALIGN

    def b(l=P, dt=1, T=4, E=16, ld=16, k=2, ids=P, counts=P, n=P, dprob=P, dloss=P, out=P, odt=1, ldd=16):
        return lib.mpm_moe_route_backward(l, dt, T, E, ld, k, 0, 1, 1.0, None, None, ids, counts, n, dprob,
                                          dloss, out, odt, ldd, None)

    assert b(l=None) == NULL and b(out=None) == NULL and b(ids=None) == NULL
    assert b(counts=None) == NULL and b(n=None) == NULL
    assert b(odt=2) == UNSUP and b(ldd=15) == SHAPE and b(T=0) == SHAPE and b(k=20) == SHAPE
    assert b(out=Q) == ALIGN and b(dprob=Q) == ALIGN

    def d(dout=P, T=4, k=2, H=64, cap=128, y=P):
        return lib.mpm_moe_combine_dprob(dout, y, P, P, T, k, H, cap, P, None)

    assert d(dout=None) == NULL and d(y=P + 8) == ALIGN
    assert d(T=0) == SHAPE and d(k=0) == SHAPE and d(H=12) == SHAPE and d(cap=0) == SHAPE

    def g(q=P, T=4, K=64, k=2, E=4, cap=128, s=P):
        return lib.mpm_moe_gather_mxfp8(q, s, T, K, k, P, P, E, cap, P, P, None)

    assert g(q=None) == NULL and g(q=P + 8) == ALIGN and g(s=Q) == ALIGN
    assert g(T=0) == SHAPE and g(K=48) == SHAPE and g(k=65) == SHAPE and g(E=0) == SHAPE and g(cap=0) == SHAPE


def test_binding_refusals(lib):
    import torch
    from microscaled_precision_moe_gb300 import ops
    bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
    x, w = torch.zeros(4, 64, dtype=bf), torch.ones(64)
    with pytest.raises(TypeError, match="x"):
        ops.add_rmsnorm(x.float(), w)
    with pytest.raises(TypeError, match="weight"):
        ops.add_rmsnorm(x, w.half())
    with pytest.raises(ValueError, match="weight"):
        ops.add_rmsnorm(x, w[:32])
    with pytest.raises(ValueError, match="residual"):
        ops.add_rmsnorm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="dense"):
        ops.add_rmsnorm(torch.zeros(64, 4, dtype=bf).t(), w)
    with pytest.raises(ValueError, match="32-value"):
        ops.add_rmsnorm(torch.zeros(4, 48, dtype=bf), torch.ones(48), quantize=True)
    with pytest.raises(ValueError, match="CUDA"):
        ops.add_rmsnorm(x, w)
    with pytest.raises(ValueError, match="y"):
        ops.add_rmsnorm(x, w, out={"y": torch.zeros(2, 64, dtype=bf)})
    with pytest.raises(ValueError, match="dh"):
        ops.add_rmsnorm_backward(x, x, torch.ones(4), w, dh=x[:, :32])
    with pytest.raises(ValueError, match="rstd"):
        ops.add_rmsnorm_backward(x, x, torch.ones(3), w)
    with pytest.raises(ValueError, match="CUDA"):
        ops.add_rmsnorm_backward(x, x, torch.ones(4), w)
    l = torch.zeros(4, 16)
    with pytest.raises(TypeError, match="logits"):
        ops.moe_route(l.half(), 2)
    with pytest.raises(ValueError, match="score"):
        ops.moe_route(l, 2, score="tanh")
    with pytest.raises(ValueError, match="bias"):
        ops.moe_route(l, 2, bias=torch.zeros(16))
    with pytest.raises(ValueError, match="bias"):
        ops.moe_route(l, 2, score="sigmoid", bias=torch.zeros(8))
    with pytest.raises(TypeError, match="token_mask"):
        ops.moe_route(l, 2, token_mask=torch.zeros(4))
    with pytest.raises(ValueError, match="token_mask"):
        ops.moe_route(l, 2, token_mask=torch.zeros(3, dtype=torch.bool))
    with pytest.raises(ValueError, match="CUDA"):
        ops.moe_route(l, 2)
    ids, c, n = torch.zeros(4, 2, dtype=i32), torch.zeros(16, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError, match="ids"):
        ops.moe_route_backward(l, ids[:3], c, n)
    with pytest.raises(ValueError, match="dprob"):
        ops.moe_route_backward(l, ids, c, n, dprob=torch.zeros(4, 3))
    with pytest.raises(TypeError, match="out"):
        ops.moe_route_backward(l, ids, c, n, out=torch.zeros(4, 16).half())
    with pytest.raises(ValueError, match="match"):
        ops.moe_combine_dprob(x, torch.zeros(128, 32, dtype=bf), ids.view(-1), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="inv_perm"):
        ops.moe_combine_dprob(x, torch.zeros(128, 64, dtype=bf), ids.view(-1)[:7], torch.zeros(4, 2))
    cap = ops.moe_row_capacity(4, 2, 4, 128)
    q, s = torch.zeros(4, 64, dtype=u8), torch.zeros(ops.scale_bytes(4, 2), dtype=u8)
    perm, seg = torch.zeros(cap, dtype=i32), torch.zeros(5, dtype=i32)
    with pytest.raises(ValueError, match="32-value"):
        ops.moe_gather_mxfp8(torch.zeros(4, 48, dtype=u8), s, perm, seg, 4, 2, cap)
    with pytest.raises(ValueError, match="seg_offsets"):
        ops.moe_gather_mxfp8(q, s, perm, seg[:4], 4, 2, cap)
    with pytest.raises(ValueError, match="out scales"):
        ops.moe_gather_mxfp8(q, s, perm, seg, 4, 2, cap, out=(torch.zeros(cap, 64, dtype=u8), s[:4]))
    with pytest.raises(ValueError, match="CUDA"):
        ops.moe_gather_mxfp8(q, s, perm, seg, 4, 2, cap)


def test_sizes_past_their_range_are_refused(lib):
    """Sizes that would wrap in the checks, or in the library's 32-bit arguments,
    are refused for what they are."""
    import torch
    from microscaled_precision_moe_gb300 import ops
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
    q, s = torch.zeros(4, 32, dtype=u8), torch.zeros(512, dtype=u8)
    perm, seg = torch.zeros(128, dtype=i32), torch.zeros(5, dtype=i32)
    for E, cap, what in ((2 ** 63 - 1, 128, "seg_offsets"), (5, 128, "seg_offsets"), (0, 128, "at least 1"),
                         (-2 ** 63, 128, "at least 1"), (4, 0, "at least 1"), (4, -2 ** 62, "at least 1")):
        with pytest.raises(ValueError, match=what):
            ops.moe_gather_mxfp8(q, s, perm, seg, E, 2, cap)
    none = lambda dtype: torch.zeros(0, 2 ** 32 + 1, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="k = 4294967297"):
        ops.moe_combine_dprob(torch.zeros(0, 64, dtype=bf), torch.zeros(4, 64, dtype=bf), torch.zeros(0, dtype=i32),
                              none(torch.float32))
    with pytest.raises(ValueError, match="k = 4294967297"):
        ops.moe_route_backward(torch.zeros(0, 8), none(i32), torch.zeros(8, dtype=i32), torch.zeros(1, dtype=i32))
