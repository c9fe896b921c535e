"""The residual RMSNorm on the GPU against its fp64 definition, and its MXFP8
output byte for byte against the quantiser.

Bounds, derived from the arithmetic: a value rounded once to bf16 is off by at
most 2^-8 of itself; rstd is an fp32 function of an fp32 sum of K positive
squares whose longest chain of additions is below 80 (5e-6); sums with
cancellation are off by their chain length times 2^-24 of the sum of their
magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import norm as N
from oracle import quant as Q
from tests.gpu_util import need_gpu, np_bf16, u8, assert_bytes_equal

pytestmark = pytest.mark.gpu

BF16, RSTD, DX, DW = 2.0 ** -8, 5e-6, 1e-5, 2e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _ops():
    from microscaled_precision_moe_gb300 import ops
    return ops


def _rows(seed, M, K, pad=0, std=1.0, off=0):
    """bf16 [M, K] inside rows of K + pad elements, starting `off` elements
    into the buffer; every eighth row 100 times as large."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(M * (K + pad) + off, device="cuda", generator=g) * std
    v = v.to(torch.bfloat16)[off:].view(M, K + pad)[:, :K]
    v[::8] *= 100
    return v


def _weight(seed, K, f32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = 1.0 + 0.2 * torch.randn(K, device="cuda", generator=g)
    return w if f32 else w.to(torch.bfloat16)


def _within(got, want, tol, what):
    bad = np.abs(np.asarray(got, np.float64) - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} out of bounds, first {np.argwhere(bad)[0]}"


def _check_forward(o, x, w, r, eps, quantize):
    ops = _ops()
    xr = np_bf16(x), None if r is None else np_bf16(r)
    h, y, rstd = N.add_rmsnorm(xr[0], w.float().cpu().numpy(), xr[1], eps)
    _within(o["rstd"].cpu().numpy(), rstd, RSTD * rstd, "rstd")
    _within(np_bf16(o["y"]), y, (BF16 + 2 * RSTD) * np.abs(y) + 1e-38, "y")
    if r is not None:
        _within(np_bf16(o["h"]), h, (BF16 + 1e-6) * np.abs(h) + 1e-38, "h")
    if quantize:
        ref = ops.mxfp8_quantize(o["y"], colwise=False)
        assert_bytes_equal(u8(o["row_q"]), u8(ref["row_q"]), "codes")
        assert_bytes_equal(u8(o["row_s"]), u8(ref["row_s"]), "tiled scales")


# widths on both sides of every vector, block and thread-count boundary
@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (129, 96), (5, 2048), (64, 7168), (2, 4096), (2, 4128),
                                 (7, 8192), (2, 16384)])
@pytest.mark.parametrize("pad", [0, 8, 5])
def test_forward_with_quantised_output(M, K, pad):
    x, r = _rows(1, M, K, pad), _rows(2, M, K, pad, 3.0)
    w = _weight(3, K, K % 64 == 0)
    o = _ops().add_rmsnorm(x, w, residual=r, eps=1e-5, quantize=True)
    _check_forward(o, x, w, r, 1e-5, True)


@pytest.mark.parametrize("M,K,pad,off", [(1, 1, 0, 0), (4, 7, 0, 0), (33, 100, 0, 0), (9, 1003, 2, 1),
                                         (3, 2056, 0, 0), (2, 4097, 0, 0), (2, 16383, 0, 0), (5, 1544, 24, 0),
                                         (5, 512, 0, 3), (6, 520, 4, 4), (6, 1030, 0, 2)])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("res", [True, False])
def test_forward_any_width_pitch_and_alignment(M, K, pad, off, f32, res):
    x, r = _rows(4, M, K, pad, off=off), _rows(5, M, K, pad) if res else None
    w = _weight(6, K, f32)
    o = _ops().add_rmsnorm(x, w, residual=r)
    assert ("h" in o) == res
    _check_forward(o, x, w, r, 1e-6, False)


def test_codes_match_the_oracle_quantiser():
    x, w = _rows(7, 40, 256), _weight(8, 256, True)
    o = _ops().add_rmsnorm(x, w, quantize=True)
    codes, scales = Q.mxfp8_quantize_rowwise(np_bf16(o["y"]))[:2]
    assert_bytes_equal(u8(o["row_q"]), codes, "codes")
    assert_bytes_equal(Q.unswizzle_scales(u8(o["row_s"]), 40, 8), scales, "scales")


def test_only_the_outputs_asked_for_and_8_bits_alone():
    ops = _ops()
    x, w = _rows(9, 6, 128), _weight(10, 128, False)
    full = ops.add_rmsnorm(x, w, quantize=True)
    o = ops.add_rmsnorm(x, w, want_y=False, quantize=True)
    assert set(o) == {"rstd", "row_q", "row_s"}
    assert torch.equal(o["row_q"], full["row_q"]) and torch.equal(o["row_s"], full["row_s"])
    assert set(ops.add_rmsnorm(x, w)) == {"y", "rstd"}


@pytest.mark.parametrize("K,pad", [(96, 32), (100, 28)])
def test_nothing_outside_the_outputs_is_written(K, pad):
    M = 5
    buf = {n: torch.full((M + 2, K + pad), 7.0, dtype=torch.bfloat16, device="cuda") for n in ("y", "h", "dx")}
    view = {n: b[1:M + 1, :K] for n, b in buf.items()}
    x, r, w = _rows(11, M, K), _rows(12, M, K), _weight(13, K, True)
    o = _ops().add_rmsnorm(x, w, residual=r, out={"y": view["y"], "h": view["h"]})
    _ops().add_rmsnorm_backward(x, o["h"], o["rstd"], w, out=(view["dx"], torch.empty(K, device="cuda")))
    torch.cuda.synchronize()
    for b in buf.values():
        assert (b[0] == 7).all() and (b[-1] == 7).all() and (b[:, K:] == 7).all()


def test_outputs_made_together_do_not_overlap():
    x, r, w = _rows(63, 3, 96), _rows(64, 3, 96), _weight(65, 96, True)
    o = _ops().add_rmsnorm(x, w, residual=r, quantize=True)
    o["dx"], o["dw"] = _ops().add_rmsnorm_backward(x, o["h"], o["rstd"], w)
    want = {n: t.clone() for n, t in o.items()}
    assert all(t.is_contiguous() for t in o.values())
    for n in o:
        o[n].zero_()
        want[n].zero_()
        assert all(torch.equal(o[m], want[m]) for m in o)


@pytest.mark.parametrize("K", [2048, 7168, 1001])
def test_in_place_residual(K):
    ops = _ops()
    x, r, w = _rows(14, 70, K), _rows(15, 70, K), _weight(16, K, False)
    ref = ops.add_rmsnorm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    o = ops.add_rmsnorm(x2, w, residual=r2, out={"h": r2, "y": x2})
    assert torch.equal(o["h"], ref["h"]) and torch.equal(o["y"], ref["y"]) and o["h"] is r2
    dx, dw = ops.add_rmsnorm_backward(x, ref["h"], ref["rstd"], w, dh=r)
    r3 = r.clone()
    dx2, dw2 = ops.add_rmsnorm_backward(x, ref["h"], ref["rstd"], w, dh=r3, out=(r3, torch.empty_like(dw)))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("M,K", [(40, 100), (700, 176), (300, 1001), (200, 2048), (20, 9001), (20, 9008)])
@pytest.mark.parametrize("onto", ["dy", "dy2", "h", "dh"])
def test_in_place_gradient(M, K, onto):
    """dx in the place of any of its operands."""
    ops = _ops()
    t = {n: _rows(40 + i, M, K, std=1e-2 if n != "h" else 1.0) for i, n in enumerate(("dy", "dy2", "h", "dh"))}
    w = _weight(44, K, True)
    rstd = ops.add_rmsnorm(t["h"], w)["rstd"]
    ref = ops.add_rmsnorm_backward(t["dy"], t["h"], rstd, w, dy2=t["dy2"], dh=t["dh"])
    dx, dw = ops.add_rmsnorm_backward(t["dy"], t["h"], rstd, w, dy2=t["dy2"], dh=t["dh"],
                                      out=(t[onto], torch.empty(K, device="cuda")))
    assert dx is t[onto] and torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])


@pytest.mark.parametrize("M,K,pad,off", [(1, 257, 0, 3), (1, 100, 0, 7), (40, 300, 0, 1), (77, 241, 5, 2), (2000, 1003, 0, 0),
                                         (700, 521, 3, 5), (3, 2048, 0, 1), (300, 4161, 8, 0), (9, 8185, 1, 7),
                                         (9, 8186, 0, 1), (2, 16377, 0, 4), (2, 16378, 0, 4)])
@pytest.mark.parametrize("two,res,f32", [(True, True, False), (False, True, True), (True, False, True),
                                         (False, False, False)])
def test_rows_off_the_alignment(M, K, pad, off, two, res, f32):
    """All operands off by the same, forward and backward; the elements beside
    the rows are NaN and stay out of them."""
    ops = _ops()

    def rows(seed, std=1.0):
        buf = torch.full((M * (K + pad) + off + 9,), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = buf[off:off + M * (K + pad)].view(M, K + pad)[:, :K]
        v.copy_(_rows(seed, M, K, std=std))
        return v

    x, r, w = rows(50), rows(51, 3.0) if res else None, _weight(52, K, f32)
    o = ops.add_rmsnorm(x, w, residual=r, out={"y": rows(53), **({"h": rows(54)} if res else {})})
    _check_forward(o, x, w, r, 1e-6, False)
    h = o["h"] if res else x
    dy, dy2, dh = rows(55, 1e-2), rows(56, 1e-2) if two else None, rows(57, 1e-2) if res else None
    dx, dw = ops.add_rmsnorm_backward(dy, h, o["rstd"], w, dy2=dy2, dh=dh, out=(rows(58), torch.empty(K, device="cuda")))
    total = np_bf16(dy).astype(np.float64) + (np_bf16(dy2) if two else 0.0)
    rx, rw, mx, mw = N.add_rmsnorm_backward(total, np_bf16(h), o["rstd"].cpu().numpy(), w.float().cpu().numpy(),
                                            np_bf16(dh) if res else None)
    _within(np_bf16(dx), rx, BF16 * np.abs(rx) + DX * mx + 1e-38, "dx")
    _within(dw.cpu().numpy(), rw, DW * mw + 1e-38, "dw")


def test_a_row_of_nan_stays_out_of_its_neighbours():
    ops = _ops()
    M, K = 600, 1003
    h, dy, w = _rows(60, M, K), _rows(61, M, K, std=1e-2), _weight(62, K, True)
    ref = ops.add_rmsnorm(h, w)
    dref, _ = ops.add_rmsnorm_backward(dy, h, ref["rstd"], w, want_dw=False)
    h[300], dy[300] = float("nan"), float("nan")
    o = ops.add_rmsnorm(h, w)
    dx, _ = ops.add_rmsnorm_backward(dy, h, o["rstd"], w, want_dw=False)
    keep = [m for m in range(M) if m != 300]
    assert torch.equal(o["y"][keep], ref["y"][keep]) and torch.equal(dx[keep], dref[keep])
    assert torch.isnan(o["y"][300]).all() and torch.isnan(dx[300]).all()


def test_rows_of_zeros_infinities_and_nan():
    """A zero row gives zeros; NaN and infinities stay in their rows."""
    K = 256
    x, w = _rows(17, 8, K), _weight(18, K, True)
    x[2] = 0
    x[3, 5] = float("inf")
    x[4, 6] = float("nan")
    x[5] = 1e30                                       # the square sum leaves fp32's range
    o = _ops().add_rmsnorm(x, w, quantize=True)
    y, rstd = np_bf16(o["y"]), o["rstd"].cpu().numpy()
    assert not y[2].any() and abs(rstd[2] - 1e3) < 1e-2
    assert not u8(o["row_q"])[2].any()
    assert rstd[3] == 0 and np.isnan(y[3, 5]) and np.isnan(y[4]).all()
    assert rstd[5] == 0 and not y[5].any()
    keep = [0, 1, 6, 7]
    ref = _ops().add_rmsnorm(x[keep].contiguous(), w)
    assert torch.equal(o["y"][keep], ref["y"]) and torch.equal(o["rstd"][keep], ref["rstd"])


@pytest.mark.parametrize("M,K,pad,off", [(1, 32, 0, 0), (2, 1, 0, 0), (17, 100, 0, 0), (129, 2048, 0, 0),
                                         (40, 7168, 8, 0), (700, 64, 0, 0), (1500, 1544, 24, 0), (9, 1003, 2, 1),
                                         (3, 4104, 0, 0), (3, 16384, 0, 0), (2, 16383, 0, 0), (30, 1030, 0, 2)])
@pytest.mark.parametrize("two,res,f32", [(True, True, True), (False, True, False), (False, False, True)])
def test_backward(M, K, pad, off, two, res, f32):
    ops = _ops()
    h, w = _rows(20, M, K, pad, 2.0, off), _weight(21, K, f32)
    dy, dy2 = _rows(22, M, K, pad, 1e-2), _rows(23, M, K, pad, 1e-2) if two else None
    dh = _rows(24, M, K, pad, 1e-2) if res else None
    rstd = ops.add_rmsnorm(h, w)["rstd"]
    dx, dw = ops.add_rmsnorm_backward(dy, h, rstd, w, dy2=dy2, dh=dh)
    total = np_bf16(dy).astype(np.float64) + (np_bf16(dy2) if two else 0.0)
    rx, rw, mx, mw = N.add_rmsnorm_backward(total, np_bf16(h), rstd.cpu().numpy(), w.float().cpu().numpy(),
                                            np_bf16(dh) if res else None)
    _within(np_bf16(dx), rx, BF16 * np.abs(rx) + DX * mx + 1e-38, "dx")
    _within(dw.cpu().numpy(), rw, DW * mw + 1e-38, "dw")
    again = ops.add_rmsnorm_backward(dy, h, rstd, w, dy2=dy2, dh=dh)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    alone, none = ops.add_rmsnorm_backward(dy, h, rstd, w, dy2=dy2, dh=dh, want_dw=False)
    assert none is None and torch.equal(alone, dx)


def test_backward_against_differences_of_the_forward():
    """<dy, y> moves by <dx, v> along v: the kernels' own forward and backward,
    fp32 rows made of bf16 values, a step large enough for bf16's rounding."""
    ops = _ops()
    M, K, eps = 64, 512, 1e-2
    x, w = _rows(25, M, K), _weight(26, K, True)
    x[::8] /= 100
    v = torch.randn(M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(27)).to(torch.bfloat16)
    dy = _rows(28, M, K)
    lo, hi = (x.float() - 0.05 * v.float()).to(torch.bfloat16), (x.float() + 0.05 * v.float()).to(torch.bfloat16)
    f = [(ops.add_rmsnorm(t, w, eps=eps)["y"].double() * dy.double()).sum(1) for t in (lo, hi)]
    o = ops.add_rmsnorm(x, w, eps=eps)
    dx, _ = ops.add_rmsnorm_backward(dy, x, o["rstd"], w)
    want = (dx.double() * (hi.double() - lo.double())).sum(1)
    # y's rounding: K independent errors of at most 2^-9 |y dy| each, twice; the
    # step's third-order term is below 1 % of the change; six standard deviations
    noise = 6 * (2 * (2.0 ** -9 * o["y"].double() * dy.double()).square().sum(1)).sqrt()
    size = (dx.double() * (hi.double() - lo.double())).square().sum(1).sqrt() * 6
    assert ((f[1] - f[0] - want).abs() <= noise + 0.02 * size).all()


def test_other_stream_and_graph_capture():
    ops = _ops()
    x, r, w = _rows(30, 33, 1024), _rows(31, 33, 1024), _weight(32, 1024, False)
    ref = ops.add_rmsnorm(x, w, residual=r, quantize=True)
    dref = ops.add_rmsnorm_backward(x, ref["h"], ref["rstd"], w, dh=r)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o = ops.add_rmsnorm(x, w, residual=r, quantize=True)
        d = ops.add_rmsnorm_backward(x, o["h"], o["rstd"], w, dh=r)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o2 = ops.add_rmsnorm(x, w, residual=r, quantize=True)
        d2 = ops.add_rmsnorm_backward(x, o2["h"], o2["rstd"], w, dh=r)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a in (o, o2):
        assert all(torch.equal(a[n], ref[n]) for n in ref)
    for a in (d, d2):
        assert all(torch.equal(s, t) for s, t in zip(a, dref))


def test_offsets_past_32_bits():
    """The last rows of a matrix of more than 2^31 elements."""
    ops = _ops()
    M, K = 270000, 8192
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    x[:] = _rows(33, 1, K)
    tail = _rows(34, 130, K)
    x[-130:] = tail
    w = _weight(35, K, True)
    o = ops.add_rmsnorm(x, w, quantize=True)
    ref = ops.add_rmsnorm(tail.contiguous(), w)
    assert torch.equal(o["y"][-130:], ref["y"])
    q = ops.mxfp8_quantize(ref["y"], colwise=False)["row_q"]
    assert torch.equal(o["row_q"][-130:], q)
    dx, _ = ops.add_rmsnorm_backward(x, x, o["rstd"], w)
    dref, _ = ops.add_rmsnorm_backward(tail, tail, ref["rstd"], w)
    assert torch.equal(dx[-130:], dref)


@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("f32", [True, False])
def test_the_quantisers_bytes_of_nan_and_infinities(pad, f32):
    """The 8-bit copy is the quantiser's whatever the rows hold: one infinity
    (rstd 0: a NaN among zeros), runs of them, whole blocks, NaN weights."""
    ops = _ops()
    inf, nan = float("inf"), float("nan")
    x, w = _rows(70, 12, 256, pad), _weight(71, 256, f32)
    x[1, 5] = inf
    x[2, 8:16] = inf
    x[3, 32:64] = inf
    x[4, 64:96:2] = inf
    x[5, 65:96:2] = -inf
    x[6, 100] = nan
    x[7, 0:32:2] = inf
    x[8, 3], x[8, 4] = inf, -inf
    for clear in (False, True):
        if clear:                                      # NaN weights in one column, a run, and a whole block
            w = w.clone()
            w[7] = w[40:48] = w[128:160] = w[161:192:2] = nan
            w[200] = inf
        o = ops.add_rmsnorm(x, w, quantize=True)
        ref = ops.mxfp8_quantize(o["y"], colwise=False)
        assert_bytes_equal(u8(o["row_q"]), u8(ref["row_q"]), "codes")
        assert_bytes_equal(u8(o["row_s"]), u8(ref["row_s"]), "tiled scales")
        alone = ops.add_rmsnorm(x, w, want_y=False, quantize=True)
        assert torch.equal(alone["row_q"], o["row_q"]) and torch.equal(alone["row_s"], o["row_s"])


def test_outputs_own_their_memory():
    """Growing one output in place leaves the others as they are."""
    ops = _ops()
    x, r, w = _rows(66, 3, 96), _rows(67, 3, 96), _weight(68, 96, True)
    o = ops.add_rmsnorm(x, w, residual=r, quantize=True)
    o["dx"], o["dw"] = ops.add_rmsnorm_backward(x, o["h"], o["rstd"], w)
    l = torch.randn(40, 16, device="cuda", generator=torch.Generator(device="cuda").manual_seed(69))
    for outs in (o, ops.moe_route(l, 2)):
        want = {n: t.clone() for n, t in outs.items()}
        for n in list(outs):
            grown = outs.pop(n)
            grown.resize_(4096).zero_()
            assert all(torch.equal(t, want[m]) for m, t in outs.items()), n


@pytest.mark.parametrize("M,K", [(40, 64), (40, 1024), (40, 1001), (9, 9000)])
def test_gradient_where_the_square_of_rstd_leaves_fp32(M, K):
    """A zero row under an eps of 1e-39 (rstd 3e19), and rows near 1e17."""
    ops = _ops()
    h, dy, w = _rows(80, M, K), _rows(81, M, K, std=1e-2), _weight(82, K, True)
    h[3] = 0
    h[5] = (h[5].float() * 1e17).to(torch.bfloat16)
    h[6] = (h[6].float() * 1e-20).to(torch.bfloat16)
    rstd = ops.add_rmsnorm(h, w, eps=1e-39)["rstd"]
    dx, dw = ops.add_rmsnorm_backward(dy, h, rstd, w)
    rx, rw, mx, mw = N.add_rmsnorm_backward(np_bf16(dy), np_bf16(h), rstd.cpu().numpy(), w.cpu().numpy())
    _within(np_bf16(dx), rx, BF16 * np.abs(rx) + DX * mx + 1e-38, "dx")
    _within(dw.cpu().numpy(), rw, DW * mw + 1e-38, "dw")
    assert float(rstd[3]) > 1e19 and torch.isfinite(dx).all()
