"""The few-token layer's and the log probabilities' entry points reject bad
arguments on the host, before any launch (CPU only)."""
import ctypes as C

import pytest

FAKE, ODD = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    from microscaled_precision_moe_gb300 import build, _lib
    build.build()
    return _lib.load()


def _desc(**k):
    from microscaled_precision_moe_gb300 import _lib as L
    d = L.FewTokensDesc()
    d.kind, d.k, d.T, d.E, d.H, d.I = L.KIND_NVFP4, 2, 4, 8, 512, 256
    d.ldx = d.ldo = 512
    for f in ("x_dev", "ids_dev", "prob_dev", "w1_q_dev", "w1_s_dev", "w1_ts_dev", "w2_q_dev", "w2_s_dev", "w2_ts_dev",
              "out_dev", "ws_dev"):
        setattr(d, f, FAKE)
    d.ws_bytes = 1 << 40
    for n, v in k.items():
        setattr(d, n, v)
    return d


@pytest.mark.parametrize("status,change", [
    (1, dict(x_dev=None)), (1, dict(w1_ts_dev=None)), (1, dict(w2_ts_dev=None)), (1, dict(ws_dev=None)), (1, dict(out_dev=None)),
    (4, dict(kind=2)), (4, dict(kind=-1)),
    (2, dict(T=0)), (2, dict(T=65)), (2, dict(k=0)), (2, dict(k=257)), (2, dict(E=0)), (2, dict(E=1025)), (2, dict(H=384)),
    (2, dict(H=0)), (2, dict(H=16640, ldx=16640, ldo=16640)), (2, dict(I=128)), (2, dict(I=0)), (2, dict(ldx=504)), (2, dict(ldo=256)),
    (2, dict(ws_bytes=1 << 10)), (2, dict(T=2 ** 62)), (2, dict(E=2 ** 62)),
    (3, dict(ldx=516)), (3, dict(ldo=516)), (3, dict(x_dev=ODD)), (3, dict(out_dev=ODD)), (3, dict(w1_q_dev=ODD)),
    (3, dict(w2_s_dev=ODD)), (3, dict(ids_dev=FAKE + 2)), (3, dict(ws_dev=FAKE + 128))])
def test_few_tokens(lib, status, change):
    assert lib.mpm_moe_few_tokens(C.byref(_desc(**change)), None) == status


def test_few_tokens_null_and_sizes(lib):
    from microscaled_precision_moe_gb300 import _lib as L
    assert lib.mpm_moe_few_tokens(None, None) == 1
    size = lib.mpm_moe_few_tokens_workspace_bytes
    assert size(L.KIND_NVFP4, 4, 2, 8, 512, 256) > 0 and size(L.KIND_MXFP8, 64, 16, 1024, 16384, 16384) > 0
    assert size(L.KIND_MXFP8, 4, 2, 8, 512, 128) > 0
    for bad in ((2, 4, 2, 8, 512, 256), (0, 0, 2, 8, 512, 256), (0, 65, 2, 8, 512, 256), (0, 4, 0, 8, 512, 256),
                (0, 4, 2, 8, 500, 256), (0, 4, 2, 8, 512, 128), (0, 64, 17, 8, 512, 256), (1, 4, 2, 8, 512, 64)):
        assert size(*bad) == 0
    # every k and T of a shape: at least what fewer tokens take of each part
    one = size(L.KIND_NVFP4, 1, 8, 256, 7168, 2048)
    assert size(L.KIND_NVFP4, 64, 8, 256, 7168, 2048) > one


def _fwd(lib, logits=FAKE, dtype=0, T=4, V=100, ld=100, targets=FAKE, tt=1, temp=1.0, top=2, logp=FAKE, lse=FAKE, H=FAKE,
         ids=FAKE, tlp=FAKE):
    v = lambda p: None if p is None else C.c_void_p(p)
    return lib.mpm_token_logprob(v(logits), dtype, T, V, ld, v(targets), tt, temp, top, v(logp), v(lse), v(H), v(ids), v(tlp), None)


@pytest.mark.parametrize("status,change", [
    (1, dict(logits=None)), (1, dict(lse=None)), (1, dict(logp=None)), (1, dict(ids=None)), (1, dict(tlp=None)),
    (4, dict(dtype=2)), (4, dict(tt=2)),
    (2, dict(T=0)), (2, dict(V=0)), (2, dict(ld=99)), (2, dict(top=-1)), (2, dict(top=33)), (2, dict(V=1, top=2)),
    (2, dict(V=2 ** 31, ld=2 ** 31)), (2, dict(T=2 ** 31)), (2, dict(targets=None)),
    (2, dict(temp=0.0)), (2, dict(temp=-1.0)), (2, dict(temp=float("inf"))), (2, dict(temp=float("nan"))), (2, dict(temp=1e-4)),
    (3, dict(logits=FAKE + 1)), (3, dict(logits=FAKE + 2, dtype=1)), (3, dict(targets=FAKE + 4)), (3, dict(lse=FAKE + 2))])
def test_token_logprob(lib, status, change):
    assert _fwd(lib, **change) == status


def _bwd(lib, logits=FAKE, dtype=0, T=4, V=100, ld=100, targets=FAKE, tt=0, lse=FAKE, dlogp=FAKE, H=FAKE, dH=FAKE, temp=1.0,
         out=FAKE, odt=0, ldd=100):
    v = lambda p: None if p is None else C.c_void_p(p)
    return lib.mpm_token_logprob_backward(v(logits), dtype, T, V, ld, v(targets), tt, v(lse), v(dlogp), v(H), v(dH), temp, v(out),
                                          odt, ldd, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(logits=None)), (1, dict(lse=None)), (1, dict(out=None)), (1, dict(H=None)), (1, dict(targets=None)),
    (4, dict(dtype=3)), (4, dict(odt=-1)), (4, dict(tt=5)),
    (2, dict(T=0)), (2, dict(V=0)), (2, dict(ld=50)), (2, dict(ldd=99)), (2, dict(temp=0.0)), (2, dict(temp=2e3)),
    (3, dict(out=FAKE + 2, odt=1)), (3, dict(dlogp=FAKE + 1)), (3, dict(targets=FAKE + 2))])
def test_token_logprob_backward(lib, status, change):
    assert _bwd(lib, **change) == status


def test_structure_mirrors_the_header(lib):
    from microscaled_precision_moe_gb300 import _lib as L
    # two ints, four sizes, two pitches, eleven pointers and the workspace's size, without padding
    assert C.sizeof(L.FewTokensDesc) == 2 * 4 + 4 * 8 + 2 * 8 + 11 * 8 + 8


def _bwd_from(lib, logits=FAKE, dtype=0, T=4, V=100, ld=100, targets=FAKE, tt=0, logp=FAKE, lse=FAKE, dlogp=FAKE, H=FAKE, dH=FAKE,
              temp=1.0, out=FAKE, odt=0, ldd=100):
    v = lambda p: None if p is None else C.c_void_p(p)
    return lib.mpm_token_logprob_backward_from(v(logits), dtype, T, V, ld, v(targets), tt, v(logp), v(lse), v(dlogp), v(H), v(dH),
                                               temp, v(out), odt, ldd, None)


@pytest.mark.parametrize("status,change", [
    (1, dict(logits=None)), (1, dict(lse=None)), (1, dict(out=None)), (1, dict(H=None)), (1, dict(targets=None)),
    (1, dict(targets=None, dlogp=None)), (4, dict(dtype=3)), (4, dict(tt=5)), (2, dict(T=0)), (2, dict(ldd=99)), (2, dict(temp=0.0)),
    (3, dict(logp=FAKE + 2)), (3, dict(lse=FAKE + 2)), (3, dict(out=FAKE + 1))])
def test_token_logprob_backward_from(lib, status, change):
    assert _bwd_from(lib, **change) == status
