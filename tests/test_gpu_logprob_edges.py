"""Token log probabilities and their gradient at the ends of what they take: masks of most of a large vocabulary at
the lowest temperature, against values known in closed form.

u = 2^-24; an exponential is off by 4 u, a logarithm by 4 u of its result at most.
"""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import need_gpu

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
