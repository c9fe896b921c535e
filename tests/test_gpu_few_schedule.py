"""The few-token layer where a block first takes a part of a cut task and then whole tasks of the same product.

A product's tasks (256 weight rows of a group of an expert's rows) go around the blocks; where a third of a round at most is
left over, those are cut along the reduction.  Each case is built from the number of SMs, and the schedule that it is for is
worked out here and asserted."""
import numpy as np
import pytest
import torch

from oracle import quant as Q
from tests.gpu_util import need_gpu
from tests.test_gpu_few import _compare, _kind, _rows, _route, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def _cut(groups, tiles, steps, blocks):
    """(tasks, how many of them are cut, in how many parts)"""
    tasks = groups * tiles
    left = tasks % blocks
    parts = min(blocks // left, 8, steps // 2) if left else 1
    return tasks, left if parts >= 3 else 0, parts


def _products(kind, groups, H, I, blocks):
    step = 256 if kind == "nvfp4" else 128
    return _cut(groups, I // 128, H // step, blocks), _cut(groups, H // 256, I // step, blocks)


def _groups(kind, nb, R, E, H, I, wanted):
    """The number of groups at which the wanted products have a cut task in front of whole ones."""
    blocks = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    for g in range(E, E + (R - E) // nb + 1):
        p = _products(kind, g, H, I, blocks)
        if all(p[w][1] > 0 and p[w][0] > blocks for w in wanted):
            return g, p
    raise AssertionError(f"no number of groups cuts the tasks of {kind} {H} x {I} on {blocks} blocks")


def _slots(T, k, E, nb, groups, seed):
    """ids, prob [T, k]: E experts with `groups` groups of up to nb rows in all, the last group of each ragged; the slots that
    are left over weigh nothing."""
    rng = np.random.default_rng(seed)
    each = np.full(E, groups // E) + (np.arange(E) < groups % E)
    spare = T * k - int(((each - 1) * nb).sum())
    last = np.minimum(rng.integers(1, nb + 1, E), spare // E)
    rows = (each - 1) * nb + last
    assert (last >= 1).all() and rows.sum() <= T * k and int(np.ceil(rows / nb).sum()) == groups
    slots = np.full(T * k, -1)
    slots[rng.permutation(T * k)[:rows.sum()]] = np.repeat(np.arange(E), rows)
    prob = np.where(slots >= 0, rng.random(T * k) + 0.1, 0.0).astype(np.float32)
    ids = np.maximum(slots, 0).astype(np.int32)
    return torch.from_numpy(ids.reshape(T, k)).cuda(), torch.from_numpy(prob.reshape(T, k)).cuda()


@pytest.mark.parametrize("kind,T,k,E,H,I,wanted", [
    ("nvfp4", 16, 40, 4, 1792, 1792, (0, 1)),      # both products, groups of 16 rows
    ("mxfp8", 16, 40, 4, 1792, 1792, (0, 1)),
    ("nvfp4", 5, 150, 4, 4096, 512, (0,)),         # in eight parts
    ("mxfp8", 16, 60, 4, 1024, 2048, (1,)),
    ("nvfp4", 64, 16, 4, 2304, 2304, (0, 1)),      # groups of 64 rows
    ("mxfp8", 64, 16, 4, 2304, 2304, (0, 1)),
    ("mxfp8", 40, 24, 6, 1280, 896, (0,)),         # groups of 48
])
def test_a_cut_task_in_front_of_whole_ones(kind, T, k, E, H, I, wanted):
    from microscaled_precision_moe_gb300 import ops
    nb = 64 if T >= 64 else (T + 15) // 16 * 16
    groups, products = _groups(kind, nb, T * k, E, H, I, wanted)
    for w in wanted:
        tasks, cut, parts = products[w]
        assert cut > 0 and parts >= 3 and tasks - cut > 0
    (w1, w2), exact = _weights(kind, E, H, I, seed=H + T)
    x = _rows(T, H, seed=T)
    ids, prob = _slots(T, k, E, nb, groups, seed=groups)
    out = ops.moe_few_tokens(_kind(kind), x, ids, prob, w1, w2, E, I)
    _compare(out, x, ids, prob, exact, kind)
    for _ in range(3):
        assert torch.equal(ops.moe_few_tokens(_kind(kind), x, ids, prob, w1, w2, E, I), out)


def _coded_nvfp4(E, R, K, seed):
    """NVFP4 weights written down as codes (rows longer than the library's own quantiser takes): for the call and decoded."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (E * R, K // 2), dtype=np.uint8)
    s = rng.integers(0x28, 0x50, (E * R, K // 16), dtype=np.uint8)       # E4M3: 0.25 to 7.5
    ts = (rng.uniform(0.5, 2.0, E) / K ** 0.5 / 8).astype(np.float32)
    d = Q.nvfp4_dequantize(q, s, np.repeat(ts.astype(np.float64), R)).reshape(E, R, K)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return (dev(q), dev(Q.swizzle_scales(s)), dev(ts)), d


@pytest.mark.parametrize("T,H,I", [(1, 16384, 256), (3, 8448, 512), (17, 256, 16384), (2, 1024, 12032), (64, 16384, 256)])
def test_nvfp4_weights_wider_than_the_quantiser_takes(T, H, I):
    """Up to the 16384 that the call accepts, on weights that another program has quantised."""
    from microscaled_precision_moe_gb300 import ops
    E, k = 3, 2
    (w1, e1), (w2, e2) = _coded_nvfp4(E, 2 * I, H, H + I), _coded_nvfp4(E, H, I, H + I + 1)
    x = _rows(T, H, seed=T)
    ids, prob = _route(T, E, k, T)
    out = ops.moe_few_tokens(_kind("nvfp4"), x, ids, prob, w1, w2, E, I)
    _compare(out, x, ids, prob, (e1, e2), "nvfp4")
    assert torch.equal(ops.moe_few_tokens(_kind("nvfp4"), x, ids, prob, w1, w2, E, I), out)
