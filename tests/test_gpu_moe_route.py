"""Routing, its gradient and the plan on the GPU against the 64-bit references.

A score is a handful of 32-bit operations on exact inputs: exp of an argument below 40 in magnitude (its rounding
alone is 40 x 2^-24 relative), a sum of ten levels, divisions; 64 x 2^-24 < 4e-6 covers one, twice that a ratio."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
RTOL = 8e-6
DEV = "cuda"


def _flags(sigmoid, renorm, sum2=False):
    return (nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0) | (nv.NVFP4_ROUTE_RENORM if renorm else 0) | \
        (nv.NVFP4_ROUTE_GROUP_SUM2 if sum2 else 0)


def _logits(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * std).to(dtype)


def _check_plan(plan, ids, E):
    offsets, rows, pos = ref.plan(ids, E)
    np.testing.assert_array_equal(plan.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(plan.rows.cpu().numpy(), rows)
    np.testing.assert_array_equal(plan.pos.cpu().numpy(), pos)


def _check(logits, k, bias=None, sigmoid=False, renorm=False, sum2=False, groups=1, group_k=1, scale=1.0, dev_logits=None):
    E = logits.shape[1]
    x = logits.to(DEV) if dev_logits is None else dev_logits
    ids, w, plan = nv.nvfp4_moe_route(x, k, _flags(sigmoid, renorm, sum2), None if bias is None else bias.to(DEV), groups,
                                      group_k, scale)
    l64 = logits.double().numpy()
    rids, rw, clear = ref.route(l64, k, sigmoid, renorm, sum2, None if bias is None else bias.double().numpy(), groups,
                                group_k, scale)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    assert clear.mean() > 0.5 or len(clear) < 20  # most tokens say something about the choice
    np.testing.assert_array_equal(ids[clear], rids[clear])
    # weights of the ids it chose, unclear tokens too
    np.testing.assert_allclose(w, ref.route_weights(l64, ids.astype(np.int64), sigmoid, renorm, scale), rtol=RTOL, atol=1e-30)
    np.testing.assert_array_equal(w[ids < 0], 0.0)
    _check_plan(plan, ids, E)
    return ids, w


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (16, 4), (17, 17), (60, 6), (64, 8), (100, 10), (160, 6), (256, 8),
                                 (384, 8), (512, 22), (512, 32), (40, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_sizes(E, k, dtype, sigmoid):
    for T in (1, 5, 67):
        # (bf16 logits tie often: the lower index wins)
        _check(_logits(T, E, dtype, E + T), k, sigmoid=sigmoid, renorm=T != 5, scale=2.5 if T == 67 else 1.0)


@pytest.mark.parametrize("E,groups,group_k,k", [(64, 8, 4, 8), (256, 8, 4, 8), (160, 8, 3, 6), (60, 4, 1, 5), (16, 16, 3, 2),
                                                (512, 16, 2, 32), (384, 3, 2, 8), (33, 11, 5, 4)])
@pytest.mark.parametrize("sum2", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_groups_and_bias(E, groups, group_k, k, sum2, sigmoid):
    bias = torch.round(torch.randn(E, generator=torch.Generator().manual_seed(9)) * 20) * 1e-3
    for T in (3, 64, 130):
        _check(_logits(T, E, torch.float32, T), k, bias, sigmoid, True, sum2, groups, group_k, 2.5)
        _check(_logits(T, E, torch.bfloat16, T + 1), k, None, sigmoid, False, sum2, groups, group_k)


@pytest.mark.parametrize("T", [64, 65, 1000, 4099, 20000])
def test_route_many_tokens(T):
    # one workgroup, one step a chunk, several steps a chunk; a ragged end
    logits = _logits(T, 48, torch.float32, 1)
    ids, w, plan = nv.nvfp4_moe_route(logits.to(DEV), 4)
    top = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :4]
    np.testing.assert_array_equal(ids.cpu().numpy(), top.numpy())
    _check_plan(plan, top.numpy(), 48)


@pytest.mark.parametrize("E", [5, 64, 250])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_closed_experts(E, sigmoid, dtype):
    g = torch.Generator().manual_seed(E)
    logits = _logits(40, E, dtype, 4)
    logits[torch.rand(40, E, generator=g) < 0.6] = -float("inf")
    logits[3] = -float("inf")                # no expert at all
    logits[4] = float("nan")                 # likewise
    logits[5] = torch.finfo(dtype).min       # the type's lowest value is an ordinary logit
    logits[6, 0], logits[6, 1] = float("inf"), float("nan")
    logits[7] = -float("inf")
    logits[7, E - 1] = 1.0                   # one expert only
    k = min(4, E)
    ids, w = _check(logits, k, sigmoid=sigmoid, renorm=True)
    assert (ids[3] == -1).all() and (ids[4] == -1).all() and (w[3] == 0).all()
    assert ids[6, 0] == 0 and ids[7].tolist() == [E - 1] + [-1] * (k - 1) and w[7, 0] == 1.0
    if not sigmoid:
        assert ids[5].tolist() == list(range(k))
    if E % 5 == 0:
        _check(logits, 1, sigmoid=sigmoid, groups=5, group_k=2, sum2=True)


def test_route_ties_take_the_lower_index():
    logits = torch.zeros(6, 96)
    ids, w = _check(logits, 8, renorm=True)
    assert (ids == np.arange(8)).all() and np.allclose(w, 1 / 8)
    logits[:, 50] = 1.0
    ids, _ = _check(logits, 3, groups=6, group_k=2)   # group 3 (48..63) leads, then group 0
    assert (ids == [50, 0, 1]).all()
    bias = torch.zeros(96)
    bias[7], bias[90] = float("-inf"), float("nan")   # closed by the bias
    bias[10] = -1e-3
    ids, _ = _check(logits, 12, bias=bias)
    assert ids[0].tolist() == [50, 0, 1, 2, 3, 4, 5, 6, 8, 9, 11, 12]


def test_route_strided_logits_and_slices():
    big = _logits(70, 300, torch.bfloat16, 8).to(DEV)
    for lo, hi in ((0, 256), (1, 257), (3, 64)):   # row starts off 16 bytes
        part = big[5:, lo:hi]
        _check(part.cpu(), 6, dev_logits=part, sigmoid=True, renorm=True)


@pytest.mark.parametrize("slots", [(0, 4), (1, 1), (700, 6), (1025, 4), (3000, 8), (40000, 3)])
@pytest.mark.parametrize("E", [1, 37, 512])
def test_plan_of_given_ids(slots, E):
    T, k = slots
    ids = torch.randint(-2, E + 3, (T, k), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    if T:
        ids[T // 2] = 2**31 - 1
        ids[-1] = -2**31
    plan = nv.nvfp4_moe_plan(ids.to(DEV), E)
    _check_plan(plan, np.where((ids.numpy() < 0) | (ids.numpy() >= E), -1, ids.numpy()), E)


@pytest.mark.parametrize("E,k", [(1, 1), (7, 3), (60, 6), (64, 8), (160, 6), (384, 8), (512, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_backward(E, k, sigmoid, renorm, dtype):
    T = 37
    logits = _logits(T, E, dtype, 21)
    if E > 7:
        logits[torch.rand(T, E, generator=torch.Generator().manual_seed(2)) < 0.2] = -float("inf")
        logits[9] = -float("inf")
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(3))
    f = _flags(sigmoid, renorm)
    ids, w, _ = nv.nvfp4_moe_route(logits.to(DEV), k, f, scale=1.5, with_plan=False)
    got = nv.nvfp4_moe_route_backward(logits.to(DEV), ids, dw.to(DEV), f, 1.5).cpu().double().numpy()
    l64, rids = logits.double().numpy(), ids.cpu().numpy().astype(np.int64)
    want = ref.route_backward(l64, rids, dw.double().numpy(), sigmoid, renorm, 1.5)
    s, _ = ref.scores(l64, sigmoid)
    total = np.where(rids >= 0, np.take_along_axis(s, np.maximum(rids, 0), 1), 0).sum(1, keepdims=True) + 1e-20
    # every term of a gradient is at most score x 1.5 |dw| (/ total), formed in a few 32-bit operations
    bound = 4 * RTOL * s * 2 * 1.5 * np.abs(dw.numpy()).max(1, keepdims=True) / (total if renorm else 1.0)
    bound = np.where(total > 1e-10, bound, 0.0)
    assert np.all(np.abs(got - want) <= bound + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0) + 1e-35)


def test_route_backward_strided_and_foreign_ids():
    logits = _logits(20, 90, torch.float32, 5)
    ids = torch.full((20, 3), -1, dtype=torch.int32)
    ids[:, 0] = torch.arange(20) * 4
    ids[:, 1] = 90          # not an expert
    ids[5] = 11             # one expert three times: its gradients add
    dw = torch.randn(20, 3, generator=torch.Generator().manual_seed(3))
    wide, out = torch.zeros(20, 128, device=DEV), torch.full((20, 100), 7.0, device=DEV)
    wide[:, 1:91] = logits.to(DEV)
    nv.nvfp4_moe_route_backward(wide[:, 1:91], ids.to(DEV), dw.to(DEV), out=out[:, 3:93])
    rids = np.where(ids.numpy() == 90, -1, ids.numpy()).astype(np.int64)
    want = ref.route_backward(logits.double().numpy(), rids, dw.double().numpy(), False, False, 1.0)
    np.testing.assert_allclose(out[:, 3:93].cpu().numpy(), want, rtol=1e-5, atol=1e-6)
    assert (out[:, :3] == 7).all() and (out[:, 93:] == 7).all()


def test_route_on_another_stream_and_twice():
    logits = _logits(3000, 128, torch.bfloat16, 6).to(DEV)
    first = nv.nvfp4_moe_route(logits, 8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        second = nv.nvfp4_moe_route(logits, 8)
    s.synchronize()
    for a, b in zip((first[0], first[1], first[2].offsets, first[2].rows, first[2].pos),
                    (second[0], second[1], second[2].offsets, second[2].rows, second[2].pos)):
        assert torch.equal(a, b)
