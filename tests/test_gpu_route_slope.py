"""The gradient of sigmoid scores far from zero, where 1 - s is much smaller than s's last bit: each element of the
gradient is held to its own size, s (1 - s) |dw|.

exp, 1 + exp, the reciprocal, the complement and three products are each within an ulp or two: 16 x 2^-24 covers
them.  Renormalised, the slots' gradients are differences of terms of up to max |dw|, whose sums over k slots add k
roundings."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _slope(l):
    """s (1 - s) without a difference: exp(-|l|) / (1 + exp(-|l|))^2."""
    e = np.exp(-np.abs(l))
    return e / (1.0 + e) ** 2


def _case(T, E, k, low, high, dtype):
    g = torch.Generator().manual_seed(E + k)
    logits = (torch.rand(T, E, generator=g) * (high - low) + low).to(dtype)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    dw = (torch.rand(T, k, generator=g) + 0.5) * torch.randn(T, k, generator=g).sign()
    return logits, ids, dw


@pytest.mark.parametrize("E,k", [(1, 1), (16, 4), (60, 6), (64, 8), (256, 8), (384, 10), (512, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("span", [2.0, 30.0, 80.0])
def test_sigmoid_gradient_of_large_logits(E, k, dtype, span):
    T = 45
    logits, ids, dw = _case(T, E, k, -span, span, dtype)
    got = nv.nvfp4_moe_route_backward(logits.to(DEV), ids.to(DEV), dw.to(DEV), nv.NVFP4_ROUTE_SIGMOID, 1.5).cpu().double().numpy()
    want = np.zeros((T, E))
    np.put_along_axis(want, ids.numpy().astype(np.int64), 1.5 * dw.double().numpy(), axis=1)
    want *= _slope(logits.double().numpy())
    tol = 16 * 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(got - want) <= tol * np.abs(want) + 1e-37)


@pytest.mark.parametrize("E,k", [(16, 4), (60, 6), (256, 8), (512, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_renormalised_sigmoid_gradient_of_large_logits(E, k, dtype):
    T = 45
    logits, ids, dw = _case(T, E, k, -12.0, 30.0, dtype)
    flags = nv.NVFP4_ROUTE_SIGMOID | nv.NVFP4_ROUTE_RENORM
    got = nv.nvfp4_moe_route_backward(logits.to(DEV), ids.to(DEV), dw.to(DEV), flags, 1.5).cpu().double().numpy()
    l, at = logits.double().numpy(), ids.numpy().astype(np.int64)
    p = np.take_along_axis(1.0 / (1.0 + np.exp(-l)), at, 1)
    total = p.sum(1, keepdims=True)
    g = 1.5 * dw.double().numpy()
    ds = (g - (g * p).sum(1, keepdims=True) / total) / total
    want, size = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, at, ds, axis=1)
    np.put_along_axis(size, at, 2 * np.abs(g).max(1, keepdims=True) / total, axis=1)
    want, size = want * _slope(l), size * _slope(l)
    rounded = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= (k + 16) * 2.0 ** -24 * size + rounded + 1e-37)


def test_saturated_and_closed_logits_have_no_gradient():
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    logits = torch.tensor([[low, high, float("inf"), -float("inf"), float("nan"), 200.0, -200.0, 0.0]])
    ids = torch.arange(8, dtype=torch.int32).reshape(1, 8)
    got = nv.nvfp4_moe_route_backward(logits.to(DEV), ids.to(DEV), torch.ones(1, 8, device=DEV), nv.NVFP4_ROUTE_SIGMOID).cpu()
    assert got[0, :7].eq(0).all() and got[0, 7] == 0.25
