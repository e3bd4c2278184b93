"""The gradient of routing weights where one expert has nearly all of the score: its own gradient is then much
smaller than the weights' gradients, and is held to that size.

An element of the exact gradient is written as a sum over the other experts, s_i sum_j s_j (ds_i - ds_j), and likewise
for the renormalised weights, so that nothing cancels; the bound is the same sum of magnitudes.  exp of a difference
is off by its rounding, span x 2^-24; sums over E experts by neighbours, k slots, and about ten further operations,
each at most doubled by a sum of magnitudes: (span + k + 64) x 2^-24 covers them."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _renorm(p, dw):
    """(gradient, bound) of the weights p_i / sum p for the scores p."""
    total = p.sum(1) + 1e-20
    g, size = np.zeros_like(p), np.zeros_like(p)
    for i in range(p.shape[1]):
        for j in range(p.shape[1]):
            if j != i:
                g[:, i] += p[:, j] * (dw[:, i] - dw[:, j])
                size[:, i] += p[:, j] * 2 * np.abs(dw).max(1)
        g[:, i] += 1e-20 * dw[:, i]
        size[:, i] += 1e-20 * np.abs(dw[:, i])
    return g / total[:, None] ** 2, size / total[:, None] ** 2


def _softmax(l, at, ds, size):
    """(gradient, bound) of the logits from those of the chosen scores."""
    e = np.exp(l - l.max(1, keepdims=True))
    s = e / e.sum(1, keepdims=True)
    full, mags = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(full, at, ds, 1)
    np.put_along_axis(mags, at, size, 1)
    d, bound = np.zeros_like(s), np.zeros_like(s)
    for j in range(s.shape[1]):
        d += s * s[:, j:j + 1] * (full - full[:, j:j + 1])
        bound += np.where(np.arange(s.shape[1]) != j, s * s[:, j:j + 1] * (mags + mags[:, j:j + 1]), 0.0)
    return d, bound


def _case(T, E, k, margin, dtype):
    g = torch.Generator().manual_seed(E * 100 + k)
    logits = torch.randn(T, E, generator=g)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    lead = torch.where(torch.arange(T) % 4 == 3, torch.randint(0, E, (T,), generator=g), ids[torch.arange(T), torch.arange(T) % k].long())
    logits[torch.arange(T), lead] += margin     # (of every fourth token an expert that may not be chosen)
    dw = (torch.rand(T, k, generator=g) + 0.5) * torch.randn(T, k, generator=g).sign()
    return logits.to(dtype), ids, dw


@pytest.mark.parametrize("E,k", [(2, 1), (16, 4), (60, 6), (64, 8), (160, 1), (256, 8), (512, 32)])
@pytest.mark.parametrize("margin", [0.0, 6.0, 20.0, 60.0])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_softmax_gradient_of_a_leading_expert(E, k, margin, renorm, dtype):
    T = 45
    logits, ids, dw = _case(T, E, k, margin, dtype)
    got = nv.nvfp4_moe_route_backward(logits.to(DEV), ids.to(DEV), dw.to(DEV), nv.NVFP4_ROUTE_RENORM if renorm else 0, 1.5)
    got = got.cpu().double().numpy()
    l, at, w = logits.double().numpy(), ids.numpy().astype(np.int64), 1.5 * dw.double().numpy()
    e = np.exp(l - l.max(1, keepdims=True))
    p = np.take_along_axis(e / e.sum(1, keepdims=True), at, 1)
    ds, size = _renorm(p, w) if renorm else (w, np.abs(w))
    want, bound = _softmax(l, at, ds, size)
    tol = (np.ptp(l, axis=1).max() + k + 64) * 2.0 ** -24
    rounded = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= tol * bound + rounded + 1e-36)


@pytest.mark.parametrize("E,k", [(2, 1), (16, 4), (60, 6), (256, 8), (512, 32)])
@pytest.mark.parametrize("margin", [0.0, 20.0, 40.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_renormalised_sigmoid_gradient_of_a_leading_expert(E, k, margin, dtype):
    T = 45
    logits, ids, dw = _case(T, E, k, margin, dtype)
    logits = (logits.float() - margin).to(dtype)    # the others are small, the leading one is near one half
    got = nv.nvfp4_moe_route_backward(logits.to(DEV), ids.to(DEV), dw.to(DEV),
                                      nv.NVFP4_ROUTE_RENORM | nv.NVFP4_ROUTE_SIGMOID, 1.5).cpu().double().numpy()
    l, at, w = logits.double().numpy(), ids.numpy().astype(np.int64), 1.5 * dw.double().numpy()
    s = 1 / (1 + np.exp(-l))
    slope = s / (1 + np.exp(l))
    ds, size = _renorm(np.take_along_axis(s, at, 1), w)
    want, bound = np.zeros_like(s), np.zeros_like(s)
    np.put_along_axis(want, at, ds * np.take_along_axis(slope, at, 1), 1)
    np.put_along_axis(bound, at, size * np.take_along_axis(slope, at, 1), 1)
    rounded = 2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0
    assert np.all(np.abs(got - want) <= (k + 64) * 2.0 ** -24 * bound + rounded + 1e-36)
