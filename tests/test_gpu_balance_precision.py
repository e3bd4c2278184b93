"""The balance loss's gradient where no expert has more than half of a token's score, against 64-bit references.

The gradient of expert e is c p_e slope_e (n_e - mean), mean = sum p n.  A probability is off by r = (|l - max l| + E / 16 + 24)
x 2^-24 of itself (see test_gpu_moe_balance.py; a sigmoid's has no first term).  The difference is taken as (n_e - ref) -
sum p (n - ref) with an integer ref next to the mean: the first part is exact up to its rounding to 32 bits, the second
adds E / 16 + 6 roundings and r to each term of sum p |n - ref| <= sum p |n - mean| + |mean - ref|; and |mean - ref| is at most
one half and the mean's own error, or the mean itself where ref is 0."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import tune_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U


def _parts(logits, counts, tokens, k, coef, sigmoid):
    """(gradient, p slope c, |n - mean|, mean, sum p |n - mean|) of one sequence whose tokens are all live."""
    l = logits.double().numpy()
    E = l.shape[1]
    p = ref.probs(l, sigmoid)[0]
    slope = 1.0 / (1.0 + np.exp(l)) if sigmoid else 1.0
    n = counts.astype(np.float64)
    mean = (p * n).sum(axis=1, keepdims=True)
    scale = coef * E / (k * float(tokens) ** 2) * p * slope
    off = np.abs(n - mean)
    return scale * (n - mean), scale, off, mean, (p * off).sum(axis=1, keepdims=True)


def _gradient(logits, ids, coef, sigmoid, counts=None, tokens=None):
    flags = nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0
    L, I = logits.to(DEV), ids.to(DEV)
    b = nv.nvfp4_moe_balance(L, I, coef, flags=flags)
    if counts is not None:
        b = nv.MoEBalance(None, torch.from_numpy(counts).to(torch.int32).view(1, -1).to(DEV), None,
                          torch.tensor([tokens], dtype=torch.int32, device=DEV))
    d = nv.nvfp4_moe_balance_backward(L, I, b, coef, flags=flags)
    return d.cpu().double().numpy(), b.counts[0].cpu().numpy(), int(b.tokens)


@pytest.mark.parametrize("T,k", [(1, 1), (4, 1)])
@pytest.mark.parametrize("E", [300, 353, 401, 505])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_equal_scores(T, k, E, sigmoid):
    """Scores of 1 (or 1/2) and their sums are exact.  What is rounded: the factor c (3 times), 1 / sum and its product, the
    difference, the product with it: 8 x 2^-24 of p |n - mean|; and of the mean 1 / sum and its product, 3 x 2^-24 with room."""
    logits = torch.zeros(T, E)
    ids = (torch.arange(T * k, dtype=torch.int32) * 7).view(T, k)
    d, counts, tokens = _gradient(logits, ids, 2.0 ** -7, sigmoid)
    want, scale, off, mean, _ = _parts(logits, counts, tokens, k, 2.0 ** -7, sigmoid)
    assert np.all(np.abs(d - want) <= scale * (8 * U * off + 3 * U * mean))


@pytest.mark.parametrize("T,E,k", [(1, 300, 1), (1, 512, 1), (4, 300, 2), (8, 401, 1), (8, 512, 4), (100, 353, 8)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_scores_without_a_leader(T, E, k, sigmoid):
    g = torch.Generator().manual_seed(T + E)
    logits = torch.randn(T, E, generator=g) * 1.5
    ids = torch.argsort(logits, dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    assert ref.probs(logits.double().numpy(), sigmoid)[0].max() < 0.5
    d, counts, tokens = _gradient(logits, ids, 0.01, sigmoid)
    _check(d, logits, counts, tokens, k, 0.01, sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_large_counts_close_to_each_other(sigmoid):
    """Counts of many ranks: their differences decide, whatever their size."""
    T, E, k = 40, 64, 2
    g = torch.Generator().manual_seed(7)
    logits = torch.randn(T, E, generator=g) * 0.5
    ids = torch.argsort(logits, dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    counts = 20_000_000 + np.random.default_rng(1).integers(-300, 300, E)
    tokens = int(counts.sum()) // k
    d, _, _ = _gradient(logits, ids, 0.01, sigmoid, counts, tokens)
    _check(d, logits, counts, tokens, k, 0.01, sigmoid)


def _check(d, logits, counts, tokens, k, coef, sigmoid):
    E = logits.shape[1]
    want, scale, off, mean, spread = _parts(logits, counts, tokens, k, coef, sigmoid)
    l = logits.double().numpy()
    deep = 0.0 if sigmoid else float((l.max(axis=1) - l.min(axis=1)).max())
    r = (deep + E / 16 + 24) * U
    away = np.minimum(mean, 0.5 + 2 * r * mean)  # |mean - ref|
    assert np.all(np.abs(d - want) <= scale * ((r + 6 * U) * off + (r + (E / 16 + 6) * U) * (spread + away)) + 2.0 ** -126)
