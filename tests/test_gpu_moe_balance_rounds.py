"""The balance loss where a workgroup takes several groups of live tokens in turn: long batches, and so many sequences that each
has one workgroup.  (The bounds of a probability and of the gradient are those of test_gpu_moe_balance.py.)"""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import tune_ref as ref
from tests.test_gpu_moe_balance import _inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U


@pytest.mark.parametrize("T,E,k,S", [(40000, 24, 2, 1), (45000, 17, 2, 300), (70001, 33, 3, 1), (36000, 130, 4, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_rounds(T, E, k, S, dtype, sigmoid, masked):
    logits, ids = _inputs(T, E, k, dtype, T + E, masked)
    flags = nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0
    got = nv.nvfp4_moe_balance(logits.to(DEV), ids.to(DEV), 0.01, flags=flags, sequences=S)
    l, i = logits.double().numpy(), ids.numpy()
    loss, counts, mean, tokens = ref.balance(l, i, 0.01, S, sigmoid)
    assert np.array_equal(got.counts[:].cpu().numpy(), counts) and np.array_equal(got.tokens.cpu().numpy(), tokens)
    deep = 0.0
    if not sigmoid:
        seen = l[~np.isnan(l).all(axis=1)]
        seen = np.where(np.isfinite(seen), seen, np.nan)
        deep = float((np.nanmax(seen, axis=1) - np.nanmin(seen, axis=1)).max())
    # the tokens of a sum in turn: those of a lane, its rows and waves (18), the workgroups (32 after another, 32 side by side)
    blocks = max(1, min(-(-(T // S) // 64), 256 // S))
    turns = -(-(T // S) // (64 * blocks)) + 18 + blocks / 32 + 32
    rel = (deep + E / 16 + 24 + turns) * U
    assert np.all(np.abs(got.probs.cpu().double().numpy() - mean) <= rel * mean + 2.0 ** -126)
    # five roundings of each term; the terms are added by 32 experts, then over all of these sums
    assert abs(float(got.loss) - loss) <= (rel + (5 + 6 + S * E / 32 + 20) * U) * abs(loss)
    given = torch.from_numpy(np.random.default_rng(T).standard_normal((T, E)) * 1e-7).to(dtype)
    d = nv.nvfp4_moe_balance_backward(logits.to(DEV), ids.to(DEV), got, 0.01, flags=flags, dlogits=given.to(DEV))
    want, tol = ref.balance_backward(l, i, counts, tokens, 0.01, sigmoid)
    total = want + given.double().numpy()
    assert np.all(np.abs(d.cpu().double().numpy() - total) <= tol + (2.0 ** -8 if dtype == torch.bfloat16 else U) * np.abs(total))
