"""Gather, combine and combine's gradients on the GPU against 64-bit references.

A sum of n products in 32 bits is within n x 2^-24 of the sum of their magnitudes; a bf16 result adds one rounding
(2^-9 of it, doubled here)."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _plan(T, k, E, seed, holes=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, k, generator=g) < holes] = -1
    offsets, rows, pos = ref.plan(ids.numpy(), E)
    to = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(torch.int32).to(DEV)
    return nv.MoEPlan(to(offsets), to(rows), to(pos)), pos


CASES = [(1, 1, 8, 0.0), (1, 8, 4096, 0.0), (5, 8, 2056, 0.3), (33, 6, 64, 0.0), (100, 9, 264, 0.5), (7, 32, 1000, 0.1),
         (3, 4, 16392, 0.0), (64, 2, 520, 1.0)]


@pytest.mark.parametrize("T,k,D,holes", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(T, k, D, holes, dtype, weighted):
    plan, pos = _plan(T, k, 11, T + k, holes)
    y = torch.randn(T * k, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    if holes:  # rows that no slot has are not read
        y[(plan.rows < 0).cpu()] = float("nan")
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(2))
    got = nv.nvfp4_moe_combine(y.to(DEV), plan, w.to(DEV) if weighted else None).cpu().double().numpy()
    rows = np.where((pos >= 0)[:, :, None], y.double().numpy()[np.maximum(pos, 0)], 0.0)
    terms = rows * (w.double().numpy()[:, :, None] if weighted else 1.0)
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    tol = k * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("T,k,D,holes", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine_backward(T, k, D, holes, dtype):
    plan, pos = _plan(T, k, 11, T + k, holes)
    g = torch.Generator().manual_seed(1)
    y, dout = torch.randn(T * k, D, generator=g).to(dtype), torch.randn(T, D, generator=g).to(dtype)
    w = torch.rand(T, k, generator=g)
    dy, dw = nv.nvfp4_moe_combine_backward(dout.to(DEV), y.to(DEV), plan, w.to(DEV))
    yd, dd, wd = y.double().numpy(), dout.double().numpy(), w.double().numpy()
    rows = np.where((pos >= 0)[:, :, None], yd[np.maximum(pos, 0)], 0.0)
    terms = rows * dd[:, None, :]
    # a lane adds at most D / 32 products in turn, then eight levels of partial sums
    assert np.all(np.abs(dw.cpu().double().numpy() - terms.sum(2)) <= (D / 32 + 8) * 2.0 ** -24 * np.abs(terms).sum(2))
    want = np.zeros((T * k, D))
    for t in range(T):
        for j in range(k):
            if pos[t, j] >= 0:
                want[pos[t, j]] = wd[t, j] * dd[t]
    tol = (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(want)
    assert np.all(np.abs(dy.cpu().double().numpy() - want) <= tol)


@pytest.mark.parametrize("T,k,D,holes", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gather(T, k, D, holes, dtype):
    plan, _ = _plan(T, k, 11, T + k, holes)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(4)).to(dtype)
    got = nv.nvfp4_moe_gather(x.to(DEV), plan).cpu()
    rows = plan.rows.cpu().long()
    want = torch.where((rows >= 0)[:, None], x[rows.clamp(min=0) // k], torch.zeros((), dtype=dtype))
    assert torch.equal(got, want)


def test_strides_and_another_stream():
    plan, pos = _plan(24, 4, 11, 3)
    x = torch.randn(24, 512, device=DEV).bfloat16()[:, 64:320]
    y = torch.full((96, 300 - 12), 5.0, device=DEV, dtype=torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        nv.nvfp4_moe_gather(x, plan, out=y[:, 8:264])
        back = nv.nvfp4_moe_combine(y[:, 8:264], plan)
    s.synchronize()
    # four equal rows: the sum is exact in 32 bits and in bf16
    assert torch.equal(back, x * 4) and (y[:, :8] == 5).all() and (y[:, 264:] == 5).all()


def test_gather_and_combine_are_transposes():
    plan, _ = _plan(50, 5, 13, 8, 0.2)
    x, z = torch.randn(50, 96, device=DEV), torch.randn(250, 96, device=DEV)
    a = (nv.nvfp4_moe_gather(x, plan).double() * z.double()).sum()
    b = (x.double() * nv.nvfp4_moe_combine(z, plan).double()).sum()
    # 24000 products of order one; each combined element is within 5 x 2^-24 of its terms' magnitudes
    assert abs(a - b) <= 5 * 2.0 ** -24 * (nv.nvfp4_moe_gather(x, plan).abs().double() * z.abs().double()).sum()
