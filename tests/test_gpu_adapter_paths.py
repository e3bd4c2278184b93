"""Adapters on each way that a call can take (the bounds are those of test_gpu_adapter.py): one launch; rows of 16, with one
and several splits of K; rows of 64, with several splits; rows gathered by expert on each of them; and the gradients of rows in the
plan's order."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import tune_ref as ref
from tests.test_gpu_adapter import _bound, _factors, _ids, _plan

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U
F32, BF16 = torch.float32, torch.bfloat16


# tokens, K, N, rank, adapters, whose: small ranks on rows of 16 (several splits of 1024) and of 64 (several splits)
@pytest.mark.parametrize("T,K,N,R,L,kind", [
    (48, 4096, 2056, 8, 64, "each"), (48, 2056, 2056, 16, 64, "each"), (60, 4104, 1544, 32, 64, "each"), (16, 14336, 33, 24, 2, "each"),
    (700, 2048, 2056, 8, 2, "segments"), (1030, 4096, 1111, 16, 4, "segments"), (900, 1544, 2056, 32, 3, "segments"),
    (1500, 1032, 1032, 24, 1, "one")])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_small_ranks(T, K, N, R, L, kind, dtype):
    w, a, b, s = _factors(L, R, K, N, T + K)
    ids = _ids(T, L, kind, T + N)
    plan, rows = _plan(ids, L)
    g = torch.Generator().manual_seed(3)
    x, base = torch.randn(T, K, generator=g).to(BF16), torch.randn(T, N, generator=g).to(dtype)
    got, h = nv.nvfp4_adapter(x.to(DEV), w, base.to(DEV), plan=plan, by_token=True, with_h=True)
    want, h64, mag = ref.adapter(x.double().numpy(), a, b, s, ids[:, 0], base.double().numpy(), np.arange(T))
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= _bound(mag, K + 2 * R + 8, dtype, want))
    at = rows[:int((ids >= 0).sum())]
    hm = np.stack([np.abs(a[ids[t, 0]]) @ np.abs(x[t].double().numpy()) for t in at])
    assert np.all(np.abs(h[:len(at)].cpu().double().numpy() - h64[at]) <= K * U * hm)


# tokens, top_k, K, N, rank, experts: rows of 16 (M <= 16 experts) with several splits; rows of 64 with eight splits and with fewer
@pytest.mark.parametrize("T,k,K,N,R,E", [(16, 8, 4096, 1536, 16, 64), (33, 5, 2056, 1032, 32, 64), (50, 2, 1544, 520, 64, 16),
                                         (1024, 4, 2048, 1032, 16, 8), (1000, 3, 4096, 520, 32, 6), (900, 3, 1032, 2056, 8, 5),
                                         (700, 2, 520, 264, 128, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gathered_rows(T, k, K, N, R, E, dtype):
    w, a, b, s = _factors(E, R, K, N, T)
    g = np.random.default_rng(T)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    ids[g.random(T) < 0.2, k - 1] = -1
    plan, rows = _plan(ids, E)
    owner = np.where(rows >= 0, ids.reshape(-1)[np.maximum(rows, 0)], -1)
    gen = torch.Generator().manual_seed(3)
    x, base = torch.randn(T, K, generator=gen).to(BF16), torch.randn(T * k, N, generator=gen).to(dtype)
    want, h64, mag = ref.adapter(x.double().numpy(), a, b, s, owner, base.double().numpy(), np.maximum(rows, 0) // k)
    n = int((ids >= 0).sum())
    hm = np.stack([np.abs(a[owner[r]]) @ np.abs(x[rows[r] // k].double().numpy()) for r in range(n)])
    # (the splits of gathered rows may be others than those of rows in order)
    for rows_x, gather in ((x.to(DEV), True), (nv.nvfp4_moe_gather(x.to(DEV), plan), False)):
        got, h = nv.nvfp4_adapter(rows_x, w, base.to(DEV), plan=plan, gather=gather, with_h=True)
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= _bound(mag, K + 2 * R + 8, dtype, want))
        assert np.all(np.abs(h[:n].cpu().double().numpy() - h64[:n]) <= K * U * hm)
        assert torch.equal(got[n:].cpu(), base[n:])


# tokens, top_k, K, N, rank, experts, experts without rows
@pytest.mark.parametrize("T,k,K,N,R,E,idle", [(1, 2, 64, 48, 16, 4, 0), (16, 8, 520, 264, 16, 64, 9), (130, 2, 264, 520, 8, 6, 2),
                                              (700, 3, 264, 328, 32, 8, 1), (900, 2, 1032, 1544, 16, 5, 2), (500, 2, 328, 264, 40, 3, 0),
                                              (2000, 1, 264, 328, 72, 2, 0), (400, 4, 520, 264, 64, 12, 3), (600, 2, 264, 520, 128, 4, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_in_the_plans_order(T, k, K, N, R, E, idle, dtype):
    """As by expert: a token has several rows, the last ones of the plan are of no expert."""
    w, a, b, s = _factors(E, R, K, N, T + K)
    g = np.random.default_rng(T)
    ids = np.stack([g.permutation(E - idle)[:k] for _ in range(T)])
    ids[g.random(T) < 0.2, k - 1] = -1
    plan, rows = _plan(ids, E)
    owner = np.where(rows >= 0, ids.reshape(-1)[np.maximum(rows, 0)], -1)
    M, n = T * k, int((ids >= 0).sum())
    gen = torch.Generator().manual_seed(4)
    x, dc, dxb = (torch.randn(M, c, generator=gen).to(t) for c, t in ((K, BF16), (N, BF16), (K, dtype)))
    _, h = nv.nvfp4_adapter(x.to(DEV), w, plan=plan, with_h=True)
    got = nv.nvfp4_adapter_backward(dc.to(DEV), x.to(DEV), w, h, dx_base=dxb.to(DEV), plan=plan)
    _, h64, _ = ref.adapter(x.double().numpy(), a, b, s, owner, np.zeros((M, N)), np.arange(M))
    want, mag = ref.adapter_backward(dc.double().numpy(), x.double().numpy(), a, b, s, owner, h64, dxb.double().numpy())
    assert np.all(np.abs(got.dx.cpu().double().numpy() - want[0]) <= _bound(mag[0], N + 3 * R + 8, dtype, want[0]))
    assert torch.equal(got.dx[n:].cpu(), dxb[n:])
    assert np.all(np.abs(got.da.cpu().double().numpy().reshape(a.shape) - want[1]) <= (N + 3 * M + 8) * U * mag[1])
    assert np.all(np.abs(got.db.cpu().double().numpy().reshape(b.shape) - want[2]) <= (K + 3 * M + 8) * U * mag[2])
    idle_rows = slice((E - idle) * R, None)
    assert not got.da[idle_rows].any() and not got.db[(E - idle) * N:].any()
