"""An adapter's h and g that are infinite, or finite beyond the largest bf16 number: both enter their second products as pieces."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests.test_gpu_adapter import _plan

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("T,K,N,R,L", [(1, 64, 48, 8, 1), (48, 4096, 2056, 16, 64), (90, 520, 264, 24, 4), (100, 264, 136, 64, 3),
                                       (700, 2048, 2056, 16, 2), (700, 264, 328, 128, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_h_and_g(T, K, N, R, L, dtype):
    """All operands are positive, so a sum with an infinite term is infinite, and no term of another row's sum is."""
    g = torch.Generator().manual_seed(T + R)
    ids = np.arange(T)[:, None] % L
    plan, _ = _plan(ids, L)
    positive = lambda *s: (torch.rand(*s, generator=g) + 0.5).to(BF16).to(DEV)
    w = nv.Adapters(positive(L * R, K), positive(L * N, R), torch.ones(L, device=DEV), R, K, N, L)
    x, dc = positive(T, K), positive(T, N)
    x[0, K // 2] = float("inf")
    c, h = nv.nvfp4_adapter(x, w, plan=plan, by_token=True, out_dtype=dtype, with_h=True)
    d = nv.nvfp4_adapter_backward(dc, x, w, h, plan=plan, by_token=True, dx_dtype=dtype)
    inf = float("inf")
    assert bool((h[0] == inf).all()) and bool((c[0] == inf).all()) and bool(torch.isfinite(c[1:]).all())
    assert bool((d.db.view(L, N, R)[0] == inf).all()) and bool(torch.isfinite(d.db.view(L, N, R)[1:]).all())
    assert bool(torch.isfinite(d.dx).all())
    x[0, K // 2] = 1.0
    dc[0, N // 2] = inf
    c, h = nv.nvfp4_adapter(x, w, plan=plan, by_token=True, out_dtype=dtype, with_h=True)
    d = nv.nvfp4_adapter_backward(dc, x, w, h, plan=plan, by_token=True, dx_dtype=dtype)
    assert bool((d.dx[0] == inf).all()) and bool(torch.isfinite(d.dx[1:]).all())
    assert bool((d.da.view(L, R, K)[0] == inf).all()) and bool(torch.isfinite(d.da.view(L, R, K)[1:]).all())


@pytest.mark.parametrize("T,K,N,R", [(1, 64, 48, 8), (200, 264, 520, 64), (700, 2048, 2056, 16)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_numbers_that_round_to_infinity(T, K, N, R, sign):
    """h = 2^128 - 2^118 and g the like are finite, and the nearest bf16 number would be infinite.  Every sum is of one product."""
    big, rest = 2.0 ** 127 * (2 - 2.0 ** -7), 1.5 * 2.0 ** 119  # (the largest bf16 number; together 2^128 - 2^118)
    a, b = torch.zeros(R, K), torch.zeros(N, R)
    a[R - 1, 3], a[R - 1, K - 2] = 2.0 ** 60, 2.0 ** 60
    b[5, R - 1], b[N - 1, R - 1] = 2.0 ** 60, 2.0 ** 60
    x, dc = torch.zeros(T, K), torch.zeros(T, N)
    x[T - 1, 3], x[T - 1, K - 2] = sign * big * 2.0 ** -60, sign * rest * 2.0 ** -60
    dc[T - 1, 5], dc[T - 1, N - 1] = sign * big * 2.0 ** -60, sign * rest * 2.0 ** -60
    small = 2.0 ** -120
    w = nv.Adapters(a.to(BF16).to(DEV), (b * small).to(BF16).to(DEV), torch.ones(1, device=DEV), R, K, N)
    x = x.to(BF16).to(DEV)
    c, h = nv.nvfp4_adapter(x, w, out_dtype=F32, with_h=True)
    assert float(h[T - 1, R - 1]) == sign * (big + rest)
    want = torch.zeros(T, N)
    want[T - 1, 5] = want[T - 1, N - 1] = sign * (big + rest) * 2.0 ** 60 * small
    assert torch.equal(c.cpu(), want)
    # the gradients of a call with small x and a, so that g is the large one
    w = nv.Adapters((a * small).to(BF16).to(DEV), b.to(BF16).to(DEV), torch.ones(1, device=DEV), R, K, N)
    d = nv.nvfp4_adapter_backward(dc.to(BF16).to(DEV), (x.float() * small).to(BF16), w, torch.zeros(T, R, device=DEV), dx_dtype=F32)
    want = torch.zeros(T, K)
    want[T - 1, 3] = want[T - 1, K - 2] = sign * (big + rest) * 2.0 ** 60 * small
    assert torch.equal(d.dx.cpu(), want)
    want = torch.zeros(R, K)
    want[R - 1, 3] = (big + rest) * (big * 2.0 ** -60 * small)
    want[R - 1, K - 2] = (big + rest) * (rest * 2.0 ** -60 * small)
    assert bool(((d.da.cpu() - want).abs() <= 2.0 ** -23 * want).all())  # (two roundings of the product's 48 bits at most)
    assert not d.db.any()
