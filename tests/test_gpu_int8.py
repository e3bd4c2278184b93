"""8-bit quantize and products on the GPU.  Both are exact by definition -- the quantize bit for bit, the sums
as integers, then three 32-bit roundings in a fixed order -- so results are compared for equality."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 64), (5, 512), (2, 1024), (9, 1040), (4, 2048), (2, 4112), (3, 8192),
                                       (2, 16384), (2, 16400), (1, 40000), (700, 48)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_bit_exact(rows, cols, dtype):
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    x[0, cols // 2] = 0.0
    if rows > 2:
        x[1] = 0.0
        x[2] = x[2].sign() * 2.0 ** -124  # scale below the normal numbers
    x = x.to(dtype)
    q = nv.nvfp4_int8_quantize(x.to(DEV))
    want, s = ref.int8_rows(x.float().numpy())
    np.testing.assert_array_equal(q.scales.cpu().numpy(), s)
    np.testing.assert_array_equal(q.data.cpu().numpy(), want)


def test_quantize_every_tie_and_every_bf16():
    # multiples of half a step: ties go to the even integer
    x = torch.cat([torch.arange(-254, 255) / 2.0, torch.tensor([127.0, 0.0, 0.0])]).reshape(1, -1)
    q = nv.nvfp4_int8_quantize(x.to(DEV))
    np.testing.assert_array_equal(q.data.cpu().numpy(), np.rint(x.numpy()).astype(np.int8))
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)  # every finite non-negative bf16, against its negative
    v = (bits << 16).view(torch.float32)
    x = torch.stack([v, -v], dim=1).repeat(1, 8)
    q = nv.nvfp4_int8_quantize(x.bfloat16().to(DEV))
    want, s = ref.int8_rows(x.numpy())
    np.testing.assert_array_equal(q.data.cpu().numpy(), want)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), s)


def test_quantize_strided():
    x = torch.randn(6, 256, device=DEV)
    q = nv.nvfp4_int8_quantize(x[1:, 64:192])
    want, s = ref.int8_rows(x[1:, 64:192].cpu().numpy())
    np.testing.assert_array_equal(q.data.cpu().numpy(), want)


def _int8(rows, k, groups=1, seed=0, extreme=False):
    g = torch.Generator().manual_seed(seed + rows * 7 + k)
    lo = -128 if extreme else -127
    q = torch.randint(lo, 128, (groups * rows, k), generator=g, dtype=torch.int16).to(torch.int8)
    if extreme:
        q[0] = -128
    return nv.Int8Tensor(q.to(DEV), (torch.rand(groups * rows, generator=g) * 0.01 + 1e-4).to(DEV), rows, k, groups)


def _want(aq, asc, bq, bsc, dtype):
    acc = (aq.double() @ bq.double().t()).cpu().numpy().astype(np.int64)  # exact: below 2^53
    scale = (asc.cpu().numpy()[:, None] * bsc.cpu().numpy()[None, :]).astype(np.float32)
    return torch.from_numpy(acc.astype(np.float32) * scale).to(dtype)


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 64, 4096), (3, 100, 48), (8, 4096, 128), (16, 33, 1040), (17, 129, 256),
                                   (33, 64, 144), (48, 300, 512), (64, 1111, 2064), (65, 65, 80), (100, 257, 640),
                                   (128, 128, 128), (200, 700, 1296), (255, 510, 112), (256, 256, 384), (300, 513, 256),
                                   (700, 1030, 528), (1000, 2050, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product(M, N, K, dtype):
    a, b = _int8(M, K, seed=1), _int8(N, K, seed=2)
    got = nv.nvfp4_int8_gemm(a, b, dtype).cpu()
    assert torch.equal(got, _want(a.data, a.scales, b.data, b.scales, dtype))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_of_extreme_values(M):
    # -128 x -128 over the longest K: the sum reaches 2^31 - 2^18
    K = (1 << 17) - 16
    a, b = _int8(M, K, extreme=True), _int8(20, K, extreme=True)
    got = nv.nvfp4_int8_gemm(a, b, torch.float32).cpu()
    assert torch.equal(got, _want(a.data, a.scales, b.data, b.scales, torch.float32))


@pytest.mark.parametrize("M,N", [(0, 8), (5, 0), (5, 24)])
def test_product_empty(M, N):
    for K in (0, 32):
        a, b = _int8(M, K), _int8(N, K)
        got = nv.nvfp4_int8_gemm(a, b)
        assert got.shape == (M, N) and (K or not got.any())


@pytest.mark.parametrize("M,N,K", [(5, 70, 64), (300, 70, 64), (300, 512, 256)])
def test_product_into_a_slice(M, N, K):
    a, b = _int8(M, K), _int8(N, K)
    for lead, dtype in ((3, torch.bfloat16), (8, torch.bfloat16), (4, torch.float32)):
        out = torch.full((M, N + 2 * lead), 9.0, dtype=dtype, device=DEV)
        nv.nvfp4_int8_gemm(a, b, out=out[:, lead:lead + N])
        assert torch.equal(out[:, lead:lead + N].cpu(), _want(a.data, a.scales, b.data, b.scales, dtype))
        assert (out[:, :lead] == 9).all() and (out[:, lead + N:] == 9).all()


@pytest.mark.parametrize("T,k,E,N,K,skew", [(1, 1, 1, 64, 64, 0), (1, 4, 8, 130, 128, 0), (8, 8, 64, 256, 512, 1.1),
                                            (40, 2, 7, 96, 80, 0), (100, 6, 60, 200, 272, 0.7), (300, 4, 5, 512, 256, 1.5),
                                            (900, 2, 3, 300, 144, 0), (33, 1, 512, 48, 64, 0), (700, 8, 100, 260, 128, 1.1)])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_product_by_expert(T, k, E, N, K, skew, gather, dtype):
    g = torch.Generator().manual_seed(T)
    load = torch.arange(1, E + 1).float().pow(-skew)
    ids = torch.multinomial(load.expand(T, E), k, generator=g, replacement=k > E).to(torch.int32)
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    offsets, rows, pos = ref.plan(ids.numpy(), E)
    to = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(torch.int32).to(DEV)
    plan = nv.MoEPlan(to(offsets), to(rows), to(pos))
    a, b = _int8(T if gather else T * k, K, seed=3), _int8(N, K, E, seed=4)
    out = torch.full((T * k, N), 3.0, dtype=dtype, device=DEV)
    nv.nvfp4_int8_gemm(a, b, plan=plan, gather=gather, out=out)
    out = out.cpu()
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            src = torch.from_numpy(rows[lo:hi] // k) if gather else torch.arange(lo, hi)
            src = src.to(DEV)
            w = slice(e * N, (e + 1) * N)
            assert torch.equal(out[lo:hi], _want(a.data[src], a.scales[src], b.data[w], b.scales[w], dtype)), e
    assert (out[offsets[-1]:] == 3).all()  # rows without an expert are not written


def test_product_after_quantize_on_another_stream():
    x, w = torch.randn(37, 512, device=DEV).bfloat16(), torch.randn(300, 512, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        qx, qw = nv.nvfp4_int8_quantize(x), nv.nvfp4_int8_quantize(w)
        got = nv.nvfp4_int8_gemm(qx, qw, torch.float32)
    s.synchronize()
    assert torch.equal(got.cpu(), _want(qx.data, qx.scales, qw.data, qw.scales, torch.float32))
    # and the product is near the unquantized one: each factor is within half a step of 1 / 127 of its row's largest
    exact = x.double() @ w.double().t()
    step = (qx.scales[:, None].double() * w.double().abs().sum(1) + qw.scales.double() * x.double().abs().sum(1)[:, None]) / 2
    assert ((got.double() - exact).abs() <= step + 512 * (qx.scales[:, None] * qw.scales).double() + 1e-4).all()
