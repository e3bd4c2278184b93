"""The operators around the quantized products where their data is larger than the 256 MiB cache (they then read it
with other loads), block norms of rows above 4096 columns with several rows a workgroup, and 8-bit products of more
than a round of 256 x 256 tiles or of few rows an expert.

Tolerances are those of the small cases: a 32-bit sum of n products is within n x 2^-24 of their magnitudes, a bf16
result adds one rounding; 8-bit products are exact."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import test_gpu_block_norm as norm
from tests.test_gpu_int8 import _want

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
CACHE = 2 ** 28


@pytest.mark.parametrize("T,D", [(520, 4104), (515, 8192), (300, 16384)])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_norm_of_long_rows(T, D, xt, yt):
    norm._run(T, D, xt, yt, norm.ALL)


def test_norm_of_long_rows_with_a_gate_by_token():
    norm._run(260, 6152, BF16, BF16, ("y", "post", "pre", "token_gate"))


@pytest.mark.parametrize("T,D", [(65543, 520), (8195, 4096), (4099, 8192), (2049, 16384)])
def test_norm_beyond_the_cache(T, D):
    assert T * D * 8 >= CACHE
    g = torch.Generator(device=DEV).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)
    x, y, dx_out, dn, gate = (r(T, D).to(BF16) for _ in range(5))
    w_post, w_pre = 1 + 0.2 * r(D), 1 + 0.2 * r(D)
    f = nv.nvfp4_block_norm(x, y, w_post, gate, w_pre, 0.7)
    b = nv.nvfp4_block_norm_backward(dx_out, dn, x, y, f.rstd_post, f.rstd_pre, w_post, gate, w_pre, 0.7)
    # rows do not depend on how many there are
    for lo in (0, T // 2, T - 64):
        s = slice(lo, lo + 64)
        fs = nv.nvfp4_block_norm(x[s], y[s], w_post, gate[s], w_pre, 0.7)
        bs = nv.nvfp4_block_norm_backward(dx_out[s], dn[s], x[s], y[s], fs.rstd_post, fs.rstd_pre, w_post, gate[s], w_pre, 0.7)
        assert torch.equal(f.x[s], fs.x) and torch.equal(f.n[s], fs.n)
        assert torch.equal(f.rstd_post[s], fs.rstd_post) and torch.equal(f.rstd_pre[s], fs.rstd_pre)
        assert torch.equal(b.dx[s], bs.dx) and torch.equal(b.dy[s], bs.dy) and torch.equal(b.dgate[s], bs.dgate)
    # the sums over all rows: dw_pre = sum dn xh, dw_post = sum q yh
    sums, mags = torch.zeros(2, D, dtype=torch.float64, device=DEV), torch.zeros(2, D, dtype=torch.float64, device=DEV)
    for lo in range(0, T, 1024):
        xd, yd, dxd, dnd, gd = (v[lo:lo + 1024].double() for v in (x, y, dx_out, dn, gate))
        yh = yd / (yd.square().mean(1, keepdim=True) + 1e-6).sqrt()
        p = 0.7 * gd * yh * w_post.double()
        rx = 1 / ((xd + p).square().mean(1, keepdim=True) + 1e-6).sqrt()
        xh, u = (xd + p) * rx, dnd * w_pre.double()
        d = dxd + rx * (u - xh * (u * xh).mean(1, keepdim=True))
        mag_xh = (xd.abs() + p.abs()) * rx
        mag_d = dxd.abs() + rx * (u.abs() + mag_xh * (u.abs() * mag_xh).mean(1, keepdim=True))
        sums += torch.stack([(dnd * xh).sum(0), (0.7 * gd * d * yh).sum(0)])
        mags += torch.stack([(dnd.abs() * mag_xh).sum(0), (0.7 * gd.abs() * mag_d * yh.abs()).sum(0)])
    assert bool(((b.dw_pre.double() - sums[0]).abs() <= norm.TOL * mags[0]).all())
    assert bool(((b.dw_post.double() - sums[1]).abs() <= norm.TOL * mags[1]).all())


@pytest.mark.parametrize("T,k,D,dtype", [(4099, 8, 4096, BF16), (16387, 2, 4096, BF16), (2051, 8, 4096, F32), (9001, 9, 2056, BF16)])
def test_combine_beyond_the_cache(T, k, D, dtype):
    g = torch.Generator(device=DEV).manual_seed(T)
    y = torch.randn(T * k, D, generator=g, device=DEV).to(dtype)
    assert y.numel() * y.element_size() >= CACHE
    dout = torch.randn(T, D, generator=g, device=DEV).to(dtype)
    ids, w, plan = nv.nvfp4_moe_route(torch.randn(T, 64, generator=g, device=DEV), k)
    out = nv.nvfp4_moe_combine(y, plan, w)
    dy, dw = nv.nvfp4_moe_combine_backward(dout, y, plan, w)
    for lo in range(0, T, 512):
        s = slice(lo, min(lo + 512, T))
        rows, wd = y[plan.pos[s].long()].double(), w[s].double()[:, :, None]
        want, mag = (rows * wd).sum(1), (rows * wd).abs().sum(1)
        tol = k * 2.0 ** -24 * mag + (2.0 ** -8 * want.abs() if dtype == BF16 else 0.0)
        assert bool(((out[s].double() - want).abs() <= tol).all()), lo
        terms = rows * dout[s].double()[:, None, :]
        assert bool(((dw[s].double() - terms.sum(2)).abs() <= (D / 32 + 8) * 2.0 ** -24 * terms.abs().sum(2)).all()), lo
        assert torch.equal(dy[plan.pos[s].long()], (w[s][:, :, None] * dout[s].float()[:, None, :]).to(dtype)), lo


def _weights(rows, k, groups, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(-127, 128, (groups * rows, k), generator=g, device=DEV, dtype=torch.int8)
    return nv.Int8Tensor(q, torch.rand(groups * rows, generator=g, device=DEV) * 0.01 + 1e-4, rows, k, groups)


@pytest.mark.parametrize("T,k,N,K", [(8, 8, 1100, 4096), (20, 3, 4200, 1024), (40, 2, 4131, 1040)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_experts_beyond_the_cache(T, k, N, K, dtype):
    E = 64
    assert E * N * K >= CACHE
    x, w = _weights(T, K, 1, 1), _weights(N, K, E, 2)
    ids, _, plan = nv.nvfp4_moe_route(torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)), k)
    got = nv.nvfp4_int8_gemm(x, w, dtype, plan=plan, gather=True).cpu()
    rows, off = plan.rows.cpu().long(), plan.offsets.cpu().tolist()
    for e in range(E):
        if off[e + 1] > off[e]:
            src, r = rows[off[e]:off[e + 1]] // k, slice(e * N, (e + 1) * N)
            want = _want(x.data[src.to(DEV)], x.scales[src.to(DEV)], w.data[r], w.scales[r], dtype)
            assert torch.equal(got[off[e]:off[e + 1]], want), e


@pytest.mark.parametrize("T,k,E,N,K", [(65, 3, 64, 130, 256), (300, 4, 64, 200, 144), (500, 2, 64, 64, 1024)])
def test_few_rows_an_expert_of_many_tokens(T, k, E, N, K):
    # one expert has nearly all tokens, so several tiles of rows of the kernel for few rows
    x, w = _weights(T, K, 1, 1), _weights(N, K, E, 2)
    logits = torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    logits[:, 5] += 6.0
    _, _, plan = nv.nvfp4_moe_route(logits, k)
    got = nv.nvfp4_int8_gemm(x, w, F32, plan=plan, gather=True).cpu()
    rows, off = plan.rows.long(), plan.offsets.cpu().tolist()
    assert off[6] - off[5] > 64 and T * k <= 24 * E
    for e in range(E):
        if off[e + 1] > off[e]:
            src, r = rows[off[e]:off[e + 1]] // k, slice(e * N, (e + 1) * N)
            assert torch.equal(got[off[e]:off[e + 1]], _want(x.data[src], x.scales[src], w.data[r], w.scales[r], F32)), e


@pytest.mark.parametrize("M,N,K", [(1, 66000, 4096), (30, 2100, 131056), (100, 4100, 65552)])
def test_weight_beyond_the_cache(M, N, K):
    assert N * K >= CACHE
    a, b = _weights(M, K, 1, 1), _weights(N, K, 1, 2)
    got = nv.nvfp4_int8_gemm(a, b, F32).cpu()
    for cols in (slice(0, 70), slice(N - 70, N)):
        assert torch.equal(got[:, cols], _want(a.data, a.scales, b.data[cols], b.scales[cols], F32))


@pytest.mark.parametrize("M,N,K", [(1999, 4000, 4096), (4500, 4096, 2064), (4096, 6100, 2048)])
def test_product_with_a_last_round_of_half_tiles(M, N, K):
    a, b = _weights(M, K, 1, 1), _weights(N, K, 1, 2)
    got = nv.nvfp4_int8_gemm(a, b, BF16).cpu()
    assert torch.equal(got, _want(a.data, a.scales, b.data, b.scales, BF16))


@pytest.mark.parametrize("T,k,E,N,K,skew", [(1024, 8, 64, 1536, 2048, 0.7), (4096, 8, 8, 1000, 1024, 0.3), (4096, 8, 64, 1536, 1040, 1.0),
                                            (1500, 2, 3, 4096, 2048, 0.0)])
def test_experts_with_a_last_round_of_half_tiles(T, k, E, N, K, skew):
    x, w = _weights(T, K, 1, 1), _weights(N, K, E, 2)
    logits = torch.randn(T, E, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    ids, _, plan = nv.nvfp4_moe_route(logits - skew * torch.log(1.0 + torch.arange(E, device=DEV)), k)
    got = nv.nvfp4_int8_gemm(x, w, BF16, plan=plan, gather=True).cpu()
    rows, off = plan.rows.long(), plan.offsets.cpu().tolist()
    for e in range(E):
        if off[e + 1] > off[e]:
            src, r = rows[off[e]:off[e + 1]] // k, slice(e * N, (e + 1) * N)
            assert torch.equal(got[off[e]:off[e + 1]], _want(x.data[src], x.scales[src], w.data[r], w.scales[r], BF16)), e
