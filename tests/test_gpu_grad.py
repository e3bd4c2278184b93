"""The norm of many gradients and their clipping on the GPU against 64-bit references.

Squares and sums are 64-bit numbers (2^-53 each, nothing beside the rest), so a norm is off by its one rounding to 32 bits,
2^-24.  The factor max_norm / (norm + eps) takes the roundings of max_norm, eps, norm, the sum and the quotient, the product
one more: 6 x 2^-24, and a bf16 result 2^-8."""
import math

import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _list(shapes, dtypes, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(*s, generator=g) * std).to(dtypes[i % len(dtypes)]).to(DEV) for i, s in enumerate(shapes)]


def _norm(ts):
    return math.sqrt(math.fsum(float((t.cpu().double() ** 2).sum()) for t in ts))


F32, BF16 = torch.float32, torch.bfloat16
LISTS = {
    "one": [(1,)], "few": [(5,), (1, 1), (8,), (7, 3)], "chunk": [(16384,), (16383,), (16385,), (32768,)],
    "ragged": [(0,), (129, 257), (0, 4), (4096, 40), (1,), (300000,)], "many": [(i % 37 + 1,) for i in range(1000)],
    "matrices": [(512, 1024)] * 7}


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("dtypes", [[F32], [BF16], [F32, BF16]], ids=["f32", "bf16", "mixed"])
def test_norm_and_clip(name, dtypes):
    ts = _list(LISTS[name], dtypes, seed=len(name))
    want = _norm(ts)
    norm = nv.nvfp4_grad_norm(ts)
    assert abs(float(norm) - want) <= 2.0 ** -24 * 1.01 * want
    top = max(float(t.abs().max()) for t in ts if t.numel())
    assert float(nv.nvfp4_grad_norm(ts, flags=nv.NVFP4_GRAD_MAX)) == top
    before = [t.clone() for t in ts]
    out = [torch.full_like(t, 7.0) for t in ts]
    got = nv.nvfp4_grad_clip(ts, 0.37 * want, out=out)
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(ts, before))
    factor = 0.37 * want / (want + 1e-6)
    for o, t in zip(out, ts):
        w = t.cpu().double() * factor
        assert bool(((o.cpu().double() - w).abs() <= (6 * 2.0 ** -24 + (2.0 ** -8 if o.dtype == BF16 else 0)) * w.abs()).all())
    nv.nvfp4_grad_clip(ts, 0.37 * want)  # in place: the same bits
    assert all(torch.equal(o, t) for o, t in zip(out, ts))


@pytest.mark.parametrize("max_norm", [2.0, math.inf])
def test_a_small_norm_changes_nothing(max_norm):
    ts = _list([(100,), (64, 64)], [F32, BF16], std=1e-3)
    before = [t.clone() for t in ts]
    out = [torch.empty_like(t) for t in ts]
    nv.nvfp4_grad_clip(ts, max_norm)
    nv.nvfp4_grad_clip(ts, max_norm, out=out)
    assert all(torch.equal(a, b) and torch.equal(a, o) for a, b, o in zip(before, ts, out))


def test_zero_is_allowed():
    ts = _list([(1000,)], [F32])
    nv.nvfp4_grad_clip(ts, 0.0)
    assert not ts[0].any()
    assert float(nv.nvfp4_grad_norm(ts)) == 0.0 and float(nv.nvfp4_grad_norm(ts, flags=nv.NVFP4_GRAD_MAX)) == 0.0
    nv.nvfp4_grad_clip(ts, 1.0)
    assert not ts[0].any()


@pytest.mark.parametrize("bad,norm,top", [(math.inf, math.inf, math.inf), (-math.inf, math.inf, math.inf), (math.nan, math.nan, math.nan)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_numbers(bad, norm, top, dtype):
    ts = _list([(20000,), (333,)], [dtype])
    ts[1][332] = bad
    if math.isnan(bad):
        ts[0][0] = math.inf  # NaN is above infinity
    same = lambda a, b: a == b or (math.isnan(a) and math.isnan(b))
    assert same(float(nv.nvfp4_grad_norm(ts)), norm) and same(float(nv.nvfp4_grad_norm(ts, flags=nv.NVFP4_GRAD_MAX)), top)
    before = [t.clone() for t in ts]
    nv.nvfp4_grad_clip(ts, 0.1)
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(before, ts))


def test_squares_beyond_32_bits():
    big = [torch.full((64,), 2.0 ** 100, device=DEV), torch.full((64,), 2.0 ** 100, device=DEV, dtype=BF16)]
    assert abs(float(nv.nvfp4_grad_norm(big)) / (2.0 ** 100 * 128 ** 0.5) - 1) <= 2.0 ** -24
    small = [torch.full((256,), 2.0 ** -140, device=DEV)]  # (denormal)
    assert float(nv.nvfp4_grad_norm(small)) == 2.0 ** -136
    nv.nvfp4_grad_clip(big, 1.0)
    assert abs(float(nv.nvfp4_grad_norm(big)) - 1.0) <= 2.0 ** -8


def test_odd_addresses_and_orders():
    """Views that start anywhere, transposed matrices and permuted tensors; nothing around them is touched."""
    for dtype in (F32, BF16):
        flat = torch.randn(70000, device=DEV).to(dtype)
        whole = flat.clone()
        ts = [flat[1:20], flat[23:16500], flat[16501:16501 + 300 * 100].view(300, 100).t(), flat[50003:50003 + 24].view(2, 3, 4).permute(2, 0, 1)]
        want = _norm(ts)
        assert abs(float(nv.nvfp4_grad_norm(ts)) - want) <= 2.0 ** -24 * 1.01 * want
        nv.nvfp4_grad_clip(ts, 0.5 * want)
        mine = torch.zeros(70000, dtype=torch.bool, device=DEV)
        for lo, n in ((1, 19), (23, 16477), (16501, 30000), (50003, 24)):
            mine[lo:lo + n] = True
        assert torch.equal(flat[~mine], whole[~mine])
        w = whole[mine].double() * (0.5 * want / (want + 1e-6))
        assert bool(((flat[mine].double() - w).abs() <= (6 * 2.0 ** -24 + (2.0 ** -8 if dtype == BF16 else 0)) * w.abs()).all())


def test_a_given_norm_of_all_ranks():
    ts = _list([(1000,)], [F32])
    whole = torch.tensor([50.0], device=DEV)
    before = ts[0].clone()
    assert nv.nvfp4_grad_clip(ts, 25.0, eps=0.0, norm=whole) is whole and torch.equal(ts[0], before * 0.5)


def test_the_same_bits_another_stream_and_graph_replays():
    ts = _list([(100000,), (4096, 129), (77,)], [F32, BF16])
    work = torch.empty(nv.lib().nvfp4_grad_workspace_size(3, sum(t.numel() for t in ts)) // 4, dtype=torch.int32, device=DEV)
    out = [torch.empty_like(t) for t in ts]
    first = nv.nvfp4_grad_clip(ts, 1.0, out=out)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert torch.equal(nv.nvfp4_grad_clip(ts, 1.0, out=out, workspace=work), first)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = nv.nvfp4_grad_clip(ts, 1.0, out=out, workspace=work)
    for i in range(4):
        for t in ts:
            t.mul_(1.0 + i)
        work.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        other = [torch.empty_like(t) for t in ts]
        assert torch.equal(norm, nv.nvfp4_grad_clip(ts, 1.0, out=other))
        assert all(torch.equal(a, b) for a, b in zip(got, other))


def test_a_large_tensor():
    """More chunks than workgroups, and byte offsets past 32 bits."""
    n = 2 ** 31 + 12345
    t = torch.zeros(n, dtype=BF16, device=DEV)
    t[-1], t[2 ** 30 + 7], t[5] = 3.0, 4.0, 12.0
    assert float(nv.nvfp4_grad_norm([t])) == 13.0
    nv.nvfp4_grad_clip([t], 6.5, eps=0.0)
    assert (float(t[-1]), float(t[2 ** 30 + 7]), float(t[5])) == (1.5, 2.0, 6.0)
    assert float(nv.nvfp4_grad_norm([t], flags=nv.NVFP4_GRAD_MAX)) == 6.0
