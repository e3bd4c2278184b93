"""The operators of fine-tuning together, as examples/moe_block.py uses them, and at sizes past 32-bit offsets."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from examples.moe_block import MoEBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def _block_and_inputs(tokens, seed=0):
    block = MoEBlock(d=256, hidden=128, experts=8, top_k=2, groups=2, group_top_k=1)
    block.add_adapters(rank=16)
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (block,) + tuple(torch.randn(tokens, 256, generator=g, device=DEV).to(BF16) for _ in range(3))


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_step_against_differentiation(tokens):
    block, x, y, dout = _block_and_inputs(tokens)
    out, balance, norm, grads, norms = block.finetune_step(x, y, dout, coef=0.5, max_norm=1e9)
    # the same function in 64 bits without any rounding of weights or activations, for the chosen experts
    _, ids, _, _ = block.route(nv.nvfp4_block_norm(x, y, w_post=block.w_post, gate=block.gate, w_pre=block.w_pre, alpha=block.alpha).n)
    E, R = block.experts, 16
    leaf = lambda t: t.double().clone().requires_grad_()
    da, db = leaf(block.down_adapters.a), leaf(block.down_adapters.b)
    ua, ub = leaf(block.up_adapters.a), leaf(block.up_adapters.b)
    router, xd, yd = leaf(block.router), leaf(x), leaf(y)
    norm_of = lambda v, w: v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + 1e-6) * w.double()
    n = norm_of(xd + block.alpha * block.gate.double() * norm_of(yd, block.w_post), block.w_pre)
    logits = n @ router.t()
    score = torch.sigmoid(logits)
    picked = score.gather(1, ids.long())
    weights = picked / (picked.sum(dim=1, keepdim=True) + 1e-20) * block.scale
    want = torch.zeros(tokens, block.d, dtype=torch.float64, device=DEV)
    up, down = block.up.double().view(E, -1, block.d), block.down.double().view(E, block.d, -1)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        A, B = ua[e * R:(e + 1) * R], ub.view(E, -1, R)[e]
        a, b = (n[t] @ (up[e] + B @ A).t()).split(block.hidden, dim=1)
        A, B = da[e * R:(e + 1) * R], db.view(E, -1, R)[e]
        v = (torch.nn.functional.silu(a) * b) @ (down[e] + B @ A).t()
        want = want.index_add(0, t, weights[t, j, None] * v)
    p = score / (score.sum(dim=1, keepdim=True) + 1e-20)
    share = torch.bincount(ids.reshape(-1).long(), minlength=E).double() * E / (ids.shape[1] * tokens)
    loss = 0.5 * (share * p.mean(dim=0)).sum()
    ((want * dout.double()).sum() + loss).backward()
    rel = lambda got, ref: float((got.double() - ref).norm() / ref.norm())
    # An 8-bit operand is off by 1% of its norm (1 / (127 sqrt(12)) x largest / typical value of a row, about 4); a chain
    # of at most four products of two such operands each, and bf16 tensors in between (2^-9 each), stays below 8 x 1.1%.
    bound = 8 * 0.011
    assert rel(out, want.detach()) < bound
    # the probabilities come from logits of bf16 norms: 2^-8 of values of order one
    assert abs(float(balance.loss) - loss.item()) <= 0.02 * loss.item()
    assert torch.equal(balance.counts[0].cpu(), torch.bincount(ids.reshape(-1).long(), minlength=E).int().cpu())
    for got, ref in zip(grads, (da, db, ua, ub, router)):
        assert rel(got, ref.grad) < bound
    assert rel(norms.dx, xd.grad) < bound and rel(norms.dy, yd.grad) < bound
    total = torch.sqrt(sum(t.double().square().sum() for t in grads))
    assert abs(float(norm) - float(total)) <= 2.0 ** -23 * float(total)


def test_clipped_step_and_graph_replays():
    block, x, y, dout = _block_and_inputs(64)
    free = block.finetune_step(x, y, dout, max_norm=1e9)
    clipped = block.finetune_step(x, y, dout, max_norm=0.5)
    assert torch.equal(free[2], clipped[2])
    factor = min(1.0, 0.5 / (float(free[2]) + 1e-6))
    for a, b in zip(free[3], clipped[3]):
        # the factor's own five roundings and one of the product
        assert bool(((b.double() - a.double() * factor).abs() <= 6 * 2.0 ** -24 * a.double().abs()).all())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block.finetune_step(x, y, dout)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block.finetune_step(x, y, dout)
    for i in range(4):
        x.mul_(-1.25)
        dout.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        want = block.finetune_step(x, y, dout)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1].loss, want[1].loss) and torch.equal(got[2], want[2])
        assert all(torch.equal(a, b) for a, b in zip(got[3], want[3])) and torch.equal(got[4].dx, want[4].dx)


def test_adapter_beside_the_4_bit_products():
    """One adapter of a request beside a frozen NVFP4 weight, for a few tokens and a prompt."""
    K, N, R = 512, 384, 32
    g = torch.Generator(device=DEV).manual_seed(4)
    weight = nv.nvfp4_quantize((torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(BF16), flags=nv.NVFP4_BLOCK2D)
    w = nv.Adapters((torch.randn(R, K, generator=g, device=DEV) * K ** -0.5).to(BF16),
                    (torch.randn(N, R, generator=g, device=DEV) * R ** -0.5).to(BF16), torch.full((1,), 2.0, device=DEV), R, K, N)
    full = nv.nvfp4_dequantize(weight).double() + 2.0 * w.b.double() @ w.a.double()
    for tokens in (3, 500):
        x = torch.randn(tokens, K, generator=g, device=DEV).to(BF16)
        y = nv.nvfp4_gemm_w4a16(x, weight)
        nv.nvfp4_adapter(x, w, y, out=y)
        want = x.double() @ full.t()
        # two roundings to bf16, of the product and of the sum; both are within 4 of values of order one
        assert bool(((y.double() - want).abs() <= 2 * 2.0 ** -8 * (want.abs() + 4)).all())


def test_rows_past_32_bit_offsets():
    """c, dc and x of more than 2^32 bytes: the last rows are right, and rows between have their own adapter's result."""
    M, N, K, R = 75000, 28672, 64, 8
    g = torch.Generator(device=DEV).manual_seed(5)
    w = nv.Adapters((torch.randn(2 * R, K, generator=g, device=DEV) * K ** -0.5).to(BF16),
                    torch.randn(2 * N, R, generator=g, device=DEV).to(BF16), torch.ones(2, device=DEV), R, K, N, 2)
    ids = torch.zeros(M, 1, dtype=torch.int32, device=DEV)
    ids[M // 2:] = 1
    ids[70000:70100] = -1
    plan = nv.nvfp4_moe_plan(ids, 2)
    x = torch.randn(M, K, generator=g, device=DEV).to(BF16)
    base = torch.ones(M, N, dtype=BF16, device=DEV)
    c, h = nv.nvfp4_adapter(x, w, base, plan=plan, by_token=True, with_h=True)
    for t in (0, 37499, 37500, 69999, 70050, 74999):
        want = 1.0 + (0.0 if ids[t] < 0 else 1.0) * (w.b.view(2, N, R)[max(int(ids[t]), 0)].double()
                                                     @ (w.a.view(2, R, K)[max(int(ids[t]), 0)].double() @ x[t].double()))
        assert bool(((c[t].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12).all()), t
    dc = torch.zeros(M, N, dtype=BF16, device=DEV)
    dc[74999, 28671], dc[0, 0] = 1.0, 1.0
    d = nv.nvfp4_adapter_backward(dc, x, w, h, plan=plan, by_token=True)
    g1 = w.b[2 * N - 1].double()
    want = g1 @ w.a.view(2, R, K)[1].double()
    assert bool(((d.dx[74999].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16).all())
    # one product each: exact but for the roundings of h and of the product
    h1 = w.a.view(2, R, K)[1].double() @ x[74999].double()
    assert bool(((d.db[2 * N - 1].double() - h1).abs() <= 80 * 2.0 ** -24 * (w.a.view(2, R, K)[1].double().abs() @ x[74999].double().abs())).all())
    assert not d.db[:N][1:].any() and not d.dx[70000:70100].any()
    del base, c, dc
    wide = nv.Adapters(torch.randn(R, N, generator=g, device=DEV).to(BF16), torch.randn(K, R, generator=g, device=DEV).to(BF16),
                       torch.ones(1, device=DEV), R, N, K)
    x = torch.zeros(M, N, dtype=BF16, device=DEV)
    x[M - 1, N - 1], x[3, 5] = 2.0, 1.0
    c = nv.nvfp4_adapter(x, wide, out_dtype=torch.float32)
    want = 2.0 * wide.b.double() @ wide.a[:, N - 1].double()
    assert bool(((c[M - 1].double() - want).abs() <= 16 * 2.0 ** -24 * 2.0 * (wide.b.double().abs() @ wide.a[:, N - 1].double().abs())).all())
    assert not c[M // 2].any()


def test_balance_past_32_bit_offsets():
    T, E, k = 4300000, 256, 2
    logits = torch.zeros(T, E, device=DEV)
    ids = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    ids[T - 1, 0], ids[T - 2, 1] = 255, 7
    logits[T - 1, 255] = 1.0
    b = nv.nvfp4_moe_balance(logits, ids, 1.0)
    assert int(b.tokens) == 2 and int(b.counts.sum()) == 2 and int(b.counts[0, 255]) == 1
    p = np.exp(1.0) / (np.exp(1.0) + 255)
    # the mean over two tokens, in 32 bits
    assert abs(float(b.probs[0, 255]) - (p + 1 / 256) / 2) <= 2.0 ** -20 * (p + 1 / 256)
    d = nv.nvfp4_moe_balance_backward(logits, ids, b, 1.0)
    assert bool(torch.isfinite(d[-2:]).all()) and float(d[T - 1, 255]) != 0.0 and not d[:-2].any()
