"""The operators together as a mixture-of-experts block (examples/moe_block.py), under a captured graph, and at
sizes past 32-bit offsets."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from examples.moe_block import MoEBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _xy(block, tokens, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + tokens)
    return [torch.randn(tokens, block.d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_block_against_the_plain_form(tokens):
    block = MoEBlock(d=512, hidden=256)
    x, y = _xy(block, tokens)
    want_x, want = block.plain(x, y)
    # an 8-bit operand is off by about 1 / (127 sqrt(12)) x its row's largest / typical value (about 4) = 1% of its
    # norm, an NVFP4 one by about 10%; two products of two operands each
    for nvfp4, bound in ((False, 0.04), (True, 0.4)):
        got_x, got = block.forward(x, y, nvfp4)
        assert ((got_x.float() - want_x).norm() / want_x.norm()) < 2.0 ** -8
        assert ((got.float() - want).norm() / want.norm()) < bound


def test_training_step_against_differentiation():
    block = MoEBlock(d=256, hidden=64, experts=8, top_k=2, groups=2, group_top_k=1)
    x, y = _xy(block, 50)
    maps = torch.randn(block.d, block.d, device=DEV) * block.d ** -0.5
    dout = torch.randn(50, block.d, device=DEV).to(torch.bfloat16)
    factor = torch.randn(block.experts, device=DEV)  # experts differ, or the renormalised weights have no gradient

    def of_row(plan):
        return factor[torch.bucketize(torch.arange(plan.rows.shape[0], device=DEV), plan.offsets[1:].long(), right=True)][:, None]

    out, grads, drouter, (ids, _) = block.train_step(x, y, lambda r, plan: (of_row(plan) * (r.float() @ maps.t())).to(r.dtype),
                                                     lambda d, plan: (of_row(plan) * (d.float() @ maps)).to(d.dtype), dout)
    # the same function in 64 bits, for the chosen experts
    leaf = {n: getattr(block, n).double().requires_grad_() for n in ("w_post", "gate", "w_pre", "router")}
    xd, yd = x.double().requires_grad_(), y.double().requires_grad_()
    norm = lambda v, w: v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + 1e-6) * w
    n = norm(xd + block.alpha * leaf["gate"] * norm(yd, leaf["w_post"]), leaf["w_pre"])
    s = torch.sigmoid(n @ leaf["router"].t()).gather(1, ids.long())
    w = s / (s.sum(dim=1, keepdim=True) + 1e-20) * block.scale
    ref = (w * factor.double()[ids.long()]).sum(dim=1, keepdim=True) * (n @ maps.double().t())
    (ref * dout.double()).sum().backward()
    rel = lambda a, b: ((a.double() - b).norm() / b.norm()).item()
    # bf16 tensors in between (n, the experts' rows and their gradients, dn): each rounds its values by up to 2^-9,
    # five of them in a chain; sums of many such terms average it out
    tol = 5 * 2.0 ** -9
    assert rel(out, ref.detach()) < tol and rel(drouter, leaf["router"].grad) < 4 * tol
    for got, want in ((grads.dx, xd), (grads.dy, yd), (grads.dw_post, leaf["w_post"]), (grads.dgate, leaf["gate"]),
                      (grads.dw_pre, leaf["w_pre"])):
        assert rel(got, want.grad) < tol


@pytest.mark.parametrize("tokens", [1, 40, 700])
def test_captured_graph_replays_with_new_inputs(tokens):
    block = MoEBlock(d=512, hidden=256)
    x, y = _xy(block, tokens)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        block.forward(x, y)  # warm
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx, gout = block.forward(x, y)
    for seed in range(3):
        nx, ny = _xy(block, tokens, seed)
        ex, eout = block.forward(nx, ny)
        torch.cuda.synchronize()
        x.copy_(nx)
        y.copy_(ny)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gx, ex) and torch.equal(gout, eout)


def _free_gib():
    return torch.cuda.mem_get_info()[0] / 2 ** 30


def test_rows_past_four_gigabytes():
    if _free_gib() < 40:
        pytest.skip("needs 40 GiB")
    # combine and gather at row offsets past 2^32 bytes: 600000 rows of 8 KB, the tokens at the far end checked
    T, k, D = 300000, 2, 4096
    ids = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    ids[:, 1] = 1
    plan = nv.nvfp4_moe_plan(ids, 2)
    x = torch.randint(-3, 4, (T, D), device=DEV, dtype=torch.int8).to(torch.bfloat16)
    y = nv.nvfp4_moe_gather(x, plan)
    assert torch.equal(y[-1], x[-1]) and torch.equal(y[T - 1], x[-1]) and torch.equal(y[T + 7], x[7])
    back = nv.nvfp4_moe_combine(y, plan)
    assert torch.equal(back[-5:], 2 * x[-5:]) and torch.equal(back[T // 2], 2 * x[T // 2])
    # 8-bit rows past 2^32 bytes (read in place) and a weight's experts past 2^32 bytes
    q = nv.nvfp4_int8_quantize(y)  # 2.4 GB
    a = nv.Int8Tensor(torch.cat([q.data, q.data]), torch.cat([q.scales, q.scales]), 4 * T, D)
    w = nv.nvfp4_int8_quantize(torch.randn(16, D, device=DEV))
    c = nv.nvfp4_int8_gemm(a, w, torch.float32)
    assert torch.equal(c[2 * T:], c[:2 * T])
    acc = (a.data[-3:].double() @ w.data.double().t()).cpu().numpy().astype(np.float32)
    scale = (a.scales[-3:].cpu().numpy()[:, None] * w.scales.cpu().numpy()[None]).astype(np.float32)
    assert np.array_equal(c[-3:].cpu().numpy(), acc * scale)


def test_gathered_rows_and_experts_past_two_gigabytes():
    if _free_gib() < 40:
        pytest.skip("needs 40 GiB")
    # a gathered operand between 2 and 4 GB, weights of 12 experts over 4 GB
    T, K, N, E = 900000, 4096, 90000, 12
    x = nv.Int8Tensor(torch.randint(-127, 128, (T, K), device=DEV, dtype=torch.int8), torch.rand(T, device=DEV), T, K)
    w = nv.Int8Tensor(torch.randint(-127, 128, (E * N, K), device=DEV, dtype=torch.int8), torch.rand(E * N, device=DEV), N, K, E)
    ids = torch.full((T, 1), -1, dtype=torch.int32, device=DEV)
    for rows in (5, 300):  # the few-row kernel cannot know how many rows an expert has; both tile kinds
        ids[-rows:, 0] = E - 1
        plan = nv.nvfp4_moe_plan(ids, E)
        small = nv.MoEPlan(plan.offsets, plan.rows[:rows].contiguous(), plan.pos)
        c = torch.empty(rows, N, dtype=torch.float32, device=DEV)
        st = nv.lib().nvfp4_int8_gemm(x.data.data_ptr(), x.scales.data_ptr(), T, w.data.data_ptr(), w.scales.data_ptr(), rows, N,
                                      K, c.data_ptr(), nv.NVFP4_F32, N, E, small.offsets.data_ptr(), small.rows.data_ptr(), 1,
                                      None, torch.cuda.current_stream().cuda_stream)
        assert st == nv.NVFP4_OK
        cols = torch.tensor([0, 1, N - 1], device=DEV)
        src = small.rows.long()
        acc = (x.data[src].double() @ w.data[(E - 1) * N + cols].double().t()).cpu().numpy().astype(np.float32)
        scale = (x.scales[src].cpu().numpy()[:, None] * w.scales[(E - 1) * N + cols].cpu().numpy()[None]).astype(np.float32)
        assert np.array_equal(c[:, cols].cpu().numpy(), acc * scale)
