"""Workspaces that the caller of the operators around the quantized products brings: one that is too small for the call
is refused before anything is enqueued (the kernels would write past its end), one of the size asked for serves.

The sizes do not grow with the problem, so a workspace from a larger call can be too small for a smaller one."""
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv


def _calls(device):
    """(name, bytes needed, call with a workspace) of every entry point of the binding that takes one."""
    L = nv.lib()
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(device)
    logits = r(70, 96)
    ids = torch.randint(0, 96, (1500, 4), generator=g, dtype=torch.int32).to(device)
    q = lambda rows, k: nv.Int8Tensor(torch.randint(-127, 128, (rows, k), generator=g, dtype=torch.int8).to(device),
                                      torch.rand(rows, generator=g).to(device), rows, k)
    a, b = q(5, 4096), q(200, 4096)
    x, y, w = r(300, 64), r(300, 64), r(64)

    def route(ws):
        i, v, plan = nv.nvfp4_moe_route(logits, 4, workspace=ws)
        return i, v, plan.offsets, plan.rows, plan.pos

    def plan(ws):
        p = nv.nvfp4_moe_plan(ids, 96, workspace=ws)
        return p.offsets, p.rows, p.pos

    def norm(ws):
        ones = torch.ones(300, device=device)
        n = nv.nvfp4_block_norm_backward(x, y, x, y, ones, ones, w, w, w, workspace=ws)
        return n.dx, n.dy, n.dw_post, n.dgate, n.dw_pre

    return [("route", L.nvfp4_moe_workspace_size(70, 96, 4), route), ("plan", L.nvfp4_moe_workspace_size(1500, 96, 4), plan),
            ("product", L.nvfp4_int8_gemm_workspace_size(5, 200, 4096), lambda ws: (nv.nvfp4_int8_gemm(a, b, workspace=ws),)),
            ("norm", L.nvfp4_block_norm_workspace_size(300, 64), norm)]


def test_refused():
    for name, size, call in _calls("cpu"):
        assert size > 0 and size % 16 == 0, name
        for wrong in (torch.empty(0, dtype=torch.uint8), torch.empty(size - 1, dtype=torch.uint8),
                      torch.empty(size // 4 - 1, dtype=torch.int32), torch.empty(size, device="meta", dtype=torch.uint8),
                      torch.empty(2 * size, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(wrong)


def test_sizes_do_not_grow_with_the_problem():
    L = nv.lib()
    assert L.nvfp4_int8_gemm_workspace_size(64, 5440, 4096) > L.nvfp4_int8_gemm_workspace_size(64, 5504, 4096) > 0
    assert L.nvfp4_int8_gemm_workspace_size(64, 8256, 4096) == 0
    assert L.nvfp4_block_norm_workspace_size(4096, 2048) > L.nvfp4_block_norm_workspace_size(4096, 2056)


@pytest.mark.gpu
def test_the_size_asked_for_serves():
    for name, size, call in _calls("cuda"):
        want = call(None)
        guarded = torch.full((size + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        for got, ref in zip(call(guarded[:size]), want):
            assert torch.equal(got, ref), name
        assert (guarded[size:] == 0x5A).all(), name
