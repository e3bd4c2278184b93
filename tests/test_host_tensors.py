"""Tensors in host memory are refused by the operators around the quantized products: their kernels would read the
addresses on the GPU."""
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv


def _calls():
    f, w, ids = torch.zeros(8, 64), torch.zeros(8, 4), torch.zeros(8, 4, dtype=torch.int32)
    y, d = torch.zeros(32, 64), torch.zeros(64)
    plan = nv.MoEPlan(torch.zeros(65, dtype=torch.int32), torch.zeros(32, dtype=torch.int32), ids)
    q = nv.Int8Tensor(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8), 8, 64)
    return dict(route=lambda: nv.nvfp4_moe_route(f, 4), route_alone=lambda: nv.nvfp4_moe_route(f, 4, with_plan=False),
                route_backward=lambda: nv.nvfp4_moe_route_backward(f, ids, w), plan=lambda: nv.nvfp4_moe_plan(ids, 64),
                gather=lambda: nv.nvfp4_moe_gather(f, plan), combine=lambda: nv.nvfp4_moe_combine(y, plan, w),
                combine_backward=lambda: nv.nvfp4_moe_combine_backward(f, y, plan, w), quantize=lambda: nv.nvfp4_int8_quantize(f),
                product=lambda: nv.nvfp4_int8_gemm(q, q), norm=lambda: nv.nvfp4_block_norm(f, f, d, d, d),
                norm_backward=lambda: nv.nvfp4_block_norm_backward(f, f, f, f, torch.ones(8), torch.ones(8), d, d, d))


@pytest.mark.parametrize("name", sorted(_calls()))
def test_refused(name):
    with pytest.raises(nv.NVFP4Error, match="cpu") as refusal:
        _calls()[name]()
    assert refusal.value.status == nv.NVFP4_ERR_UNSUPPORTED
