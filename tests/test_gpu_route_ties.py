"""Routing of rows where some scores are equal, within a lane's experts and across lanes, next to rows without any.

Scores rise with the logits, and logits 1/4 apart have scores that differ, so the choice is the stable order of the
logits from the largest on."""
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("E,k", [(7, 7), (40, 8), (64, 6), (100, 20), (160, 8), (256, 8), (256, 32), (384, 17), (512, 10)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [3, 500, 5000])
def test_ties_among_the_chosen(E, k, dtype, T):
    g = torch.Generator().manual_seed(E + k + T)
    logits = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() / 4  # no ties
    some = torch.rand(T, generator=g)
    few = torch.randint(0, max(2, E // 2), (T, E), generator=g).float() / 4              # some
    many = torch.randint(0, 3, (T, E), generator=g).float()                              # nearly all
    logits = torch.where((some < 0.3)[:, None], few, torch.where((some > 0.9)[:, None], many, logits))
    logits[T // 2] = 1.0
    # (as the operator reads them: bf16 rounds 511 / 4, which makes more ties)
    want = torch.sort(logits.to(dtype).float(), dim=1, descending=True, stable=True).indices[:, :k]
    ids, weights, plan = nv.nvfp4_moe_route(logits.to(dtype).to(DEV), k)
    assert torch.equal(ids.cpu().long(), want)
    flat = ids.cpu().flatten()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(plan.rows.cpu().long(), order)
    assert torch.equal(plan.offsets.cpu().long(), torch.cat([torch.zeros(1, dtype=torch.long), torch.bincount(flat, minlength=E).cumsum(0)]))
