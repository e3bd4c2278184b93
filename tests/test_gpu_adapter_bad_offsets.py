"""Offsets that no plan gives (a plan of more rows, or of none of these): no row outside of the call's is read or written, and
the gradients are the sums over the rows that there are."""
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def _step(offsets, x, dc, w):
    T, R, K, N, L = x.shape[0], w.rank, w.k, w.n, w.count
    rows = torch.arange(T, dtype=torch.int32, device=DEV)
    plan = nv.MoEPlan(torch.tensor(offsets, dtype=torch.int32, device=DEV), rows, rows[:, None].contiguous())
    back = torch.full((nv.lib().nvfp4_adapter_backward_workspace_size(T, N, K, R, L) // 4,), -1, dtype=torch.int32, device=DEV)
    _, h = nv.nvfp4_adapter(x, w, plan=plan, with_h=True)
    return nv.nvfp4_adapter_backward(dc, x, w, h, plan=plan, workspace=back)


@pytest.mark.parametrize("T", [90, 3000])
@pytest.mark.parametrize("R", [16, 72])
def test_offsets_beyond_the_rows(T, R):
    K, N, L = 264, 328, 3
    g = torch.Generator(device=DEV).manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)
    w = nv.Adapters(r(L * R, K), r(L * N, R), torch.ones(L, device=DEV), R, K, N, L)
    x, dc = r(T, K), r(T, N)
    half = T // 2
    good = _step([0, half, T, T], x, dc, w)
    for offsets in ([0, half, T, 2 * T], [0, half, 5 * T, 6 * T], [0, half, 1 << 30, (1 << 31) - 1]):
        got = _step(offsets, x, dc, w)
        assert torch.equal(got.dx, good.dx) and torch.equal(got.da, good.da) and torch.equal(got.db, good.db), offsets
    # an adapter whose rows start far before the first (no workgroup meets the others' then), and offsets that fall
    for offsets in ([-(1 << 20), half, T, T], [T, half, 0, 0]):
        got = _step(offsets, x, dc, w)
        assert not got.da.any() and not got.db.any(), offsets
