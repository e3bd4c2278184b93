"""8-bit products by expert, read through a plan, where an expert has more rows than there are tokens: ids that
name an expert several times in a token (unavoidable with more choices than experts), and row maps of any kind.  The
sums are exact, so every row is compared for equality, and rows without an expert stay as they were."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import block_ref as ref
from tests.test_gpu_int8 import _int8, _want

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _check_rows(out, offsets, source, a, b, N):
    for e in range(len(offsets) - 1):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            src, w = torch.as_tensor(source[lo:hi]).to(DEV), slice(e * N, (e + 1) * N)
            want = _want(a.data[src], a.scales[src], b.data[w], b.scales[w], out.dtype)
            wrong = (out[lo:hi] != want).any(dim=1).nonzero().flatten().tolist()
            assert not wrong, f"expert {e}: rows {wrong[:8]}.. of {hi - lo}"
    assert (out[int(offsets[-1]):] == 3).all()


def _ids(kind, T, k, E):
    if kind == "one":       # all slots on one expert
        return torch.full((T, k), E - 1, dtype=torch.int32)
    g = torch.Generator().manual_seed(T + k)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    if kind == "two":       # an unequal pair of experts
        ids = (torch.rand(T, k, generator=g) < 0.2).to(torch.int32) * (E - 1)
    ids[torch.rand(T, k, generator=g) < 0.1] = -1
    return ids


# tokens up to 16, 32, 64 (one tile of rows for distinct experts) and more (at most 24 rows an expert on average)
@pytest.mark.parametrize("T,k,E", [(17, 2, 1), (40, 2, 4), (64, 8, 3), (3, 8, 5), (10, 8, 4), (20, 8, 2), (60, 8, 6), (1, 32, 2),
                                   (100, 8, 64), (70, 2, 7), (300, 3, 40)])
@pytest.mark.parametrize("kind", ["one", "two", "any"])
@pytest.mark.parametrize("N,K,dtype", [(70, 272, torch.bfloat16), (130, 1040, torch.float32)])
def test_repeated_experts(T, k, E, kind, N, K, dtype):
    ids = _ids(kind, T, k, E)
    plan = nv.nvfp4_moe_plan(ids.to(DEV), E)
    offsets, rows, _ = ref.plan(ids.numpy(), E)
    a, b = _int8(T, K, seed=3), _int8(N, K, E, seed=4)
    out = torch.full((T * k, N), 3.0, dtype=dtype, device=DEV)
    nv.nvfp4_int8_gemm(a, b, plan=plan, gather=True, out=out)
    _check_rows(out.cpu(), offsets, rows // k, a, b, N)


def test_repeated_experts_with_weights_beyond_the_cache():
    T, k, E, N, K = 10, 8, 512, 1024, 512
    assert E * N * K >= 2 ** 28
    ids = _ids("two", T, k, E)
    g = torch.Generator(device=DEV).manual_seed(7)
    b = nv.Int8Tensor(torch.randint(-127, 128, (E * N, K), generator=g, device=DEV, dtype=torch.int8),
                      torch.rand(E * N, generator=g, device=DEV) * 0.01 + 1e-4, N, K, E)
    a = _int8(T, K, seed=3)
    plan = nv.nvfp4_moe_plan(ids.to(DEV), E)
    offsets, rows, _ = ref.plan(ids.numpy(), E)
    out = torch.full((T * k, N), 3.0, dtype=torch.bfloat16, device=DEV)
    nv.nvfp4_int8_gemm(a, b, plan=plan, gather=True, out=out)
    _check_rows(out.cpu(), offsets, rows // k, a, b, N)


@pytest.mark.parametrize("a_rows,M,row_div,offsets", [(10, 80, 2, [0, 50, 80]), (1, 200, 1, [0, 0, 200]), (70, 190, 3, [0] + [3] * 7 + [180]),
                                                      (33, 400, 4, [0, 1, 390])])
def test_any_map_of_rows(a_rows, M, row_div, offsets):
    E, N, K = len(offsets) - 1, 100, 400
    rows = torch.randint(0, a_rows * row_div, (M,), generator=torch.Generator().manual_seed(M), dtype=torch.int32)
    a, b = _int8(a_rows, K, seed=5), _int8(N, K, E, seed=6)
    out = torch.full((M, N), 3.0, device=DEV)
    dev_rows, dev_offsets = rows.to(DEV), torch.tensor(offsets, dtype=torch.int32, device=DEV)
    status = nv.lib().nvfp4_int8_gemm(a.data.data_ptr(), a.scales.data_ptr(), a_rows, b.data.data_ptr(), b.scales.data_ptr(), M, N,
                                      K, out.data_ptr(), nv.NVFP4_F32, N, E, dev_offsets.data_ptr(), dev_rows.data_ptr(), row_div,
                                      None, torch.cuda.current_stream().cuda_stream)
    assert status == nv.NVFP4_OK
    _check_rows(out.cpu(), np.array(offsets), rows.numpy() // row_div, a, b, N)
