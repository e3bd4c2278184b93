"""Workspace of an adapter's backward call: the rows of a workgroup of the factors' gradients are whole steps of 32."""
import pytest

import nvfp4_bit_block_quantize_amd as nv


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 48, 56, 64, 72, 80, 88, 96, 104, 112, 120, 128])
def test_chunks_are_whole_steps(rank):
    """M rows of K = N = 8 for which the smallest chunk is taken: twice the rank or 64 rows, in steps of 32."""
    chunk = max(64, -(-2 * rank // 32) * 32)
    M, N, K, adapters = 200 * chunk, 8, 8, 2
    up = lambda n: -(-n // 256) * 256
    tiles = M // chunk + adapters
    want = up(adapters * rank * K * 2) + 2 * up(M * rank * 6) + up(M * rank * 4) + 2 * up(tiles * N * rank * 4)
    assert nv.lib().nvfp4_adapter_backward_workspace_size(M, N, K, rank, adapters) == want
