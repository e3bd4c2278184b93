"""The bf16 pieces of an adapter's h and g: all 24 bits of a number reach fp32 results.

The factors are one power of two by rank column, alpha_q at the elements k with k mod R = q (beta_q likewise), so that every
element of c and dx is ONE product, and x and dc have in each row three groups of elements of 1, 2^-9 and 2^-18: h and g are a power
of two times 1 + 2^-9 + 2^-18, which takes exactly three pieces, each 2^-9 of the one before.  Rows that share their groups
add equal powers with signs; at most 63 of them make sums of fewer than 2^24 units of 2^-18, so every sum is exact in 32 bits in
whatever order, and results have to be equal."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests.test_gpu_adapter import _plan

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _factor(count, n, R):
    """[count, R, n]: powers of two at n mod R = q."""
    f = torch.zeros(count, R, n, dtype=torch.float64)
    i = torch.arange(n)
    for g in range(count):
        f[g, i % R, i] = 2.0 ** ((i % R + g) % 3 - 1).double()
    return f


def _sparse(T, n, R, ids, L, turn):
    """[T, n]: three groups of R elements a row; rows of an adapter share them in turn.  The sign changes every `turn` rows."""
    triples = n // (3 * R)
    v = torch.zeros(T, n, dtype=torch.float64)
    seen = np.zeros(L, dtype=int)
    for t in range(T):
        g = max(int(ids[t, 0]), 0)
        first = seen[g] % triples * 3
        for j in range(3):
            v[t, (first + j) * R:(first + j + 1) * R] = 2.0 ** (-9 * j) * (1 - 2 * (t // turn % 2))
        seen[g] += 1
    assert seen.max() <= 63 * triples
    return v


# tokens, K, N, rank, adapters: one launch up to rank 32; rows of 16 with one and several splits; rows of 64
CASES = [(5, 256, 128, 8, 1), (16, 256, 264, 16, 2), (40, 512, 264, 24, 3), (30, 512, 520, 32, 2),
         (48, 4096, 2056, 16, 64), (48, 4096, 2056, 24, 64), (100, 2048, 512, 64, 4), (200, 1032, 1544, 128, 2),
         (700, 2048, 2056, 8, 2), (700, 2048, 2056, 16, 2), (700, 1544, 2056, 24, 3), (600, 1544, 2056, 40, 2),
         (900, 2560, 1032, 64, 3), (500, 2048, 2056, 72, 2), (600, 4096, 2056, 128, 2)]


@pytest.mark.parametrize("T,K,N,R,L", CASES)
def test_all_bits_of_h_and_g(T, K, N, R, L):
    ids = (np.arange(T) * 7 % L)[:, None]
    ids[T // 2:T // 2 + 3] = -1
    plan, _ = _plan(ids, L)
    a, b = _factor(L, K, R), _factor(L, N, R).transpose(1, 2).contiguous()  # [L, R, K], [L, N, R]
    x, dc = _sparse(T, K, R, ids, L, 3), _sparse(T, N, R, ids, L, 5)
    w = nv.Adapters(a.reshape(L * R, K).to(BF16).to(DEV), b.reshape(L * N, R).to(BF16).to(DEV), torch.ones(L, device=DEV), R, K, N, L)
    want_c, want_dx = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    want_da, want_db = torch.zeros(L, R, K, dtype=torch.float64), torch.zeros(L, N, R, dtype=torch.float64)
    for g in range(L):
        at = torch.from_numpy(np.flatnonzero(ids[:, 0] == g))
        h, dh = x[at] @ a[g].t(), dc[at] @ b[g]
        want_c[at], want_dx[at] = h @ b[g].t(), dh @ a[g]
        want_da[g], want_db[g] = dh.t() @ x[at], dc[at].t() @ h
    c, h = nv.nvfp4_adapter(x.to(BF16).to(DEV), w, plan=plan, by_token=True, out_dtype=F32, with_h=True)
    d = nv.nvfp4_adapter_backward(dc.to(BF16).to(DEV), x.to(BF16).to(DEV), w, h, plan=plan, by_token=True, dx_dtype=F32)
    for name, got, want in (("c", c, want_c), ("dx", d.dx, want_dx), ("da", d.da, want_da.view(L * R, K)),
                            ("db", d.db, want_db.reshape(L * N, R))):
        assert torch.equal(want.float().double(), want) and want.any()
        assert torch.equal(got.cpu(), want.float()), name
