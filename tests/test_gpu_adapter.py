"""Low-rank adapters and their gradients on the GPU against 64-bit references.

Every result is a sum of products of exact bf16 numbers over two contractions.  In 32 bits a sum of n terms is within n x
2^-24 of the sum of their magnitudes (whatever its order); here n is the longer of the sums, and the first sum's error goes
through the second: (n1 + n2) x 2^-24 of the magnitudes' product bounds it, with n the terms that one accumulator takes in
turn.  Between the two, a value is replaced by bf16 pieces: two leave 2^-16 of it, three 2^-24.  A bf16 result adds its
rounding, 2^-8."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import block_ref, tune_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U
F32, BF16 = torch.float32, torch.bfloat16


def _plan(ids, L):
    offsets, rows, pos = block_ref.plan(ids, L)
    to = lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(torch.int32).to(DEV)
    return nv.MoEPlan(to(offsets), to(rows), to(pos)), rows


def _factors(L, R, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    a = (torch.randn(L * R, K, generator=g) * K ** -0.5).to(BF16)
    b = (torch.randn(L * N, R, generator=g) * R ** -0.5).to(BF16)
    s = torch.rand(L, generator=g) + 0.5
    return nv.Adapters(a.to(DEV), b.to(DEV), s.to(DEV), R, K, N, L), a.double().numpy().reshape(L, R, K), \
        b.double().numpy().reshape(L, N, R), s.double().numpy()


def _bound(mag, terms, dtype, want):
    if dtype == BF16:
        return (terms * U + 2.0 ** -16) * mag + 2.0 ** -8 * np.abs(want)
    return ((terms + 4) * U) * mag


def _ids(T, L, kind, seed):
    g = np.random.default_rng(seed)
    if kind == "each":      # a request a token
        return g.integers(-1, L, (T, 1))
    if kind == "segments":  # ragged requests, some with none, some adapters without rows
        ends = np.sort(g.integers(0, T + 1, min(T, 6)))
        of = g.integers(-1, max(1, L - 1), len(ends) + 1)
        return of[np.searchsorted(ends, np.arange(T), side="right")][:, None]
    if kind == "none":
        return np.full((T, 1), -1)
    return np.zeros((T, 1), dtype=np.int64)


# tokens, K, N, rank, adapters, whose
CASES = [(1, 64, 32, 8, 1, "one"), (1, 8, 1, 16, 3, "each"), (5, 72, 40, 24, 4, "each"), (16, 520, 257, 16, 16, "each"),
         (17, 1000, 300, 32, 2, "segments"), (48, 2048, 512, 16, 64, "each"), (64, 136, 33, 128, 3, "segments"),
         (200, 256, 100, 64, 5, "none"), (257, 512, 264, 16, 1, "one"), (300, 200, 520, 8, 4, "segments"),
         (500, 1032, 271, 40, 7, "segments"), (1100, 264, 528, 112, 3, "segments"), (1200, 4096, 72, 128, 2, "segments"),
         (777, 328, 1024, 64, 9, "segments"), (600, 64, 128, 48, 512, "each")]


@pytest.mark.parametrize("T,K,N,R,L,kind", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("based", [True, False])
def test_by_token(T, K, N, R, L, kind, dtype, based):
    w, a, b, s = _factors(L, R, K, N, T + K)
    ids = _ids(T, L, kind, T + N)
    plan, rows = _plan(ids, L)
    g = torch.Generator().manual_seed(3)
    x, base = torch.randn(T, K, generator=g).to(BF16), torch.randn(T, N, generator=g).to(dtype)
    got, h = nv.nvfp4_adapter(x.to(DEV), w, base.to(DEV) if based else None, plan=plan, by_token=True, out_dtype=dtype, with_h=True)
    want, h64, mag = ref.adapter(x.double().numpy(), a, b, s, ids[:, 0], base.double().numpy() if based else np.zeros((T, N)), np.arange(T))
    assert got.dtype == dtype and np.all(np.abs(got.cpu().double().numpy() - want) <= _bound(mag, K + 2 * R + 8, dtype, want))
    n = int((ids >= 0).sum())
    at = rows[:n]
    xa = np.abs(x.double().numpy()[at])
    hm = np.stack([np.abs(a[ids[t, 0]]) @ xa[i] for i, t in enumerate(at)]) if n else np.zeros((0, R))
    assert np.all(np.abs(h[:n].cpu().double().numpy() - h64[at]) <= K * U * hm)
    if based:  # in place: the same bits
        c = base.to(DEV)
        assert nv.nvfp4_adapter(x.to(DEV), w, c, plan=plan, by_token=True, out=c) is c and torch.equal(c, got)


@pytest.mark.parametrize("T,k,K,N,R,E", [(1, 2, 64, 48, 16, 4), (9, 2, 136, 33, 16, 4), (130, 4, 512, 256, 8, 16), (700, 3, 264, 72, 32, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_by_expert(T, k, K, N, R, E, dtype):
    """Rows in the plan's order, gathered in the call or before it."""
    w, a, b, s = _factors(E, R, K, N, T)
    g = np.random.default_rng(T)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)])
    ids[g.random(T) < 0.2, k - 1] = -1
    plan, rows = _plan(ids, E)
    owner = np.where(rows >= 0, ids.reshape(-1)[np.maximum(rows, 0)], -1)
    gen = torch.Generator().manual_seed(3)
    x, base = torch.randn(T, K, generator=gen).to(BF16), torch.randn(T * k, N, generator=gen).to(dtype)
    want, _, mag = ref.adapter(x.double().numpy(), a, b, s, owner, base.double().numpy(), np.maximum(rows, 0) // k)
    got = nv.nvfp4_adapter(x.to(DEV), w, base.to(DEV), plan=plan, gather=True)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= _bound(mag, K + 2 * R + 8, dtype, want))
    sorted_x = nv.nvfp4_moe_gather(x.to(DEV), plan)
    assert torch.equal(nv.nvfp4_adapter(sorted_x, w, base.to(DEV), plan=plan), got)


@pytest.mark.parametrize("T,K,N,R,L,kind", [c for c in CASES if c[2] % 8 == 0])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients(T, K, N, R, L, kind, dtype):
    w, a, b, s = _factors(L, R, K, N, T + K)
    ids = _ids(T, L, kind, T + N)
    plan, rows = _plan(ids, L)
    g = torch.Generator().manual_seed(4)
    x, dc, dxb = torch.randn(T, K, generator=g).to(BF16), torch.randn(T, N, generator=g).to(BF16), torch.randn(T, K, generator=g).to(dtype)
    _, h = nv.nvfp4_adapter(x.to(DEV), w, plan=plan, by_token=True, with_h=True)
    got = nv.nvfp4_adapter_backward(dc.to(DEV), x.to(DEV), w, h, dx_base=dxb.to(DEV), plan=plan, by_token=True)
    _, h64, _ = ref.adapter(x.double().numpy(), a, b, s, ids[:, 0], np.zeros((T, N)), np.arange(T))
    want, mag = ref.adapter_backward(dc.double().numpy(), x.double().numpy(), a, b, s, ids[:, 0], h64, dxb.double().numpy())
    assert np.all(np.abs(got.dx.cpu().double().numpy() - want[0]) <= _bound(mag[0], N + 3 * R + 8, dtype, want[0]))
    assert np.all(np.abs(got.da.cpu().double().numpy().reshape(a.shape) - want[1]) <= (N + 3 * T + 8) * U * mag[1])
    assert np.all(np.abs(got.db.cpu().double().numpy().reshape(b.shape) - want[2]) <= (K + 3 * T + 8) * U * mag[2])


def test_one_adapter_without_a_plan_and_rows_in_order():
    T, K, N, R = 333, 264, 136, 16
    w, a, b, s = _factors(1, R, K, N, 1)
    x, dc, base = (torch.randn(T, n, device=DEV).to(BF16) for n in (K, N, N))
    plan = nv.nvfp4_moe_plan(torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1)
    c, h = nv.nvfp4_adapter(x, w, base, with_h=True)
    d = nv.nvfp4_adapter_backward(dc, x, w, h)
    for how in (dict(by_token=True), {}):
        c2, h2 = nv.nvfp4_adapter(x, w, base, plan=plan, with_h=True, **how)
        d2 = nv.nvfp4_adapter_backward(dc, x, w, h2, plan=plan, **how)
        assert torch.equal(c, c2) and torch.equal(h, h2)
        assert torch.equal(d.dx, d2.dx) and torch.equal(d.da, d2.da) and torch.equal(d.db, d2.db)


def test_gradients_against_differences():
    """The loss sum(c z) is linear in each of x, A and B: its difference quotient is the gradient up to rounding."""
    T, K, N, R, L = 20, 32, 24, 8, 3
    w, a, b, s = _factors(L, R, K, N, 2)
    ids = _ids(T, L, "each", 5)
    plan, _ = _plan(ids, L)
    x, z = torch.randn(T, K).to(BF16), torch.randn(T, N).to(BF16)
    _, h = nv.nvfp4_adapter(x.to(DEV), w, plan=plan, by_token=True, with_h=True)
    d = nv.nvfp4_adapter_backward(z.to(DEV), x.to(DEV), w, h, plan=plan, by_token=True, dx_dtype=F32)
    loss = lambda x, a, b: (ref.adapter(x, a, b, s, ids[:, 0], np.zeros((T, N)), np.arange(T))[0] * z.double().numpy()).sum()
    x64 = x.double().numpy()
    for which, grad, shape in ((0, d.dx, x64.shape), (1, d.da, a.shape), (2, d.db, b.shape)):
        grad = grad.cpu().double().numpy().reshape(shape)
        for i in np.random.default_rng(which).integers(0, grad.size, 12):
            at = np.unravel_index(i, shape)
            parts = [x64, a, b]
            up, down = parts[which].copy(), parts[which].copy()
            up[at] += 0.5
            down[at] -= 0.5
            q = loss(*[up if j == which else p for j, p in enumerate(parts)]) - loss(*[down if j == which else p for j, p in enumerate(parts)])
            # terms of order one, at most T N R of them
            assert abs(q - grad[at]) <= (T + N + K) * U * np.sqrt(T * N * R) + 1e-12


def test_strides_in_place_and_untouched_rows():
    T, K, N, R, L = 300, 128, 96, 16, 4
    w, a, b, s = _factors(L, R, K, N, 7)
    ids = _ids(T, L, "segments", 11)
    ids[50:90] = -1
    plan, _ = _plan(ids, L)
    wide = torch.randn(T, K + 64, device=DEV).to(BF16)
    x = wide[:, 24:24 + K]
    big = torch.randn(T, N + 40, device=DEV).to(BF16)
    before = big.clone()
    c = big[:, 16:16 + N]
    want = nv.nvfp4_adapter(x.contiguous(), w, c.contiguous(), plan=plan, by_token=True)
    nv.nvfp4_adapter(x, w, c, plan=plan, by_token=True, out=c)
    assert torch.equal(c, want) and torch.equal(c[50:90], before[50:90, 16:16 + N])
    assert torch.equal(big[:, :16], before[:, :16]) and torch.equal(big[:, 16 + N:], before[:, 16 + N:])
    # columns that start anywhere take the element path: the same bits
    odd = torch.zeros(T, N + 3, device=DEV, dtype=BF16)
    nv.nvfp4_adapter(x, w, before[:, 16:16 + N], plan=plan, by_token=True, out=odd[:, 1:1 + N])
    assert torch.equal(odd[:, 1:1 + N], want) and not odd[:, 0].any() and not odd[:, 1 + N:].any()


def test_rows_without_an_adapter_are_not_read():
    """NaN in x, dc and the poisoned workspace of tokens without an adapter reach nothing."""
    T, K, N, R, L = 400, 256, 64, 32, 3
    w, *_ = _factors(L, R, K, N, 7)
    ids = _ids(T, L, "segments", 2)
    ids[100:180] = -1
    ids[300:301] = -1
    plan, _ = _plan(ids, L)
    x, dc = torch.randn(T, K, device=DEV).to(BF16), torch.randn(T, N, device=DEV).to(BF16)
    none = torch.from_numpy(ids[:, 0] < 0).to(DEV)
    clean = [torch.where(none[:, None], torch.zeros_like(t), t) for t in (x, dc)]
    dirty = [torch.where(none[:, None], torch.full_like(t, float("nan")), t) for t in (x, dc)]
    L_ = nv.lib()
    out = []
    for x_, dc_ in (clean, dirty):
        work = torch.full((L_.nvfp4_adapter_workspace_size(T, N, K, R, L) // 4,), -1, dtype=torch.int32, device=DEV)
        back = torch.full((L_.nvfp4_adapter_backward_workspace_size(T, N, K, R, L) // 4,), -1, dtype=torch.int32, device=DEV)
        c, h = nv.nvfp4_adapter(x_, w, plan=plan, by_token=True, with_h=True, workspace=work)
        d = nv.nvfp4_adapter_backward(dc_, x_, w, h, plan=plan, by_token=True, workspace=back)
        out.append((c, d.dx, d.da, d.db))
    for p, q in zip(*out):
        assert bool(torch.isfinite(q.float()).all()) and torch.equal(p, q)
    assert not out[1][0][none].any() and not out[1][1][none].any()


@pytest.mark.parametrize("T,K,N,R,L", [(3, 64, 48, 16, 2), (90, 520, 264, 24, 4), (700, 264, 328, 64, 3)])
def test_no_numbers_stay_in_their_rows(T, K, N, R, L):
    """Infinities and NaN of a token, or of an adapter's factors, reach no other token and no other adapter's gradients."""
    w, *_ = _factors(L, R, K, N, 7)
    ids = np.arange(T)[:, None] % L
    plan, _ = _plan(ids, L)
    x, dc, base = (torch.randn(T, n, device=DEV).to(BF16) for n in (K, N, N))
    mine = torch.from_numpy(ids[:, 0] == 1).to(DEV)

    def step(w, x, dc, base):
        c, h = nv.nvfp4_adapter(x, w, base, plan=plan, by_token=True, with_h=True)
        d = nv.nvfp4_adapter_backward(dc, x, w, h, plan=plan, by_token=True)
        return c, d.dx, d.da.view(L, R, K), d.db.view(L, N, R)

    clean = step(w, x, dc, base)
    for bad in (float("inf"), float("nan")):
        x2, dc2, base2 = x.clone(), dc.clone(), base.clone()
        x2[1, 3], dc2[1, N - 1], base2[1, 5] = bad, bad, bad  # (token 1 has adapter 1)
        dirty = step(w, x2, dc2, base2)
        for p, q in zip(clean[:2], dirty[:2]):
            assert torch.equal(p[2:], q[2:]) and torch.equal(p[0], q[0]) and not bool(torch.isfinite(q[1].float()).all())
        for p, q in zip(clean[2:], dirty[2:]):
            assert torch.equal(p[0], q[0]) and torch.equal(p[2:], q[2:])
        a2, b2 = w.a.clone(), w.b.clone()
        a2.view(L, R, K)[1] = bad
        b2.view(L, N, R)[1] = bad
        dirty = step(nv.Adapters(a2, b2, w.scales, R, K, N, L), x, dc, base)
        for p, q in zip(clean[:2], dirty[:2]):
            assert torch.equal(p[~mine], q[~mine]) and not bool(torch.isfinite(q[mine].float()).any())
        for p, q in zip(clean[2:], dirty[2:]):
            assert torch.equal(p[0], q[0]) and torch.equal(p[2:], q[2:])


def test_no_rows():
    w, *_ = _factors(3, 16, 64, 32, 1)
    x = torch.empty(0, 64, dtype=BF16, device=DEV)
    plan = nv.nvfp4_moe_plan(torch.empty(0, 1, dtype=torch.int32, device=DEV), 3)
    c, h = nv.nvfp4_adapter(x, w, plan=plan, by_token=True, with_h=True)
    d = nv.nvfp4_adapter_backward(torch.empty(0, 32, dtype=BF16, device=DEV), x, w, h, plan=plan, by_token=True)
    assert c.shape == (0, 32) and d.dx.shape == (0, 64) and not d.da.any() and not d.db.any()


@pytest.mark.parametrize("T", [40, 700])
def test_another_stream_and_graph_replays(T):
    K, N, R, L = 512, 256, 16, 8
    w, *_ = _factors(L, R, K, N, 1)
    ids = torch.from_numpy(_ids(T, L, "each", 2)).to(torch.int32).to(DEV)
    x, dc, base = (torch.randn(T, n, device=DEV).to(BF16) for n in (K, N, N))

    def step():
        plan = nv.nvfp4_moe_plan(ids, L)
        c, h = nv.nvfp4_adapter(x, w, base, plan=plan, by_token=True, with_h=True)
        d = nv.nvfp4_adapter_backward(dc, x, w, h, plan=plan, by_token=True)
        return c, d.dx, d.da, d.db

    first = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = step()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.mul_(-1.5)
        ids.copy_((ids + 2) % (L + 1) - 1)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


def test_bad_rows_are_skipped():
    """Rows outside the tokens (no plan gives them) write nothing."""
    T, K, N, R = 80, 64, 32, 16
    w, *_ = _factors(1, R, K, N, 1)
    plan = nv.nvfp4_moe_plan(torch.zeros(T, 1, dtype=torch.int32, device=DEV), 1)
    x, base = torch.randn(T, K, device=DEV).to(BF16), torch.randn(T, N, device=DEV).to(BF16)
    want = nv.nvfp4_adapter(x, w, base, plan=plan, by_token=True)
    plan.rows[5], plan.rows[7] = T + 3, -4
    out = torch.full_like(base, 9.0)
    nv.nvfp4_adapter(x, w, base, plan=plan, by_token=True, out=out)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[5] = keep[7] = False
    assert torch.equal(out[keep], want[keep]) and bool((out[~keep] == 9.0).all())
