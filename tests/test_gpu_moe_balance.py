"""The balance loss, its counts and gradient on the GPU against 64-bit references.

A probability in 32 bits is off, relative to itself, by the rounding of l - max l (|l - max l| x 2^-24 in the exponent; a
sigmoid has none), two roundings of an exponential, those of a sum of E positive terms (a lane's E / 16 and four levels),
and a handful of single operations: (|l - max l| + E / 16 + 24) x 2^-24 bounds it.  A sum of N positive terms adds at
most N x 2^-24.  In the gradient c p (n_e - mean n) both differences are taken from the count of the likeliest expert, so
their errors are relative to |n_e - ref| and to sum p |n - ref|."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import tune_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = ref.U


def _inputs(T, E, k, dtype, seed, masked=False, std=1.5):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(T, E, generator=g) * std).to(dtype)
    ids = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k].to(torch.int32).contiguous()
    if masked:
        shut = torch.rand(T, E, generator=g) < 0.1
        logits = logits.masked_fill(shut, -np.inf)
        logits[torch.rand(T, generator=g) < 0.1] = float("nan")   # tokens with nothing open
        ids[shut.gather(1, ids.long())] = -1
        ids[torch.isnan(logits).all(dim=1)] = -1
    return logits, ids


def _check_forward(got, logits, ids, coef, S, sigmoid):
    loss, counts, mean, tokens = ref.balance(logits.double().numpy(), ids.numpy(), coef, S, sigmoid)
    assert np.array_equal(got.counts.cpu().numpy(), counts) and np.array_equal(got.tokens.cpu().numpy(), tokens)
    E, seq = logits.shape[1], logits.shape[0] // S
    l = logits.double().numpy()
    deep = 0.0
    if not sigmoid:
        fin = np.where(np.isfinite(l), l, np.nan)
        with np.errstate(all="ignore"):
            import warnings
            with warnings.catch_warnings():
                warnings.simplefilter("ignore")
                spans = np.nanmax(fin, axis=1) - np.nanmin(fin, axis=1)
        deep = min(float(np.nan_to_num(spans).max(initial=0.0)), 110.0)
    rel = (deep + E / 16 + 24 + seq) * U
    assert np.all(np.abs(got.probs.cpu().double().numpy() - mean) <= rel * mean + 2.0 ** -126)
    # the shares are positive too: the loss adds S E terms of five roundings each
    assert abs(float(got.loss) - loss) <= (rel + (5 + S + E / 64 + 20) * U) * abs(loss) + 2.0 ** -126
    return counts, tokens


CASES = [(1, 4, 1, 1), (1, 512, 32, 1), (63, 64, 8, 1), (64, 64, 8, 1), (65, 64, 8, 1), (100, 160, 6, 4), (1000, 100, 3, 5),
         (4097, 256, 8, 1), (48, 17, 2, 48), (600, 384, 10, 300), (2048, 33, 4, 2)]


@pytest.mark.parametrize("T,E,k,S", CASES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_and_gradient(T, E, k, S, dtype, sigmoid, masked):
    logits, ids = _inputs(T, E, k, dtype, T + E, masked)
    flags = nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0
    got = nv.nvfp4_moe_balance(logits.to(DEV), ids.to(DEV), 0.01, flags=flags, sequences=S)
    counts, tokens = _check_forward(got, logits, ids, 0.01, S, sigmoid)
    dloss = torch.tensor([1.7])
    d = nv.nvfp4_moe_balance_backward(logits.to(DEV), ids.to(DEV), got, 0.01, flags=flags, dloss=dloss.to(DEV))
    want, tol = ref.balance_backward(logits.double().numpy(), ids.numpy(), counts, tokens, 0.01, sigmoid, float(dloss))
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(d.cpu().double().numpy() - want) <= tol)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_gradient_against_differences(sigmoid):
    T, E, k, S = 24, 12, 3, 2
    logits, ids = _inputs(T, E, k, torch.float32, 5)
    flags = nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0
    b = nv.nvfp4_moe_balance(logits.to(DEV), ids.to(DEV), 1.0, flags=flags, sequences=S)
    d = nv.nvfp4_moe_balance_backward(logits.to(DEV), ids.to(DEV), b, 1.0, flags=flags).cpu().double().numpy()
    l, i, h = logits.double().numpy(), ids.numpy(), 1e-5
    for t, e in ((0, 0), (5, 11), (13, 4), (23, 7)):
        up, down = l.copy(), l.copy()
        up[t, e] += h
        down[t, e] -= h
        slope = (ref.balance(up, i, 1.0, S, sigmoid)[0] - ref.balance(down, i, 1.0, S, sigmoid)[0]) / (2 * h)
        # a central difference is off by h^2 / 6 x the third derivative (below 10 here) and 64-bit rounding / h
        assert abs(d[t, e] - slope) <= 10 * h * h + 1e-15 * 50 / h + 1e-6 * abs(slope)


def test_one_expert_with_nearly_all_of_the_score():
    """Its gradient is the others' terms, far below the rounding of a difference from its own."""
    T, E, k = 32, 64, 2
    logits, ids = _inputs(T, E, k, torch.float32, 9)
    logits[:, 5] += 18.0
    ids[:, 0] = 5
    ids[:, 1] = 6 + torch.arange(T, dtype=torch.int32) % 8
    b = nv.nvfp4_moe_balance(logits.to(DEV), ids.to(DEV), 1.0)
    d = nv.nvfp4_moe_balance_backward(logits.to(DEV), ids.to(DEV), b, 1.0).cpu().double().numpy()
    _, counts, _, tokens = ref.balance(logits.double().numpy(), ids.numpy(), 1.0, 1, False)
    want, tol = ref.balance_backward(logits.double().numpy(), ids.numpy(), counts, tokens, 1.0, False)
    assert np.all(np.abs(d - want) <= tol) and np.all(tol[:, 5] < 2e-5 * np.abs(want[:, 5]))


@pytest.mark.parametrize("sigmoid", [False, True])
def test_infinities_and_lowest_values(sigmoid):
    low = float(np.finfo(np.float32).min)
    logits = torch.tensor([[np.inf, 0.0, -np.inf, 1.0, np.nan, low],
                           [low, low, low, low, low, low],
                           [-np.inf] * 6,
                           [90.0, -90.0, 104.0, -104.0, 3e38, -3e38],
                           [np.inf, np.inf, 0.0, 0.0, 0.0, 0.0]], dtype=torch.float32)
    ids = torch.tensor([[0, 3], [1, 0], [2, 5], [4, 2], [0, 1]], dtype=torch.int32)  # (a closed expert may be named)
    flags = nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0
    b = nv.nvfp4_moe_balance(logits.to(DEV), ids.to(DEV), 1.0, flags=flags)
    counts, tokens = _check_forward(b, logits, ids, 1.0, 1, sigmoid)
    assert tokens[0] == 5
    d = nv.nvfp4_moe_balance_backward(logits.to(DEV), ids.to(DEV), b, 1.0, flags=flags).cpu().double().numpy()
    with np.errstate(all="ignore"):
        want, tol = ref.balance_backward(logits.double().numpy(), ids.numpy(), counts, tokens, 1.0, sigmoid)
    assert np.all(np.isfinite(d)) and np.all(np.abs(d - want) <= tol)


def test_added_in_place_with_strides_and_padding_untouched():
    T, E, k = 70, 40, 3
    logits, ids = _inputs(T, E, k, torch.float32, 3)
    ids[10:20] = -1
    wide = torch.randn(T, E + 9)
    view = wide.to(DEV)[:, 4:4 + E]
    big = torch.zeros(T, E + 5, device=DEV)
    big[:, 2:2 + E] = logits.to(DEV)
    b = nv.nvfp4_moe_balance(big[:, 2:2 + E], ids.to(DEV), 0.5)
    before = view.clone()
    out = nv.nvfp4_moe_balance_backward(big[:, 2:2 + E], ids.to(DEV), b, 0.5, dlogits=view, out=view)
    assert out.data_ptr() == view.data_ptr() and torch.equal(view[10:20], before[10:20])
    _, counts, _, tokens = ref.balance(logits.double().numpy(), ids.numpy(), 0.5, 1, False)
    want, tol = ref.balance_backward(logits.double().numpy(), ids.numpy(), counts, tokens, 0.5, False)
    got, was = view.cpu().double().numpy(), before.cpu().double().numpy()
    assert np.all(np.abs(got - (was + want)) <= tol + U * np.abs(was + want))
    # nothing beside the view
    whole = view._base.cpu()
    assert torch.equal(whole[:, :4], wide[:, :4]) and torch.equal(whole[:, 4 + E:], wide[:, 4 + E:])


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_masked_places_of_a_loss_that_is_no_number(sigmoid, bad):
    T, E, k = 37, 24, 2
    logits, ids = _inputs(T, E, k, torch.float32, 11)
    logits[:, 3] = -np.inf
    logits[5, :] = np.nan
    ids[7:9] = -1
    flags = nv.NVFP4_ROUTE_SIGMOID if sigmoid else 0
    b = nv.nvfp4_moe_balance(logits.to(DEV), ids.to(DEV), 1.0, flags=flags)
    given = torch.randn(T, E).to(DEV)
    d = nv.nvfp4_moe_balance_backward(logits.to(DEV), ids.to(DEV), b, 1.0, flags=flags, dloss=torch.tensor([bad]).to(DEV), dlogits=given)
    assert torch.equal(d[:, 3], given[:, 3]) and torch.equal(d[5], given[5]) and torch.equal(d[7:9], given[7:9])
    assert not torch.isfinite(d[0, 0]) and not torch.isfinite(d[36, 23])


def test_counts_of_all_ranks():
    """Counts and tokens summed over two halves give each half its part of the whole batch's gradient."""
    logits, ids = _inputs(128, 24, 2, torch.float32, 21)
    L, I = logits.to(DEV), ids.to(DEV)
    whole = nv.nvfp4_moe_balance(L, I, 1.0)
    halves = [nv.nvfp4_moe_balance(L[i:i + 64], I[i:i + 64], 1.0) for i in (0, 64)]
    both = nv.MoEBalance(None, halves[0].counts + halves[1].counts, None, halves[0].tokens + halves[1].tokens)
    assert torch.equal(both.counts, whole.counts) and torch.equal(both.tokens, whole.tokens)
    d = nv.nvfp4_moe_balance_backward(L, I, whole, 1.0)
    parts = torch.cat([nv.nvfp4_moe_balance_backward(L[i:i + 64], I[i:i + 64], both, 1.0) for i in (0, 64)])
    assert torch.equal(d, parts)


def test_the_same_bits_and_another_stream():
    logits, ids = _inputs(3000, 100, 6, torch.bfloat16, 2)
    L, I = logits.to(DEV), ids.to(DEV)
    a = nv.nvfp4_moe_balance(L, I, 0.1, sequences=3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = nv.nvfp4_moe_balance(L, I, 0.1, sequences=3)
    s.synchronize()
    assert torch.equal(a.loss, b.loss) and torch.equal(a.probs, b.probs) and torch.equal(a.counts, b.counts)


def test_graph_replays():
    logits, ids = _inputs(2000, 64, 4, torch.float32, 2)
    L, I = logits.to(DEV), ids.to(DEV)
    work = torch.empty(nv.lib().nvfp4_moe_balance_workspace_size(2000, 64, 2) // 4, dtype=torch.int32, device=DEV)

    def step():
        b = nv.nvfp4_moe_balance(L, I, 0.1, sequences=2, workspace=work)
        return b, nv.nvfp4_moe_balance_backward(L, I, b, 0.1)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b, d = step()
    for i in range(4):
        L.copy_(logits * (1 + 0.25 * i))
        work.fill_(-1)  # whatever the workspace holds
        graph.replay()
        torch.cuda.synchronize()
        eb, ed = step()
        assert torch.equal(b.loss, eb.loss) and torch.equal(b.counts, eb.counts) and torch.equal(d, ed)


def test_no_tokens():
    L, I = torch.empty(0, 8, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    for S in (1, 3):
        b = nv.nvfp4_moe_balance(L, I, 1.0, sequences=S)
        assert float(b.loss) == 0.0 and not b.counts.any() and not b.probs.any() and not b.tokens.any()
        assert nv.nvfp4_moe_balance_backward(L, I, b, 1.0).shape == (0, 8)
