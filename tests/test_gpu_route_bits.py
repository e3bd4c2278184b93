"""The bits of a routing key.  Each tested expert A stands between two others of lower and higher index whose keys are
exactly the score that A has by IEEE division: the row's order is then B, A, C (ties to the lower index) only if A's
key has exactly those bits.  Checked alone, and beside a token whose scores need the general division.

The sigmoid's reciprocals are taken at every significand where one Newton step from a start that is an ulp off would
miss (found here by trying them all), and at random ones."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32_MAX = torch.finfo(torch.float32).max
TRIPLES = 10


def _hard_significands():
    """x in [1, 2) where r + r (1 - x r), exactly summed and rounded once, misses RN(1 / x) for r = RN(1 / x) + or - an ulp."""
    x = np.arange(1 << 23, 1 << 24, dtype=np.uint32)
    x = (x & 0x7FFFFF | 0x3F800000).view(np.float32)
    t = np.float32(1) / x
    hard = np.zeros(x.shape, dtype=bool)
    for step in (-1, 1):
        r = (t.view(np.int32) + step).view(np.float32)
        e = np.longdouble(1) - x.astype(np.longdouble) * r.astype(np.longdouble)   # exact in 64 bits
        e = e.astype(np.float32).astype(np.longdouble)
        hard |= (e * r + r).astype(np.float32) != t
    return x[hard]


def _order(logits, bias, mate, flags):
    """Order of the token's experts by key, alone and with a token in the same wave that needs the general division."""
    rows = [logits[None], torch.stack([logits, mate]), torch.stack([mate, logits, mate])]
    got = [nv.nvfp4_moe_route(r, r.shape[1], flags, bias, with_plan=False)[:2] for r in rows]
    ids, w = zip(got[0], (got[1][0][:1], got[1][1][:1]), (got[2][0][1:2], got[2][1][1:2]))
    assert torch.equal(ids[0], ids[1]) and torch.equal(ids[0], ids[2])
    assert torch.equal(w[0], w[1]) and torch.equal(w[0], w[2])
    return ids[0][0].tolist(), w[0][0]


def _check(order, weights, scores, tested):
    place = {e: i for i, e in enumerate(order)}
    for i, e in enumerate(tested):
        assert place[e] == place[e - 1] + 1 and place[e + 1] == place[e] + 1, (e, scores[i].item().hex())
        assert weights[place[e]] == scores[i]


def test_sigmoid_scores_have_the_bits_of_a_division():
    hard = _hard_significands()
    assert 30 <= len(hard) <= 100
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.from_numpy(hard), 1 + torch.rand(300, generator=g)]).to(DEV)
    # logits whose 1 + exp(-l) is x: neighbours of -log(x - 1)
    near = (-torch.log(x.double() - 1)).float()[:, None].view(torch.int32) + torch.arange(-200, 201, device=DEV, dtype=torch.int32)
    near = near.view(torch.float32)
    hits = (1 + torch.exp(-near)) == x[:, None]
    found = hits.any(dim=1)
    assert found.float().mean() > 0.8
    l = near.gather(1, hits.int().argmax(dim=1, keepdim=True))[found, 0]
    scores = 1 / (1 + torch.exp(-l))
    mate = torch.full((3 * TRIPLES,), -200.0, device=DEV)
    for at in range(0, len(l), TRIPLES):
        s, n = scores[at:at + TRIPLES], len(l[at:at + TRIPLES])
        if len(torch.unique(s)) < n:
            continue
        logits = torch.full((3 * n,), F32_MAX, device=DEV)   # score 1, so the key 1 + (s - 1) is s exactly
        bias = torch.repeat_interleave(s - 1, 3)
        logits[1::3], bias[1::3] = l[at:at + TRIPLES], 0.0
        order, w = _order(logits, bias, mate[:3 * n], nv.NVFP4_ROUTE_SIGMOID)
        _check(order, w, s, range(1, 3 * n, 3))


@pytest.mark.parametrize("spread", [1.5, 12.0])
def test_softmax_scores_have_the_bits_of_a_division(spread):
    g = torch.Generator().manual_seed(2)
    n = TRIPLES
    mate = torch.full((3 * n,), -80.0, device=DEV)           # exp(-80) is below what the quotient takes
    mate[0] = 0.0
    for _ in range(60):
        l = (torch.randn(n, generator=g) * spread).to(DEV)
        logits = torch.full((3 * n,), -F32_MAX, device=DEV)  # score 0: the key is the bias
        logits[1::3] = l
        e = torch.zeros(32, device=DEV)
        e[:3 * n] = torch.exp(logits - l.max())
        total = e
        while len(total) > 1:
            total = total[0::2] + total[1::2]
        s = (e[:3 * n] / total)[1::3]
        if len(torch.unique(s)) < n:
            continue
        bias = torch.repeat_interleave(s, 3)
        bias[1::3] = 0.0
        order, w = _order(logits, bias, mate, 0)
        _check(order, w, s, range(1, 3 * n, 3))
