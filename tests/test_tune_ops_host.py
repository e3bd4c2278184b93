"""Refusals of the operators of fine-tuning: every bad argument is named on the host, before anything is enqueued (the
fake device addresses here are never read)."""
import ctypes
import math

import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv

P = 0x10000   # 16-byte aligned fake device address
ODD = 0x10002
OK, NULL, SHAPE, ALIGN, UNSUPPORTED = (nv.NVFP4_OK, nv.NVFP4_ERR_NULL, nv.NVFP4_ERR_SHAPE, nv.NVFP4_ERR_ALIGN,
                                       nv.NVFP4_ERR_UNSUPPORTED)


def _call(name, defaults, **changes):
    args = dict(defaults)
    assert set(changes) <= set(args), changes
    args.update(changes)
    return getattr(nv.lib(), name)(*args.values())


BALANCE = dict(logits=P, dtype=nv.NVFP4_F32, tokens=80, experts=64, ld=64, ids=P, top_k=4, sequences=2, flags=0, coef=0.01, loss=P,
               counts=P, probs=P, live=P, workspace=P, stream=None)
BBWD = dict(logits=P, dtype=nv.NVFP4_F32, tokens=80, experts=64, ld=64, ids=P, top_k=4, sequences=2, flags=0, coef=0.01, counts=P,
            live=P, dloss=None, dlogits_in=None, ld_in=0, dlogits=P, ldd=64, stream=None)
COMMON = [(dict(logits=None), NULL), (dict(ids=None), NULL), (dict(dtype=2), UNSUPPORTED), (dict(flags=8), UNSUPPORTED),
          (dict(coef=math.nan), UNSUPPORTED), (dict(coef=math.inf), UNSUPPORTED), (dict(tokens=-2), SHAPE), (dict(tokens=81), SHAPE),
          (dict(experts=0), SHAPE), (dict(experts=513, ld=513), SHAPE), (dict(ld=63), SHAPE), (dict(top_k=0), SHAPE),
          (dict(top_k=33), SHAPE), (dict(experts=3, ld=3), SHAPE), (dict(sequences=0), SHAPE), (dict(sequences=65536, tokens=65536), SHAPE),
          (dict(tokens=2**30), SHAPE), (dict(ld=2**62), SHAPE), (dict(logits=ODD), ALIGN), (dict(ids=ODD), ALIGN), (dict(live=ODD), ALIGN),
          (dict(counts=ODD), ALIGN), (dict(counts=None), NULL), (dict(live=None), NULL)]


@pytest.mark.parametrize("changes,status", COMMON + [
    (dict(loss=None), NULL), (dict(probs=None), NULL), (dict(workspace=None), NULL), (dict(workspace=0x10008), ALIGN),
    (dict(loss=ODD), ALIGN), (dict(probs=ODD), ALIGN)])
def test_balance(changes, status):
    assert _call("nvfp4_moe_balance", BALANCE, **changes) == status


@pytest.mark.parametrize("changes,status", COMMON + [
    (dict(dlogits=None), NULL), (dict(ldd=63), SHAPE), (dict(dlogits_in=P, ld_in=60), SHAPE), (dict(dlogits=ODD), ALIGN),
    (dict(dloss=ODD), ALIGN), (dict(dlogits_in=ODD, ld_in=64), ALIGN), (dict(tokens=0, logits=None, ids=None, dlogits=None), OK)])
def test_balance_backward(changes, status):
    assert _call("nvfp4_moe_balance_backward", BBWD, **changes) == status


def _grads(*ranges, dtype=nv.NVFP4_F32):
    n = len(ranges)
    return ((ctypes.c_void_p * n)(*[a for a, _ in ranges]), (ctypes.c_int64 * n)(*[c for _, c in ranges]),
            (ctypes.c_int32 * n)(*[dtype] * n), n)


def _norm(g, flags=0, norm=P, workspace=P):
    return nv.lib().nvfp4_grad_norm(*g, flags, norm, workspace, None)


def _clip(g, outs=None, norm=P, max_norm=1.0, eps=1e-6):
    a, c, d, n = g
    return nv.lib().nvfp4_grad_clip(a, a if outs is None else (ctypes.c_void_p * n)(*outs), c, d, n, norm, max_norm, eps, None)


def test_grad_norm():
    good = _grads((P, 8), (P + 64, 3))
    assert _norm(good, flags=2) == UNSUPPORTED and _norm(good, norm=None) == NULL and _norm(good, workspace=None) == NULL
    assert _norm(good, norm=ODD) == ALIGN and _norm(good, workspace=P + 8) == ALIGN
    assert _norm(_grads((P, 8), (None, 3))) == NULL and _norm(_grads((P, -1))) == SHAPE and _norm(_grads((P, 2**40 + 1))) == SHAPE
    assert _norm(_grads((P, 2**39), (P, 2**39), (P, 1))) == SHAPE
    assert _norm(_grads((ODD, 8))) == ALIGN and _norm(_grads((P + 1, 8), dtype=nv.NVFP4_BF16)) == ALIGN
    assert _norm(_grads((P, 8), dtype=5)) == UNSUPPORTED
    assert nv.lib().nvfp4_grad_norm(None, None, None, 2, 0, P, P, None) == NULL
    assert nv.lib().nvfp4_grad_norm(None, None, None, -1, 0, P, P, None) == SHAPE


def test_grad_clip():
    good = _grads((P, 8), (P + 64, 3))
    for bad in (-1.0, math.nan):
        assert _clip(good, max_norm=bad) == UNSUPPORTED and _clip(good, eps=bad) == UNSUPPORTED
    assert _clip(good, max_norm=0.0, eps=0.0) == UNSUPPORTED
    assert _clip(good, norm=None) == NULL and _clip(good, norm=ODD) == ALIGN
    assert _clip(good, outs=[P, None]) == NULL and _clip(good, outs=[P, ODD]) == ALIGN
    # one tensor twice, tensors that share bytes, an output over another tensor's input or its own
    assert _clip(_grads((P, 8), (P, 8))) == UNSUPPORTED and _clip(_grads((P, 8), (P + 28, 3))) == UNSUPPORTED
    assert _clip(good, outs=[P + 4096, P + 4100]) == UNSUPPORTED and _clip(good, outs=[P + 4096, P]) == UNSUPPORTED
    assert _clip(good, outs=[P + 4, P + 4096]) == UNSUPPORTED


ADAPTER = dict(x=P, x_dtype=nv.NVFP4_BF16, x_rows=80, ldx=64, a=P, b=P, scales=P, M=80, N=40, K=64, rank=48, adapters=3, offsets=P,
               rows=P, pos=P, row_div=1, flags=nv.NVFP4_ADAPTER_BY_TOKEN, base=P, ldb=40, c=P + 4096, c_dtype=nv.NVFP4_BF16, ldc=40, h=P,
               workspace=P, stream=None)
ABWD = dict(dc=P, dc_dtype=nv.NVFP4_BF16, lddc=40, x=P, x_dtype=nv.NVFP4_BF16, ldx=64, a=P, b=P, scales=P, M=80, N=40, K=64, rank=16,
            adapters=3, offsets=P, rows=P, pos=P, flags=nv.NVFP4_ADAPTER_BY_TOKEN, h=P, dx_base=P, ldb=64, dx=P + 4096,
            dx_dtype=nv.NVFP4_BF16, lddx=64, da=P, db=P, workspace=P, stream=None)
BOTH = [(dict(x=None), NULL), (dict(a=None), NULL), (dict(b=None), NULL), (dict(scales=None), NULL), (dict(rows=None), NULL),
        (dict(pos=None), NULL), (dict(workspace=None), NULL), (dict(x_dtype=nv.NVFP4_F32), UNSUPPORTED), (dict(flags=4), UNSUPPORTED),
        (dict(flags=3), UNSUPPORTED), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=2**24 + 8, ldx=2**24 + 8), SHAPE), (dict(K=0), SHAPE), (dict(K=60), SHAPE), (dict(ldx=56), SHAPE),
        (dict(rank=0), SHAPE), (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(adapters=0), SHAPE), (dict(adapters=513), SHAPE),
        (dict(offsets=None), SHAPE), (dict(offsets=None, adapters=1), SHAPE), (dict(ldb=8), SHAPE), (dict(ldx=2**62), SHAPE),
        (dict(M=2**31), SHAPE), (dict(x=P + 8), ALIGN), (dict(ldx=68), ALIGN), (dict(a=P + 8), ALIGN), (dict(b=P + 8), ALIGN),
        (dict(scales=ODD), ALIGN), (dict(offsets=ODD), ALIGN), (dict(rows=ODD), ALIGN), (dict(pos=ODD), ALIGN), (dict(h=P + 8), ALIGN),
        (dict(workspace=P + 8), ALIGN)]


@pytest.mark.parametrize("changes,status", BOTH + [
    (dict(c=None), NULL), (dict(c_dtype=2), UNSUPPORTED), (dict(ldc=39), SHAPE), (dict(x_rows=79), SHAPE), (dict(c=P, ldc=48), SHAPE),
    (dict(flags=nv.NVFP4_ADAPTER_GATHER, row_div=0), SHAPE), (dict(c=P + 1), ALIGN), (dict(base=P + 1), ALIGN),
    (dict(c=ODD, c_dtype=nv.NVFP4_F32), ALIGN), (dict(M=2**30, x_rows=2**30), SHAPE),
    (dict(M=0, x_rows=0, x=None, base=None, c=None, h=None, workspace=None), OK)])
def test_adapter(changes, status):
    assert _call("nvfp4_adapter", ADAPTER, **changes) == status


@pytest.mark.parametrize("changes,status", BOTH + [
    (dict(dc=None), NULL), (dict(dx=None), NULL), (dict(da=None), NULL), (dict(db=None), NULL), (dict(h=None), NULL),
    (dict(dc_dtype=nv.NVFP4_F32), UNSUPPORTED), (dict(flags=nv.NVFP4_ADAPTER_GATHER), UNSUPPORTED), (dict(dx_dtype=2), UNSUPPORTED),
    (dict(N=44, lddc=48), SHAPE), (dict(lddc=32), SHAPE), (dict(lddx=56), SHAPE), (dict(dx=P, lddx=72), SHAPE), (dict(dc=P + 8), ALIGN),
    (dict(lddc=44), ALIGN), (dict(da=P + 8), ALIGN), (dict(db=P + 8), ALIGN), (dict(M=2**30), SHAPE)])
def test_adapter_backward(changes, status):
    assert _call("nvfp4_adapter_backward", ABWD, **changes) == status


def test_workspace_sizes():
    L = nv.lib()
    assert L.nvfp4_moe_balance_workspace_size(64, 64, 1) == 0 and L.nvfp4_moe_balance_workspace_size(65, 64, 1) > 0
    assert L.nvfp4_moe_balance_workspace_size(64, 64, 2) > 0 and L.nvfp4_moe_balance_workspace_size(64, 0, 1) == 0
    assert L.nvfp4_grad_workspace_size(1, 1) == 16 and L.nvfp4_grad_workspace_size(-1, 1) == 0
    assert L.nvfp4_grad_workspace_size(3, 1 << 40) <= 2048 * 8
    assert L.nvfp4_adapter_workspace_size(4, 64, 512, 64, 2) >= 4 * 64 * 4 and L.nvfp4_adapter_workspace_size(4, 64, 512, 0, 2) == 0
    assert L.nvfp4_adapter_backward_workspace_size(4, 64, 512, 16, 2) >= 2 * 2 * 16 * (64 + 512)
    assert L.nvfp4_adapter_backward_workspace_size(-1, 64, 512, 16, 2) == 0


def test_binding_refuses_wrong_tensors():
    f, i = torch.zeros(8, 64), torch.zeros(8, 4, dtype=torch.int32)
    b = nv.MoEBalance(torch.zeros(1), torch.zeros(1, 64, dtype=torch.int32), torch.zeros(1, 64), torch.zeros(1, dtype=torch.int32))
    h, one = f.bfloat16(), torch.ones(1)
    w = nv.Adapters(torch.zeros(16, 64).bfloat16(), torch.zeros(24, 16).bfloat16(), one, 16, 64, 24)
    w2 = nv.Adapters(torch.zeros(32, 64).bfloat16(), torch.zeros(48, 16).bfloat16(), torch.ones(2), 16, 64, 24, 2)
    z = torch.zeros(8, dtype=torch.int32)
    plan = nv.MoEPlan(torch.zeros(3, dtype=torch.int32), z, z[:, None].contiguous())
    r = torch.zeros(8, 16)
    for error, call in [
            (TypeError, lambda: nv.nvfp4_adapter(f, w)),
            (ValueError, lambda: nv.nvfp4_adapter(h[:, :32], w)),
            (ValueError, lambda: nv.nvfp4_adapter(h.t(), w)),
            (ValueError, lambda: nv.nvfp4_adapter(h, w2)),
            (ValueError, lambda: nv.nvfp4_adapter(h, w, plan=plan)),
            (ValueError, lambda: nv.nvfp4_adapter(h, w2, plan=plan, gather=True, by_token=True)),
            (ValueError, lambda: nv.nvfp4_adapter(h[:7], w2, plan=plan)),
            (ValueError, lambda: nv.nvfp4_adapter(h, w, f[:, :20])),
            (ValueError, lambda: nv.nvfp4_adapter(h, w, f[:, :24], out=h[:, :24])),
            (TypeError, lambda: nv.nvfp4_adapter(h, w, out_dtype=torch.float16)),
            (nv.NVFP4Error, lambda: nv.nvfp4_adapter(h, w)),  # host memory
            (TypeError, lambda: nv.nvfp4_adapter_backward(f[:, :24], h, w, r)),
            (ValueError, lambda: nv.nvfp4_adapter_backward(h[:, :20], h, w, r)),
            (ValueError, lambda: nv.nvfp4_adapter_backward(h[:, :24], h, w, r[:, :8])),
            (nv.NVFP4Error, lambda: nv.nvfp4_adapter_backward(h[:, :24], h, w, r)),
            (TypeError, lambda: nv.nvfp4_moe_balance(f, i.long())),
            (TypeError, lambda: nv.nvfp4_moe_balance(f.double(), i)),
            (ValueError, lambda: nv.nvfp4_moe_balance(f, i[:7])),
            (ValueError, lambda: nv.nvfp4_moe_balance(f.t(), i)),
            (nv.NVFP4Error, lambda: nv.nvfp4_moe_balance(f, i)),   # host memory
            (ValueError, lambda: nv.nvfp4_moe_balance_backward(f, i, b, dlogits=f[:, :60])),
            (ValueError, lambda: nv.nvfp4_moe_balance_backward(f, i, b, out=f.bfloat16())),
            (ValueError, lambda: nv.nvfp4_moe_balance_backward(f, i, b, dloss=torch.zeros(2))),
            (ValueError, lambda: nv.nvfp4_moe_balance_backward(f[:, :32], i, b)),
            (ValueError, lambda: nv.nvfp4_grad_norm([])),
            (ValueError, lambda: nv.nvfp4_grad_norm(f)),
            (ValueError, lambda: nv.nvfp4_grad_norm([f[:, :32]])),
            (ValueError, lambda: nv.nvfp4_grad_norm([torch.zeros(1).expand(4)])),
            (TypeError, lambda: nv.nvfp4_grad_norm([f.half()])),
            (nv.NVFP4Error, lambda: nv.nvfp4_grad_norm([f])),
            (nv.NVFP4Error, lambda: nv.nvfp4_grad_clip([f], 1.0)),
            (ValueError, lambda: nv.nvfp4_grad_clip([f], 1.0, out=[])),
            (ValueError, lambda: nv.nvfp4_grad_clip([f], 1.0, out=[f.t()])),
            (ValueError, lambda: nv.nvfp4_grad_clip([f], 1.0, norm=torch.zeros(())))]:
        with pytest.raises(error):
            call()
