"""Refusals of the operators around the quantized products: every bad argument is named on the host, before
anything is enqueued (the fake device addresses here are never read)."""
import ctypes

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


ROUTE = dict(logits=P, dtype=nv.NVFP4_F32, tokens=80, experts=64, ld=64, bias=None, num_groups=1, group_top_k=1, top_k=4,
             flags=0, scale=1.0, ids=P, weights=P, offsets=P, rows=P, pos=P, workspace=P, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(weights=None), NULL), (dict(offsets=None), NULL),
    (dict(rows=None), NULL), (dict(pos=None), NULL), (dict(workspace=None), NULL), (dict(dtype=7), UNSUPPORTED),
    (dict(flags=8), UNSUPPORTED), (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(experts=513, ld=513), SHAPE),
    (dict(ld=63), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=33), SHAPE), (dict(experts=3, ld=3, top_k=4), SHAPE),
    (dict(num_groups=3), SHAPE), (dict(num_groups=0), SHAPE), (dict(num_groups=32), SHAPE), (dict(num_groups=4, group_top_k=5), SHAPE),
    (dict(num_groups=4, group_top_k=0), SHAPE), (dict(num_groups=16, group_top_k=1, top_k=5), SHAPE),
    (dict(tokens=2**31 // 4), SHAPE), (dict(tokens=2**62), SHAPE), (dict(ld=2**62), SHAPE),
    (dict(logits=ODD), ALIGN), (dict(ids=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(workspace=0x10004), ALIGN),
    (dict(logits=0x10001, dtype=nv.NVFP4_BF16), ALIGN)])
def test_route(changes, status):
    assert _call("nvfp4_moe_route", ROUTE, **changes) == status


def test_route_without_tokens_or_plan_needs_no_buffers():
    assert _call("nvfp4_moe_route", ROUTE, tokens=0, logits=None, ids=None, weights=None, offsets=None, rows=None, pos=None,
                 workspace=None) == OK


BWD = dict(logits=P, dtype=nv.NVFP4_BF16, tokens=8, experts=64, ld=64, ids=P, dweights=P, top_k=4, flags=0, scale=1.0,
           dlogits=P, ldd=64, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(dweights=None), NULL), (dict(dlogits=None), NULL),
    (dict(ldd=63), SHAPE), (dict(top_k=65), SHAPE), (dict(flags=16), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED),
    (dict(dlogits=0x10001), ALIGN), (dict(tokens=0, logits=None, ids=None, dweights=None, dlogits=None), OK)])
def test_route_backward(changes, status):
    assert _call("nvfp4_moe_route_backward", BWD, **changes) == status


PLAN = dict(ids=P, tokens=80, top_k=4, experts=64, offsets=P, rows=P, pos=P, workspace=P, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(ids=None), NULL), (dict(offsets=None), NULL), (dict(rows=None), NULL), (dict(workspace=None), NULL),
    (dict(experts=513), SHAPE), (dict(top_k=40), SHAPE), (dict(tokens=2**30), SHAPE), (dict(ids=ODD), ALIGN),
    (dict(workspace=0x10008), ALIGN)])
def test_plan(changes, status):
    assert _call("nvfp4_moe_plan", PLAN, **changes) == status


GATHER = dict(x=P, dtype=nv.NVFP4_BF16, tokens=8, d=64, ldx=64, rows=P, top_k=4, y=P, ldy=64, stream=None)
COMBINE = dict(y=P, dtype=nv.NVFP4_BF16, tokens=8, d=64, ldy=64, pos=P, weights=None, top_k=4, out=P, ldo=64, stream=None)
CBWD = dict(dout=P, ldo=64, y=P, ldy=64, dtype=nv.NVFP4_BF16, tokens=8, d=64, pos=P, rows=P, weights=P, top_k=4, dy=P, lddy=64,
            dweights=P, stream=None)


@pytest.mark.parametrize("name,args,changes,status", [
    ("gather", GATHER, dict(x=None), NULL), ("gather", GATHER, dict(rows=None), NULL), ("gather", GATHER, dict(y=None), NULL),
    ("gather", GATHER, dict(d=60), ALIGN), ("gather", GATHER, dict(ldx=63), SHAPE), ("gather", GATHER, dict(ldy=68), ALIGN),
    ("gather", GATHER, dict(x=0x10008), ALIGN), ("gather", GATHER, dict(dtype=3), UNSUPPORTED),
    ("gather", GATHER, dict(top_k=0), SHAPE), ("gather", GATHER, dict(tokens=-4), SHAPE), ("gather", GATHER, dict(tokens=0), OK),
    ("combine", COMBINE, dict(y=None), NULL), ("combine", COMBINE, dict(pos=None), NULL), ("combine", COMBINE, dict(out=None), NULL),
    ("combine", COMBINE, dict(weights=ODD), ALIGN), ("combine", COMBINE, dict(ldo=32), SHAPE), ("combine", COMBINE, dict(tokens=0), OK),
    ("combine_backward", CBWD, dict(weights=None), NULL), ("combine_backward", CBWD, dict(dweights=None), NULL),
    ("combine_backward", CBWD, dict(rows=None), NULL), ("combine_backward", CBWD, dict(dy=0x10008), ALIGN),
    ("combine_backward", CBWD, dict(lddy=60), SHAPE), ("combine_backward", CBWD, dict(d=0, ldo=0, ldy=0, lddy=0), SHAPE)])
def test_rows(name, args, changes, status):
    assert _call("nvfp4_moe_" + name, args, **changes) == status


QUANT = dict(x=P, dtype=nv.NVFP4_BF16, rows=8, cols=64, ldx=64, q=P, scales=P, stream=None)
GEMM = dict(a=P, a_scales=P, a_rows=8, b=P, b_scales=P, M=8, N=64, K=64, c=P, c_dtype=nv.NVFP4_BF16, ldc=64, num_groups=1,
            offsets=None, rows=None, row_div=1, workspace=None, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(scales=None), NULL), (dict(cols=40), SHAPE), (dict(ldx=48), SHAPE),
    (dict(ldx=68), ALIGN), (dict(x=0x10008), ALIGN), (dict(q=0x10008), ALIGN), (dict(scales=ODD), ALIGN), (dict(dtype=2), UNSUPPORTED),
    (dict(rows=-1), SHAPE), (dict(rows=0), OK)])
def test_int8_quantize(changes, status):
    assert _call("nvfp4_int8_quantize", QUANT, **changes) == status


@pytest.mark.parametrize("changes,status", [
    (dict(a=None), NULL), (dict(b=None), NULL), (dict(c=None), NULL), (dict(a_scales=None), NULL), (dict(b_scales=None), NULL),
    (dict(K=72), SHAPE), (dict(K=1 << 17), SHAPE), (dict(K=-16), SHAPE), (dict(N=2**26), SHAPE), (dict(ldc=63), SHAPE),
    (dict(a_rows=7), SHAPE), (dict(num_groups=2), SHAPE), (dict(num_groups=0), SHAPE), (dict(num_groups=513, offsets=P), SHAPE),
    (dict(rows=P), SHAPE), (dict(rows=P, offsets=P, row_div=0), SHAPE), (dict(rows=P, offsets=P, a_rows=0), SHAPE),
    (dict(a=0x10008), ALIGN), (dict(b=0x10008), ALIGN), (dict(c=0x10001), ALIGN), (dict(offsets=ODD, num_groups=2), ALIGN),
    (dict(c_dtype=2), UNSUPPORTED), (dict(M=0, a_rows=0), OK), (dict(N=0, ldc=1), OK)])
def test_int8_gemm(changes, status):
    assert _call("nvfp4_int8_gemm", GEMM, **changes) == status


NORM = dict(x=P, x_dtype=nv.NVFP4_BF16, y=P, y_dtype=nv.NVFP4_BF16, tokens=4, d=64, w_post=P, gate=P, w_pre=P, alpha=1.0,
            eps=1e-6, flags=0, x_out=P, n=P, rstd_post=P, rstd_pre=P, stream=None)
NBWD = dict(dx_out=P, dn=P, x=P, x_dtype=nv.NVFP4_BF16, y=P, y_dtype=nv.NVFP4_BF16, tokens=4, d=64, w_post=P, gate=P, w_pre=P,
            alpha=1.0, flags=0, rstd_post=P, rstd_pre=P, dx=P, dy=P, dw_post=P, dgate=P, dw_pre=P, workspace=P, stream=None)


@pytest.mark.parametrize("changes,status", [
    (dict(x=None), NULL), (dict(x_out=None), NULL), (dict(n=None), NULL), (dict(w_pre=None), NULL),
    (dict(y=None, x_out=None), UNSUPPORTED), (dict(y=None, w_post=None, gate=None), NULL), (dict(d=60), SHAPE), (dict(d=0), SHAPE),
    (dict(d=16392), SHAPE), (dict(tokens=-1), SHAPE), (dict(eps=0.0), UNSUPPORTED), (dict(eps=-1e-6), UNSUPPORTED),
    (dict(eps=float("nan")), UNSUPPORTED), (dict(flags=4), UNSUPPORTED), (dict(x_dtype=5), UNSUPPORTED), (dict(w_post=0x10008), ALIGN),
    (dict(n=0x10008), ALIGN), (dict(y=None, w_post=None, gate=None, w_pre=None, x_out=None, n=None), UNSUPPORTED),
    (dict(tokens=0), OK)])
def test_block_norm(changes, status):
    assert _call("nvfp4_block_norm", NORM, **changes) == status


@pytest.mark.parametrize("changes,status", [
    (dict(dx=None), NULL), (dict(dy=None), NULL), (dict(dn=None), NULL), (dict(dw_post=None), NULL), (dict(dgate=None), NULL),
    (dict(dw_pre=None), NULL), (dict(rstd_post=None), NULL), (dict(rstd_pre=None), NULL), (dict(workspace=None), NULL),
    (dict(w_pre=None), NULL), (dict(d=12), SHAPE), (dict(workspace=0x10004), ALIGN), (dict(dx_out=0x10008), ALIGN),
    (dict(flags=64), UNSUPPORTED)])
def test_block_norm_backward(changes, status):
    assert _call("nvfp4_block_norm_backward", NBWD, **changes) == status


def test_workspace_sizes():
    L = nv.lib()
    assert L.nvfp4_moe_workspace_size(100, 64, 4) >= 64 * 4 and L.nvfp4_moe_workspace_size(100, 0, 4) == 0
    assert L.nvfp4_moe_workspace_size(16, 512, 32) == 0
    assert L.nvfp4_block_norm_workspace_size(4, 64) >= 2 * 4 * 64 * 4 and L.nvfp4_block_norm_workspace_size(4, 0) == 0


def test_binding_refuses_wrong_tensors():
    f, b, i = torch.zeros(8, 64), torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8, 4, dtype=torch.int32)
    plan = nv.MoEPlan(torch.zeros(9, dtype=torch.int32), torch.zeros(32, dtype=torch.int32), i)
    q = nv.Int8Tensor(torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8), 8, 64)
    for error, call in [
            (TypeError, lambda: nv.nvfp4_moe_route(f.double(), 4)),
            (ValueError, lambda: nv.nvfp4_moe_route(f.t(), 4)),
            (TypeError, lambda: nv.nvfp4_moe_route(f, 4, bias=torch.zeros(64, dtype=torch.float64))),
            (ValueError, lambda: nv.nvfp4_moe_route(f, 4, bias=torch.zeros(63))),
            (nv.NVFP4Error, lambda: nv.nvfp4_moe_route(f, 65)),
            (TypeError, lambda: nv.nvfp4_moe_route_backward(f, i.long(), torch.zeros(8, 4))),
            (ValueError, lambda: nv.nvfp4_moe_route_backward(f, i, torch.zeros(8, 5))),
            (ValueError, lambda: nv.nvfp4_moe_plan(i[0], 8)),
            (ValueError, lambda: nv.nvfp4_moe_gather(f[:7], plan)),
            (ValueError, lambda: nv.nvfp4_moe_combine(f, plan)),
            (ValueError, lambda: nv.nvfp4_moe_combine_backward(f, torch.zeros(32, 64, dtype=torch.bfloat16), plan, torch.zeros(8, 4))),
            (ValueError, lambda: nv.nvfp4_int8_quantize(f[0])),
            (ValueError, lambda: nv.nvfp4_int8_gemm(q, q, gather=True)),
            (ValueError, lambda: nv.nvfp4_int8_gemm(q, q, plan=plan)),
            (ValueError, lambda: nv.nvfp4_block_norm(f, w_post=torch.zeros(64))),
            (TypeError, lambda: nv.nvfp4_block_norm(f, f, w_post=torch.zeros(64, dtype=torch.bfloat16))),
            (ValueError, lambda: nv.nvfp4_block_norm(f, b[:, :32])),
            (ValueError, lambda: nv.nvfp4_block_norm_backward(f, None, f, f, w_pre=torch.zeros(64)))]:
        with pytest.raises(error):
            call()
