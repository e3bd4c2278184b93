"""Block norms and their gradients on the GPU against the 64-bit formulas.

Every 32-bit sum here adds at most 64 terms in turn and a few levels of partial sums, every value a handful of
operations: TOL = 2^-16 of the magnitudes that enter covers them many times over and is 2^7 times finer than bf16."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_quantize_amd as nv
from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 2.0 ** -16
F32, BF16 = torch.float32, torch.bfloat16


def _inputs(T, D, xt, yt, parts, seed=0):
    g = torch.Generator().manual_seed(seed + T * 31 + D)
    r = lambda *s: torch.randn(*s, generator=g)
    v = {"x": (2 * r(T, D)).to(xt), "y": r(T, D).to(yt) if "y" in parts else None,
         "w_post": 1 + 0.2 * r(D) if "post" in parts else None, "w_pre": 1 + 0.2 * r(D) if "pre" in parts else None,
         "gate": 0.5 + 0.3 * r(D) if "gate" in parts else (0.5 + 0.3 * r(T, D)).to(yt) if "token_gate" in parts else None,
         "dx_out": r(T, D).to(xt), "dn": r(T, D).to(yt) if "pre" in parts else None}
    return v


def _close(got, want, mag, what):
    if want is None:
        assert got is None, what
        return
    got64 = got.cpu().double().numpy()
    tol = TOL * mag + (2.0 ** -8 * np.abs(want) if got.dtype == BF16 else 0.0) + 1e-30
    assert got64.shape == want.shape, what
    bad = np.abs(got64 - want) > tol
    assert not bad.any(), (what, int(bad.sum()), float(np.max(np.abs(got64 - want) / tol)))


def _run(T, D, xt, yt, parts, one_plus=False, alpha=0.7, eps=1e-6, v=None, dx_none=False):
    v = v or _inputs(T, D, xt, yt, parts)
    dev = {k: None if t is None else t.to(DEV) for k, t in v.items()}
    n = {k: None if t is None else t.double().numpy() for k, t in v.items()}
    flags = nv.NVFP4_NORM_ONE_PLUS if one_plus else 0
    f = nv.nvfp4_block_norm(dev["x"], dev["y"], dev["w_post"], dev["gate"], dev["w_pre"], alpha, eps, flags, n_dtype=yt)
    x1, nn, r1, r2 = ref.block_norm(n["x"], n["y"], n["w_post"], n["gate"], n["w_pre"], alpha, eps, one_plus)
    shift = 1.0 if one_plus else 0.0
    part = 0.0 if n["y"] is None else np.abs(x1 - n["x"])
    mag1 = np.abs(n["x"]) + part
    if n["y"] is not None:
        _close(f.x, x1, mag1, "x")
    _close(f.rstd_post, r1, r1, "rstd_post")
    _close(f.rstd_pre, r2, None if r2 is None else r2, "rstd_pre")
    _close(f.n, nn, None if nn is None else mag1 * r2[:, None] * np.abs(n["w_pre"] + shift) + np.abs(nn), "n")

    dx_out = None if dx_none else n["dx_out"]
    b = nv.nvfp4_block_norm_backward(None if dx_none else dev["dx_out"], dev["dn"], dev["x"], dev["y"], f.rstd_post,
                                     f.rstd_pre, dev["w_post"], dev["gate"], dev["w_pre"], alpha, flags)
    want = ref.block_norm_backward(dx_out, n["dn"], n["x"], n["y"], n["w_post"], n["gate"], n["w_pre"], alpha, eps, one_plus)
    # magnitudes: the same formulas with every term's absolute value
    d = np.zeros_like(n["x"]) if dx_none else np.abs(n["dx_out"])
    mags = {}
    if n["w_pre"] is not None:
        xh = mag1 * r2[:, None]
        mags["dw_pre"] = (np.abs(n["dn"]) * xh).sum(0)
        u = np.abs(n["dn"] * (n["w_pre"] + shift))
        d = d + r2[:, None] * (u + xh * (u * xh).mean(1, keepdims=True))
    mags["dx"] = d
    if n["y"] is not None:
        yh = np.abs(n["y"]) * (1 if r1 is None else r1[:, None])
        wp = 1 if n["w_post"] is None else np.abs(n["w_post"] + shift)
        q = abs(alpha) * d
        if n["gate"] is not None:
            mags["dgate"] = (q * yh * wp).sum(0) if n["gate"].ndim == 1 else q * yh * wp
            q = q * np.abs(n["gate"])
        if n["w_post"] is not None:
            mags["dw_post"] = (q * yh).sum(0)
            u = q * wp
            q = r1[:, None] * (u + yh * (u * yh).mean(1, keepdims=True))
        mags["dy"] = q
    for name in ("dx", "dy", "dw_post", "dgate", "dw_pre"):
        _close(getattr(b, name), want.get(name), mags.get(name), name)
    return f, b


ALL = ("y", "post", "pre", "gate")


@pytest.mark.parametrize("T,D", [(1, 8), (3, 64), (5, 512), (9, 520), (6, 1024), (2, 1032), (4, 2048), (3, 2056), (1, 4096),
                                 (5, 4104), (2, 8192), (3, 8200), (2, 16384), (1030, 64), (300, 1096)])
@pytest.mark.parametrize("xt,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_sizes_and_types(T, D, xt, yt):
    _run(T, D, xt, yt, ALL)


@pytest.mark.parametrize("parts", [("y",), ("y", "gate"), ("y", "token_gate"), ("y", "post"), ("y", "pre"), ("pre",),
                                   ("y", "post", "gate"), ("y", "post", "token_gate"), ("y", "pre", "gate"),
                                   ("y", "post", "pre"), ("y", "post", "pre", "token_gate")])
@pytest.mark.parametrize("D", [72, 1536, 8200])
@pytest.mark.parametrize("one_plus", [False, True])
def test_parts(parts, D, one_plus):
    _run(7, D, BF16, BF16, parts, one_plus)
    if len(parts) > 1 and "pre" in parts:
        _run(6, D, F32, BF16, parts, one_plus, dx_none=True)


def test_rows_of_zeros_and_a_large_row():
    v = _inputs(6, 512, F32, F32, ALL)
    v["y"][1] = 0.0
    v["x"][2] = 0.0
    v["y"][2] = 0.0
    v["x"][3] *= 1e15
    v["y"][4] *= 1e-12
    f, b = _run(6, 512, F32, F32, ALL, v=v)
    assert (f.n[2] == 0).all() and torch.isfinite(b.dy).all() and torch.isfinite(b.dx).all()


def test_no_rows():
    x = torch.empty(0, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    f = nv.nvfp4_block_norm(x, x.clone(), w, w, w)
    b = nv.nvfp4_block_norm_backward(x, x, x, x.clone(), f.rstd_post, f.rstd_pre, w, w, w)
    assert f.n.shape == (0, 64) and (b.dw_post == 0).all() and (b.dw_pre == 0).all() and (b.dgate == 0).all()


def test_in_place_another_stream_and_same_bits():
    v = _inputs(600, 768, BF16, BF16, ALL)
    dev = {k: t.to(DEV) for k, t in v.items()}
    a = nv.nvfp4_block_norm(dev["x"], dev["y"], dev["w_post"], dev["gate"], dev["w_pre"])
    ga = nv.nvfp4_block_norm_backward(dev["dx_out"], dev["dn"], dev["x"], dev["y"], a.rstd_post, a.rstd_pre, dev["w_post"],
                                      dev["gate"], dev["w_pre"])
    x = dev["x"].clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gb = nv.nvfp4_block_norm_backward(dev["dx_out"], dev["dn"], x, dev["y"], a.rstd_post, a.rstd_pre, dev["w_post"],
                                          dev["gate"], dev["w_pre"])
        b = nv.nvfp4_block_norm(x, dev["y"], dev["w_post"], dev["gate"], dev["w_pre"], x_out=x)
    s.synchronize()
    assert b.x is x and torch.equal(x, a.x) and torch.equal(b.n, a.n)
    for name in ("dx", "dy", "dw_post", "dgate", "dw_pre"):
        assert torch.equal(getattr(ga, name), getattr(gb, name)), name
