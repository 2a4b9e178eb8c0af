"""Refusals of the linear layers' and norms' entry points: every bad call is
turned down before anything is launched.  CPU only: no call here reaches the GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def fa():
    from nvfp4_precision_b200 import build
    build.build()
    from nvfp4_precision_b200 import fp4attn
    return fp4attn


P, WS, BIG = 1 << 20, 1 << 21, 1 << 40  # aligned addresses that are never read


def quantize(fa, x=P, t=0, ld=64, rows=4, K=64, g=None, flags=0, codes=P, scales=P, ws=WS, wsb=BIG):
    return fa.lib.fp4attn_quantize_rows(x, t, ld, rows, K, g, flags, codes, scales, ws, wsb, None)


def test_sizes_of_scale_tiles(fa):
    f = fa.lib.fp4attn_scale_tile_bytes
    assert f(1, 32) == 512 and f(128, 64) == 512 and f(129, 64) == 1024 and f(128, 96) == 1024 and f(0, 64) == 0
    assert f(-1, 64) == 0 and f(4, 33) == 0 and f(4, 0) == 0 and f(1 << 40, 64) == 0


def test_quantize_rows_refusals(fa):
    inv, uns, wsp = fa.ERR_INVALID_ARG, fa.ERR_UNSUPPORTED, fa.ERR_WORKSPACE
    assert quantize(fa, rows=-1) == inv and quantize(fa, K=0) == inv and quantize(fa, K=-32) == inv
    assert quantize(fa, K=48) == uns and quantize(fa, K=1048608) == uns and quantize(fa, rows=4194305) == uns
    assert quantize(fa, t=2) == inv and quantize(fa, flags=1) == inv and quantize(fa, flags=8) == inv
    assert quantize(fa, flags=fa.DYNAMIC_GSCALE) == inv  # no place for the computed scale
    assert quantize(fa, g=P + 2) == inv
    assert quantize(fa, ws=None) == wsp and quantize(fa, ws=WS + 8) == wsp and quantize(fa, wsb=255) == wsp
    assert quantize(fa, x=None) == inv and quantize(fa, x=P + 8) == inv
    assert quantize(fa, codes=None) == inv and quantize(fa, codes=P + 4) == inv and quantize(fa, scales=None) == inv
    assert quantize(fa, ld=63) == inv and quantize(fa, ld=68) == inv and quantize(fa, ld=0) == inv
    assert quantize(fa, ld=66, t=fa.F32) == inv and quantize(fa, ld=1 << 38) == inv


def test_dequant_rows_refusals(fa):
    def f(codes=P, scales=P, g=None, rows=4, K=64, out=P, t=0):
        return fa.lib.fp4attn_dequant_rows(codes, scales, g, rows, K, out, t, None)
    inv, uns = fa.ERR_INVALID_ARG, fa.ERR_UNSUPPORTED
    assert f(rows=-1) == inv and f(K=16) == uns and f(t=7) == inv and f(g=P + 1) == inv
    for k in ("codes", "scales", "out"):
        assert f(**{k: None}) == inv and f(**{k: P + 8}) == inv
    assert f(rows=0, codes=None, out=None) == fa.OK


def test_gemm_and_linear_refusals(fa):
    def gemm(xc=P, xs=P, gx=None, wc=P, wsc=P, gw=None, b=None, M=4, N=8, K=64, y=P, ld=8, ws=WS, wsb=BIG):
        return fa.lib.fp4attn_gemm(xc, xs, gx, wc, wsc, gw, b, M, N, K, y, ld, ws, wsb, None)

    def linear(x=P, ldx=64, gx=None, flags=0, wc=P, wsc=P, gw=None, b=None, M=4, N=8, K=64, y=P, ld=8, ws=WS, wsb=BIG):
        return fa.lib.fp4attn_linear(x, ldx, gx, flags, wc, wsc, gw, b, M, N, K, y, ld, ws, wsb, None)

    inv, uns, wsp = fa.ERR_INVALID_ARG, fa.ERR_UNSUPPORTED, fa.ERR_WORKSPACE
    for f in (gemm, linear):
        assert f(M=-1) == inv and f(N=-1) == inv and f(K=0) == inv and f(K=40) == uns and f(N=4194305) == uns
        assert f(ws=None) == wsp and f(wsb=16) == wsp
        assert f(gx=P + 2) == inv and f(gw=P + 2) == inv and f(b=P + 2) == inv
        assert f(wc=None) == inv and f(wsc=P + 8) == inv and f(y=None) == inv and f(y=P + 2) == inv
        assert f(ld=7) == inv and f(ld=1 << 38) == inv
    assert gemm(xc=None) == inv and gemm(xs=P + 4) == inv
    assert linear(x=None) == inv and linear(x=P + 2) == inv and linear(ldx=60) == inv and linear(ldx=68) == inv
    assert linear(flags=2) == inv
    assert linear(M=1000, wsb=1000 * 32) == wsp  # x's codes do not fit
    assert gemm(M=0) == fa.OK and gemm(N=0) == fa.OK and linear(M=0) == fa.OK and linear(N=0) == fa.OK


def test_linear_backward_refusals(fa):
    def f(dy=P, ld=8, xc=P, xs=P, gx=None, wc=P, wsc=P, gw=None, M=4, N=8, K=64, dx=P, ldx=64, dw=P, db=P, ws=WS, wsb=BIG):
        return fa.lib.fp4attn_linear_backward(dy, ld, xc, xs, gx, wc, wsc, gw, M, N, K, dx, ldx, dw, db, ws, wsb, None)
    inv, uns, wsp = fa.ERR_INVALID_ARG, fa.ERR_UNSUPPORTED, fa.ERR_WORKSPACE
    assert f(M=-1) == inv and f(K=0) == inv and f(K=100) == uns and f(M=4194305) == uns
    assert f(ws=None) == wsp and f(wsb=1024) == wsp
    assert f(dy=None) == inv and f(dy=P + 2) == inv and f(ld=7) == inv and f(ld=12) == inv
    assert f(dx=P + 2) == inv and f(ldx=60) == inv and f(ldx=68) == inv and f(dw=P + 8) == inv and f(db=P + 1) == inv
    assert f(gx=P + 1) == inv and f(gw=P + 3) == inv
    assert f(xc=None) == inv and f(xs=P + 4) == inv and f(wc=None) == inv and f(wsc=None) == inv
    assert f(dx=None, dw=None, db=None) == fa.OK  # nothing asked for
    need = fa.lib.fp4attn_linear_backward_workspace_bytes
    assert need(8, 8, 64) % 256 == 0 and need(4096, 8, 64) > need(8, 8, 64) and need(-1, 8, 64) == 256


def norm_args(fa, **kw):
    v = fa.NormVectors(P, P, P, 64, P, 64, P, 64)
    a = dict(x=P, t=0, ldx=64, h=P, ldh=64, v=v, rows=4, C=64, G=2, eps=1e-6, flags=0, y=P, ldy=64, z=P, ldz=64, zc=None,
             zs=None, gz=None, ws=WS, wsb=BIG)
    a.update(kw)
    return list(a.values()) + [None]


def test_norm_gate_refusals(fa):
    def f(**kw):
        return fa.lib.fp4attn_norm_gate(*norm_args(fa, **kw))
    inv, uns, wsp = fa.ERR_INVALID_ARG, fa.ERR_UNSUPPORTED, fa.ERR_WORKSPACE
    assert f(rows=-1) == inv and f(C=0) == inv and f(G=0) == inv and f(rows=5) == inv  # 5 rows of 2 samples
    assert f(C=60) == uns and f(C=16392) == uns and f(rows=1 << 23) == uns and f(rows=1 << 21, G=1 << 21) == uns
    assert f(t=3) == inv and f(flags=4) == inv and f(eps=-1.0) == inv and f(eps=float("nan")) == inv and f(eps=float("inf")) == inv
    assert f(v=None) == inv
    assert f(x=None) == inv and f(x=P + 8) == inv and f(h=P + 8) == inv and f(y=P + 8) == inv and f(z=P + 8) == inv
    assert f(y=None, z=None) == inv  # no output
    for k in ("ldx", "ldh", "ldy", "ldz"):
        assert f(**{k: 56}) == inv and f(**{k: 65}) == inv and f(**{k: 1 << 38}) == inv
    assert f(zc=P, zs=P) == inv  # z twice
    assert f(z=None, zc=P) == inv and f(z=None, zc=P, zs=P, gz=P + 1) == inv and f(z=None, zc=P + 8, zs=P) == inv
    assert f(z=None, zc=P, zs=P, C=72, ldx=72, ldh=72, ldy=72) == uns
    assert f(z=None, zc=P, zs=P, ws=None) == wsp and f(ws=WS + 4) == wsp and f(wsb=8) == wsp
    good = dict(post_weight=P, pre_weight=P, gate=P, gate_stride=64, scale=P, scale_stride=64, shift=P, shift_stride=64)
    for bad in (dict(post_weight=P + 2), dict(pre_weight=P + 8), dict(gate=P + 4), dict(gate_stride=56),
                dict(scale_stride=65), dict(shift_stride=0), dict(shift=P + 2)):
        assert f(v=fa.NormVectors(**{**good, **bad})) == inv
    assert f(rows=0) == fa.OK


def test_norm_gate_backward_refusals(fa):
    def f(**kw):
        v = fa.NormVectors(P, P, P, 64, P, 64, P, 64)
        a = dict(dz=P, lddz=64, dy=P, lddy=64, y=P, ldy=64, t=0, h=P, ldh=64, v=v, rows=4, C=64, G=2, eps=1e-6, flags=0,
                 dx=P, lddx=64, dh=P, lddh=64, dshift=P, dscale=P, dgate=P, dpre=P, dpost=P, ws=WS, wsb=BIG)
        a.update(kw)
        return fa.lib.fp4attn_norm_gate_backward(*a.values(), None)
    inv, uns, wsp = fa.ERR_INVALID_ARG, fa.ERR_UNSUPPORTED, fa.ERR_WORKSPACE
    assert f(rows=3) == inv and f(C=20) == uns and f(t=5) == inv and f(flags=1) == inv and f(eps=-0.5) == inv
    assert f(ws=None) == wsp and f(wsb=256) == wsp
    assert f(dz=None) == inv and f(y=None) == inv and f(dx=None) == inv and f(dh=None) == inv
    for k in ("dz", "dy", "y", "h", "dx", "dh"):
        assert f(**{k: P + 8}) == inv
    for k in ("lddz", "lddy", "ldy", "ldh", "lddx", "lddh"):
        assert f(**{k: 60}) == inv
    for k in ("dshift", "dscale", "dgate", "dpre", "dpost"):
        assert f(**{k: P + 2}) == inv
    # without the forward's branch there is nothing to differentiate in it
    assert f(h=None) == inv and f(h=None, dh=None) == inv and f(h=None, dh=None, dgate=None) == inv
    need = fa.lib.fp4attn_norm_gate_backward_workspace_bytes
    assert need(4, 64, 3) == 256 and need(4, 60, 1) == 256 and need(4, 64, 2) > 256


def test_tensors_off_the_current_device_are_refused(fa):
    import torch
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: fa.fp4attn_quantize_rows(bf), lambda: fa.fp4attn_dequant_rows(codes, scales),
                 lambda: fa.fp4attn_gemm(codes, scales, codes, scales), lambda: fa.fp4attn_linear(bf, codes, scales),
                 lambda: fa.fp4attn_linear_backward(bf, codes, scales, codes, scales),
                 lambda: fa.fp4attn_norm_gate(bf, bf), lambda: fa.fp4attn_norm_gate_backward(bf, None, bf)):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    with pytest.raises(AssertionError):
        fa.norm_gate(bf, gate=bf)
    with pytest.raises(AssertionError):
        fa.fp4_linear(bf, bf.float().t())


def test_an_empty_batch_of_samples_is_no_error(fa):
    f = lambda **kw: fa.lib.fp4attn_norm_gate(*norm_args(fa, **kw))
    assert f(rows=0, G=0) == fa.OK and f(rows=0, G=7) == fa.OK
    assert f(rows=4, G=0) == fa.ERR_INVALID_ARG and f(rows=0, G=-1) == fa.ERR_INVALID_ARG
    v = fa.NormVectors(P, P, P, 64, P, 64, P, 64)

    def back(rows, G):  # no sums asked for: nothing to clear
        return fa.lib.fp4attn_norm_gate_backward(P, 64, P, 64, P, 64, 0, P, 64, v, rows, 64, G, 1e-6, 0, P, 64, P, 64, None,
                                                 None, None, None, None, WS, BIG, None)
    assert back(0, 0) == fa.OK and back(4, 0) == fa.ERR_INVALID_ARG and back(0, -1) == fa.ERR_INVALID_ARG
    assert fa.lib.fp4attn_norm_gate_backward_workspace_bytes(0, 64, 0) == 256
