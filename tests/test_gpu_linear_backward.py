"""The straight-through gradients of the NVFP4 linear layer on the GPU against
the products in 64 bits."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


def _fa():
    from nvfp4_precision_b200 import fp4attn
    return fp4attn


def _case(M, N, K, pad=0):
    """Packed x and w with their 64-bit values, and a dy of rows `pad` elements wider than a multiple of 8."""
    _, xc, xs, xg = ref.make_packed(M, K, M + K)
    _, wc, ws_, wg = ref.make_packed(N, K, N + K + 1, std=K ** -0.5, outliers=0)
    gen = torch.Generator().manual_seed(M + N)
    ld = (N + 7) // 8 * 8 + pad
    dy = torch.full((M, ld), float("nan"))
    dy[:, :N] = torch.randn(M, N, generator=gen)
    return dict(x=ref.packed_to("cuda", xc, xs, xg), w=ref.packed_to("cuda", wc, ws_, wg),
                xv=ref.values(xc, xs, xg).cuda(), wv=ref.values(wc, ws_, wg).cuda(), dy=dy.bfloat16().cuda()[:, :N])


def _check(got, a, b):
    """a @ b in 64 bits.  Products of bf16 values are exact in fp32; the contraction's L terms and at most 16
    parts add with L + 18 roundings (or truncations, 2^-23) relative to the sum of magnitudes; the factor g
    rounds once, the store by half a bf16 step."""
    want = a @ b
    bound = (a.abs() @ b.abs()) * (a.shape[1] + 20) * 2.0 ** -23
    assert torch.isfinite(got).all()
    assert ref.worst(got, want, bound) <= 1.0


SHAPES = [(1, 1, 32), (1, 200, 96), (7, 1, 64), (5, 1003, 544), (64, 64, 64), (130, 257, 288), (333, 8, 2080),
          (256, 256, 256), (300, 520, 1056), (3001, 200, 544), (2000, 1500, 320), (4097, 72, 32), (1000, 6000, 512),
          (600, 4100, 4128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("pad", [0, 8])
def test_gradients_against_64_bits(M, N, K, pad):
    fa = _fa()
    c = _case(M, N, K, pad)
    ws = fa.new_linear_backward_workspace(M, N, K)
    args = (c["dy"], c["x"][0], c["x"][1], c["w"][0], c["w"][1])
    kw = dict(x_gscale=c["x"][2], w_gscale=c["w"][2], workspace=ws)
    dx, dw, dbias = fa.fp4attn_linear_backward(*args, **kw)
    assert fa.fp4attn_read_status(ws) == 0
    dy = c["dy"].double()
    _check(dx, dy, c["wv"])
    _check(dw, dy.t(), c["xv"])
    assert ref.worst(dbias, dy.sum(0), dy.abs().sum(0) * M * ref.U) <= 1.0
    again = fa.fp4attn_linear_backward(*args, **kw)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, dbias), again))
    # each gradient alone (its own split of the work)
    for want in ((True, False, False), (False, True, False), (False, False, True)):
        got = fa.fp4attn_linear_backward(*args, want_dx=want[0], want_dw=want[1], want_dbias=want[2], **kw)
        assert [g is not None for g in got] == list(want)
        if got[0] is not None:
            _check(got[0], dy, c["wv"])
        if got[1] is not None:
            _check(got[1], dy.t(), c["xv"])
        if got[2] is not None:
            assert torch.equal(got[2], dbias)
    assert fa.fp4attn_read_status(ws) == 0


def test_empty_sums_are_zero():
    fa = _fa()
    for M, N in ((0, 5), (5, 0), (0, 0)):
        _, wc, ws_, wg = ref.make_packed(N, 64, 1)
        _, xc, xs, xg = ref.make_packed(M, 64, 2)
        w, x = ref.packed_to("cuda", wc, ws_, wg), ref.packed_to("cuda", xc, xs, xg)
        dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        dx, dw, db = fa.fp4attn_linear_backward(dy, x[0], x[1], w[0], w[1])
        assert dx.shape == (M, 64) and (dx == 0).all() and dw.shape == (N, 64) and (dw == 0).all()
        assert db.shape == (N,) and (db == 0).all()


def test_bad_scales_are_reported():
    fa = _fa()
    c = _case(64, 64, 64)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        g = torch.tensor([bad], device="cuda")
        for kw in (dict(x_gscale=g), dict(w_gscale=g)):
            ws = fa.new_linear_backward_workspace(64, 64, 64)
            fa.fp4attn_linear_backward(c["dy"], c["x"][0], c["x"][1], c["w"][0], c["w"][1], workspace=ws, **kw)
            assert fa.fp4attn_read_status(ws) == fa.ERR_RANGE


def test_infinities_stay_in_their_rows():
    """An infinite dy[m, n] reaches row m of dx and row n of dw only."""
    fa = _fa()
    M, N, K = 300, 200, 96
    c = _case(M, N, K)
    dy = c["dy"].clone()
    dy[7, 11] = float("inf")
    dx, dw, db = fa.fp4attn_linear_backward(dy, c["x"][0], c["x"][1], c["w"][0], c["w"][1])
    for g, at in ((dx, 7), (dw, 11)):
        ok = torch.isfinite(g).all(1)
        assert not ok[at] and ok.sum() == g.shape[0] - 1
    assert not torch.isfinite(db[11]) and torch.isfinite(db).sum() == N - 1


def test_graph_replay():
    fa = _fa()
    M, N, K = 700, 264, 544
    c = _case(M, N, K)
    ws = fa.new_linear_backward_workspace(M, N, K)
    dy = c["dy"].clone()
    args = (dy, c["x"][0], c["x"][1], c["w"][0], c["w"][1])
    want = [t.clone() for t in fa.fp4attn_linear_backward(*args, workspace=ws)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.fp4attn_linear_backward(*args, workspace=ws)
    dy.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, -q) for p, q in zip(got, want))
    assert fa.fp4attn_read_status(ws) == 0


@pytest.mark.parametrize("M,N,K", [(2400, 2000, 1632), (2401, 2000, 1536), (9000, 5000, 1728), (5000, 9001, 1184), (6000, 7777, 2048),
                                   (12000, 700, 3200), (28972, 976, 928), (100, 15912, 3328), (12652, 18, 2048)])
def test_gradients_of_large_and_uneven_products(M, N, K):
    """Tiles of every width, whole and split, the last column's second half absent; many tiles a pair."""
    fa = _fa()
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = fa.fp4attn_quantize_rows(torch.randn(M, K, generator=gen, device="cuda").bfloat16(), dynamic_gscale=True)
    w = fa.fp4attn_quantize_rows(torch.randn(N, K, generator=gen, device="cuda").bfloat16() * 0.05, dynamic_gscale=True)
    dy = torch.randn(M, (N + 7) // 8 * 8, generator=gen, device="cuda").bfloat16()[:, :N]
    ws = fa.new_linear_backward_workspace(M, N, K)
    out = fa.fp4attn_linear_backward(dy, x["codes"], x["scales"], w["codes"], w["scales"], x["gscale"], w["gscale"],
                                     workspace=ws)
    assert fa.fp4attn_read_status(ws) == 0
    d = dy.double()
    # the unit-scale values are exact in fp32 (g 1), the factor g rounds once in the kernel and not here
    for got, a, q in ((out[0], d, w), (out[1], d.t(), x)):
        v = fa.fp4attn_dequant_rows(q["codes"], q["scales"], dtype=torch.float32).double() * q["gscale"].double()
        _check(got, a, v)
        del v
    assert ref.worst(out[2], d.sum(0), d.abs().sum(0) * M * ref.U) <= 1.0
    again = fa.fp4attn_linear_backward(dy, x["codes"], x["scales"], w["codes"], w["scales"], x["gscale"], w["gscale"],
                                       workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(out, again))


@pytest.mark.parametrize("M,N,K", [(64, 64, 64), (700, 264, 544), (2400, 2000, 1632)])
def test_the_scale_of_an_absent_product_is_not_judged(M, N, K):
    """x_gscale belongs to dw and w_gscale to dx: without the one the other may be anything."""
    fa = _fa()
    c = _case(M, N, K)
    args = (c["dy"], c["x"][0], c["x"][1], c["w"][0], c["w"][1])
    for alone, scale, other in (("want_dx", "w_gscale", "x_gscale"), ("want_dw", "x_gscale", "w_gscale")):
        want = {k: k == alone for k in ("want_dx", "want_dw", "want_dbias")}
        good = {scale: c["w" if scale == "w_gscale" else "x"][2]}
        ref_out = next(t for t in fa.fp4attn_linear_backward(*args, **good, **want) if t is not None)
        for bad in (float("nan"), 0.0, float("inf")):
            ws = fa.new_linear_backward_workspace(M, N, K)
            got = fa.fp4attn_linear_backward(*args, **good, **want, workspace=ws,
                                             **{other: torch.tensor([bad], device="cuda")})
            assert fa.fp4attn_read_status(ws) == 0
            assert torch.equal(next(t for t in got if t is not None), ref_out)
