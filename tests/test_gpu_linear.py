"""The NVFP4 linear layers on the GPU: rows quantised bit for bit as defined,
the product against the same values multiplied in 64 bits."""
import numpy as np
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu


def _fa():
    from nvfp4_precision_b200 import fp4attn
    return fp4attn


def _source(rows, K, seed, dtype=torch.bfloat16, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=gen) * scale
    x[:, torch.randperm(K, generator=gen)[:2]] *= 20.0
    return x.to(dtype)


SHAPES = [(1, 32), (1, 6144), (3, 96), (31, 64), (128, 256), (129, 544), (333, 2080), (1000, 1056), (257, 4128)]


@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g", [None, 0.037, "dynamic"])
def test_quantize_rows_bit_exact(rows, K, dtype, g):
    fa = _fa()
    x = _source(rows, K, rows * 7 + K, dtype)
    gv = ref.computed_g(x) if g == "dynamic" else 1.0 if g is None else g
    gt = torch.tensor([gv], dtype=torch.float32, device="cuda") if isinstance(g, float) else None
    out = fa.fp4attn_quantize_rows(x.cuda(), gscale=gt, dynamic_gscale=g == "dynamic")
    assert fa.fp4attn_read_status(out["workspace"]) == 0
    gf = float(np.float32(gv))
    c, s = ref.quantize(x, gf)
    if g == "dynamic":
        assert float(out["gscale"].item()) == gf
    assert np.array_equal(out["codes"].cpu().numpy(), ref.pack_codes(c))
    got = fa.untile_scales(out["scales"], rows, K).cpu().numpy()
    assert np.array_equal(got, s)
    # channels past K have scale 0 (the product reads those bytes)
    words = out["scales"].cpu().numpy()
    want = ref.tile(s)
    r = np.arange(-(-rows // 128) * 128)[:, None]
    b = np.arange(-(-K // 64) * 4)[None, :]
    at = ((r // 128) * (-(-K // 64)) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    assert np.array_equal(words[at[:rows]], want[at[:rows]])
    # read back: fl(fl(g s) e2m1) in fp32, one more rounding to bf16
    f = np.float32
    v = ref.MAGS[c & 7] * np.where(c & 8, -1.0, 1.0)
    gs = (f(gf) * ref.UE4M3[s].astype(f)).astype(f)
    v = (v.reshape(rows, -1, 16).astype(f) * gs[..., None]).astype(f).reshape(rows, K)
    back = fa.fp4attn_dequant_rows(out["codes"], out["scales"], gt if gt is not None else out["gscale"],
                                   dtype=torch.float32)
    assert np.array_equal(back.cpu().numpy(), v)
    back = fa.fp4attn_dequant_rows(out["codes"], out["scales"], gt if gt is not None else out["gscale"])
    assert torch.equal(back.cpu(), torch.from_numpy(v).bfloat16())


def test_quantize_rows_extremes():
    """Zeros, subnormals, the largest finite values, ties and tiny blocks beside huge ones."""
    fa = _fa()
    x = torch.zeros(40, 64)
    x[1] = 3.0e38
    x[2] = 1e-40
    x[3, ::2], x[3, 1::2] = 6.0, -0.25
    x[4, :16] = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
    x[5] = -0.0
    for i in range(6, 40):
        x[i] = torch.randn(64, generator=torch.Generator().manual_seed(i)) * 10.0 ** (i - 24)
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        out = fa.fp4attn_quantize_rows(y.cuda())
        assert fa.fp4attn_read_status(out["workspace"]) == 0
        c, s = ref.quantize(y)
        assert np.array_equal(out["codes"].cpu().numpy(), ref.pack_codes(c))
        assert np.array_equal(fa.untile_scales(out["scales"], 40, 64).cpu().numpy(), s)


def test_quantize_rows_equals_the_attention_prologue():
    """With both transforms off the prologue's quantiser and this one are the same function."""
    fa = _fa()
    gen = torch.Generator().manual_seed(5)
    q = torch.randn(1, 2, 300, 128, generator=gen).bfloat16().cuda()
    g = torch.tensor([0.3], device="cuda")
    out = fa.fp4attn_quantize_qk(q, q, g, g, flags=fa.NO_SMOOTH_K | fa.NO_HADAMARD)
    rows = fa.fp4attn_quantize_rows(q.view(600, 128), gscale=g)
    assert torch.equal(out["q_codes"].view(600, 64), rows["codes"])
    assert torch.equal(out["q_scales"].view(600, 8), fa.untile_scales(rows["scales"], 600, 128))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dynamic", [False, True])
@pytest.mark.parametrize("rows", [2, 700])
def test_quantize_rows_reports_non_finite(bad, dynamic, rows):
    fa = _fa()
    x = torch.randn(rows, 96).bfloat16()
    x[rows - 1, 95] = bad
    out = fa.fp4attn_quantize_rows(x.cuda(), dynamic_gscale=dynamic)
    assert fa.fp4attn_read_status(out["workspace"]) == fa.ERR_RANGE


def test_bad_scales_are_reported():
    fa = _fa()
    x = torch.randn(4, 64).bfloat16().cuda()
    w = fa.fp4attn_quantize_rows(x)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        g = torch.tensor([bad], device="cuda")
        out = fa.fp4attn_quantize_rows(x, gscale=g)
        assert fa.fp4attn_read_status(out["workspace"]) == fa.ERR_RANGE
        ws = fa.new_linear_workspace(4, 4, 64)
        fa.fp4attn_gemm(w["codes"], w["scales"], w["codes"], w["scales"], w_gscale=g, workspace=ws)
        assert fa.fp4attn_read_status(ws) == fa.ERR_RANGE


def product_bound(xv, wv, y64):
    """How far a bf16 product may be from the 64-bit one.

    Every term is exact in fp32 (a 4-bit by 4-bit significand under two 4-bit
    scale significands: 16 bits) up to the factor g_x g_w applied at the end
    (two roundings).  The K terms are added in fp32 in some tree or chain: at
    most K + 2 roundings or truncations of 2^-23 relative to the sum of
    magnitudes.  The store rounds to bf16, 2^-9 relative to the result (half a
    step is eps / 2 = 2^-8 at most)."""
    K = xv.shape[1]
    mag = xv.abs() @ wv.abs().t()
    return mag * (K + 4) * 2.0 ** -23 + y64.abs() * 2.0 ** -8 + 1e-30


def check_product(y, x, w, g, bias=None):
    xv, wv = ref.values(x[0], x[1], x[2]), ref.values(w[0], w[1], w[2])
    y64 = xv @ wv.t()
    bound = product_bound(xv, wv, y64)
    if bias is not None:
        y64 = y64 + bias.double()
        bound = bound + y64.abs() * 2.0 ** -8 + bias.double().abs() * 2.0 ** -23
    diff = (y.double().cpu() - y64).abs()
    assert torch.isfinite(y).all()
    worst = (diff / bound).max().item() if diff.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.3g} of the bound"


GEMMS = [(1, 64, 32), (1, 129, 96), (1, 1000, 6144), (5, 384, 2080), (16, 16, 256), (17, 257, 544), (64, 128, 64),
         (65, 100, 8224), (100, 1003, 1056), (128, 256, 256), (129, 256, 512), (130, 255, 288), (333, 1003, 2080),
         (1000, 520, 96), (257, 4104, 544), (2000, 3000, 1056), (4097, 6000, 320), (6001, 3501, 64)]


@pytest.mark.parametrize("M,N,K", GEMMS)
def test_gemm_against_64_bits(M, N, K):
    fa = _fa()
    _, xc, xs, xg = ref.make_packed(M, K, M + 3 * K)
    _, wc, ws_, wg = ref.make_packed(N, K, N + 5 * K, std=K ** -0.5, outliers=0)
    x, w = ref.packed_to("cuda", xc, xs, xg), ref.packed_to("cuda", wc, ws_, wg)
    work = fa.new_linear_workspace(M, N, K)
    y = fa.fp4attn_gemm(x[0], x[1], w[0], w[1], x_gscale=x[2], w_gscale=w[2], workspace=work)
    assert fa.fp4attn_read_status(work) == 0
    check_product(y, (xc, xs, xg), (wc, ws_, wg), None)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(N)).bfloat16()
    # an output of a wider row stride: what lies between its rows is left alone
    for pad in (8, 3):
        big = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        out = fa.fp4attn_gemm(x[0], x[1], w[0], w[1], x_gscale=x[2], w_gscale=w[2], bias=bias.cuda(), y=big[:, :N],
                              workspace=work)
        assert out.data_ptr() == big.data_ptr() and (big[:, N:] == 7.0).all()
        check_product(big[:, :N], (xc, xs, xg), (wc, ws_, wg), None, bias)
    assert fa.fp4attn_read_status(work) == 0


@pytest.mark.parametrize("M,N,K", [(1, 777, 6144), (33, 384, 544), (500, 1536, 2080)])
@pytest.mark.parametrize("g", [None, 0.02, "dynamic"])
def test_linear_quantises_and_multiplies(M, N, K, g):
    fa = _fa()
    x = _source(M, K, M + N)
    big = torch.zeros(M, K + 24, dtype=torch.bfloat16)
    big[:, :K] = x
    xin = big.cuda()[:, :K]  # strided rows
    gv = float(np.float32(ref.computed_g(x) if g == "dynamic" else 1.0 if g is None else g))
    xc, xs = ref.quantize(x, gv)
    _, wc, ws_, wg = ref.make_packed(N, K, N, std=K ** -0.5, outliers=0)
    w = ref.packed_to("cuda", wc, ws_, wg)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(3)).bfloat16()
    gt = torch.tensor([gv], device="cuda") if isinstance(g, float) else None
    ws = fa.new_linear_workspace(M, N, K)
    y = fa.fp4attn_linear(xin, w[0], w[1], w_gscale=w[2], x_gscale=gt, dynamic_gscale=g == "dynamic",
                          bias=bias.cuda(), workspace=ws)
    assert fa.fp4attn_read_status(ws) == 0
    check_product(y, (xc, xs, gv), (wc, ws_, wg), None, bias)
    again = fa.fp4attn_linear(xin, w[0], w[1], w_gscale=w[2], x_gscale=gt, dynamic_gscale=g == "dynamic",
                              bias=bias.cuda(), workspace=ws)
    assert torch.equal(y, again)


def test_scale_bytes_of_rows_past_the_end_do_not_matter():
    """The tiles cover 128 rows: bytes of rows that do not exist may be anything, a NaN pattern too."""
    fa = _fa()
    M, N, K = 70, 200, 288
    _, xc, xs, xg = ref.make_packed(M, K, 1)
    _, wc, ws_, wg = ref.make_packed(N, K, 2)
    x, w = ref.packed_to("cuda", xc, xs, xg), ref.packed_to("cuda", wc, ws_, wg)
    y = fa.fp4attn_gemm(x[0], x[1], w[0], w[1], x_gscale=x[2], w_gscale=w[2])
    for p, rows in ((x, M), (w, N)):
        R, C = -(-rows // 128), -(-K // 64)
        t = p[1].view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4).clone()
        t[rows:] = 0x7F
        p[1].copy_(t.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1))
    assert torch.equal(y, fa.fp4attn_gemm(x[0], x[1], w[0], w[1], x_gscale=x[2], w_gscale=w[2]))


def test_empty_sizes():
    fa = _fa()
    _, wc, ws_, wg = ref.make_packed(10, 64, 2)
    w = ref.packed_to("cuda", wc, ws_, wg)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    q = fa.fp4attn_quantize_rows(none, dynamic_gscale=True)
    assert float(q["gscale"].item()) == 2.0 ** -64
    assert fa.fp4attn_dequant_rows(q["codes"], q["scales"]).shape == (0, 64)
    assert fa.fp4attn_linear(none, w[0], w[1]).shape == (0, 10)
    x = torch.randn(3, 64).bfloat16().cuda()
    assert fa.fp4attn_linear(x, w[0][:0], w[1][:0]).shape == (3, 0)


def test_graph_and_stream():
    """A captured linear replays on new inputs; a call on another stream works there."""
    fa = _fa()
    M, N, K = 130, 512, 544
    _, wc, ws_, wg = ref.make_packed(N, K, 2)
    w = ref.packed_to("cuda", wc, ws_, wg)
    a, b = _source(M, K, 1).cuda(), _source(M, K, 2).cuda()
    want = [fa.fp4attn_linear(v, w[0], w[1], w_gscale=w[2], dynamic_gscale=True) for v in (a, b)]
    x, ws = a.clone(), fa.new_linear_workspace(M, N, K)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.fp4attn_linear(x, w[0], w[1], w_gscale=w[2], dynamic_gscale=True, y=y, workspace=ws)
    s.synchronize()
    assert torch.equal(y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fp4attn_linear(x, w[0], w[1], w_gscale=w[2], dynamic_gscale=True, y=y, workspace=ws)
    for v, z in ((b, want[1]), (a, want[0])):
        x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    assert fa.fp4attn_read_status(ws) == 0


# the kernel with 16, 64 and 128 columns a tile, whole and split, and the pairs with either operand on the lanes
@pytest.mark.parametrize("M,N,K", [(3, 200, 96), (3, 200, 4128), (40, 200, 96), (40, 200, 4128), (100, 300, 288),
                                   (100, 300, 4128), (2100, 2100, 96), (2104, 2104, 96)])
@pytest.mark.parametrize("gx,gw,byte", [(1.3 * 2.0 ** -74, 1.7 * 2.0 ** -74, 0x7E), (1.1e24, 1.3e15, 0x01),
                                        (2.0 ** -149, 3.0e38, 0x38), (1.9 * 2.0 ** 20, 3.1, 0x38)])
@pytest.mark.parametrize("bias", [False, True])
def test_scales_whose_product_leaves_the_range(M, N, K, gx, gw, byte, bias):
    """Each scale and each result is an ordinary number; g_x g_w in fp32 has lost its digits or is infinite."""
    fa = _fa()
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    gx, gw = float(np.float32(gx)), float(np.float32(gw))
    mags = torch.tensor(ref.MAGS, device="cuda")
    table = torch.cat([mags, -mags])
    packed, values = [], []
    for rows in (M, N):
        codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
        codes[rows // 2] = 0  # a row of zeros: its results are zero, not NaN
        v = table[torch.stack([codes & 15, codes >> 4], -1).view(rows, K).long()]
        packed += [codes, torch.full((-(-rows // 128) * -(-K // 64) * 512,), byte, dtype=torch.uint8, device="cuda")]
        values.append(v * float(ref.UE4M3[byte]))
    want = (values[0] @ values[1].t()) * (gx * gw)
    mag = (values[0].abs() @ values[1].abs().t()) * (gx * gw)
    b = None
    if bias:  # of the results' size
        b = (torch.randn(N, generator=gen, device="cuda") * float(want.std())).bfloat16()
        want = want + b.double()
    ws = fa.new_linear_workspace(M, N, K)
    y = fa.fp4attn_gemm(*packed, x_gscale=torch.tensor([gx], device="cuda"), w_gscale=torch.tensor([gw], device="cuda"),
                        bias=b, workspace=ws)
    assert fa.fp4attn_read_status(ws) == 0 and torch.isfinite(y).all()
    # the terms are exact in fp32: K additions and three roundings of the scales and the bias, 2^-23 each; the
    # store by half a bf16 step, at least that of bf16's subnormals
    bound = (mag + want.abs()) * (K + 4) * 2.0 ** -23 + want.abs() * 2.0 ** -8 + 2.0 ** -134
    assert ((y.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("M,N,K", [(3, 200, 4128), (40, 200, 4128), (100, 300, 4128), (2100, 2100, 288), (2104, 2101, 288)])
def test_scale_bytes_of_rows_past_the_end_do_not_matter_to_any_kernel(M, N, K):
    """As above, for split products and for pairs with either operand on the lanes."""
    fa = _fa()
    _, xc, xs, xg = ref.make_packed(M, K, 1)
    _, wc, ws_, wg = ref.make_packed(N, K, 2)
    x, w = ref.packed_to("cuda", xc, xs, xg), ref.packed_to("cuda", wc, ws_, wg)
    y = fa.fp4attn_gemm(x[0], x[1], w[0], w[1], x_gscale=x[2], w_gscale=w[2])
    for p, rows in ((x, M), (w, N)):
        R, C = -(-rows // 128), -(-K // 64)
        t = p[1].view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4).clone()
        t[rows:] = 0x7F
        p[1].copy_(t.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1))
    assert torch.equal(y, fa.fp4attn_gemm(x[0], x[1], w[0], w[1], x_gscale=x[2], w_gscale=w[2]))
