"""Linear layers and norms on tensors of more than 2^31 elements.

The rows repeat with a period of 384 (three scale tiles, one and a half of the
largest row tiles), so every period's results are known from the first, whose
own come from a small reference.  Operands of the products are small multiples
of 1/2: every partial sum is exact in fp32, in whatever order it is taken, and
the stored result has one right value."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

PERIOD, TIMES, WIDE = 384, 1400, 4096
ROWS = PERIOD * TIMES
assert ROWS * WIDE > 2 ** 31


def _fa():
    from nvfp4_precision_b200 import fp4attn
    return fp4attn


@pytest.fixture(autouse=True)
def _give_memory_back():
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _periods_equal(t, first):
    """Whether t [TIMES * rows, ...] is first [rows, ...] again and again."""
    n = first.shape[0]
    return all(torch.equal(t[i:i + n], first) for i in range(0, t.shape[0], n))


def _packed(rows, K, gen):
    """Random codes under scales of 1 and their values."""
    codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    mags = torch.tensor(ref.MAGS, device="cuda")
    table = torch.cat([mags, -mags])
    values = table[torch.stack([codes & 15, codes >> 4], -1).view(rows, K).long()]
    scales = torch.full((-(-rows // 128) * -(-K // 64) * 512,), 0x38, dtype=torch.uint8, device="cuda")
    return codes, scales, values


@pytest.mark.parametrize("N", [32776, 32777])
def test_gemm(N):
    fa = _fa()
    gen, K, times = _gen(N), 32, 174
    assert PERIOD * times * N > 2 ** 31
    xc, xs, xv = _packed(PERIOD, K, gen)
    wc, ws, wv = _packed(N, K, gen)
    work = fa.new_linear_workspace(PERIOD * times, N, K)
    y = fa.fp4attn_gemm(xc.repeat(times, 1), xs.repeat(times), wc, ws, workspace=work)
    assert fa.fp4attn_read_status(work) == 0
    assert _periods_equal(y, (xv @ wv.t()).bfloat16())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dynamic", [False, True])
def test_quantise_and_back(dtype, dynamic):
    fa = _fa()
    part = torch.randn(PERIOD, WIDE, device="cuda", generator=_gen(1)).to(dtype)
    x = part.repeat(TIMES, 1)
    if dynamic:  # the largest value stands at the very end
        x[-1, -1] = 1000.0
    out = fa.fp4attn_quantize_rows(x, dynamic_gscale=dynamic)
    assert fa.fp4attn_read_status(out["workspace"]) == 0
    g = 1.0
    if dynamic:
        g = ref.computed_g(torch.tensor([[1000.0]]))
        assert float(out["gscale"]) == g
    codes, scales = ref.quantize(part.cpu(), g)
    want = ref.packed_to("cuda", codes, scales, g)
    assert _periods_equal(out["codes"][:-PERIOD], want[0])
    per = want[1].numel()
    assert _periods_equal(out["scales"][:-per], want[1])
    codes, scales = ref.quantize(x[-PERIOD:].cpu(), g)
    last = ref.packed_to("cuda", codes, scales, g)
    assert torch.equal(out["codes"][-PERIOD:], last[0]) and torch.equal(out["scales"][-per:], last[1])
    gs = out["gscale"] if dynamic else None
    back = fa.fp4attn_dequant_rows(out["codes"], out["scales"], gscale=gs, dtype=dtype)
    one = fa.fp4attn_dequant_rows(want[0], want[1], gscale=gs, dtype=dtype)
    assert _periods_equal(back[:-PERIOD], one)


def test_linear_backward():
    fa = _fa()
    gen, K, N = _gen(2), WIDE, WIDE
    xc, xs, xv = _packed(PERIOD, K, gen)
    wc, ws, wv = _packed(N, K, gen)
    part = torch.randint(-1, 2, (PERIOD, N), device="cuda", generator=gen).bfloat16()
    dy = part.repeat(TIMES, 1)
    # 6 * ROWS halves and 6 * N halves both stay below 2^24: exact
    assert 12 * ROWS < 2 ** 24
    work = fa.new_linear_backward_workspace(ROWS, N, K)
    dx, dw, dbias = fa.fp4attn_linear_backward(dy, xc.repeat(TIMES, 1), xs.repeat(TIMES), wc, ws, workspace=work)
    assert fa.fp4attn_read_status(work) == 0
    p = part.double()
    assert _periods_equal(dx, (p @ wv).to(dx.dtype))
    assert torch.equal(dw, (TIMES * (p.t() @ xv)).to(dw.dtype))
    assert torch.equal(dbias, (TIMES * p.sum(0)).float())


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_and_its_gradients(layer, dtype):
    fa = _fa()
    gen, C, flags = _gen(3), WIDE, fa.LAYER_NORM if layer else 0
    rows = lambda t=torch.bfloat16: torch.randn(PERIOD, C, device="cuda", generator=gen).to(t)
    vec = lambda: (1.0 + 0.1 * torch.randn(C, device="cuda", generator=gen)).bfloat16()
    mod = lambda: (0.3 * torch.randn(1, C, device="cuda", generator=gen)).bfloat16()
    v = dict(post_weight=vec(), gate=mod(), pre_weight=vec(), scale=mod(), shift=mod())
    x, h = rows(dtype), rows()
    out = fa.fp4attn_norm_gate(x.repeat(TIMES, 1), h.repeat(TIMES, 1), flags=flags, eps=1e-6, **v)
    want, bound = ref.norm_gate64(x, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], v["shift"], 1, layer,
                                  1e-6)
    for k in ("y", "z"):
        assert ref.worst(out[k][:PERIOD], want[k], bound[k]) <= 1.0
        assert _periods_equal(out[k], out[k][:PERIOD])
    y = out["y"][:PERIOD].clone()
    v.pop("shift")
    del out, x
    dz, dy = rows(), rows(dtype)
    work = fa.new_norm_backward_workspace(ROWS, C, 1)
    out = fa.fp4attn_norm_gate_backward(dz.repeat(TIMES, 1), dy.repeat(TIMES, 1), y.repeat(TIMES, 1),
                                        h.repeat(TIMES, 1), flags=flags, eps=1e-6, workspace=work, **v)
    assert fa.fp4attn_read_status(work) == 0
    want, bound = ref.norm_gate_backward64(dz, dy, y, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], 1,
                                           layer, 1e-6)
    for k in want:
        if k in ("dx", "dh"):
            assert ref.worst(out[k][:PERIOD], want[k], bound[k]) <= 1.0
            assert _periods_equal(out[k], out[k][:PERIOD])
        else:
            # the period's bound counts PERIOD + 16 roundings of its sum; here they are ROWS + 16
            grown = bound[k] * TIMES * (ROWS + 16) / (PERIOD + 16)
            assert ref.worst(out[k], want[k] * TIMES, grown) <= 1.0, k


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_column_sums_miss_no_row(layer, dtype):
    """The norms' sums down ROWS rows to less than the rows beyond 2^31 elements add to them.

    dshift sums small integers: exact.  The others: a CTA of this width is one team, which adds the rows of a
    part one after the other; the parts (their number shows in the workspace's size) are added in order."""
    fa = _fa()
    gen, C, flags = _gen(4), WIDE, fa.LAYER_NORM if layer else 0
    rows = lambda t=torch.bfloat16: torch.randn(PERIOD, C, device="cuda", generator=gen).to(t)
    vec = lambda: (1.0 + 0.1 * torch.randn(C, device="cuda", generator=gen)).bfloat16()
    mod = lambda: (0.3 * torch.randn(1, C, device="cuda", generator=gen)).bfloat16()
    v = dict(post_weight=vec(), gate=mod(), pre_weight=vec(), scale=mod())
    y, h, dy = rows(dtype), rows(), rows(dtype)
    dz = torch.randint(-1, 2, (PERIOD, C), device="cuda", generator=gen).bfloat16()
    work = fa.new_norm_backward_workspace(ROWS, C, 1)
    parts = (work.numel() - 256) // (12 * C)
    depth = -(-ROWS // parts) + parts + 16
    assert 100 <= parts <= 600
    out = fa.fp4attn_norm_gate_backward(dz.repeat(TIMES, 1), dy.repeat(TIMES, 1), y.repeat(TIMES, 1), h.repeat(TIMES, 1),
                                        flags=flags, eps=1e-6, workspace=work, **v)
    assert fa.fp4attn_read_status(work) == 0
    assert torch.equal(out["dshift"], TIMES * dz.double().sum(0, keepdim=True).float())
    want, bound = ref.norm_gate_backward64(dz, dy, y, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], 1, layer,
                                           1e-6)
    beyond = 1.0 - 2 ** 31 / (ROWS * C)  # the share of a column's rows that lies there
    for k in ("dscale", "dgate", "dpre_weight", "dpost_weight"):
        # the period's bound counts PERIOD + 16 roundings of each term, and the terms' own errors
        grown = bound[k] * TIMES * (depth / (PERIOD + 16))
        assert ref.worst(out[k], want[k] * TIMES, grown) <= 1.0, k
        # without those rows the sums would be off by more, in most columns
        assert (want[k].abs() * TIMES * beyond > grown).double().mean() > 0.5, k


@pytest.mark.parametrize("M,N,K", [(28972, 976, 928), (12652, 18, 2048), (100, 15912, 3328), (9000, 5000, 1728)])
def test_long_contractions_are_whole(M, N, K):
    """Operands whose sums are exact in fp32 in any order: every gradient has one right value."""
    fa = _fa()
    gen = _gen(M)
    xc, xs, xv = _packed(M, K, gen)
    wc, ws, wv = _packed(N, K, gen)
    dy = torch.randint(-1, 2, (M, -(-N // 8) * 8), device="cuda", generator=gen).bfloat16()[:, :N]
    assert 12 * max(M, N) < 2 ** 24  # halves
    work = fa.new_linear_backward_workspace(M, N, K)
    args = (dy, xc, xs, wc, ws)
    d = dy.double()
    want = ((d @ wv).bfloat16(), (d.t() @ xv).bfloat16(), d.sum(0).float())
    for only in ((True, True, True), (True, False, False), (False, True, False)):
        got = fa.fp4attn_linear_backward(*args, want_dx=only[0], want_dw=only[1], want_dbias=only[2], workspace=work)
        assert fa.fp4attn_read_status(work) == 0
        assert all(g is None or torch.equal(g, w) for g, w in zip(got, want))
