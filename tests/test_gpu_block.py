"""The operators around the attention as they are used together: a block of
quantised QKV projection, FP4 attention, output projection and gated norms, its
training step, and the differentiable forms against 64-bit references."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _fa():
    from nvfp4_precision_b200 import fp4attn
    return fp4attn


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape, std=1.0, dtype=BF):
    return (std * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)


def _values(fa, q):
    return fa.fp4attn_dequant_rows(q["codes"], q["scales"], q["gscale"], dtype=torch.float32).double()


@pytest.mark.parametrize("lead,K,N", [((7,), 96, 40), ((2, 33), 256, 513), ((300,), 544, 200)])
@pytest.mark.parametrize("wdtype", [BF, torch.float32])
@pytest.mark.parametrize("bias", [False, True])
def test_fp4_linear_and_its_gradients(lead, K, N, wdtype, bias):
    fa = _fa()
    gen = _gen(K + N)
    x = _randn(gen, *lead, K).requires_grad_()
    w = _randn(gen, N, K, std=K ** -0.5, dtype=wdtype).requires_grad_()
    b = _randn(gen, N).requires_grad_() if bias else None
    dy = _randn(gen, *lead, N)
    y = fa.fp4_linear(x, w, b)
    y.backward(dy)
    xv = _values(fa, fa.fp4attn_quantize_rows(x.detach().view(-1, K), dynamic_gscale=True))
    wv = _values(fa, fa.fp4attn_quantize_rows(w.detach(), dynamic_gscale=True))
    g = dy.double().view(-1, N)

    def check(got, a, c, add=None):
        # the values are fl(fl(g s) e): two roundings each beside the exact products', then the fp32 sums
        want, mag = a @ c, a.abs() @ c.abs()
        if add is not None:
            want, mag = want + add, mag + add.abs()
        assert ref.worst(got, want, mag * (a.shape[1] + 24) * 2.0 ** -23) <= 1.0

    check(y.detach().view(-1, N), xv, wv.t(), b.detach().double() if bias else None)
    check(x.grad.view(-1, K), g, wv)
    # a bf16 gradient, widened where the weight is fp32
    check(w.grad.to(BF) if wdtype == torch.float32 else w.grad, g.t(), xv)
    assert torch.equal(w.grad, w.grad.to(BF).to(wdtype))
    if bias:
        assert ref.worst(b.grad, g.sum(0), g.abs().sum(0) * g.shape[0] * ref.U) <= 1.0


def test_fp4_linear_takes_views_and_skips_what_is_not_needed():
    fa = _fa()
    gen = _gen(2)
    big = _randn(gen, 5, 40, 128)
    x = big[:, ::2, :96]  # strided rows
    w = _randn(gen, 72, 96, std=0.1).requires_grad_()
    y = fa.fp4_linear(x, w)
    assert torch.equal(y, fa.fp4_linear(x.contiguous(), w))
    y.sum().backward()
    assert w.grad is not None and big.grad is None
    with torch.no_grad():
        assert torch.equal(fa.fp4_linear(x, w), y)


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_norm_gate_autograd(layer, dtype):
    fa = _fa()
    gen = _gen(4)
    B, n, C = 3, 21, 200
    x = _randn(gen, B, n, C, std=2.0, dtype=dtype).requires_grad_()
    h = _randn(gen, B, n, C).requires_grad_()
    mod = _randn(gen, B, 3 * C, std=0.3).requires_grad_()
    w = [(1 + _randn(gen, C, std=0.1, dtype=torch.float32)).to(BF).requires_grad_() for _ in range(2)]
    gate, scale, shift = mod.chunk(3, 1)
    y, z = fa.norm_gate(x, h, w[0], gate, w[1], scale, shift, eps=1e-6, layer_norm=layer)
    dy, dz = _randn(gen, B, n, C, dtype=dtype), _randn(gen, B, n, C)
    torch.autograd.backward([y, z], [dy, dz])
    two = lambda t: t.detach().reshape(B * n, C)
    v = [t.detach() for t in (gate, scale, shift)]
    want, bound = ref.norm_gate64(two(x), two(h), w[0].detach(), v[0], w[1].detach(), v[1], v[2], B, layer, 1e-6)
    assert ref.worst(two(y), want["y"], bound["y"]) <= 1.0 and ref.worst(two(z), want["z"], bound["z"]) <= 1.0
    want, bound = ref.norm_gate_backward64(two(dz), two(dy), two(y), two(h), w[0].detach(), v[0], w[1].detach(), v[1], B,
                                           layer, 1e-6)
    got = dict(dx=two(x.grad), dh=two(h.grad), dpost_weight=w[0].grad, dpre_weight=w[1].grad)
    got.update(zip(("dgate", "dscale", "dshift"), mod.grad.chunk(3, 1)))
    for k in want:
        assert ref.worst(got[k], want[k], bound[k]) <= 1.0, k


def test_norm_gate_autograd_of_one_output():
    fa = _fa()
    gen = _gen(6)
    x, h = _randn(gen, 9, 64).requires_grad_(), _randn(gen, 9, 64).requires_grad_()
    y, z = fa.norm_gate(x, h)
    (gz,) = torch.autograd.grad(z, h, torch.ones_like(z), retain_graph=True)
    ref_out = fa.fp4attn_norm_gate_backward(torch.ones_like(z), None, y.detach(), h.detach())
    assert torch.equal(gz, ref_out["dh"])
    (gy,) = torch.autograd.grad(y, x, torch.ones_like(y))
    assert torch.equal(gy, torch.ones_like(y))  # z not used: the residual passes dy on
    a, b = fa.norm_gate(x.detach().requires_grad_())
    assert torch.equal(a, x)


def test_differentiable_forms_refuse_a_capture():
    fa = _fa()
    x = torch.randn(4, 64, device="cuda").to(BF)
    w = torch.randn(8, 64, device="cuda").to(BF)
    for call in (lambda: fa.fp4_linear(x, w), lambda: fa.norm_gate(x)):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = x + 1  # a capture with something in it
            with pytest.raises(RuntimeError, match="captured"):
                call()
        graph.replay()
        assert torch.equal(held, x + 1)


def _block(fa, p, x, h, B, n, H, D):
    """norm -> NVFP4 QKV -> FP4 attention -> NVFP4 output projection -> gated norm."""
    C = H * D
    a = fa.fp4attn_norm_gate(x, h, quantize=True, z_gscale=p["gz"], workspace=p["ws"], **p["norm"])
    qkv = fa.fp4attn_gemm(a["z_codes"], a["z_scales"], *p["wqkv"], x_gscale=p["gz"], w_gscale=p["gqkv"], bias=p["bqkv"],
                          workspace=p["ws"])
    q, k, v = (t.view(B, n, H, D).transpose(1, 2) for t in qkv.chunk(3, 1))
    packed = fa.fp4attn_quantize_qk(q, k, workspace=p["aws"])
    o, _ = fa.fp4attn_forward(packed["q_codes"], packed["q_scales"], packed["k_codes"], packed["k_scales"], v,
                              o=p["o"].view(B, n, H, D).transpose(1, 2), workspace=p["aws"])
    out = fa.fp4attn_linear(p["o"], *p["wo"], w_gscale=p["go"], dynamic_gscale=True, workspace=p["ws"])
    return a["y"], qkv, out, fa.fp4attn_norm_gate(a["y"], out, workspace=p["ws"], **p["norm"])


def test_a_block_end_to_end_and_replayed():
    fa = _fa()
    B, n, H, D = 2, 150, 2, 128
    C, M = H * D, B * n
    gen = _gen(9)
    mod = _randn(gen, B, 3 * C, std=0.3)
    gate, scale, shift = mod.chunk(3, 1)
    ones = torch.ones(C, device="cuda").to(BF)
    p = dict(norm=dict(post_weight=ones, gate=gate, pre_weight=ones, scale=scale, shift=shift),
             gz=torch.tensor([0.01], device="cuda"), bqkv=_randn(gen, 3 * C), ws=fa.new_linear_workspace(M, 3 * C, C),
             aws=fa.new_workspace(B, H, n), o=torch.empty(M, C, dtype=BF, device="cuda"))
    for name, N in (("qkv", 3 * C), ("o", C)):
        q = fa.fp4attn_quantize_rows(_randn(gen, N, C, std=C ** -0.5), dynamic_gscale=True)
        p["w" + name], p["g" + name] = (q["codes"], q["scales"]), q["gscale"]
    x, h = _randn(gen, M, C, std=2.0, dtype=torch.float32), _randn(gen, M, C)
    y, qkv, out, last = _block(fa, p, x, h, B, n, H, D)
    assert fa.fp4attn_read_status(p["ws"]) == 0 and fa.fp4attn_read_status(p["aws"]) == 0
    # each step against its reference on the inputs that it had
    nrm = (p["norm"][k] for k in ("post_weight", "gate", "pre_weight", "scale", "shift"))
    nrm = list(nrm)
    want, bound = ref.norm_gate64(x, h, *nrm, B, False, 1e-6)
    assert ref.worst(y, want["y"], bound["y"]) <= 1.0
    z = fa.fp4attn_norm_gate(x, h, **p["norm"])["z"]
    zq = fa.fp4attn_quantize_rows(z, gscale=p["gz"])
    zv, wv = _values(fa, zq), fa.fp4attn_dequant_rows(*p["wqkv"], p["gqkv"], dtype=torch.float32).double()
    want, mag = zv @ wv.t() + p["bqkv"].double(), zv.abs() @ wv.abs().t() + p["bqkv"].double().abs()
    assert ref.worst(qkv, want, mag * (C + 24) * 2.0 ** -23) <= 1.0
    ov = _values(fa, fa.fp4attn_quantize_rows(p["o"], dynamic_gscale=True))
    wv = fa.fp4attn_dequant_rows(*p["wo"], p["go"], dtype=torch.float32).double()
    assert ref.worst(out, ov @ wv.t(), (ov.abs() @ wv.abs().t()) * (C + 24) * 2.0 ** -23) <= 1.0
    want, bound = ref.norm_gate64(y, out, *nrm, B, False, 1e-6)
    assert ref.worst(last["y"], want["y"], bound["y"]) <= 1.0 and ref.worst(last["z"], want["z"], bound["z"]) <= 1.0
    # the whole chain captured once and replayed on other inputs
    first = [t.clone() for t in (y, qkv, out, last["y"], last["z"])]
    xs, hs = x.clone(), h.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ry, rqkv, rout, rlast = _block(fa, p, xs, hs, B, n, H, D)
    for a, b in ((-x, -h), (x, h)):
        xs.copy_(a)
        hs.copy_(b)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (ry, rqkv, rout, rlast["y"], rlast["z"])))
    assert fa.fp4attn_read_status(p["ws"]) == 0


def test_a_training_step_has_gradients():
    """Differentiable norm, projections and attention in one graph: finite gradients of every leaf, the same twice."""
    fa = _fa()
    B, n, H, D = 1, 130, 2, 128
    C = H * D

    def step():
        gen = _gen(12)
        x, h = (_randn(gen, B, n, C).requires_grad_() for _ in range(2))
        wqkv, wo = (_randn(gen, N, C, std=C ** -0.5, dtype=torch.float32).requires_grad_() for N in (3 * C, C))
        mod = _randn(gen, B, 3 * C, std=0.3).requires_grad_()
        gate, scale, shift = mod.chunk(3, 1)
        y, z = fa.norm_gate(x, h, None, gate, None, scale, shift)
        q, k, v = (t.view(B, n, H, D).transpose(1, 2) for t in fa.fp4_linear(z, wqkv).chunk(3, -1))
        o = fa.fp4_attention(q, k, v).transpose(1, 2).reshape(B, n, C)
        y2, z2 = fa.norm_gate(y, fa.fp4_linear(o, wo))
        (y2.float().square().mean() + z2.float().mean()).backward()
        return [t.grad for t in (x, h, wqkv, wo, mod)]

    a, b = step(), step()
    for p, q in zip(a, b):
        assert torch.isfinite(p).all() and p.abs().sum() > 0
    # the attention's gradient of K passes through sums whose order may vary; the rest of the chain does not
    assert torch.equal(a[3], b[3])


def test_two_streams_with_a_workspace_each():
    fa = _fa()
    gen = _gen(14)
    K, N = 544, 264
    w = fa.fp4attn_quantize_rows(_randn(gen, N, K, std=0.05), dynamic_gscale=True)
    xs = [_randn(gen, 300 + i, K) for i in range(2)]
    want = [fa.fp4attn_linear(x, w["codes"], w["scales"], w["gscale"], dynamic_gscale=True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [fa.new_linear_workspace(x.shape[0], N, K) for x in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(fa.fp4attn_linear(xs[i], w["codes"], w["scales"], w["gscale"], dynamic_gscale=True,
                                            workspace=ws[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i]) and fa.fp4attn_read_status(ws[i]) == 0


def test_weights_quantised_right_before_they_are_used():
    """Back to back on one stream, with launches that overlap: no kernel reads what the one before still writes."""
    fa = _fa()
    gen = _gen(15)
    K, N, M = 2048, 1536, 64
    x = fa.fp4attn_quantize_rows(_randn(gen, M, K))
    xb = _randn(gen, M, K)
    ws = fa.new_linear_workspace(M, N, K)
    master = [_randn(gen, N, K, std=0.02, dtype=torch.float32) for _ in range(4)]
    packed = [fa.fp4attn_quantize_rows(m, dynamic_gscale=True) for m in master]
    torch.cuda.synchronize()
    want = []
    for q in packed:
        want.append((fa.fp4attn_gemm(x["codes"], x["scales"], q["codes"], q["scales"], w_gscale=q["gscale"], workspace=ws),
                     fa.fp4attn_linear(xb, q["codes"], q["scales"], q["gscale"], workspace=ws)))
        torch.cuda.synchronize()
    codes, scales = torch.empty_like(packed[0]["codes"]), torch.empty_like(packed[0]["scales"])
    g = torch.empty(1, device="cuda")
    for _ in range(10):
        got = []
        for m in master:
            fa.fp4attn_quantize_rows(m, gscale=g, dynamic_gscale=True, codes=codes, scales=scales, workspace=ws)
            a = fa.fp4attn_gemm(x["codes"], x["scales"], codes, scales, w_gscale=g, workspace=ws)
            got.append((a, fa.fp4attn_linear(xb, codes, scales, g, workspace=ws)))
        torch.cuda.synchronize()
        for (a, b), (p, q) in zip(got, want):
            assert torch.equal(a, p) and torch.equal(b, q)
    assert fa.fp4attn_read_status(ws) == 0


def test_wrong_kinds_are_refused():
    """Types, shapes and layouts that the calls cannot take, and tensors off the device among those on it."""
    fa = _fa()
    gen = _gen(16)
    x = _randn(gen, 4, 64)
    w = fa.fp4attn_quantize_rows(_randn(gen, 8, 64))
    c, s = w["codes"], w["scales"]
    g = torch.ones(1, device="cuda")
    nb = dict(dz=x, dy=x, y=x, h=x)
    bad = [lambda: fa.fp4attn_quantize_rows(x.half()), lambda: fa.fp4attn_quantize_rows(x.t()),
           lambda: fa.fp4attn_quantize_rows(x, gscale=g.double()), lambda: fa.fp4attn_quantize_rows(x, codes=c),
           lambda: fa.fp4attn_quantize_rows(x, workspace=g), lambda: fa.fp4attn_dequant_rows(c, s[:-1]),
           lambda: fa.fp4attn_dequant_rows(c.int(), s), lambda: fa.fp4attn_gemm(c, s, c[:, :16].contiguous(), s),
           lambda: fa.fp4attn_gemm(c, s, c, s, bias=g), lambda: fa.fp4attn_gemm(c, s, c, s, y=x),
           lambda: fa.fp4attn_linear(x.float(), c, s), lambda: fa.fp4attn_linear(x[:, :32], c, s),
           lambda: fa.fp4attn_linear_backward(x, c, s, c, s), lambda: fa.fp4attn_norm_gate(x, x.float()),
           lambda: fa.fp4attn_norm_gate(x, x[:2]), lambda: fa.fp4attn_norm_gate(x, x, post_weight=x),
           lambda: fa.fp4attn_norm_gate(x, x, gate=x[:2], scale=x[:1]), lambda: fa.fp4attn_norm_gate(x, x, gate=x[:2], groups=4),
           lambda: fa.fp4attn_norm_gate(x, x, pre_weight=x[0].float()), lambda: fa.fp4attn_norm_gate(x, y=x.float()),
           lambda: fa.fp4attn_norm_gate_backward(**{**nb, "dz": x.float()}),
           lambda: fa.fp4attn_norm_gate_backward(**{**nb, "dy": x.float()}),
           lambda: fa.fp4attn_norm_gate_backward(**{**nb, "h": x[:3]})]
    for call in bad:
        with pytest.raises(AssertionError):
            call()
    for call in (lambda: fa.fp4attn_linear(x, c, s.cpu()), lambda: fa.fp4attn_linear(x, c, s, g.cpu()),
                 lambda: fa.fp4attn_norm_gate(x, x.cpu()), lambda: fa.fp4attn_norm_gate(x, x, gate=x[:1].cpu()),
                 lambda: fa.fp4attn_gemm(c, s, c, s, workspace=torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    for call in (lambda: fa.fp4attn_quantize_rows(_randn(gen, 4, 72)[:, :40]), lambda: fa.fp4attn_norm_gate(_randn(gen, 4, 60)),
                 lambda: fa.fp4attn_norm_gate(_randn(gen, 4, 72), quantize=True),
                 lambda: fa.fp4attn_norm_gate(x, gate=x[:3]), lambda: fa.fp4attn_norm_gate(x, eps=-1.0),
                 lambda: fa.fp4attn_linear(x, c, s, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa.Fp4AttnError):
            call()


def test_results_in_place_and_strided_through_the_c_abi():
    """What the header allows and the binding never asks for: gradients over their inputs, rows of other strides."""
    fa = _fa()
    gen = _gen(18)
    M, C, G = 50, 1160, 2
    for dtype in (BF, torch.float32):
        y, dy = _randn(gen, M, C, dtype=dtype), _randn(gen, M, C, dtype=dtype)
        h, dz = _randn(gen, M, C), _randn(gen, M, C)
        gate = _randn(gen, G, C)
        ws = fa.new_norm_backward_workspace(M, C, G)
        want = fa.fp4attn_norm_gate_backward(dz, dy, y, h, gate=gate, workspace=ws)
        vec = fa.NormVectors(gate=gate.data_ptr(), gate_stride=C)
        t = fa.F32 if dtype == torch.float32 else fa.BF16
        for over in ("dz", "h"):
            dx, dzc, hc = dy.clone(), dz.clone(), h.clone()
            dh = dzc if over == "dz" else hc
            rc = fa.lib.fp4attn_norm_gate_backward(dzc.data_ptr(), C, dx.data_ptr(), C, y.data_ptr(), C, t, hc.data_ptr(), C,
                                                   vec, M, C, G, 1e-6, 0, dx.data_ptr(), C, dh.data_ptr(), C, None, None, None,
                                                   None, None, ws.data_ptr(), ws.numel(), fa._stream(None))
            assert rc == 0 and torch.equal(dx, want["dx"]) and torch.equal(dh, want["dh"])
        # outputs between rows of other data
        big = {k: torch.full((M, C + 16), 3.0, dtype=want[k].dtype, device="cuda") for k in ("dx", "dh")}
        rc = fa.lib.fp4attn_norm_gate_backward(dz.data_ptr(), C, dy.data_ptr(), C, y.data_ptr(), C, t, h.data_ptr(), C, vec, M, C,
                                               G, 1e-6, 0, big["dx"].data_ptr(), C + 16, big["dh"].data_ptr(), C + 16, None, None,
                                               None, None, None, ws.data_ptr(), ws.numel(), fa._stream(None))
        assert rc == 0
        for k, b in big.items():
            assert torch.equal(b[:, :C], want[k]) and (b[:, C:] == 3.0).all()
        z = torch.full((M, C + 8), 3.0, dtype=BF, device="cuda")
        rc = fa.lib.fp4attn_norm_gate(y.data_ptr(), t, C, h.data_ptr(), C, vec, M, C, G, 1e-6, 0, None, 0, z.data_ptr(), C + 8,
                                      None, None, None, None, 0, fa._stream(None))
        assert rc == 0 and (z[:, C:] == 3.0).all()
        assert torch.equal(z[:, :C], fa.fp4attn_norm_gate(y, h, gate=gate)["z"])
    # dx of the linear layer, whole tiles and split ones
    for M, N, K in ((700, 264, 96), (5000, 4000, 544)):
        x, w = fa.fp4attn_quantize_rows(_randn(gen, M, K)), fa.fp4attn_quantize_rows(_randn(gen, N, K))
        dy = _randn(gen, M, N)
        ws = fa.new_linear_backward_workspace(M, N, K)
        want = fa.fp4attn_linear_backward(dy, x["codes"], x["scales"], w["codes"], w["scales"], want_dw=False, want_dbias=False)[0]
        big = torch.full((M, K + 24), 3.0, dtype=BF, device="cuda")
        rc = fa.lib.fp4attn_linear_backward(dy.data_ptr(), N, None, None, None, w["codes"].data_ptr(), w["scales"].data_ptr(), None,
                                            M, N, K, big.data_ptr(), K + 24, None, None, ws.data_ptr(), ws.numel(),
                                            fa._stream(None))
        assert rc == 0 and torch.equal(big[:, :K], want) and (big[:, K:] == 3.0).all()
        assert fa.fp4attn_read_status(ws) == 0


def test_chains_through_launches_that_overlap():
    """Each call reads what the one before has just written, on one stream with no wait between them."""
    fa = _fa()
    gen = _gen(19)
    M, C = 640, 512
    w = fa.fp4attn_quantize_rows(_randn(gen, C, C, std=C ** -0.5), dynamic_gscale=True)
    x, h = _randn(gen, M, C), _randn(gen, M, C)
    ws = fa.new_linear_workspace(M, C, C)
    bws, nws = fa.new_linear_backward_workspace(M, C, C), fa.new_norm_backward_workspace(M, C, 1)

    def chain(wait):
        outs, t = [], h
        for i in range(6):
            n = fa.fp4attn_norm_gate(x, t, workspace=ws)
            wait()
            q = fa.fp4attn_quantize_rows(n["z"], dynamic_gscale=i % 2 == 0, workspace=ws)
            wait()
            t = fa.fp4attn_gemm(q["codes"], q["scales"], w["codes"], w["scales"], q["gscale"], w["gscale"], workspace=ws)
            wait()
            t = fa.fp4attn_linear(t, w["codes"], w["scales"], w["gscale"], dynamic_gscale=i % 2 == 1, workspace=ws)
            wait()
            g = fa.fp4attn_linear_backward(t, q["codes"], q["scales"], w["codes"], w["scales"], q["gscale"], w["gscale"],
                                           workspace=bws)
            wait()
            b = fa.fp4attn_norm_gate_backward(g[0], None, n["y"], t, workspace=nws)
            wait()
            outs += [t, *g, *b.values()]
        return outs

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        got = chain(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(fa.fp4attn_read_status(v) == 0 for v in (ws, bws, nws))


def test_copies_and_other_streams_are_waited_for():
    """Launches that may start early behind a kernel do not do so past a copy, a memset or an event of another stream."""
    fa = _fa()
    gen = _gen(21)
    M, K, N = 3000, 1024, 512
    w = fa.fp4attn_quantize_rows(_randn(gen, N, K, std=0.03), dynamic_gscale=True)
    ws, nws = fa.new_linear_workspace(M, N, K), fa.new_norm_backward_workspace(M, K)
    host = [torch.randn(M, K).to(BF).pin_memory() for _ in range(4)]

    def use(x):
        a = fa.fp4attn_linear(x, w["codes"], w["scales"], w["gscale"], workspace=ws)
        b = fa.fp4attn_norm_gate(x, x)
        return [a, b["y"], b["z"], fa.fp4attn_norm_gate_backward(x, None, x, x, workspace=nws)["dh"]]

    want = []
    for h in host:
        want.append(use(h.cuda()))
        torch.cuda.synchronize()
    x = torch.empty(M, K, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(5):
        got = []
        for h in host:  # a copy between two calls
            x.copy_(h, non_blocking=True)
            got.append(use(x))
            x.zero_()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, v in zip(got, want) for p, q in zip(g, v))
        got = []
        for i, h in enumerate(host):  # another stream's work between two calls
            done = torch.cuda.Event()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(20):
                    x.copy_(host[(i + 1) % 4], non_blocking=True)
                x.copy_(h, non_blocking=True)
                done.record()
            torch.cuda.current_stream().wait_event(done)
            got.append(use(x))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, v in zip(got, want) for p, q in zip(g, v))
    assert fa.fp4attn_read_status(ws) == 0


@pytest.mark.parametrize("lead", [(12,), (3, 4)])
def test_results_of_the_differentiable_forms_take_operations_in_place(lead):
    """An activation or a residual in place on what they return, and the gradients of the same out of place."""
    fa = _fa()
    gen = _gen(23)
    K, N = 64, 72
    x, r = _randn(gen, *lead, K), _randn(gen, *lead, N)
    w = _randn(gen, N, K, std=0.1)
    pre = _randn(gen, K)
    grads = []
    for inplace in (True, False):
        leaves = [t.clone().requires_grad_() for t in (x, w, pre)]
        a = fa.fp4_linear(leaves[0], leaves[1])
        a = a.add_(r) if inplace else a + r
        a = torch.nn.functional.silu(a, inplace=inplace)
        y, z = fa.norm_gate(leaves[0], None, None, None, leaves[2])
        z = z.mul_(2.0) if inplace else z * 2.0
        (a.float().square().sum() + z.float().square().sum() + y.float().sum()).backward()
        grads.append([t.grad for t in leaves] + [a.detach(), z.detach()])
    assert all(torch.equal(p, q) for p, q in zip(*grads))
    # y is what the backward reads: a change of it is allowed, and reported where a gradient would need the old one
    y, z = fa.norm_gate(x.clone().requires_grad_())
    y.add_(x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.float().sum().backward()


def test_the_norms_write_z_where_the_caller_says():
    fa = _fa()
    gen = _gen(26)
    x, h = _randn(gen, 9, 64), _randn(gen, 9, 64)
    want = fa.fp4attn_norm_gate(x, h)
    big = torch.full((9, 80), 3.0, dtype=BF, device="cuda")
    out = fa.fp4attn_norm_gate(x, h, z=big[:, :64], want_z=False)
    assert out["z"].data_ptr() == big.data_ptr() and torch.equal(out["y"], want["y"])
    assert torch.equal(big[:, :64], want["z"]) and (big[:, 64:] == 3.0).all()
    for call in (lambda: fa.fp4attn_norm_gate(x, h, z=big), lambda: fa.fp4attn_norm_gate(x, h, z=x.float()),
                 lambda: fa.fp4attn_norm_gate(x, h, z=x.clone(), quantize=True)):
        with pytest.raises(AssertionError):
            call()


def test_differentiable_forms_take_vectors_at_any_offset():
    """Slices of a fused bias or weight that do not start on 16 bytes."""
    fa = _fa()
    gen = _gen(24)
    K, N = 96, 1003
    x, w = _randn(gen, 5, K), _randn(gen, N, K, std=0.1)
    for dtype in (BF, torch.float32):
        fused = _randn(gen, 2 * N, dtype=dtype).requires_grad_()
        y = fa.fp4_linear(x, w, fused[N:])
        assert torch.equal(y, fa.fp4_linear(x, w, fused[N:].detach().clone()))
        y.backward(_randn(gen, 5, N))
        assert (fused.grad[:N] == 0).all() and fused.grad[N:].abs().sum() > 0
    fused = _randn(gen, 2 * K + 3).requires_grad_()
    post, pre = fused[1:K + 1], fused[K + 3:]
    got = fa.norm_gate(x, x, post, None, pre)
    want = fa.norm_gate(x, x, post.detach().clone(), None, pre.detach().clone())
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    got[1].float().sum().backward()
    assert fused.grad[1:].abs().sum() > 0 and fused.grad[0] == 0


def test_an_argument_without_a_truth_value_is_refused():
    fa = _fa()
    x = torch.ones(4, 64, dtype=BF, device="cuda")
    two = torch.zeros(2, device="cuda")
    for call in (lambda: fa.fp4attn_quantize_rows(x, dynamic_gscale=two),
                 lambda: fa.fp4attn_norm_gate(x, want_z=two)):
        with pytest.raises(RuntimeError, match="ambiguous"):
            call()


def test_every_call_on_a_stream_that_is_named():
    """stream= gives the results of the current stream."""
    fa = _fa()
    gen = _gen(25)
    M, K, N, G = 60, 96, 40, 3
    x, h, dy = _randn(gen, M, K), _randn(gen, M, K), _randn(gen, M, N)
    wt = _randn(gen, N, K, std=0.1)
    v = dict(zip(("post_weight", "pre_weight"), _randn(gen, 2, K)), **dict(zip(("gate", "scale", "shift"), _randn(gen, 3, G, K))))
    bias, g = _randn(gen, N), torch.tensor([0.02], device="cuda")

    def every(**kw):
        w = fa.fp4attn_quantize_rows(wt, dynamic_gscale=True, **kw)
        q = fa.fp4attn_quantize_rows(x, g, **kw)
        packed, gs = (q["codes"], q["scales"], w["codes"], w["scales"]), (g, w["gscale"])
        n = fa.fp4attn_norm_gate(x, h, groups=G, eps=1e-3, flags=fa.LAYER_NORM, **v, **kw)
        nq = fa.fp4attn_norm_gate(x, h, quantize=True, z_gscale=g, want_y=False, **v, **kw)
        back = {k: t for k, t in v.items() if k != "shift"}
        b = fa.fp4attn_norm_gate_backward(x, h, n["y"], h, groups=G, eps=1e-3, flags=fa.LAYER_NORM, **back, **kw)
        # scale bytes of rows that do not exist are not the norm's to write
        return [q["codes"], fa.fp4attn_dequant_rows(q["codes"], q["scales"], g, torch.float32, **kw),
                fa.fp4attn_gemm(*packed, *gs, bias, **kw), fa.fp4attn_linear(x, *packed[2:], gs[1], g, bias=bias, **kw),
                *fa.fp4attn_linear_backward(dy, *packed, *gs, **kw), n["y"], n["z"], nq["z_codes"], *b.values()]

    want = every()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for name in (s, s.cuda_stream):
        got = every(stream=name)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_large_and_wide_calls_captured():
    """Launches of clusters and pairs in a graph, replayed on other inputs: large products, rows of two and three CTAs."""
    fa = _fa()
    gen = _gen(27)
    M, N, K = 2104, 2096, 544
    w = fa.fp4attn_quantize_rows(_randn(gen, N, K, std=0.05), dynamic_gscale=True)
    ws, bws = fa.new_linear_workspace(M, N, K), fa.new_linear_backward_workspace(M, N, K)
    wide = [(60, 8192), (40, 16384)]
    nws = [fa.new_norm_backward_workspace(*s) for s in wide]
    sources = [[_randn(gen, M, K), _randn(gen, M, N)] + [_randn(gen, *s) for s in wide] for _ in range(2)]

    def every(x, dy, *rows):
        q = fa.fp4attn_quantize_rows(x, dynamic_gscale=True, workspace=ws)
        packed = (q["codes"], q["scales"], w["codes"], w["scales"])
        out = [fa.fp4attn_gemm(*packed, q["gscale"], w["gscale"], workspace=ws),
               fa.fp4attn_linear(x[:5], *packed[2:], w["gscale"], dynamic_gscale=True, workspace=ws),
               *fa.fp4attn_linear_backward(dy, *packed, q["gscale"], w["gscale"], workspace=bws)]
        for r, b in zip(rows, nws):
            n = fa.fp4attn_norm_gate(r, r, flags=fa.LAYER_NORM)
            out += [n["y"], n["z"], *fa.fp4attn_norm_gate_backward(r, r, n["y"], r, flags=fa.LAYER_NORM, workspace=b).values()]
        return out

    want = [[t.clone() for t in every(*s)] for s in sources]
    held = [t.clone() for t in sources[0]]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = every(*held)
    for s, v in ((sources[1], want[1]), (sources[0], want[0])):
        for t, u in zip(held, s):
            t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, v))
    assert all(fa.fp4attn_read_status(t) == 0 for t in (ws, bws, *nws))


def test_an_output_that_finds_no_memory():
    """torch's own exception, and nothing launched: 2^22 x 2^22 results are 35 TB."""
    fa = _fa()
    rows = 1 << 22
    codes = torch.zeros(rows, 16, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(fa.fp4attn_scale_tile_bytes(rows, 32), dtype=torch.uint8, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        fa.fp4attn_gemm(codes, scales, codes, scales)
    del codes, scales
    torch.cuda.empty_cache()
    x = torch.ones(2, 64, dtype=BF, device="cuda")
    assert torch.isfinite(fa.fp4attn_norm_gate(x)["z"]).all()
