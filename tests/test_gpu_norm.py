"""The norms around a branch and their gradients on the GPU against the
formulas in 64 bits, within bounds derived from the fp32 arithmetic."""
import pytest
import torch

import linear_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def _fa():
    from nvfp4_precision_b200 import fp4attn
    return fp4attn


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(M, C, gen, dtype=BF, at=0.0, std=1.0, pad=0):
    x = at + std * torch.randn(M, C + pad, generator=gen, device="cuda")
    if C >= 8:
        x[:, torch.randint(0, C, (1,), generator=gen, device="cuda")] *= 20.0
    return x.to(dtype)[:, :C]


def _vectors(C, G, gen):
    mod = (0.3 * torch.randn(G, 3 * C, generator=gen, device="cuda")).to(BF)
    gate, scale, shift = mod.chunk(3, 1)
    w = (1.0 + 0.1 * torch.randn(2, C, generator=gen, device="cuda")).to(BF)
    return dict(post_weight=w[0], gate=gate, pre_weight=w[1], scale=scale, shift=shift)


# rows, channels, samples: every team size and register count, rows short of
# the teams, parts of samples, a sample per row
SHAPES = [(1, 8, 1), (1, 6144, 1), (5, 128, 5), (77, 264, 7), (640, 520, 2), (300, 776, 3), (129, 1024, 1), (66, 1160, 6),
          (40, 1536, 4), (33, 2048, 1), (31, 2504, 1), (50, 4096, 2), (20, 5000, 1), (1500, 6144, 2), (9, 7168, 3),
          (64, 8192, 1), (12, 10240, 1), (7, 12288, 1), (10, 16384, 5), (5000, 96, 1)]


@pytest.mark.parametrize("M,C,G", SHAPES)
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_forward_against_64_bits(M, C, G, layer, dtype):
    fa = _fa()
    gen = _gen(M + C)
    x, h = _rows(M, C, gen, dtype, at=0.5, std=3.0, pad=8), _rows(M, C, gen, pad=16)
    v = _vectors(C, G, gen)
    ws = fa.new_linear_workspace(0, 0, 32)
    out = fa.fp4attn_norm_gate(x, h, eps=EPS, flags=fa.LAYER_NORM if layer else 0, workspace=ws, **v)
    want, bound = ref.norm_gate64(x, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], v["shift"], G, layer, EPS)
    assert out["y"].dtype == dtype and out["z"].dtype == BF
    for k in ("y", "z"):
        assert ref.worst(out[k], want[k], bound[k]) <= 1.0, k
    again = fa.fp4attn_norm_gate(x, h, eps=EPS, flags=fa.LAYER_NORM if layer else 0, **v)
    assert torch.equal(out["y"], again["y"]) and torch.equal(out["z"], again["z"])
    assert fa.fp4attn_read_status(ws) == 0


@pytest.mark.parametrize("M,C,G", SHAPES)
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_against_64_bits(M, C, G, layer, dtype):
    fa = _fa()
    gen = _gen(M + C + 1)
    y, h = _rows(M, C, gen, dtype, at=0.5, std=3.0, pad=8), _rows(M, C, gen, pad=16)
    dz, dy = _rows(M, C, gen, pad=24), _rows(M, C, gen, dtype, pad=8)
    v = _vectors(C, G, gen)
    v.pop("shift")
    ws = fa.new_norm_backward_workspace(M, C, G)
    out = fa.fp4attn_norm_gate_backward(dz, dy, y, h, eps=EPS, flags=fa.LAYER_NORM if layer else 0, workspace=ws, **v)
    want, bound = ref.norm_gate_backward64(dz, dy, y, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], G,
                                           layer, EPS)
    assert set(out) == set(want)
    for k in want:
        assert out[k].shape == want[k].shape
        assert ref.worst(out[k], want[k], bound[k]) <= 1.0, k
    again = fa.fp4attn_norm_gate_backward(dz, dy, y, h, eps=EPS, flags=fa.LAYER_NORM if layer else 0, workspace=ws, **v)
    for k in want:
        assert torch.equal(out[k], again[k]), k
    assert fa.fp4attn_read_status(ws) == 0


@pytest.mark.parametrize("layer", [False, True])
def test_absent_vectors_and_branch(layer):
    fa = _fa()
    M, C = 37, 512
    gen = _gen(3)
    x, h, dz = _rows(M, C, gen, F32), _rows(M, C, gen), _rows(M, C, gen)
    v = _vectors(C, 1, gen)
    flags = fa.LAYER_NORM if layer else 0
    none = dict(post_weight=None, gate=None, pre_weight=None, scale=None, shift=None)
    cases = [(h, none), (None, none), (None, dict(none, pre_weight=v["pre_weight"], shift=v["shift"]))]
    cases += [(h, dict(none, **{k: v[k]})) for k in none]
    for hh, vec in cases:
        out = fa.fp4attn_norm_gate(x, hh, eps=EPS, flags=flags, **vec)
        want, bound = ref.norm_gate64(x, hh, vec["post_weight"], vec["gate"], vec["pre_weight"], vec["scale"],
                                      vec["shift"], 1, layer, EPS)
        for k in ("y", "z"):
            assert ref.worst(out[k], want[k], bound[k]) <= 1.0, k
        args = {k: vec[k] for k in vec if k != "shift"}
        for dy in (None, x):
            got = fa.fp4attn_norm_gate_backward(dz, dy, x, hh, eps=EPS, flags=flags, **args)
            want, bound = ref.norm_gate_backward64(dz, dy, x, hh, args["post_weight"], args["gate"], args["pre_weight"],
                                                   args["scale"], 1, layer, EPS)
            for k in got:
                if got[k] is None:
                    assert hh is None and k in ("dh", "dgate", "dpost_weight")
                else:
                    assert ref.worst(got[k], want[k], bound[k]) <= 1.0, k
    # one output alone is the same output
    both = fa.fp4attn_norm_gate(x, h, eps=EPS, flags=flags, **v)
    assert torch.equal(fa.fp4attn_norm_gate(x, h, eps=EPS, flags=flags, want_y=False, **v)["z"], both["z"])
    assert torch.equal(fa.fp4attn_norm_gate(x, h, eps=EPS, flags=flags, want_z=False, **v)["y"], both["y"])
    # in place
    mine = x.clone()
    out = fa.fp4attn_norm_gate(mine, h, eps=EPS, flags=flags, y=mine, **v)
    assert torch.equal(mine, both["y"]) and torch.equal(out["z"], both["z"])


@pytest.mark.parametrize("M,C,G", [(1, 32, 1), (1, 6144, 1), (130, 96, 2), (500, 544, 1), (257, 1056, 1), (300, 2080, 3),
                                   (129, 4128, 1), (1000, 6144, 1), (16, 12288, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantised_z_is_the_quantiser_of_z(M, C, G, dtype):
    fa = _fa()
    gen = _gen(M * 3 + C)
    x, h = _rows(M, C, gen, dtype, std=3.0), _rows(M, C, gen)
    v = _vectors(C, G, gen)
    g = torch.tensor([0.013], device="cuda")
    for gz in (None, g):
        z = fa.fp4attn_norm_gate(x, h, eps=EPS, **v)
        q = fa.fp4attn_norm_gate(x, h, eps=EPS, quantize=True, z_gscale=gz, **v)
        want = fa.fp4attn_quantize_rows(z["z"], gscale=gz)
        assert torch.equal(q["y"], z["y"]) and torch.equal(q["z_codes"], want["codes"])
        assert torch.equal(fa.untile_scales(q["z_scales"], M, C), fa.untile_scales(want["scales"], M, C))
        assert fa.fp4attn_read_status(q["workspace"]) == 0


def test_quantised_z_reports_errors_and_plain_z_propagates():
    fa = _fa()
    gen = _gen(5)
    x, h = _rows(4, 64, gen), _rows(4, 64, gen)
    bad = h.clone()
    bad[2, 5] = float("nan")
    out = fa.fp4attn_norm_gate(x, bad)
    assert out["z"][2].isnan().all() and torch.isfinite(out["z"][[0, 1, 3]]).all()
    assert fa.fp4attn_read_status(fa.fp4attn_norm_gate(x, bad, quantize=True)["workspace"]) == fa.ERR_RANGE
    for g in (0.0, -1.0, float("inf"), float("nan")):
        q = fa.fp4attn_norm_gate(x, h, quantize=True, z_gscale=torch.tensor([g], device="cuda"))
        assert fa.fp4attn_read_status(q["workspace"]) == fa.ERR_RANGE


def test_zero_rows_and_constant_rows():
    """A row of zeros has norm 0; a constant row has layer norm 0 up to the rounding of its mean."""
    fa = _fa()
    x = torch.zeros(3, 256, device="cuda")
    x[1] = 7.0
    out = fa.fp4attn_norm_gate(x, eps=EPS)
    assert (out["z"][0] == 0).all() and ref.worst(out["z"][1:2], torch.ones(1, 256, device="cuda").double(),
                                                  torch.full((1, 256), 8e-6, device="cuda").double()) <= 1.0
    assert (fa.fp4attn_norm_gate(x, eps=EPS, flags=fa.LAYER_NORM)["z"] == 0).all()


def test_empty_rows():
    fa = _fa()
    x = torch.empty(0, 64, device="cuda")
    z = torch.empty(0, 64, dtype=BF, device="cuda")
    assert fa.fp4attn_norm_gate(x)["z"].shape == (0, 64)
    out = fa.fp4attn_norm_gate_backward(z, None, x, z, groups=3)
    assert out["dx"].shape == (0, 64) and (out["dgate"] == 0).all() and (out["dpost_weight"] == 0).all()
    assert out["dshift"].shape == (3, 64) and (out["dshift"] == 0).all()


@pytest.mark.parametrize("layer", [False, True])
def test_gradients_against_differences(layer):
    """(L(p + e d) - L(p - e d)) / 2e in 64 bits, for L = <dz, z> + <dy, y>, against <gradient, d>."""
    fa = _fa()
    M, C, G = 24, 136, 3
    gen = _gen(11)
    x, h = _rows(M, C, gen, F32, std=2.0), _rows(M, C, gen)
    v = _vectors(C, G, gen)
    dz, dy = _rows(M, C, gen), _rows(M, C, gen, F32)
    p = {"x": x.double(), "h": h.double(), **{k: t.double() for k, t in v.items()}}

    def fwd(q):
        out, _ = ref.norm_gate64(q["x"], q["h"], q["post_weight"], q["gate"], q["pre_weight"], q["scale"], q["shift"],
                                 G, layer, EPS)
        return out["y"], out["z"]

    y = fwd(p)[0].float()  # an fp32 residual: what the forward keeps, rounded by 2^-24
    vec = {k: t for k, t in v.items() if k != "shift"}
    got = fa.fp4attn_norm_gate_backward(dz, dy, y, h, eps=EPS, flags=fa.LAYER_NORM if layer else 0, **vec)
    _, bound = ref.norm_gate_backward64(dz, dy, y, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], G, layer,
                                        EPS)
    e = 1e-5
    for name in p:
        key = "d" + name
        d = torch.randn(p[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        loss = []
        for s in (e, -e):
            yy, zz = fwd({**p, name: p[name] + s * d})
            loss.append((dz.double() * zz).sum() + (dy.double() * yy).sum())
        diff = (loss[0] - loss[1]) / (2 * e)
        dot = (got[key].double() * d).sum()
        # the gradient's own bound, its rounding, the rounding of y (2^-24 relative, within the
        # bound's constants by a factor above 10), and the differences' own error: e^2 and 2^-53 / e
        tol = ((bound[key] * 2 + got[key].double().abs() * ref.half_step(got[key].dtype)) * d.abs()).sum() \
            + 1e-6 * (got[key].double() * d).abs().sum()
        assert (diff - dot).abs() <= tol, (name, float(diff), float(dot), float(tol))


def test_norm_graph_and_stream():
    fa = _fa()
    M, C, G = 96, 1160, 3
    gen = _gen(8)
    a, b = [(_rows(M, C, gen, F32), _rows(M, C, gen), _rows(M, C, gen)) for _ in range(2)]
    v = _vectors(C, G, gen)
    vec = {k: t for k, t in v.items() if k != "shift"}

    def both(x, h, dz, ws):
        out = fa.fp4attn_norm_gate(x, h, eps=EPS, **v)
        return [*out.values(), *fa.fp4attn_norm_gate_backward(dz, x, out["y"], h, eps=EPS, workspace=ws, **vec).values()]

    ws = fa.new_norm_backward_workspace(M, C, G)
    want = [[t.clone() for t in both(*i, ws)] for i in (a, b)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = both(*a, ws)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want[0]))
    held = [t.clone() for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both(*held, ws)
    for src, w in ((b, want[1]), (a, want[0])):
        for t, u in zip(held, src):
            t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, w))


TEAMS = [104, 264, 520, 776, 1160, 1536, 2048, 2504, 4096, 5000, 6144, 7168, 8192, 10240, 12288, 16384]


@pytest.mark.parametrize("C", TEAMS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layer", [False, True])
def test_equal_rows_have_equal_results(C, dtype, layer):
    """Whichever team of a CTA takes a row: the same bits, also where the mean is many deviations off."""
    fa = _fa()
    gen = _gen(C)
    M, flags = 700, fa.LAYER_NORM if layer else 0
    v = _vectors(C, 1, gen)
    for at in (0.5, 100.0):
        x, h = (_rows(1, C, gen, t, at=at).repeat(M, 1) for t in (dtype, BF))
        dz, dy = (_rows(1, C, gen, t).repeat(M, 1) for t in (BF, dtype))
        out = fa.fp4attn_norm_gate(x, h, eps=EPS, flags=flags, **v)
        vec = {k: t for k, t in v.items() if k != "shift"}
        out.update(fa.fp4attn_norm_gate_backward(dz, dy, out["y"], h, eps=EPS, flags=flags, **vec))
        for k in ("y", "z", "dx", "dh"):
            assert (out[k] == out[k][:1]).all(), (k, at)


def test_an_empty_batch_of_samples():
    """No samples at all: x [0, C] with modulation [0, C]."""
    fa = _fa()
    for dtype in (BF, F32):
        x, h = torch.empty(0, 64, dtype=dtype, device="cuda"), torch.empty(0, 64, dtype=BF, device="cuda")
        v = dict(post_weight=torch.ones(64, dtype=BF, device="cuda"), gate=h, pre_weight=None, scale=h)
        out = fa.fp4attn_norm_gate(x, h, shift=h, **v)
        assert out["y"].shape == out["z"].shape == (0, 64)
        assert fa.fp4attn_norm_gate(x, h, shift=h, quantize=True, **v)["z_codes"].shape == (0, 32)
        got = fa.fp4attn_norm_gate_backward(h, x, x, h, **v)
        for k in ("dshift", "dscale", "dgate", "dx", "dh"):
            assert got[k].shape == (0, 64)
        assert (got["dpre_weight"] == 0).all() and (got["dpost_weight"] == 0).all()
        leaf = torch.empty(0, 5, 64, dtype=dtype, device="cuda", requires_grad=True)
        w = torch.ones(64, dtype=BF, device="cuda", requires_grad=True)
        y, z = fa.norm_gate(leaf, torch.empty(0, 5, 64, dtype=BF, device="cuda"), w, h, None, h, h)
        (y.float().sum() + z.float().sum()).backward()
        assert y.shape == z.shape == leaf.grad.shape == (0, 5, 64) and (w.grad == 0).all()


def _off_centre(M, C, gen, dtype, kind):
    """Rows whose moments lose bits about 0 or about a few of their own values."""
    if kind == "pivot":  # outliers where the kernels look for a first guess of the mean, in each CTA's columns
        x = torch.randn(M, C, generator=gen, device="cuda")
        ctas = -(-C // 6144)
        cols = C if ctas == 1 else -(-C // (64 * ctas)) * 64
        for r in range(ctas):
            mid = cols * r + (min(cols, C - cols * r) // 2)
            x[:, max(mid - 8, 0):mid + 8] += 300.0
        return x.to(dtype)
    return (float(kind) + torch.randn(M, C, generator=gen, device="cuda")).to(dtype)


@pytest.mark.parametrize("C", TEAMS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["pivot", 10, -1000])
def test_layer_norm_of_rows_far_from_zero(C, dtype, kind):
    fa = _fa()
    gen = _gen(C + 7)
    M = 37
    x, h = _off_centre(M, C, gen, dtype, kind), _off_centre(M, C, gen, BF, kind)
    v = _vectors(C, 1, gen)
    out = fa.fp4attn_norm_gate(x, h, eps=EPS, flags=fa.LAYER_NORM, **v)
    want, bound = ref.norm_gate64(x, h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], v["shift"], 1, True, EPS)
    for k in ("y", "z"):
        assert ref.worst(out[k], want[k], bound[k]) <= 1.0, k
    dz, dy = _rows(M, C, gen), _rows(M, C, gen, dtype)
    vec = {k: t for k, t in v.items() if k != "shift"}
    got = fa.fp4attn_norm_gate_backward(dz, dy, out["y"], h, eps=EPS, flags=fa.LAYER_NORM, **vec)
    want, bound = ref.norm_gate_backward64(dz, dy, out["y"], h, v["post_weight"], v["gate"], v["pre_weight"], v["scale"], 1,
                                           True, EPS)
    for k in want:
        assert ref.worst(got[k], want[k], bound[k]) <= 1.0, k


@pytest.mark.parametrize("M,C,G", [(1, 32, 1), (1, 6144, 1), (130, 96, 2), (64, 256, 4), (500, 544, 1), (90, 768, 3),
                                   (257, 1056, 1), (70, 1536, 1), (300, 2080, 3), (200, 2048, 2), (60, 4096, 1),
                                   (129, 4128, 1), (1000, 6144, 2), (33, 8192, 1), (16, 12288, 1), (5, 16384, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantised_layer_norm_is_the_quantiser_of_z(M, C, G, dtype):
    fa = _fa()
    gen = _gen(M * 5 + C)
    x, h = _rows(M, C, gen, dtype, at=0.5, std=3.0), _rows(M, C, gen)
    v = _vectors(C, G, gen)
    g = torch.tensor([0.013], device="cuda")
    for gz in (None, g):
        for hh in (h, None):
            vec = v if hh is not None else {**v, "gate": None, "post_weight": None}
            z = fa.fp4attn_norm_gate(x, hh, eps=EPS, flags=fa.LAYER_NORM, **vec)
            q = fa.fp4attn_norm_gate(x, hh, eps=EPS, flags=fa.LAYER_NORM, quantize=True, z_gscale=gz, **vec)
            want = fa.fp4attn_quantize_rows(z["z"], gscale=gz)
            assert torch.equal(q["y"], z["y"]) and torch.equal(q["z_codes"], want["codes"])
            assert torch.equal(fa.untile_scales(q["z_scales"], M, C), fa.untile_scales(want["scales"], M, C))
            assert fa.fp4attn_read_status(q["workspace"]) == 0


@pytest.mark.parametrize("C", [8192, 16384])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("branch", [False, True])
def test_clusters_meet_row_after_row(C, layer, branch):
    """Rows shared by two and three CTAs, thousands of meetings on the same barriers, every row known."""
    fa = _fa()
    gen = _gen(C + 1)
    M, period, flags = 7777, 11, fa.LAYER_NORM if layer else 0
    at = torch.arange(M, device="cuda") % period
    x, h, dz, dy = (_rows(period, C, gen, at=0.5) for _ in range(4))
    h = h if branch else None
    one = fa.fp4attn_norm_gate(x, h, eps=EPS, flags=flags)
    few = fa.fp4attn_norm_gate_backward(dz, dy, one["y"], h, eps=EPS, flags=flags)
    ws, nws = fa.new_linear_workspace(0, 0, 32), fa.new_norm_backward_workspace(M, C)
    big = lambda t: None if t is None else t[at].contiguous()
    out = fa.fp4attn_norm_gate(big(x), big(h), eps=EPS, flags=flags, workspace=ws)
    got = fa.fp4attn_norm_gate_backward(big(dz), big(dy), out["y"], big(h), eps=EPS, flags=flags, workspace=nws)
    assert torch.equal(out["y"], big(one["y"])) and torch.equal(out["z"], big(one["z"]))
    assert torch.equal(got["dx"], big(few["dx"])) and (not branch or torch.equal(got["dh"], big(few["dh"])))
    assert fa.fp4attn_read_status(ws) == 0 and fa.fp4attn_read_status(nws) == 0


def test_calls_of_several_threads():
    """The C entry points from threads of their own, on streams and rows of their own: each call is accepted."""
    import threading
    fa = _fa()
    gen = _gen(30)
    shapes = [(3, 4352), (2, 6144), (5, 5000), (4, 4608)]
    wrong, start = [], threading.Barrier(len(shapes))

    def work(M, C, s):
        x, h, z, dx, dh, want = s["t"]
        vec, ws, stream = fa.NormVectors(), s["ws"], s["stream"].cuda_stream
        start.wait()
        for _ in range(1500):
            rc = fa.lib.fp4attn_norm_gate(x.data_ptr(), fa.BF16, C, h.data_ptr(), C, vec, M, C, 1, EPS, 0, None, 0,
                                          z.data_ptr(), C, None, None, None, None, 0, stream)
            rc = rc or fa.lib.fp4attn_norm_gate_backward(z.data_ptr(), C, None, 0, x.data_ptr(), C, fa.BF16, h.data_ptr(), C, vec,
                                                         M, C, 1, EPS, 0, dx.data_ptr(), C, dh.data_ptr(), C, None, None, None,
                                                         None, None, ws.data_ptr(), ws.numel(), stream)
            if rc:
                wrong.append((C, rc))
                return

    state = []
    for M, C in shapes:
        x, h = _rows(M, C, gen), _rows(M, C, gen)
        want = fa.fp4attn_norm_gate(x, h, eps=EPS)["z"]
        state.append(dict(t=(x, h, torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), want),
                          ws=fa.new_norm_backward_workspace(M, C), stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(M, C, s)) for (M, C), s in zip(shapes, state)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong
    for s in state:
        assert torch.equal(s["t"][2], s["t"][5]) and fa.fp4attn_read_status(s["ws"]) == 0
