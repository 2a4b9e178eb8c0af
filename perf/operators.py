"""The operators around the FP4 attention of a transformer block, as they are measured.

A block's linear layers in NVFP4 and the norms between them:

  quantize      rows of bf16 or fp32 -> NVFP4 (E2M1 values, one E4M3 scale per 16
                channels, an fp32 per-tensor scale g) and the values read back
  linear        y = (quantised x) (NVFP4 weight)^T + bias, x and y bf16
  linear_bwd    its straight-through gradients: dx = dy W^, dw = dy^T x^, dbias
  norm          y = x + gate * (post_weight * norm(h)),
                z = norm(y) * pre_weight * (1 + scale) + shift,
                norm(v) = v / sqrt(mean(v^2) + eps) (RMS) or the same of v - mean(v)
                (layer norm); `qkv` cases quantise z and go on into the product that
                reads it
  norm_bwd      the gradients of both norms, of the gate, the modulation and the weights

The quantiser's definition (all four roundings are part of it, since the codes
depend on them): block scale s = E4M3(fl32(fl32(amax / 6) / g)), reciprocal
i = fl32(1 / fl32(g s)) (0 when s is 0), code = E2M1(fl32(v i)), rounding to
nearest even and saturating; the code's value is g * s * e2m1.  A computed
per-tensor scale is g = fl32(amax of the tensor / (6 * 448)), at least 2^-64.

`own` selects the calls a user makes of the library; otherwise the plain form
below runs, in elementary fp32 torch operations.
"""
import math

import torch

own = False

HIDDEN = 48 * 128  # 48 heads of 128 channels, the width of the repository's clip workloads
CLIP5S, CLIP15S, MID = 36864, 109568, 8192  # their sequence lengths

MAX_COST = {"quantize": 4 * HIDDEN * HIDDEN, "linear": CLIP15S * HIDDEN * HIDDEN,
            "linear_bwd": MID * HIDDEN * HIDDEN, "norm": CLIP15S * HIDDEN, "norm_bwd": CLIP5S * HIDDEN}


def listed():
    return [
        # the NVFP4 form of an outlier-heavy activation at 8192 tokens, static scale of 1
        dict(name="quantize activations", op="quantize", M=MID, K=HIDDEN, dtype="bf16", g="one"),
        # the master weights of an MLP layer, requantised after an optimiser step with a scale of their own
        dict(name="quantize weights", op="quantize", M=4 * HIDDEN + 10, K=HIDDEN, dtype="fp32", g="dynamic"),
        # the modulation of one sample's block (shift, scale and gate of two norms): one row in, latency
        dict(name="linear one row", op="linear", M=1, K=HIDDEN, N=6 * HIDDEN, bias=True, g="static"),
        # odd and ragged everywhere: a short prompt, a width whose last 64 channels are half there
        dict(name="linear ragged", op="linear", M=333, K=2080, N=1003, bias=True, g="dynamic"),
        # the projection of the attention's output over the 15-second clip
        dict(name="linear clip15s", op="linear", M=CLIP15S, K=HIDDEN, N=HIDDEN, bias=False, g="dynamic"),
        # a training step's gradients of that layer at 8192 tokens
        dict(name="linear backward", op="linear_bwd", M=MID, K=HIDDEN, N=HIDDEN, bias=True, g="static"),
        # the same of a narrow adapter over a ragged batch
        dict(name="linear backward ragged", op="linear_bwd", M=3001, K=544, N=200, bias=True, g="dynamic"),
        # one token: residual, gate, both norms
        dict(name="norm one row", op="norm", M=1, C=HIDDEN, groups=1, layer=False, residual="bf16", qkv=0),
        # the 15-second clip with the residual stream held in fp32
        dict(name="norm clip15s", op="norm", M=CLIP15S, C=HIDDEN, groups=1, layer=False, residual="fp32", qkv=0),
        # the entry of an attention layer at 5 seconds: the norm hands NVFP4 rows to the Q, K and V projection
        dict(name="norm into qkv", op="norm", M=CLIP5S, C=HIDDEN, groups=1, layer=True, residual="bf16",
             qkv=HIDDEN),
        # a training step's gradients over two clips of different modulation
        dict(name="norm backward", op="norm_bwd", M=CLIP5S, C=HIDDEN, groups=2, layer=False, residual="bf16"),
        # layer norm, odd lengths, many short samples, fp32 residual
        dict(name="norm backward ragged", op="norm_bwd", M=31 * 77, C=1160, groups=31, layer=True, residual="fp32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "linear", "linear", "linear_bwd", "norm", "norm_bwd"])
    top = MAX_COST[op]
    if op in ("norm", "norm_bwd"):
        C = 8 * log(16, 1536)
        qkv = log(16, 4096) if op == "norm" and rng.random() < 0.4 else 0
        if qkv:
            C = (C + 31) // 32 * 32
        groups = rng.choice([1, 1, 2, 3, 5, 17])
        most = min(CLIP15S, top // C, CLIP5S * HIDDEN * HIDDEN // (C * qkv) if qkv else CLIP15S)
        rows = log(1, max(1, most // groups))
        c = dict(op=op, M=rows * groups, C=C, groups=groups, layer=rng.random() < 0.5,
                 residual=rng.choice(["bf16", "fp32"]))
        if op == "norm":
            c["qkv"] = qkv
        return c
    K = 32 * log(2, 384)
    if op == "quantize":
        return dict(op=op, M=log(1, min(CLIP15S, top // K)), K=K, dtype=rng.choice(["bf16", "fp32"]),
                    g=rng.choice(["one", "static", "dynamic"]))
    N = log(8, 4 * HIDDEN)
    M = log(1, max(1, min(CLIP15S, top // (K * N), CLIP15S * HIDDEN // K)))
    return dict(op=op, M=M, K=K, N=N, bias=rng.random() < 0.5, g=rng.choice(["static", "dynamic"]))


# ---------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _activations(M, K, gen, dtype=torch.bfloat16):
    """N(0, 1) with two channels 20 times as large, as a block's activations have them."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x[:, torch.randint(0, K, (2,), generator=gen, device="cuda")] *= 20.0
    return x.to(dtype)


def _round_e2m1(r):
    """Nearest E2M1 value, ties to the even code, saturating at 6."""
    a = r.abs()
    m = 0.5 * (a > 0.25).float()
    for at, step, tie_up in ((0.75, 0.5, True), (1.25, 0.5, False), (1.75, 0.5, True), (2.5, 1.0, False),
                             (3.5, 1.0, True), (5.0, 2.0, False)):
        m += step * ((a >= at) if tie_up else (a > at)).float()
    return torch.copysign(m, r)


def _quantize(v, g):
    """(values / (g s), s): E2M1 values [M, K] and block scales [M, K / 16] of fp32 rows v."""
    M, K = v.shape
    b = v.view(M, K // 16, 16)
    six = torch.full_like(g, 6.0)  # a tensor: a division by a number would multiply by its rounded reciprocal
    s = (b.abs().amax(-1) / six / g).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    gs = g * s
    inv = torch.where(s > 0, 1.0 / gs, torch.zeros_like(gs))
    return _round_e2m1(b * inv[..., None]).view(M, K), s


def _computed_g(v):
    a = v.abs().amax().float().reshape(1)
    return (a / torch.full_like(a, 2688.0)).clamp(min=2.0 ** -64)


def _scale_of(case, x, gen):
    """The per-tensor scale the caller holds: None (1), a calibrated one, or None with `dynamic`."""
    if case["g"] != "static":
        return None
    return _computed_g(x) * (0.5 + torch.rand(1, generator=gen, device="cuda"))


def _pack(values, s):
    """A checkpoint's layout: two codes per byte (the first in the low nibble) and the scales in
    tiles of 128 rows x 4 blocks, 512 bytes each: row r, block b of a tile at 16 (r % 32) + 4 (r / 32) + b."""
    M, K = values.shape
    mag = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], dtype=torch.uint8, device=values.device)
    codes = mag[(values.abs() * 2).long()] | (torch.signbit(values).to(torch.uint8) << 3)
    codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
    R, B = -(-M // 128), -(-K // 64)
    t = torch.zeros(R * 128, B * 4, dtype=torch.uint8, device=values.device)
    t[:M, :K // 16] = s.to(torch.float8_e4m3fn).view(torch.uint8)
    tiles = t.view(R, 4, 32, B, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes.contiguous(), tiles.view(-1)


def _unpack(codes, scales, g, M, K):
    """The values of packed rows, fp32."""
    R, B = -(-M // 128), -(-K // 64)
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).view(M, K // 16, 16)
    s = scales.view(torch.float8_e4m3fn).float().view(R, B, 32, 4, 4).permute(0, 3, 2, 1, 4)
    s = s.reshape(R * 128, B * 4)[:M, :K // 16]
    return (v * (g * s)[..., None]).view(M, K)


def _pack_weight(N, K, gen):
    w = torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)
    g = _computed_g(w)
    codes, scales = _pack(*_quantize(w, g))
    return dict(w_codes=codes, w_scales=scales, gw=g)


def prepare(case, seed):
    gen, op, s = _gen(seed), case["op"], {"case": case}
    if op == "quantize":
        s["x"] = _activations(case["M"], case["K"], gen, torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["gx"] = _scale_of(case, s["x"], gen)
        return s
    if op in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(M, K, gen)
        s["gx"] = _scale_of(case, x, gen)
        s.update(_pack_weight(N, K, gen))
        if op == "linear":
            s["x"] = x
            s["bias"] = torch.randn(N, generator=gen, device="cuda").bfloat16() if case["bias"] else None
        else:  # what the forward kept: the quantised input
            if s["gx"] is None:
                s["gx"] = _computed_g(x)
            s["x_codes"], s["x_scales"] = _pack(*_quantize(x.float(), s["gx"]))
            ld = (N + 7) // 8 * 8  # rows of dy start on 16 bytes
            s["dy"] = torch.randn(M, ld, generator=gen, device="cuda").bfloat16()[:, :N]
        return s
    M, C, G = case["M"], case["C"], case["groups"]
    res = torch.bfloat16 if case["residual"] == "bf16" else torch.float32

    def vec(n, at, spread):
        return (at + spread * torch.randn(n, C, generator=gen, device="cuda")).bfloat16()

    s["h"] = _activations(M, C, gen)
    s["post_weight"], s["pre_weight"] = vec(1, 1.0, 0.1)[0], vec(1, 1.0, 0.1)[0]
    mod = torch.cat([vec(G, 0.0, 0.3) for _ in range(3)], 1)  # a modulation layer's output, taken apart
    s["gate"], s["scale"], s["shift"] = mod.chunk(3, 1)
    stream = 3.0 * torch.randn(M, C, generator=gen, device="cuda") + 0.5
    if op == "norm":
        s["x"] = stream.to(res)
        if case["qkv"]:
            s["gz"] = torch.full((1,), 0.01, device="cuda")
            s.update(_pack_weight(3 * case["qkv"], C, gen))
    else:
        s["y"] = stream.to(res)
        s["dz"] = torch.randn(M, C, generator=gen, device="cuda").bfloat16()
        s["dy"] = torch.randn(M, C, generator=gen, device="cuda").to(res)
    return s


# ------------------------------------------------------------------- run --

EPS = 1e-6


def run(s):
    if own:
        return _own(s)
    op, case = s["case"]["op"], s["case"]
    if op == "quantize":
        x = s["x"].float()
        g = _computed_g(x) if case["g"] == "dynamic" else torch.ones(1, device=x.device) if s["gx"] is None else s["gx"]
        v, sc = _quantize(x, g)
        v = (v.view(case["M"], -1, 16) * (g * sc)[..., None]).view_as(x)
        return {"values": v.bfloat16(), "g": g}
    if op == "linear":
        x = s["x"].float()
        g = _computed_g(x) if case["g"] == "dynamic" else s["gx"]
        y = _product(x, g, s)
        return y.bfloat16() if s["bias"] is None else (y + s["bias"].float()).bfloat16()
    if op == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        dy = s["dy"].float()
        dx = dy @ _unpack(s["w_codes"], s["w_scales"], s["gw"], N, K)
        dw = dy.t() @ _unpack(s["x_codes"], s["x_scales"], s["gx"], M, K)
        out = {"dx": dx.bfloat16(), "dw": dw.bfloat16()}
        return out | {"dbias": dy.sum(0)} if case["bias"] else out
    return _plain_norm(s) if op == "norm" else _plain_norm_bwd(s)


def _product(x, g, s):
    M, K = x.shape
    v, sc = _quantize(x, g)
    v = (v.view(M, -1, 16) * (g * sc)[..., None]).view(M, K)
    return v @ _unpack(s["w_codes"], s["w_scales"], s["gw"], s["w_codes"].shape[0], K).t()


def _norm(v, layer):
    v = v - v.mean(-1, keepdim=True) if layer else v
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)


def _rows(v):
    """The samples' vectors [groups, C], for each of their rows [groups, 1, C]."""
    return v.float()[:, None, :]


def _plain_norm(s):
    case = s["case"]
    M, C, G = case["M"], case["C"], case["groups"]
    h, x = s["h"].float().view(G, M // G, C), s["x"].float().view(G, M // G, C)
    y = x + _rows(s["gate"]) * (s["post_weight"].float() * _norm(h, case["layer"]))
    z = _norm(y, case["layer"]) * s["pre_weight"].float() * (1.0 + _rows(s["scale"])) + _rows(s["shift"])
    y = y.view(M, C).to(s["x"].dtype)
    if not case["qkv"]:
        return {"y": y, "z": z.view(M, C).bfloat16()}
    # the quantiser reads the norm's bf16 output
    return {"y": y, "qkv": _product(z.view(M, C).bfloat16().float(), s["gz"], s).bfloat16()}


def _norm_grad(v, dn, layer):
    """The gradient of _norm at v for the gradient dn of its result, and that result."""
    v = v - v.mean(-1, keepdim=True) if layer else v
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    n = v * r
    d = dn - n * (dn * n).mean(-1, keepdim=True)
    return r * (d - dn.mean(-1, keepdim=True) if layer else d), n


def _plain_norm_bwd(s):
    case, t = s["case"], torch.float32
    M, C, G = case["M"], case["C"], case["groups"]
    h, y, dz, dy = (s[k].to(t).view(G, M // G, C) for k in ("h", "y", "dz", "dy"))
    gate, scale = (s[k].to(t)[:, None, :] for k in ("gate", "scale"))
    post, pre = s["post_weight"].to(t), s["pre_weight"].to(t)
    dv, n = _norm_grad(y, dz * (pre * (1.0 + scale)), case["layer"])
    dzn = (dz * n).sum(1)
    dx = dy + dv
    dh, m = _norm_grad(h, dx * (gate * post), case["layer"])
    dxm = (dx * m).sum(1)
    return {"dx": dx.view(M, C).to(s["y"].dtype), "dh": dh.view(M, C).bfloat16(), "dshift": dz.sum(1),
            "dscale": dzn * pre, "dpre_weight": (dzn * (1.0 + scale[:, 0])).sum(0), "dgate": dxm * post,
            "dpost_weight": (dxm * gate[:, 0]).sum(0)}


def _own(s):
    from nvfp4_precision_b200 import fp4attn as fa

    op, case = s["case"]["op"], s["case"]
    if op == "quantize":
        if "ws" not in s:
            s["ws"] = fa.new_linear_workspace(case["M"], 0, case["K"])
        q = fa.fp4attn_quantize_rows(s["x"], gscale=s["gx"], dynamic_gscale=case["g"] == "dynamic", workspace=s["ws"])
        g = torch.ones(1, device=s["x"].device) if q["gscale"] is None else q["gscale"]
        return {"values": fa.fp4attn_dequant_rows(q["codes"], q["scales"], gscale=q["gscale"]), "g": g}
    if op == "linear":
        if "ws" not in s:
            s["ws"] = fa.new_linear_workspace(case["M"], case["N"], case["K"])
        return fa.fp4attn_linear(s["x"], s["w_codes"], s["w_scales"], w_gscale=s["gw"], x_gscale=s["gx"],
                                 dynamic_gscale=case["g"] == "dynamic", bias=s["bias"], workspace=s["ws"])
    if op == "linear_bwd":
        if "ws" not in s:
            s["ws"] = fa.new_linear_backward_workspace(case["M"], case["N"], case["K"])
        dx, dw, dbias = fa.fp4attn_linear_backward(s["dy"], s["x_codes"], s["x_scales"], s["w_codes"], s["w_scales"],
                                                   x_gscale=s["gx"], w_gscale=s["gw"], want_dbias=case["bias"],
                                                   workspace=s["ws"])
        return {"dx": dx, "dw": dw, "dbias": dbias} if case["bias"] else {"dx": dx, "dw": dw}
    flags = fa.LAYER_NORM if case["layer"] else 0
    vectors = dict(post_weight=s["post_weight"], gate=s["gate"], pre_weight=s["pre_weight"], scale=s["scale"])
    if op == "norm":
        if not case["qkv"]:
            out = fa.fp4attn_norm_gate(s["x"], s["h"], shift=s["shift"], eps=EPS, flags=flags, **vectors)
            return {"y": out["y"], "z": out["z"]}
        if "ws" not in s:
            s["ws"] = fa.new_linear_workspace(case["M"], 3 * case["qkv"], case["C"])
        out = fa.fp4attn_norm_gate(s["x"], s["h"], shift=s["shift"], eps=EPS, flags=flags, quantize=True,
                                   z_gscale=s["gz"], workspace=s["ws"], **vectors)
        qkv = fa.fp4attn_gemm(out["z_codes"], out["z_scales"], s["w_codes"], s["w_scales"], x_gscale=s["gz"],
                              w_gscale=s["gw"], workspace=s["ws"])
        return {"y": out["y"], "qkv": qkv}
    if "ws" not in s:
        s["ws"] = fa.new_norm_backward_workspace(case["M"], case["C"], case["groups"])
    return fa.fp4attn_norm_gate_backward(s["dz"], s["dy"], s["y"], s["h"], eps=EPS, flags=flags, workspace=s["ws"],
                                         **vectors)


# ------------------------------------------------------------------ work --

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["M"] * case["K"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + 2), "flops": 4 * n}
    if op in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        packed = (M + N) * K * 9 / 16
        if op == "linear":
            return {"bytes": 2 * M * (K + N) + N * K * 9 / 16 + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}
        return {"bytes": 2 * M * (N + K) + 2 * N * K + packed + (4 * N if case["bias"] else 0), "flops": 4 * M * N * K}
    M, C, res = case["M"], case["C"], 2 if case["residual"] == "bf16" else 4
    vectors = 2 * C * (2 + 3 * case["groups"])
    if op == "norm":
        N = 3 * case["qkv"]
        out = 2 * M * N + N * C * 9 / 16 if N else 2 * M * C
        return {"bytes": M * C * (2 * res + 2) + vectors + out, "flops": 16 * M * C + 2 * M * N * C}
    return {"bytes": M * C * (3 * res + 6) + vectors + 4 * C * (2 + 3 * case["groups"]), "flops": 30 * M * C}


# ----------------------------------------------------------------- exact --

F64 = torch.float64


def _fl(v):
    """The fp32 rounding of a value in 64 bits, where the quantiser's definition has one."""
    return v.float().double()


def _nearest(a, step_bits):
    """a rounded to a binary float of `step_bits` fraction bits, ties to even (a > 0 normal)."""
    e = torch.floor(torch.log2(a))
    e = e + (torch.exp2(e + 1) <= a).double() - (torch.exp2(e) > a).double()
    step = torch.exp2(e - step_bits)
    return torch.round(a / step) * step


def _exact_quantize(x, g):
    """The quantised values of x in 64 bits."""
    M, K = x.shape
    v = x.double().view(M, K // 16, 16)
    t = _fl(_fl(v.abs().amax(-1) / 6.0) / g)
    small = torch.round(t * 512.0) / 512.0  # below 2^-6 the E4M3 steps are 2^-9
    s = torch.where(t < 2.0 ** -6, small, _nearest(t.clamp(min=2.0 ** -6), 3)).clamp(max=448.0)
    gs = _fl(g * s)
    r = v.mul_(torch.where(s > 0, _fl(1.0 / gs), torch.zeros_like(gs))[..., None])
    r = _fl(r)
    a = r.abs()
    step = 0.5 + 0.5 * (a >= 2.0) + 1.0 * (a >= 4.0)
    q = torch.copysign((torch.round(a / step) * step).clamp(max=6.0), r)
    return (q * (g * s)[..., None]).view(M, K)


def _exact_unpack(codes, scales, g, M, K):
    c = torch.stack((codes & 15, codes >> 4), -1).view(M, K).double()
    sign = 1.0 - 2.0 * (c >= 8)
    m = c - 8.0 * (c >= 8)
    mag = torch.where(m < 2, m / 2, torch.exp2(torch.floor(m / 2) - 1) * (1.0 + 0.5 * torch.remainder(m, 2)))
    r = torch.arange(M, device=codes.device)[:, None]
    b = torch.arange(K // 16, device=codes.device)[None, :]
    tile = (r // 128) * (-(-K // 64)) + b // 4
    byte = scales[tile * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4].double()
    e = torch.floor(byte / 8)
    f = byte - 8 * e
    s = torch.where(e > 0, torch.exp2(e - 7) * (1 + f / 8), f / 512)
    return (sign * mag).view(M, K // 16, 16).mul(g * s[..., None]).view(M, K)


def _exact_norm(v, layer):
    if layer:
        v = v - v.sum(-1, keepdim=True) / v.shape[-1]
    return v / torch.sqrt(v.square().sum(-1, keepdim=True) / v.shape[-1] + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    g = s.get("gx")
    if op in ("quantize", "linear"):
        x = s["x"]
        if case["g"] == "dynamic":
            g = _fl(x.double().abs().amax() / 2688.0).clamp(min=2.0 ** -64).reshape(1)
        g = torch.ones(1, dtype=F64, device="cuda") if g is None else g.double()
        q = _exact_quantize(x, g)
        if op == "quantize":
            return {"values": q, "g": g}
        y = q @ _exact_unpack(s["w_codes"], s["w_scales"], s["gw"].double(), case["N"], case["K"]).t()
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "linear_bwd":
        M, N, K = case["M"], case["N"], case["K"]
        dy = s["dy"].double()
        out = {"dx": dy @ _exact_unpack(s["w_codes"], s["w_scales"], s["gw"].double(), N, K),
               "dw": dy.t() @ _exact_unpack(s["x_codes"], s["x_scales"], s["gx"].double(), M, K)}
        return out | {"dbias": dy.sum(0)} if case["bias"] else out
    M, C, G = case["M"], case["C"], case["groups"]
    if op == "norm":
        h, x = s["h"].double(), s["x"].double()
        each = [s[k].double().repeat_interleave(M // G, 0) if G > 1 else s[k].double() for k in ("gate", "scale", "shift")]
        y = x + each[0] * s["post_weight"].double() * _exact_norm(h, case["layer"])
        z = _exact_norm(y, case["layer"]) * (s["pre_weight"].double() * (1 + each[1])) + each[2]
        if not case["qkv"]:
            return {"y": y, "z": z}
        q = _exact_quantize(z.bfloat16(), s["gz"].double())  # the quantiser reads the norm's bf16 output
        return {"y": y, "qkv": q @ _exact_unpack(s["w_codes"], s["w_scales"], s["gw"].double(), 3 * case["qkv"], C).t()}
    # the gradients of L = sum(dz z) + sum(dy y) by automatic differentiation of the definition in 64 bits
    rows = max(1, M // G)
    out = {"dx": [], "dh": [], "dshift": [], "dscale": [], "dgate": []}
    dpre = torch.zeros(C, dtype=F64, device="cuda")
    dpost = torch.zeros(C, dtype=F64, device="cuda")
    for i in range(G):
        part = slice(i * rows, (i + 1) * rows)
        y0, h = s["y"][part].double(), s["h"][part].double().requires_grad_()
        leaves = [s[k].double().requires_grad_() for k in ("post_weight", "pre_weight")]
        gate, scale, shift = (s[k][i].double().requires_grad_() for k in ("gate", "scale", "shift"))
        branch = gate * leaves[0] * _exact_norm(h, case["layer"])
        # x is what makes y the given one
        x = (y0 - branch.detach()).requires_grad_()
        y = x + branch
        z = _exact_norm(y, case["layer"]) * leaves[1] * (1 + scale) + shift
        grads = torch.autograd.grad([z, y], [x, h, shift, scale, gate, leaves[1], leaves[0]],
                                    [s["dz"][part].double(), s["dy"][part].double()])
        for k, v in zip(out, grads):
            out[k].append(v)
        dpre += grads[5]
        dpost += grads[6]
    return {"dx": torch.cat(out["dx"]), "dh": torch.cat(out["dh"]), "dshift": torch.stack(out["dshift"]),
            "dscale": torch.stack(out["dscale"]), "dgate": torch.stack(out["dgate"]), "dpre_weight": dpre,
            "dpost_weight": dpost}
