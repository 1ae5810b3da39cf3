"""What is measured of the 8-bit training operators: tensors of E4M3 elements
with a scale per block of 128 (F8 tensors), as quantised for a product and as
the checkpoint of an activation, their products, and the layer norm that feeds
them, with its gradient.

An F8 tensor of rows x cols values is, per row, ``pitch(cols)`` E4M3 codes
(cols rounded up to 128, the codes past cols zero) and ``scale_pitch(cols)``
bytes of power-of-two scales (E8M0: 2^(byte - 127)), one per block of 128
codes, the bytes past the last block zero.  A block's scale is the least power
of two that brings its values within 448.  ``listed`` gives the cases,
``prepare`` their inputs, ``run`` one pass: elementary torch operations in 32
bits, or with ``own`` the calls a user makes of the package.  ``exact`` is the
definition in 64 bits.
"""
import math

import torch

own = False

_EPS = 1e-5
_BLOCK = 128


def pitch(k):
    """Bytes of one row of codes."""
    return -(-k // _BLOCK) * _BLOCK


def scale_pitch(k):
    """Bytes of one row of scales."""
    return -(-(-(-k // _BLOCK)) // 16) * 16


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoding step of four sequences: the residual's addition, the norm and the
        # 8-bit blocks that the next product reads
        dict(name="norm_4x16384", op="norm", rows=4, cols=16384, type="bf16", residual=True, out="F8", kept=False),
        # a training step's norm: 8-bit blocks for the product, the normalised rows kept in 8 bits for the gradient
        dict(name="norm_kept_8192x8192", op="norm", rows=8192, cols=8192, type="bf16", residual=True, out="F8", kept=True),
        # its gradient, from what was kept in 8 bits, with the residual stream's gradient added
        dict(name="norm_grad_kept_8192x8192", op="norm_grad", rows=8192, cols=8192, type="bf16", residual=True, kept=True),
        # the gradient in 32 bits from the kept stream; a width that is no multiple of anything
        dict(name="norm_grad_1021x5123", op="norm_grad", rows=1021, cols=5123, type="f32", residual=False, kept=False),
        # an output's gradient on its way into both products of the backward pass: by rows and transposed
        dict(name="quantize_both_8192x13312", op="quantize", rows=8192, cols=13312, type="bf16", form="both"),
        # a short ragged batch of activations by rows, for the forward product and as the checkpoint
        dict(name="quantize_rows_777x3584", op="quantize", rows=777, cols=3584, type="bf16", form="rows"),
        # an activation's checkpoint, read in the backward pass: transposed for the weight's gradient
        dict(name="transpose_8192x16384", op="transpose", rows=8192, cols=16384),
        dict(name="transpose_777x3584", op="transpose", rows=777, cols=3584),
        # single-token decoding against a layer's 8-bit weights
        dict(name="product_1x13312x16384", op="product", M=1, N=13312, K=16384, weight=True, bias=False),
        # a decoding batch of 200 sequences, the down projection's share
        dict(name="product_200x8192x3584", op="product", M=200, N=8192, K=3584, weight=True, bias=True),
        # a weight's gradient over a ragged batch of 8100 tokens, both operands transposed
        dict(name="product_grad_8192x3584x8100", op="product", M=8192, N=3584, K=8100, weight=False, bias=False),
        # the forward pass of the all-gather GEMM's per-GPU shape
        dict(name="product_16384x13312x16384", op="product", M=16384, N=13312, K=16384, weight=True, bias=False),
    ]


def _log(rng, lo, hi):
    """A size spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "transpose", "product"])
    if op == "product":
        return dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 64, 13312), K=_log(rng, 64, 16384),
                    weight=rng.random() < 0.6, bias=rng.random() < 0.3)
    cols = _log(rng, 64, 16384)
    rows = _log(rng, 1, min(16384, 8192 * (8192 if op in ("norm", "norm_grad") else 13312) // cols))
    if op == "transpose":
        return dict(op=op, rows=rows, cols=cols)
    typ = rng.choice(["bf16", "bf16", "f32"])
    if typ == "f32":
        rows = max(1, rows // 2)
    if op == "quantize":
        return dict(op=op, rows=rows, cols=cols, type=typ, form=rng.choice(["rows", "both", "tiles"]))
    c = dict(op=op, rows=rows, cols=cols, type=typ, residual=rng.random() < 0.6, kept=rng.random() < 0.5)
    if op == "norm":
        c["out"] = rng.choice(["SAME", "E4M3", "F8"])
    return c


# ------------------------------------------------------------------ F8 tensors in elementary operations

def _power(e):
    """2^e in 32 bits for whole e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _to_f8(x, tiles=False):
    """The F8 tensor (codes, scales) of x (rows x cols); tiles: blocks of 128 x 128 share a scale."""
    rows, cols = x.shape
    b = torch.nn.functional.pad(x.float(), (0, pitch(cols) - cols)).view(rows, -1, _BLOCK)
    amax = b.abs().amax(-1)
    if tiles:
        t = torch.nn.functional.pad(amax, (0, 0, 0, pitch(rows) - rows)).view(-1, _BLOCK, amax.shape[1]).amax(1)
        amax = t.repeat_interleave(_BLOCK, 0)[:rows]
    m, e = torch.frexp(amax)  # amax = m 2^e, 448 = 0.875 2^9
    e = torch.where(amax > 0, e.int() - 9 + (m > 0.875).int(), -127).clamp(-127, 127)
    codes = (b * _power(-e)[..., None]).view(rows, -1).to(torch.float8_e4m3fn)
    scales = torch.zeros((rows, scale_pitch(cols)), dtype=torch.uint8, device=x.device)
    scales[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    return codes, scales


def _e8m0(scales):
    return scales.view(torch.float8_e8m0fnu)


def _values(codes, scales, cols=None):
    """The 32-bit values of an F8 tensor (exact), with its padding or its first cols."""
    rows, k = codes.shape
    s = _e8m0(scales[:, :k // _BLOCK].contiguous()).float()
    v = (codes.float().view(rows, -1, _BLOCK) * s[..., None]).view(rows, k)
    return v if cols is None else v[:, :cols]


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _hidden(g, rows, cols):
    """Hidden states: unit normal with a few loud channels."""
    loud = 1 + 15 * (torch.rand(cols, generator=g, device="cuda") < 0.01).float()
    return _normal(g, rows, cols) * loud


def _codes_of(rows, cols):
    """Room for an F8 tensor."""
    return (torch.empty((rows, pitch(cols)), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.empty((rows, scale_pitch(cols)), dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], s["A_scales"] = _to_f8(_hidden(g, M, K))
        s["B"], s["B_scales"] = _to_f8(0.02 * _normal(g, N, K), tiles=True) if case["weight"] else _to_f8(_hidden(g, N, K))
        s["bias"] = _normal(g, N).to(torch.bfloat16) if case["bias"] else None
        s["D"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        if own:
            import communication_tensor_gemm_amd as dg
            s["workspace"] = torch.empty(dg.dist_gemm_f8_product_workspace(M, N, pitch(K)), dtype=torch.uint8, device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    if op == "transpose":
        s["codes"], s["scales"] = _to_f8(_hidden(g, rows, cols))
        s["codes_t"], s["scales_t"] = _codes_of(cols, rows)
        return s
    t = _TYPES[case["type"]]
    if op == "quantize":
        s["x"] = _hidden(g, rows, cols).to(t)
        s["codes"], s["scales"] = _codes_of(rows, cols)
        s["codes_t"], s["scales_t"] = (None, None) if case["form"] == "rows" else _codes_of(cols, rows)
        return s
    # a stream whose channels have means of their own
    s["x"] = (_hidden(g, rows, cols) + 0.5 * _normal(g, cols)).to(t)
    s["weight"] = (1 + 0.1 * _normal(g, cols)).to(t)
    if op == "norm":
        s["bias"] = (0.1 * _normal(g, cols)).to(t)
        s["residual"] = _hidden(g, rows, cols).to(t) if case["residual"] else None
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["scale"] = 0.0625
        s["scales"] = None
        if case["out"] == "SAME":
            s["y"] = torch.empty_like(s["x"])
        elif case["out"] == "E4M3":
            s["y"] = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device="cuda")
        else:
            s["y"], s["scales"] = _codes_of(rows, cols)
        s["kept"], s["kept_scales"] = _codes_of(rows, cols) if case["kept"] else (None, None)
        s["mean"], s["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        return s
    # the gradient gets what the forward pass kept: the rows' statistics, and the stream or its normalised rows in 8 bits
    f = s.pop("x").float()
    s["mean"] = f.mean(-1)
    f = f - s["mean"][:, None]
    s["rstd"] = torch.rsqrt(f.square().mean(-1) + _EPS)
    if case["kept"]:
        s["h"], s["h_scales"] = _to_f8(f * s["rstd"][:, None])
    else:
        s["h"], s["h_scales"] = (f + s["mean"][:, None]).to(t), None
    s["dy"] = (0.01 * _normal(g, rows, cols)).to(t)
    s["dh"] = (0.01 * _normal(g, rows, cols)).to(t) if case["residual"] else None
    s["dx"] = torch.empty((rows, cols), dtype=t, device="cuda")
    s["dweight"], s["dbias"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    if own:
        import communication_tensor_gemm_amd as dg
        s["workspace"] = torch.empty(dg.dist_gemm_layer_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        import communication_tensor_gemm_amd as dg
        return {"norm": _own_norm, "norm_grad": _own_norm_grad, "quantize": _own_quantize, "transpose": _own_transpose,
                "product": _own_product}[op](dg, state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "quantize": _plain_quantize, "transpose": _plain_transpose,
            "product": _plain_product}[op](state)


def _own_norm(dg, s):
    c = s["case"]
    dg.dist_gemm_layer_norm(s["x"], s["weight"], s["bias"], s["y"], eps=_EPS, output=c["out"], residual=s["residual"],
                            h=s["h"], mean=s["mean"], rstd=s["rstd"], scales=s["scales"], scale=s["scale"],
                            kept=s["kept"], kept_scales=s["kept_scales"])
    r = dict(y=s["y"], mean=s["mean"], rstd=s["rstd"])
    if c["residual"]:
        r["h"] = s["h"]
    if c["out"] == "F8":
        r["scales"] = _e8m0(s["scales"])
    if c["kept"]:
        r.update(kept=s["kept"], kept_scales=_e8m0(s["kept_scales"]))
    return r


def _plain_norm(s):
    c = s["case"]
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = h.float()
    mean = f.mean(-1)
    f = f - mean[:, None]
    rstd = torch.rsqrt(f.square().mean(-1) + _EPS)
    n = f * rstd[:, None]
    y = n * s["weight"].float() + s["bias"].float()
    r = dict(mean=mean, rstd=rstd)
    if c["residual"]:
        r["h"] = h
    if c["out"] == "SAME":
        r["y"] = y.to(h.dtype)
    elif c["out"] == "E4M3":
        r["y"] = (y / s["scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    else:
        r["y"], scales = _to_f8(y)
        r["scales"] = _e8m0(scales)
    if c["kept"]:
        r["kept"], scales = _to_f8(n)
        r["kept_scales"] = _e8m0(scales)
    return r


def _own_norm_grad(dg, s):
    kept = s["case"]["kept"]
    dg.dist_gemm_layer_norm_backward(s["dy"], s["h"], None if kept else s["mean"], s["rstd"], s["weight"], s["dx"],
                                     s["dweight"], s["dbias"], s["workspace"], dh=s["dh"], h_scales=s["h_scales"])
    return dict(dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"])


def _plain_norm_grad(s):
    c, dy, rstd = s["case"], s["dy"].float(), s["rstd"][:, None]
    n = _values(s["h"], s["h_scales"], c["cols"]) if c["kept"] else (s["h"].float() - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True)) * rstd
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(dx=dx.to(s["dy"].dtype), dweight=(dy * n).sum(0), dbias=dy.sum(0))


def _own_quantize(dg, s):
    form = s["case"]["form"]
    dg.dist_gemm_f8_quantize(s["x"], s["codes"], s["scales"], s["codes_t"], s["scales_t"],
                             block_rows=128 if form == "tiles" else 1)
    r = dict(codes=s["codes"], scales=_e8m0(s["scales"]))
    if form != "rows":
        r.update(codes_t=s["codes_t"], scales_t=_e8m0(s["scales_t"]))
    return r


def _plain_quantize(s):
    form = s["case"]["form"]
    codes, scales = _to_f8(s["x"], form == "tiles")
    r = dict(codes=codes, scales=_e8m0(scales))
    if form != "rows":
        codes, scales = _to_f8(s["x"].t(), form == "tiles")
        r.update(codes_t=codes, scales_t=_e8m0(scales))
    return r


def _own_transpose(dg, s):
    dg.dist_gemm_f8_transpose(s["codes"], s["scales"], s["codes_t"], s["scales_t"])
    return dict(codes_t=s["codes_t"], scales_t=_e8m0(s["scales_t"]))


def _plain_transpose(s):
    codes, scales = _to_f8(_values(s["codes"], s["scales"], s["case"]["cols"]).t())
    return dict(codes_t=codes, scales_t=_e8m0(scales))


def _own_product(dg, s):
    dg.dist_gemm_f8_product(s["A"], s["A_scales"], s["B"], s["B_scales"], s["D"], bias=s["bias"], workspace=s["workspace"])
    return s["D"]


def _plain_product(s):
    d = _values(s["A"], s["A_scales"]) @ _values(s["B"], s["B_scales"]).t()
    if s["bias"] is not None:
        d = d + s["bias"].float()
    return d.to(torch.bfloat16)


# ------------------------------------------------------------------ the least a pass reads, writes and computes

def work(case):
    op = case["op"]
    f8 = 1 + 1 / 128
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=(M + N) * K * f8 + 2 * M * N, flops=2 * M * N * K)
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if op == "transpose":
        return dict(bytes=2 * n * f8, flops=3 * n)
    es = 2 if case["type"] == "bf16" else 4
    if op == "quantize":
        return dict(bytes=n * (es + f8 * (1 if case["form"] == "rows" else 2)), flops=3 * n)
    if op == "norm":
        out = {"SAME": es, "E4M3": 1, "F8": f8}[case["out"]] + (f8 if case["kept"] else 0)
        return dict(bytes=n * (es * (3 if case["residual"] else 1) + out) + 2 * cols * es + 8 * rows, flops=9 * n)
    kept = f8 if case["kept"] else es
    return dict(bytes=n * (es * (3 if case["residual"] else 2) + kept) + cols * (es + 8) + 8 * rows, flops=13 * n)


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_values(codes, scales):
    """The values of an F8 tensor from its bit fields, padding included."""
    bits = codes.view(torch.uint8).int()
    exponent, fraction = (bits & 127) >> 3, (bits & 7).double() / 8
    v = torch.where(exponent > 0, (1 + fraction) * torch.exp2((exponent - 7).double()), fraction * 2.0 ** -6)
    v = torch.where(bits >= 128, -v, v)
    return v * torch.exp2(scales[:, :codes.shape[1] // _BLOCK].double() - 127).repeat_interleave(_BLOCK, -1)


def _exact_f8(x, tiles=False):
    """(x over its block's scale, padded; scales, padded): nothing rounded yet."""
    rows, cols = x.shape
    blocks = pitch(cols) // _BLOCK
    v = torch.zeros((rows, pitch(cols)), dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    most = v.view(rows, blocks, _BLOCK).abs().amax(-1)
    if tiles:
        for r in range(0, rows, _BLOCK):
            most[r:r + _BLOCK] = most[r:r + _BLOCK].amax(0, keepdim=True)
    # the least power of two with most <= 448 times it
    s = torch.exp2(torch.floor(torch.log2(most.clamp(min=2.0 ** -1000) / 448)))
    s = torch.where(most > 448 * s, 2 * s, s)
    s = torch.where(most <= 224 * s, s / 2, s).clamp(min=2.0 ** -127)
    scales = torch.full((rows, scale_pitch(cols)), 2.0 ** -127, dtype=torch.float64, device=x.device)
    scales[:, :blocks] = s
    return v / s.repeat_interleave(_BLOCK, -1), scales


def _exact_round(v):
    """Nearest E4M3 value, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        d = _exact_values(s["A"], s["A_scales"]) @ _exact_values(s["B"], s["B_scales"]).t()
        return d if s["bias"] is None else d + s["bias"].double()
    if op == "transpose":
        x = _exact_values(s["codes"], s["scales"])[:, :case["cols"]]
        v, scales = _exact_f8(x.t())
        return dict(codes_t=_exact_round(v), scales_t=scales)
    if op == "quantize":
        tiles = case["form"] == "tiles"
        v, scales = _exact_f8(s["x"].double(), tiles)
        r = dict(codes=_exact_round(v), scales=scales)
        if case["form"] != "rows":
            v, scales = _exact_f8(s["x"].double().t(), tiles)
            r.update(codes_t=_exact_round(v), scales_t=scales)
        return r
    cols = case["cols"]
    if op == "norm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        # the norm is of the stream as it is kept, in its own type
        f = h if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype).double()
        mean = f.sum(-1) / cols
        var = ((f - mean[:, None]) ** 2).sum(-1) / cols
        n = (f - mean[:, None]) / torch.sqrt(var + _EPS)[:, None]
        y = n * s["weight"].double() + s["bias"].double()
        r = dict(mean=mean, rstd=1 / torch.sqrt(var + _EPS))
        if case["residual"]:
            r["h"] = h
        # 8-bit outputs: the values before their rounding; the blocks' exponents are no computed numbers
        if case["out"] == "SAME":
            r["y"] = y
        elif case["out"] == "E4M3":
            r["y"] = (y / s["scale"]).clamp(-448, 448)
        else:
            r.update(y=_exact_f8(y)[0], scales=None)
        if case["kept"]:
            r.update(kept=_exact_f8(n)[0], kept_scales=None)
        return r
    dy, r = s["dy"].double(), s["rstd"].double()[:, None]
    if case["kept"]:
        n = _exact_values(s["h"], s["h_scales"])[:, :cols]
    else:
        n = (s["h"].double() - s["mean"].double()[:, None]) * r
    g = dy * s["weight"].double()
    dx = r * (g - g.sum(-1, keepdim=True) / cols - n * ((g * n).sum(-1, keepdim=True) / cols))
    return dict(dx=dx if s["dh"] is None else dx + s["dh"].double(), dweight=(dy * n).sum(0), dbias=dy.sum(0))
