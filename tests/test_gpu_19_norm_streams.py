"""GPU tests of the RMS norm, its gradient and dequantising on a stream of their
own and captured: every replay against the eager result, bit for bit, with
eager work and synchronisation between the replays."""
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import mx

pytestmark = pytest.mark.gpu


def twice_and_captured(call, outs):
    """`call` writes `outs` (its inputs stay as they are): eager, on another stream, replayed."""
    import torch
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]

    def clear():
        for t in outs:
            t.view(torch.uint8).fill_(0x5A)

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t, w in zip(outs, want))

    clear()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        clear()
        g.replay()
        assert same()
        clear()
        call()
        assert same()


SIZES = [(4, 16384), (37, 96), (300, 5120), (2100, 1024)]


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("out", ["SAME", "E4M3", "MX_E2M1", "MX_E4M3"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm(rows, cols, out, typ):
    import torch
    log("norm captured", rows, cols, out, typ)
    t = torch.bfloat16 if typ == "BF16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(2))
    w = torch.randn(cols, generator=g, device="cuda").to(t)
    y = torch.empty((rows, cols // 2 if out == "MX_E2M1" else cols), dtype=t if out == "SAME" else torch.uint8, device="cuda")
    h, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    scales = torch.empty((rows, mx.scale_pitch(cols)), dtype=torch.uint8, device="cuda") if out.startswith("MX") else None
    twice_and_captured(lambda: dg.dist_gemm_rms_norm(x, w, y, output=out, residual=r, h=h, rstd=rstd, scales=scales, scale=0.25),
                       [v for v in (y, h, rstd, scales) if v is not None])


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", SIZES + [(0, 96), (5, 20000)])
def test_gradient(rows, cols, typ):
    import torch
    log("norm gradient captured", rows, cols, typ)
    t = torch.bfloat16 if typ == "BF16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(2)
    dy, h, dh = (torch.randn(rows, cols, generator=g, device="cuda").to(t) for _ in range(3))
    w, rstd = torch.randn(cols, generator=g, device="cuda").to(t), torch.rand(rows, generator=g, device="cuda")
    dx, dw = torch.empty_like(h), torch.empty(cols, device="cuda")
    ws = torch.empty(dg.dist_gemm_rms_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    twice_and_captured(lambda: dg.dist_gemm_rms_norm_backward(dy, h, rstd, w, dx, dw, ws, dh=dh),
                       [dx, dw] if rows else [dw])


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_dequantize(rows, cols, fmt, typ):
    import torch
    log("dequantize captured", rows, cols, fmt, typ)
    t = torch.bfloat16 if typ == "BF16" else torch.float32
    x = torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    codes = torch.empty((rows, cols if fmt == "E4M3" else cols // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, mx.scale_pitch(cols)), dtype=torch.uint8, device="cuda")
    dg.dist_gemm_mx_quantize(x, fmt, codes, scales)
    y = torch.empty((rows, cols), dtype=t, device="cuda")
    twice_and_captured(lambda: dg.dist_gemm_mx_dequantize(codes, scales, fmt, y), [y])
