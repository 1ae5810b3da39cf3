"""GPU tests of quantising to an MX tensor and back, bit for bit against the
fp64 oracle: both element formats, both plain types, ragged sizes, pitches,
unaligned bases, the ends of the exponent range, infinities and NaN."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import codecs, mx

pytestmark = pytest.mark.gpu


def buffers(rows, cols, fmt, fill=0xA5):
    import torch
    codes = torch.full((rows, cols // 2 if fmt == "E2M1" else cols), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, mx.scale_pitch(cols)), fill, dtype=torch.uint8, device="cuda")
    return codes, scales


def draw(rows, cols, typ, seed, pitch=None, skew=0):
    """A matrix whose rows are `pitch` apart, `skew` elements into its buffer, and its fp64 values."""
    import torch
    pitch = pitch or cols
    g = np.random.default_rng(seed)
    v = g.standard_normal((rows, cols)) * np.exp2(g.integers(-40, 40, (rows, 1)))
    t = torch.from_numpy(v).to(torch.float32).to(torch.bfloat16 if typ == "BF16" else torch.float32)
    buf = torch.zeros(skew + rows * pitch, dtype=t.dtype, device="cuda")
    x = buf[skew:].as_strided((rows, cols), (pitch, 1))
    x.copy_(t)
    return x, t.to(torch.float64).numpy()


def check(x, x64, fmt):
    import torch
    rows, cols = x64.shape
    codes, scales = buffers(rows, cols, fmt)
    dg.dist_gemm_mx_quantize(x, fmt, codes, scales)
    want, want_s = mx.quantize(x64, fmt)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want)
    v = mx.values(want, want_s, fmt, cols)
    for t in (torch.float32, torch.bfloat16):
        y = torch.full((rows, cols + 3), -7.0, dtype=t, device="cuda")
        dg.dist_gemm_mx_dequantize(codes, scales, fmt, y[:, :cols])
        ref = torch.from_numpy(v).to(torch.float32).to(t)
        got = y[:, :cols].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))
        assert (y[:, cols:] == -7.0).all()          # nothing past the row


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (65, 480), (7, 512), (5, 3584), (33, 8160), (2, 8192), (3, 8224),
                                       (2, 16416), (1000, 64)])
def test_against_the_oracle(fmt, typ, rows, cols):
    log("quantize", fmt, typ, rows, cols)
    x, x64 = draw(rows, cols, typ, rows + cols)
    check(x, x64, fmt)


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("pitch,skew", [(136, 0), (131, 0), (128, 1), (160, 8)])
def test_pitches_and_bases(fmt, typ, pitch, skew):
    log("quantize pitch", fmt, typ, pitch, skew)
    x, x64 = draw(9, 128, typ, 7, pitch, skew)
    check(x, x64, fmt)


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
def test_ends_of_the_range(fmt):
    """Zeros of both signs, subnormals, every power of two, every rounding midpoint, the largest floats."""
    import torch
    rows = [np.zeros(32), np.full(32, -0.0), np.full(32, 1e-45), np.full(32, 2.0 ** -126), np.full(32, 2.0 ** -127)]
    rows += [np.full(32, 3.4028234663852886e38), np.linspace(-1, 1, 32) * 3e38]
    rows += [np.where(np.arange(32) == 5, 1.0, 2.0 ** -np.arange(32))]
    rows += [np.where(np.arange(32) == 0, 2.0 ** e, 1.5 * 2.0 ** (e - 3)) for e in range(-126, 128, 7)]
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    rows += [np.concatenate([mid, -mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])]
    e4 = np.concatenate([448 + np.arange(-24, 64, 8.0), 17 + np.arange(0, 14, 2.0)])
    rows += [np.resize(e4, 32), np.resize(2.0 ** -10 * np.arange(0.0, 33, 1.0), 32) + np.where(np.arange(32) == 0, 300, 0)]
    x32 = np.stack(rows).astype(np.float32)
    check(torch.from_numpy(x32).cuda(), x32.astype(np.float64), fmt)


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
def test_infinities_and_nan_poison_their_block_alone(fmt):
    import torch
    x = np.random.default_rng(1).standard_normal((4, 128)).astype(np.float32)
    x[0, 0], x[1, 63], x[2, 100], x[3, 31] = np.inf, -np.inf, np.nan, np.inf
    x[3, 5] = np.nan
    check(torch.from_numpy(x).cuda(), x.astype(np.float64), fmt)


def test_every_e4m3_and_e2m1_code_back():
    import torch
    c = np.arange(256, dtype=np.uint8).reshape(1, 256)
    for fmt, cols in (("E4M3", 256), ("E2M1", 512)):
        s = np.zeros((1, mx.scale_pitch(cols)), dtype=np.uint8)
        s[0, :cols // 32] = np.resize([127, 0, 1, 254, 255, 100, 130], cols // 32)
        y = torch.empty((1, cols), dtype=torch.float32, device="cuda")
        dg.dist_gemm_mx_dequantize(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), fmt, y)
        with np.errstate(over="ignore"):
            ref = mx.values(c, s, fmt, cols).astype(np.float32)
        assert np.array_equal(y.cpu().numpy(), ref, equal_nan=True)


def test_offsets_past_32_bits():
    """The last row starts more than 2^32 elements into the buffer."""
    import torch
    rows, cols, pitch = 3, 64, (1 << 31) + 64
    buf = torch.empty(2 * pitch + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, cols), (pitch, 1))
    v = torch.from_numpy(np.random.default_rng(2).standard_normal((rows, cols))).to(torch.bfloat16)
    x.copy_(v)
    check(x, v.to(torch.float64).numpy(), "E2M1")


def test_refusals_of_tensors():
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    codes, scales = buffers(4, 64, "E2M1")
    for bad in (dict(x=x.half()), dict(x=x.t()), dict(x=x[0]), dict(codes=codes[:, :31].contiguous()),
                dict(scales=scales[:3]), dict(codes=codes.t()), dict(format="E5M2"), dict(scales=scales.float())):
        a = {**dict(x=x, format="E2M1", codes=codes, scales=scales), **bad}
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_mx_quantize(**a)
    with pytest.raises(dg.DistGemmError) as ei:
        y = torch.zeros((4, 48), dtype=torch.bfloat16, device="cuda")
        dg.dist_gemm_mx_quantize(y, "E2M1", torch.zeros((4, 24), dtype=torch.uint8, device="cuda"), scales)
    assert ei.value.status == -2


def test_on_a_stream_of_its_own_and_in_a_graph():
    import torch
    x, x64 = draw(64, 512, "BF16", 3)
    codes, scales = buffers(64, 512, "E4M3")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dg.dist_gemm_mx_quantize(x, "E4M3", codes, scales)
    s.synchronize()
    want, want_s = mx.quantize(x64, "E4M3")
    assert np.array_equal(codes.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.dist_gemm_mx_quantize(x, "E4M3", codes, scales)
    for k in range(3):
        codes.fill_(0)
        scales.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
def test_matrices_past_the_cache_equal_their_parts(fmt, typ):
    """Above the last-level cache's size the accesses go past the caches: the same bytes."""
    import torch
    rows, cols = 20000, 8224
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16 if typ == "BF16" else torch.float32)
    codes, scales = buffers(rows, cols, fmt)
    dg.dist_gemm_mx_quantize(x, fmt, codes, scales)
    y = torch.empty_like(x)
    dg.dist_gemm_mx_dequantize(codes, scales, fmt, y)
    for lo in range(0, rows, 4000):
        c, s = buffers(4000, cols, fmt)
        part = x[lo:lo + 4000]
        dg.dist_gemm_mx_quantize(part, fmt, c, s)
        z = torch.empty_like(part)
        dg.dist_gemm_mx_dequantize(c, s, fmt, z)
        assert torch.equal(c, codes[lo:lo + 4000]) and torch.equal(s, scales[lo:lo + 4000])
        assert torch.equal(z, y[lo:lo + 4000])
