"""GPU tests of F8 tensors (quantised by rows, transposed, in square blocks;
transposed from one another; back to values), bit for bit against the fp64
oracle: both plain types, ragged sizes, pitches, unaligned bases, the ends of
the exponent range, infinities and NaN."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log
from oracle import f8

pytestmark = pytest.mark.gpu


def torch_type(typ):
    import torch
    return torch.bfloat16 if typ == "BF16" else torch.float32


def room(rows, cols, fill=0xA5):
    import torch
    return (torch.full((rows, f8.pitch(cols)), fill, dtype=torch.uint8, device="cuda"),
            torch.full((rows, f8.scale_pitch(cols)), fill, dtype=torch.uint8, device="cuda"))


def draw(rows, cols, typ, seed, pitch=None, skew=0):
    """A matrix whose rows are `pitch` apart, `skew` elements into its buffer, and its fp64 values."""
    import torch
    pitch = pitch or cols
    g = np.random.default_rng(seed)
    v = g.standard_normal((rows, cols)) * np.exp2(g.integers(-20, 20, (rows, 1))) * np.exp2(g.integers(-20, 20, (1, cols)))
    t = torch.from_numpy(v).to(torch.float32).to(torch_type(typ))
    buf = torch.zeros(skew + rows * pitch, dtype=t.dtype, device="cuda")
    x = buf[skew:].as_strided((rows, cols), (pitch, 1))
    x.copy_(t)
    return x, t.to(torch.float64).numpy()


def same(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def check(x, x64):
    """Every form of the quantiser, and every form's values back."""
    import torch
    rows, cols = x64.shape
    for block in (1, 128):
        want, want_t = f8.quantize(x64, block == 128), f8.quantize(x64.T, block == 128)
        a, b = room(rows, cols), room(cols, rows)
        dg.dist_gemm_f8_quantize(x, *a, *b, block_rows=block)
        same(a, want)
        same(b, want_t)
        a, b = room(rows, cols), room(cols, rows)
        dg.dist_gemm_f8_quantize(x, *a, block_rows=block)
        same(a, want)
        dg.dist_gemm_f8_quantize(x, codes_t=b[0], scales_t=b[1], block_rows=block)
        same(b, want_t)
    check_back(*f8.quantize(x64), cols)


def check_back(codes, scales, cols):
    """The values of a tensor and its transpose."""
    import torch
    rows = codes.shape[0]
    up = [torch.from_numpy(t).cuda() for t in (codes, scales)]
    v = f8.values(codes, scales, cols)
    with np.errstate(over="ignore"):
        v32 = v.astype(np.float32)
    for t in (torch.float32, torch.bfloat16):
        y = torch.full((rows, cols + 3), -7.0, dtype=t, device="cuda")
        dg.dist_gemm_f8_dequantize(*up, y[:, :cols])
        ref = torch.from_numpy(v32).to(t)
        got = y[:, :cols].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(ref))
        assert (y[:, cols:] == -7.0).all()          # nothing past the row
    b = room(cols, rows)
    dg.dist_gemm_f8_transpose(*up, *b)
    same(b, f8.quantize(v32.T))


SIZES = [(1, 1), (1, 128), (3, 96), (65, 480), (7, 513), (130, 127), (128, 128), (129, 257), (300, 1000), (5, 3584), (2, 8224),
         (1000, 64), (2100, 130), (127, 2049)]


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_against_the_oracle(typ, rows, cols):
    log("f8 quantize", typ, rows, cols)
    check(*draw(rows, cols, typ, rows + cols))


@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("pitch,skew", [(208, 0), (203, 0), (200, 1), (216, 8)])
def test_pitches_and_bases(typ, pitch, skew):
    log("f8 quantize pitch", typ, pitch, skew)
    check(*draw(139, 200, typ, 7, pitch, skew))


def test_ends_of_the_range():
    """Zeros of both signs, subnormals, every power of two, every rounding midpoint, scale borders, the largest floats."""
    import torch
    n = 128
    rows = [np.zeros(n), np.full(n, -0.0), np.full(n, 1e-45), np.full(n, 2.0 ** -126), np.full(n, 2.0 ** -127)]
    rows += [np.full(n, 3.4028234663852886e38), np.linspace(-1, 1, n) * 3e38]
    rows += [np.where(np.arange(n) == 5, 1.0, 2.0 ** -(np.arange(n) / 4.0))]
    rows += [np.where(np.arange(n) == 0, 2.0 ** e, 1.5 * 2.0 ** (e - 3)) for e in range(-126, 128, 7)]
    rows += [np.where(np.arange(n) == 0, 1.75 * 2.0 ** e, 2.0 ** (e - 4)) for e in range(-126, 127, 11)]
    rows += [np.where(np.arange(n) == 0, np.nextafter(np.float32(1.75 * 2.0 ** e), np.float32(np.inf)), 2.0 ** (e - 4))
             for e in range(-126, 127, 11)]
    e4 = np.concatenate([448 - np.arange(0, 192, 8.0), 17 + np.arange(0, 14, 2.0)])
    rows += [np.resize(e4, n), np.resize(2.0 ** -10 * np.arange(0.0, 33, 1.0), n) + np.where(np.arange(n) == 0, 300, 0)]
    x32 = np.stack(rows).astype(np.float32)
    check(torch.from_numpy(x32).cuda(), x32.astype(np.float64))
    xb = torch.from_numpy(x32).to(torch.bfloat16)
    check(xb.cuda(), xb.to(torch.float64).numpy())


def test_every_bf16_value_in_a_block_of_its_own_scale():
    """All 65536 patterns, each the largest of its block."""
    import torch
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.zeros((65536, 128), dtype=torch.bfloat16)
    x[:, 17] = bits
    x[:, 18] = bits / 3
    want, want_s = f8.quantize(x.to(torch.float64).numpy())
    codes, scales = room(65536, 128)
    dg.dist_gemm_f8_quantize(x.cuda(), codes, scales)
    same((codes, scales), (want, want_s))


@pytest.mark.parametrize("typ", ["BF16", "F32"])
def test_infinities_and_nan_poison_their_block_alone(typ):
    import torch
    x = np.random.default_rng(1).standard_normal((260, 390)).astype(np.float32)
    x[0, 0], x[1, 163], x[2, 300], x[200, 131], x[259, 389] = np.inf, -np.inf, np.nan, np.inf, np.nan
    t = torch.from_numpy(x).to(torch_type(typ))
    check(t.cuda(), t.to(torch.float64).numpy())


def test_every_code_and_scale_back_and_transposed():
    """All codes at scales over the whole range: values past fp32's range count as infinite, those below it round."""
    import torch
    codes = np.tile(np.arange(256, dtype=np.uint8), (140, 1))
    scales = np.zeros((140, 16), dtype=np.uint8)
    scales[:, 0] = np.resize([127, 0, 1, 2, 246, 247, 255, 100, 130], 140)
    scales[:, 1] = np.resize([120, 3, 240, 12, 127], 140)
    check_back(codes, scales, 256)
    codes[:, 0x7F] = codes[:, 0xFF] = 0             # no NaN element: the other blocks' values count
    scales[scales == 255] = 9
    check_back(codes, scales, 256)


def test_a_checkpoint_read_transposed_is_its_values():
    """Powers of two as scales: what stays in E4M3's normal range of the new block is moved exactly."""
    import torch
    x = torch.randn(300, 500, generator=torch.Generator().manual_seed(3)).cuda()
    a, b = room(300, 500), room(500, 300)
    dg.dist_gemm_f8_quantize(x, *a)
    dg.dist_gemm_f8_transpose(*a, *b)
    y, z = torch.empty_like(x), torch.empty((500, 300), device="cuda")
    dg.dist_gemm_f8_dequantize(*a, y)
    dg.dist_gemm_f8_dequantize(*b, z)
    step = torch.exp2(b[1][:, :3].float() - 127).repeat_interleave(128, 1)[:, :300].t()
    assert bool(((y == z.t()) | ((y.abs() < step * 2.0 ** -6) & ((y - z.t()).abs() <= step * 2.0 ** -10))).all())
    assert (y == z.t()).float().mean() > 0.9


def test_offsets_past_32_bits():
    """The last row starts more than 2^32 elements into the buffer."""
    import torch
    rows, cols, pitch = 3, 130, (1 << 31) + 64
    buf = torch.empty(2 * pitch + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, cols), (pitch, 1))
    v = torch.from_numpy(np.random.default_rng(2).standard_normal((rows, cols))).to(torch.bfloat16)
    x.copy_(v)
    check(x, v.to(torch.float64).numpy())


def test_tensors_past_4_gib():
    """Codes whose last rows lie past 2^32 bytes, by rows, transposed and back."""
    import torch
    rows, cols = 34000, 130000
    codes = torch.randint(0, 120, (rows, f8.pitch(cols)), dtype=torch.uint8, device="cuda")
    codes[:, cols:] = 0
    scales = torch.full((rows, f8.scale_pitch(cols)), 127, dtype=torch.uint8, device="cuda")
    b = room(cols, rows)
    dg.dist_gemm_f8_transpose(codes, scales, *b)
    for r0, c0 in ((0, 0), (33900, 129900), (33000, 5), (7, 129990)):
        r1, c1 = min(rows, r0 + 128), min(cols, c0 + 128)
        v = codes[r0:r1, c0:c1].contiguous().view(torch.float8_e4m3fn).float()
        s = torch.exp2(b[1][c0:c1].float() - 127)[:, torch.arange(r0, r1, device="cuda") // 128]
        w = b[0][c0:c1, r0:r1].contiguous().view(torch.float8_e4m3fn).float() * s
        assert bool(((w - v.t()).abs() <= torch.maximum(v.t() * 0, s * 2.0 ** -10)).all())
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    dg.dist_gemm_f8_dequantize(codes, scales, y)
    assert torch.equal(y[-1].float(), codes[-1, :cols].view(torch.float8_e4m3fn).float())
    del codes, scales
    c, s = room(rows, cols, 7)
    dg.dist_gemm_f8_quantize(y, c, s)
    z = torch.empty((50, cols), dtype=torch.bfloat16, device="cuda")
    dg.dist_gemm_f8_dequantize(c[-50:], s[-50:], z)
    assert bool(((z.float() - y[-50:].float()).abs() <= 2.0 ** -10).all())


def test_refusals_of_tensors():
    import torch
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    (c, s), (ct, st) = room(4, 64), room(64, 4)
    good = dict(x=x, codes=c, scales=s, codes_t=ct, scales_t=st)
    for bad in (dict(x=x.half()), dict(x=x.t()), dict(x=x[0]), dict(codes=c[:, :64].contiguous()), dict(scales=s[:3]),
                dict(codes_t=c), dict(scales_t=None), dict(codes=None), dict(block_rows=64), dict(scales=s.float()),
                dict(x=x.cpu()), dict(codes=x)):
        with pytest.raises((ValueError, dg.DistGemmError)):
            dg.dist_gemm_f8_quantize(**{**good, **bad})
    with pytest.raises(dg.DistGemmError):
        dg.dist_gemm_f8_quantize(x)
    for bad in (dict(codes_t=ct[:63]), dict(codes=c[:3]), dict(scales_t=st.cpu()), dict(codes=c[0])):
        with pytest.raises(ValueError):
            dg.dist_gemm_f8_transpose(**{**dict(codes=c, scales=s, codes_t=ct, scales_t=st), **bad})
    with pytest.raises(ValueError):
        dg.dist_gemm_f8_dequantize(c, s, torch.empty((4, 200), device="cuda"))


def test_on_a_stream_of_its_own_and_in_a_graph():
    import torch
    x, x64 = draw(300, 500, "BF16", 3)
    want, want_t = f8.quantize(x64), f8.quantize(x64.T)
    a, b, c = room(300, 500), room(500, 300), room(500, 300)
    moved = f8.quantize(f8.values(*want, 500).T)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dg.dist_gemm_f8_quantize(x, *a, *b)
        dg.dist_gemm_f8_transpose(*a, *c)
    s.synchronize()
    same(a, want), same(b, want_t), same(c, moved)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.dist_gemm_f8_quantize(x, *a, *b)
        dg.dist_gemm_f8_transpose(*a, *c)
    for k in range(3):
        for t in (*a, *b, *c):
            t.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        same(a, want), same(b, want_t), same(c, moved)


@pytest.mark.parametrize("typ", ["BF16", "F32"])
def test_matrices_past_the_cache_equal_their_parts(typ):
    """Above the last-level cache's size the accesses go past the caches: the same bytes."""
    import torch
    rows, cols = 20480, 8232
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch_type(typ))

    def run(x):
        n = x.size(0)
        a, b, c, r = room(n, cols), room(cols, n), room(cols, n), room(n, cols)
        dg.dist_gemm_f8_quantize(x, *a, *b)
        dg.dist_gemm_f8_quantize(x, *r)
        assert torch.equal(a[0], r[0]) and torch.equal(a[1], r[1])
        dg.dist_gemm_f8_transpose(*a, *c)
        y = torch.empty_like(x)
        dg.dist_gemm_f8_dequantize(*a, y)
        return a, b, c, y

    a, b, c, y = run(x)
    for lo in range(0, rows, 4096):
        pa, pb, pc, py = run(x[lo:lo + 4096])
        assert all(torch.equal(p, w[lo:lo + 4096]) for p, w in zip(pa, a)) and torch.equal(py, y[lo:lo + 4096])
        for p, w in ((pb, b), (pc, c)):
            assert torch.equal(p[0], w[0][:, lo:lo + 4096]) and torch.equal(p[1][:, :32], w[1][:, lo // 128:lo // 128 + 32])
