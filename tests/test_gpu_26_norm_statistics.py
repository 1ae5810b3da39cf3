"""GPU tests of the statistics that the norms return for their gradients, with
every row accounted for: where the formula gives a number, that number, and
where it gives a NaN or an infinity, the same.  Every layout of rows on lanes
and waves, aligned and not.

Tolerances as in the norms' own tests (u = 2^-24, N = 64 u, A = mean|h| rstd):
the mean N mean|h|, layer norm's rstd N (1 + 2 A) relative, RMS norm's 48 u
relative.  A row whose sum of squares is past fp32's range has rstd 0 and is the
bias alone: exact."""
import numpy as np
import pytest

import communication_tensor_gemm_amd as dg
from gpu_helpers import log, within
from oracle import codecs, f8, mx

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
N = 64 * U
EPS = 1e-5

# rows of 16 and 32 lanes, of one and several waves, of one, two and four pieces to a lane
SIZES = [(9, 8), (9, 100), (9, 128), (9, 130), (9, 256), (9, 264), (7, 500), (7, 512), (7, 1000), (7, 2048), (7, 5123), (7, 8192),
         (7, 16384), (7, 20000), (7, 32768), (2051, 520), (2051, 1025), (2051, 4104), (2049, 20000)]


def draw(rows, cols, typ, skew):
    import torch
    t = torch.bfloat16 if typ == "BF16" else torch.float32
    v = np.random.default_rng(rows + cols).standard_normal((rows, cols)).astype(np.float32) + 0.5
    v[1, cols // 3] = np.nan
    v[2, cols - 1] = np.inf
    v[3] = np.where(np.arange(cols) % 2, -1e20, 1e20)
    v[4] = 0.0
    buf = torch.zeros(skew + rows * cols, dtype=t, device="cuda")
    x = buf[skew:].view(rows, cols)
    x.copy_(torch.from_numpy(v))
    return x, x.to(torch.float64).cpu().numpy()


def f64(t):
    import torch
    return t.to(torch.float64).cpu().numpy()


@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_layer_norm(rows, cols, typ, skew):
    import torch
    log("layer norm's statistics", rows, cols, typ, skew)
    x, x64 = draw(rows, cols, typ, skew)
    w, b = (torch.from_numpy(np.random.default_rng(s).standard_normal(cols).astype(np.float32)).to(x.dtype).cuda() for s in (1, 2))
    with np.errstate(invalid="ignore"):
        _, _, mean, rstd = f8.layer_norm(x64, np.ones(cols), None, EPS)
    size = np.abs(x64).mean(-1)
    rstd[3] = 0.0
    room = lambda n: (torch.full((rows, f8.pitch(cols)), n, dtype=torch.uint8, device="cuda"),  # noqa: E731
                      torch.full((rows, f8.scale_pitch(cols)), n, dtype=torch.uint8, device="cuda"))
    for out in ("SAME", "E4M3", "F8"):
        m, s = torch.full((rows,), 7.0, device="cuda"), torch.full((rows,), 7.0, device="cuda")
        k, ks = room(0xA5)
        y, scales = room(0xA5) if out == "F8" else (torch.empty((rows, cols), dtype=x.dtype if out == "SAME" else torch.uint8, device="cuda"), None)
        dg.dist_gemm_layer_norm(x, w, b, y, eps=EPS, output=out, mean=m, rstd=s, scales=scales, kept=k, kept_scales=ks)
        assert within(f64(m), mean, N * size)
        assert within(f64(s), rstd, N * (1 + 2 * size * rstd) * rstd)
        if out == "F8":
            bad = (scales.cpu().numpy()[:, :-(-cols // 128)] == 255)
            assert bad[1:3].all() and not bad[0].any() and not bad[3:].any()
        else:
            got = f64(y) if out == "SAME" else codecs.e4m3_to_f64(y.cpu().numpy())
            assert np.isnan(got[1:3]).all() and np.isfinite(got[0]).all() and np.isfinite(got[3:]).all()
            if out == "SAME":
                assert np.array_equal(got[3:5], np.tile(f64(b), (2, 1)))
        bad = (ks.cpu().numpy()[:, :-(-cols // 128)] == 255)
        assert bad[1:3].all() and not bad[0].any() and not bad[3:].any() and not (k[3:5] & 127).any()  # (a zero has a sign)


@pytest.mark.parametrize("skew", [0, 1])
@pytest.mark.parametrize("typ", ["BF16", "F32"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rms_norm(rows, cols, typ, skew):
    import torch
    log("RMS norm's statistics", rows, cols, typ, skew)
    x, x64 = draw(rows, cols, typ, skew)
    with np.errstate(invalid="ignore"):
        _, rstd = mx.rms_norm(x64, np.ones(cols), EPS)
    rstd[3] = 0.0
    y, s = torch.empty_like(x), torch.full((rows,), 7.0, device="cuda")
    dg.dist_gemm_rms_norm(x, torch.ones(cols, dtype=x.dtype, device="cuda"), y, eps=EPS, rstd=s)
    assert within(f64(s), rstd, 48 * U * rstd)
    assert torch.isnan(y[1]).any() and not y[3:5].any() and torch.isfinite(y[5:]).all()
