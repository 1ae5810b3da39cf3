"""GPU tests of quantising bf16 at the ends of its range, bit for bit against the
fp64 oracle: bf16 takes instructions of its own, with the block's scale as an
operand."""
import numpy as np
import pytest

from gpu_helpers import log
from test_gpu_11_mx_quantize import check

pytestmark = pytest.mark.gpu


def bf16(bits):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(bits).astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    return t.cuda(), t.to(torch.float64).numpy()


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
def test_every_bf16_value(fmt):
    """Each of the 65536 values under every block maximum that its exponent is near: the value alone, under a
    maximum of up to 14 binary orders above it, and in a block of its neighbours."""
    log("every bf16", fmt)
    every = np.arange(65536, dtype=np.int64)
    check(*bf16(np.repeat(every, 32).reshape(4096, 512)), fmt)        # alone
    check(*bf16(every.reshape(128, 512)), fmt)                        # with its neighbours
    for up in (1, 2, 3, 5, 7, 9, 11, 14):
        b = np.repeat(every[:, None], 32, 1)
        # one element of the block `up` orders above, where there is such a number
        top = np.minimum((every & 0x7F80) + (up << 7), 0x7F00)
        b[:, 7] = top | np.where(every & 1, 0x8000, 0) | (every & 0x40)
        check(*bf16(b.reshape(4096, 512)), fmt)


@pytest.mark.parametrize("fmt", ["E2M1", "E4M3"])
def test_random_bits(fmt):
    log("random bf16 bits", fmt)
    g = np.random.default_rng(4)
    b = g.integers(0, 65536, (2000, 512))
    b = np.where((b & 0x7F80) == 0x7F80, b & 0x3FFF, b)               # finite ones
    check(*bf16(b), fmt)
    small = (b & 0x807F) | g.integers(0, 12, b.shape) << 7             # down to the smallest, where the scale is 2^-127
    check(*bf16(small), fmt)
    check(*bf16((b & 0x807F) | g.integers(242, 255, b.shape) << 7), fmt)
    check(*bf16(g.integers(0, 65536, (2000, 512))), fmt)              # infinities and NaN among them
