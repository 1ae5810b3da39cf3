"""One training step of a linear layer behind a layer norm, at 8 bits.

  h = x + residual, a = layer_norm(h)     dist_gemm_layer_norm: a as an F8 tensor, and the
                                          normalised rows kept as another (8-bit checkpoints)
  y = a W^T + b                           dist_gemm_f8_product, W in 128 x 128 blocks

  dy by rows and transposed               dist_gemm_f8_quantize, one pass
  da = dy W                               dist_gemm_f8_product with W's transposed tensor
  a^T                                     dist_gemm_f8_transpose of the checkpoint
  dW = dy^T a                             dist_gemm_f8_product of the two transposed tensors
  dx, dweight, dbias of the norm          dist_gemm_layer_norm_backward from what it kept

Between forward and backward only 8-bit tensors and one fp32 number per row
are kept.  Run it on an MI355X:  python examples/f8_linear.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import communication_tensor_gemm_amd as dg  # noqa: E402


def f8_empty(rows, cols):
    """Room for an F8 tensor of rows x cols values."""
    return (torch.empty((rows, dg.dist_gemm_f8_pitch(cols)), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.empty((rows, dg.dist_gemm_f8_scale_pitch(cols)), dtype=torch.uint8, device="cuda"))


def product_workspace(M, N, K):
    return torch.empty(dg.dist_gemm_f8_product_workspace(M, N, K), dtype=torch.uint8, device="cuda")


class NormLinear:
    """A layer norm and a linear layer width -> out over `tokens` rows, in bf16."""

    def __init__(self, tokens, width, out, eps=1e-5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.tokens, self.width, self.out, self.eps = tokens, width, out, eps
        self.norm_weight = (1 + 0.1 * torch.randn(width, generator=g, device="cuda")).bfloat16()
        self.norm_bias = (0.1 * torch.randn(width, generator=g, device="cuda")).bfloat16()
        self.weight = (torch.randn(out, width, generator=g, device="cuda") * width ** -0.5).bfloat16()
        self.bias = (0.1 * torch.randn(out, generator=g, device="cuda")).bfloat16()
        # the weight and its transpose as F8 tensors: once per update of the weight
        self.w8, self.w8_t = f8_empty(out, width), f8_empty(width, out)
        self.quantize_weight()
        # what the step keeps and what it returns
        self.h, self.rstd, self.y = bf16(tokens, width), f32(tokens), bf16(tokens, out)
        self.act, self.kept, self.act_t = f8_empty(tokens, width), f8_empty(tokens, width), f8_empty(width, tokens)
        self.dy8, self.dy8_t = f8_empty(tokens, out), f8_empty(out, tokens)
        self.dact, self.dx, self.dweight = bf16(tokens, width), bf16(tokens, width), bf16(out, width)
        self.dnorm_weight, self.dnorm_bias = f32(width), f32(width)
        pitch = dg.dist_gemm_f8_pitch
        self.ws_y = product_workspace(tokens, out, pitch(width))
        self.ws_a = product_workspace(tokens, width, pitch(out))
        self.ws_w = product_workspace(out, width, pitch(tokens))
        self.ws_n = torch.empty(dg.dist_gemm_layer_norm_workspace(tokens, width), dtype=torch.uint8, device="cuda")

    def quantize_weight(self):
        dg.dist_gemm_f8_quantize(self.weight, *self.w8, *self.w8_t, block_rows=128)

    def forward(self, x, residual):
        dg.dist_gemm_layer_norm(x, self.norm_weight, self.norm_bias, self.act[0], eps=self.eps, output="F8", residual=residual,
                                h=self.h, rstd=self.rstd, scales=self.act[1], kept=self.kept[0], kept_scales=self.kept[1])
        dg.dist_gemm_f8_product(*self.act, *self.w8, self.y, bias=self.bias, workspace=self.ws_y)
        return self.y

    def backward(self, dy, dh):
        """The gradient of x (and of the residual) from y's and, along the residual stream, h's."""
        dg.dist_gemm_f8_quantize(dy, *self.dy8, *self.dy8_t)
        dg.dist_gemm_f8_product(*self.dy8, *self.w8_t, self.dact, workspace=self.ws_a)
        dg.dist_gemm_f8_transpose(*self.act, *self.act_t)
        dg.dist_gemm_f8_product(*self.dy8_t, *self.act_t, self.dweight, workspace=self.ws_w)
        dg.dist_gemm_layer_norm_backward(self.dact, self.kept[0], None, self.rstd, self.norm_weight, self.dx, self.dnorm_weight,
                                         self.dnorm_bias, self.ws_n, dh=dh, h_scales=self.kept[1])
        return self.dx


def main(tokens=4096, width=4096, out=8192):
    layer = NormLinear(tokens, width, out)
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r, dh = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    dy = torch.randn(tokens, out, generator=g, device="cuda").bfloat16()
    y = layer.forward(x, r)
    dx = layer.backward(dy, dh)
    torch.cuda.synchronize()
    for name, t in (("y", y), ("dx", dx), ("dweight", layer.dweight), ("norm's dweight", layer.dnorm_weight)):
        print(f"{name}: {tuple(t.shape)}, rms {t.float().square().mean().sqrt().item():.4f}")
    kept = sum(t.numel() * t.element_size() for t in (*layer.act, *layer.kept, layer.rstd))
    print(f"kept between forward and backward: {kept / tokens / width:.3f} bytes per value of the stream")


if __name__ == "__main__":
    main()
