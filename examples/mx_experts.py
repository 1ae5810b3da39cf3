"""The low-precision operators together, as a layer of experts would use them.

  h = x + residual                        dist_gemm_rms_norm, which also keeps h
  n = rms_norm(h) in MX E4M3              ... and its 1 / rms, for the gradient
  u = n W_up[e]^T, by expert              MxPlan with groups, weights in MX E2M1
  a = relu(u)^2 in MX E4M3                dist_gemm_mx_quantize
  o = a W_down[e]^T, by expert            MxPlan with groups
  h', m = rms_norm(o + h) in MX E2M1      dist_gemm_rms_norm, o the next residual
  logits = m W_head^T                     MxPlan

`tensor_parallel` takes the norm's e4m3 output with one scale into a
tensor-parallel step of the library (Plan), and `norm_gradient` is the norm's
backward pass.  Run it on an MI355X:  python examples/mx_experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import communication_tensor_gemm_amd as dg  # noqa: E402


def mx_empty(rows, cols, fmt):
    """Room for the codes and scales of a rows x cols MX tensor."""
    codes = torch.empty(rows, cols if fmt == "E4M3" else cols // 2, dtype=torch.uint8, device="cuda")
    return codes, torch.empty(rows, dg.dist_gemm_mx_scale_pitch(cols), dtype=torch.uint8, device="cuda")


def mx_weight(w):
    """A weight (any number of rows x cols matrices on top of each other) in MX E2M1: done once."""
    w = w.reshape(-1, w.shape[-1])
    codes, scales = mx_empty(*w.shape, "E2M1")
    dg.dist_gemm_mx_quantize(w, "E2M1", codes, scales)
    return codes, scales


class Experts:
    """`experts` feed-forward experts width -> hidden -> width and a head width -> vocab, for up to `tokens` tokens."""

    def __init__(self, tokens, experts, width, hidden, vocab, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return torch.randn(*shape, device="cuda", generator=g).mul_(shape[-1] ** -0.5).bfloat16()

        self.tokens, self.width, self.hidden, self.vocab, self.experts = tokens, width, hidden, vocab, experts
        self.gain = torch.rand(width, device="cuda", generator=g).add_(0.5).bfloat16()
        self.head_gain = torch.rand(width, device="cuda", generator=g).add_(0.5).bfloat16()
        self.up = mx_weight(weight(experts, hidden, width))
        self.down = mx_weight(weight(experts, width, hidden))
        self.head = mx_weight(weight(vocab, width))
        self.up_plan = dg.MxPlan(tokens, hidden, width, groups=experts, a_format="E4M3")
        self.down_plan = dg.MxPlan(tokens, width, hidden, groups=experts, a_format="E4M3")
        self.head_plan = dg.MxPlan(tokens, vocab, width, a_format="E2M1", out_dtype="F32")

    def forward(self, x, residual, offsets):
        """x, residual: tokens x width, the tokens in the order of their experts; expert e has
        rows offsets[e] .. offsets[e + 1] (int32, on the GPU: no host wait).  Every stage's tensors."""
        t = x.shape[0]
        s = {"h": torch.empty_like(x), "rstd": torch.empty(t, dtype=torch.float32, device="cuda"),
             "n": mx_empty(t, self.width, "E4M3"), "a": mx_empty(t, self.hidden, "E4M3"),
             "h2": torch.empty_like(x), "m": mx_empty(t, self.width, "E2M1")}
        s["u"] = torch.empty(t, self.hidden, dtype=torch.bfloat16, device="cuda")
        s["o"] = torch.empty(t, self.width, dtype=torch.bfloat16, device="cuda")
        s["logits"] = torch.empty(t, self.vocab, dtype=torch.float32, device="cuda")
        dg.dist_gemm_rms_norm(x, self.gain, s["n"][0], output="MX_E4M3", scales=s["n"][1], residual=residual, h=s["h"],
                              rstd=s["rstd"])
        self.up_plan.run(*s["n"], *self.up, s["u"], offsets=offsets)
        s["r"] = torch.relu(s["u"]).square_()
        dg.dist_gemm_mx_quantize(s["r"], "E4M3", *s["a"])
        self.down_plan.run(*s["a"], *self.down, s["o"], offsets=offsets)
        dg.dist_gemm_rms_norm(s["o"], self.head_gain, s["m"][0], output="MX_E2M1", scales=s["m"][1], residual=s["h"],
                              h=s["h2"])
        self.head_plan.run(*s["m"], *self.head, s["logits"])
        return s

    def norm_gradient(self, dn, s, dh):
        """dx (also the residual's gradient) and the gain's gradient, from dn and what reaches h elsewhere."""
        t, w = dn.shape
        dx, dgain = torch.empty_like(dn), torch.empty(w, dtype=torch.float32, device="cuda")
        work = torch.empty(dg.dist_gemm_rms_norm_workspace(t, w), dtype=torch.uint8, device="cuda")
        dg.dist_gemm_rms_norm_backward(dn, s["h"], s["rstd"], self.gain, dx, dgain, work, dh=dh)
        return dx, dgain


def tensor_parallel(x, gain, weight, scale, TP=8):
    """rms_norm(x) in e4m3 times weight^T (e4m3 bytes, N x width) by the all-gather schedule over TP steps."""
    t, w = x.shape
    y = torch.empty(t, w, dtype=torch.uint8, device="cuda")
    dg.dist_gemm_rms_norm(x, gain, y, output="E4M3", scale=scale)
    out = torch.empty(t, weight.shape[0], dtype=torch.bfloat16, device="cuda")
    with dg.Plan(t, weight.shape[0], w, TP=TP, schedule="AG_ROT_A", dtype="E4M3_BF16") as p:
        p.set_scales(scale, 1.0)
        p.run(y, weight, None, out)
        torch.cuda.synchronize()
    return y, out


def main():
    tokens, experts, width, hidden, vocab = 512, 16, 4096, 2048, 8192
    layer = Experts(tokens, experts, width, hidden, vocab)
    x, residual = (torch.randn(tokens, width, device="cuda").bfloat16() for _ in range(2))
    for t in (tokens, 1):  # a batch, and one token of it (of expert 3)
        if t == 1:
            offsets = torch.tensor([0] * 4 + [1] * (experts - 3), dtype=torch.int32, device="cuda")
        else:
            cuts = torch.sort(torch.randint(0, t + 1, (experts - 1,))).values.tolist()
            offsets = torch.tensor([0] + cuts + [t], dtype=torch.int32, device="cuda")
        s = layer.forward(x[:t], residual[:t], offsets)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            s = layer.forward(x[:t], residual[:t], offsets)
        end.record()
        torch.cuda.synchronize()
        print(f"{t} tokens, {experts} experts {width} -> {hidden} -> {width}, head {vocab}: "
              f"{start.elapsed_time(end) / 20 * 1e3:.0f} us, logits {s['logits'].std().item():.3f} rms")
    dx, dgain = layer.norm_gradient(torch.randn(1, width, device="cuda").bfloat16(), s, None)
    print(f"norm gradient: dx {dx.float().norm().item():.3f}, gain {dgain.norm().item():.3f}")
    weight = torch.randint(0, 0x50, (4096, width), dtype=torch.uint8, device="cuda")
    _, out = tensor_parallel(x, layer.gain, weight, 1 / 64)
    print(f"tensor-parallel step of {tuple(out.shape)}: finite {bool(out.isfinite().all())}")


if __name__ == "__main__":
    main()
