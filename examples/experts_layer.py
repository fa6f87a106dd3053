"""A layer of experts in 8 bits, forward and backward, from this package's calls alone.

    z = silu(W1g x) * (W1u x);  y = W2 z        for each of a token's chosen experts
    out = sum over them of weight * y

Weights stay in FP32 and are quantised to e4m3 by 128 x 128 tiles; activations
and gradients by blocks of 128 of the summed axis. Run it on an MI355X from the
repository root:

    python examples/experts_layer.py
    python examples/experts_layer.py --tokens 8192 --width 2048 --hidden 1024 --experts 32 --rate 0.05

It fits the layer to a fixed target and prints the loss and the time of a step.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_02_amd as sg  # noqa: E402


def quantized(w):
    """(Q, S) of weights experts x n x k (n a multiple of 128), and the same of their transposes: a tile's scale is
    that of the transposed tile."""
    e, n, k = w.shape
    q, s = sg.quantize_fp8(w.view(e * n, k), blocks=True)
    q, s = q.unflatten(0, (e, n)), s.unflatten(0, (e, n // 128))
    back = q.view(torch.uint8).transpose(1, 2).contiguous().view(q.dtype)
    return (q, s), (back, s.transpose(1, 2).contiguous())


class ExpertsLayer:
    """Weights of the router (experts x width), W1 (experts x 2 hidden x width) and W2 (experts x width x hidden)."""

    def __init__(self, width, hidden, experts, choices, seed=0, device="cuda"):
        if width % 128 or hidden % 128:
            raise ValueError("width and hidden must be multiples of 128")
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

        self.choices = choices
        self.router, self.w1, self.w2 = normal(experts, width), normal(experts, 2 * hidden, width), normal(experts, width, hidden)
        self.load_weights()

    def load_weights(self):
        """Quantises the weights; after each change of them."""
        (self.q1, self.q1t), (self.q2, self.q2t) = quantized(self.w1), quantized(self.w2)

    def forward(self, x):
        """x: tokens x width, bfloat16. Returns the output and what backward needs."""
        logits = sg.matmul(x.float(), self.router.t().contiguous())
        weights, experts = sg.route(logits, self.choices)
        offsets, tokens, place = sg.route_plan(experts, self.router.shape[0])
        h = sg.gemm_fp8_experts(*sg.quantize_fp8(x, index=tokens), *self.q1, offsets)
        gate, up = h.float().chunk(2, dim=1)
        z = (torch.sigmoid(gate) * gate * up).to(x.dtype)
        y = sg.gemm_fp8_experts(*sg.quantize_fp8(z), *self.q2, offsets)
        out = sg.route_combine(y, place, weights)
        return out, dict(x=x, logits=logits, weights=weights, experts=experts, offsets=offsets, tokens=tokens, place=place,
                         h=h, z=z, y=y)

    def backward(self, dout, saved):
        """Gradients of x, the router's weights, W1 and W2 for the gradient of the output."""
        x, offsets, tokens, place = (saved[k] for k in ("x", "offsets", "tokens", "place"))
        dy, dweights = sg.route_combine_backward(dout, saved["y"], place, saved["weights"])
        dz = sg.gemm_fp8_experts(*sg.quantize_fp8(dy), *self.q2t, offsets).float()
        gate, up = saved["h"].float().chunk(2, dim=1)
        open_ = torch.sigmoid(gate)
        dh = torch.cat([dz * up * open_ * (1 + gate * (1 - open_)), dz * open_ * gate], 1).to(x.dtype)
        dx_rows = sg.gemm_fp8_experts(*sg.quantize_fp8(dh), *self.q1t, offsets)
        dw2 = sg.gemm_fp8_experts_wgrad(*sg.quantize_fp8_cols(dy, offsets=offsets),
                                        *sg.quantize_fp8_cols(saved["z"], offsets=offsets), offsets)
        dw1 = sg.gemm_fp8_experts_wgrad(*sg.quantize_fp8_cols(dh, offsets=offsets),
                                        *sg.quantize_fp8_cols(x, index=tokens, offsets=offsets), offsets)
        dlogits = sg.route_backward(saved["logits"], saved["experts"], dweights)
        dx = sg.route_combine(dx_rows, place, torch.ones_like(saved["weights"])).float()
        dx += sg.matmul(dlogits, self.router)
        drouter = sg.gemm(dlogits, x.float(), opA=1)
        return dict(x=dx, router=drouter, w1=dw1, w2=dw2, dy=dy, dweights=dweights, dh=dh, dz=dz, dlogits=dlogits)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 2048), ("width", 512), ("hidden", 256), ("experts", 16), ("choices", 4), ("steps", 5)):
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--rate", type=float, default=0.5)
    a = p.parse_args(argv)
    layer = ExpertsLayer(a.width, a.hidden, a.experts, a.choices)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.width, generator=g, device="cuda").bfloat16()
    target = torch.randn(a.tokens, a.width, generator=g, device="cuda") * 0.1
    losses = []
    for step in range(a.steps):
        torch.cuda.synchronize()
        start = time.perf_counter()
        out, saved = layer.forward(x)
        miss = out.float() - target
        grads = layer.backward((miss / a.tokens).bfloat16(), saved)
        for name in ("router", "w1", "w2"):
            getattr(layer, name).sub_(grads[name], alpha=a.rate)
        layer.load_weights()
        losses.append(float(miss.square().mean()))
        torch.cuda.synchronize()
        print(f"step {step}: loss {losses[-1]:.6f}, {(time.perf_counter() - start) * 1e3:.2f} ms", flush=True)
    return losses


if __name__ == "__main__":
    main()
