"""A residual layer in 8-bit floating point: trained for some steps, then asked one token at a time.

    h = x + r,  y = rmsnorm(h) * w,  out = y @ W.T

The forward pass normalises and quantises in one launch and multiplies; the backward pass quantises the output's
gradient for both of its products in one launch, multiplies by W for the input's gradient and by y for W's, and goes
back through the norm.  W is kept in float32 and quantised in 128 x 128 blocks after each update; what the layer has
to learn is a fixed random W.

    python examples/fp8_layer.py [--tokens 2048] [--inputs 1024] [--outputs 1536] [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_matrix_10_gb300 as sg  # noqa: E402


class Layer:
    """W (outputs x inputs) and the norm's weights w in float32, W's 8-bit blocks beside it."""

    def __init__(self, inputs, outputs, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.W = torch.randn(outputs, inputs, generator=g, device="cuda") / inputs ** 0.5
        self.w = torch.ones(inputs, device="cuda")
        self.quantise()

    def quantise(self):
        self.qW, self.sW = sg.quantize_fp8(self.W, block=(128, 128))

    def forward(self, x, r, training=True):
        """The layer's output in bfloat16, and what backward wants."""
        o = sg.rms_norm_fp8(x, self.w, residual=r, training=training)
        return sg.gemm_fp8(o.q, o.scale, self.qW, self.sW, transB=True), o

    def backward(self, dout, o):
        """(gradient of x and of r alike, gradient of W, gradient of w)"""
        q_rows, s_rows, q_cols, s_cols = sg.quantize_fp8_both(dout)
        dy = sg.gemm_fp8(q_rows, s_rows, self.qW, self.sW)                            # dout @ W
        qy, sy = sg.quantize_fp8(o.y, block=(128, 1))
        dW = sg.gemm_fp8(q_cols, s_cols, qy, sy, transA=True, out_dtype=torch.float32)   # dout.T @ y
        dx, dw = sg.rms_norm_backward(dy, o.h, self.w, o.rstd)
        return dx, dW, dw

    def step(self, dW, dw, rate):
        self.W.sub_(dW, alpha=rate)
        self.w.sub_(dw, alpha=rate)
        self.quantise()


def train(tokens=2048, inputs=1024, outputs=1536, steps=40, rate=0.4):
    """The mean squared error before each step, against a layer with other weights."""
    layer, goal = Layer(inputs, outputs, 1), Layer(inputs, outputs, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x, r = (torch.randn(tokens, inputs, generator=g, device="cuda").bfloat16() for _ in range(2))
    with torch.no_grad():
        want = goal.forward(x, r)[0].float()
        errors = []
        for _ in range(steps):
            out, o = layer.forward(x, r)
            diff = out.float() - want
            errors.append(diff.square().mean())
            _, dW, dw = layer.backward((diff / tokens).bfloat16(), o)
            layer.step(dW, dw, rate)
    return layer, goal, torch.stack(errors).tolist()


def decode(layer, tokens=8):
    """One token after the other, and all of them at once: the same rows."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r = (torch.randn(tokens, layer.W.shape[1], generator=g, device="cuda").bfloat16() for _ in range(2))
    one_by_one = torch.cat([layer.forward(x[i:i + 1], r[i:i + 1], training=False)[0] for i in range(tokens)])
    return one_by_one, layer.forward(x, r, training=False)[0]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 2048), ("inputs", 1024), ("outputs", 1536), ("steps", 40)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    layer, _, errors = train(a.tokens, a.inputs, a.outputs, a.steps)
    for i in sorted({*range(0, a.steps, max(1, a.steps // 8)), a.steps - 1}):
        print(f"step {i:4d}  mean squared error {errors[i]:.5f}")
    one, all_ = decode(layer)
    print(f"one token at a time against all at once: largest difference "
          f"{(one.float() - all_.float()).abs().max().item():.2e}")
    status = sg.sgemm_last_device_status()
    if status != 0:
        raise SystemExit(f"device status {status} ({sg.sgemm_status_string(status)})")


if __name__ == "__main__":
    main()
