"""One training step of a LoRA MLP block whose frozen weights are kept in 4 bits
and whose activations are checkpointed in 8, and one new token through it:

    h = x W1^T + (x A^T) B^T + bias,  y = gelu(h),  out = y W2^T

W1 [F, d] and W2 [d, F] frozen, stored in "fp4" (blocks along their rows); the
adapter A [r, d], B [F, r] and the bias are trained.  The forward pass keeps x
and h as "int8" checkpoints instead of 16-bit tensors; the backward pass uses
them for the adapter's gradient and for gelu's.

    python examples/lora_mlp_block.py            # T=512 d=2048 F=5632 r=32, fp16
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_gemm_tiled_gb300 import binding as g  # noqa: E402


class Block:
    def __init__(self, d=2048, F=5632, r=32, dtype=torch.float16, seed=0, fmt="fp4"):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=0.02, dt=torch.float32):
            return (torch.randn(shape, generator=gen, device="cuda") * std).to(dt)

        self.d, self.F, self.r, self.dtype = d, F, r, dtype
        self.W1, self.W2 = g.mx_empty(F, d, fmt), g.mx_empty(d, F, fmt)
        g.mx_quantize(normal(F, d), self.W1)
        g.mx_quantize(normal(d, F), self.W2)
        self.A, self.B = normal(r, d, dt=dtype), normal(F, r, dt=dtype)
        self.bias = normal(F, dt=dtype)

    def new(self, *shape):
        return torch.empty(shape, dtype=self.dtype, device="cuda")

    def forward(self, x):
        """Returns out and what the backward pass needs."""
        T = x.shape[0]
        x8, h8 = g.mx_empty(T, self.d, "int8"), g.mx_empty(T, self.F, "int8")
        g.mx_quantize(x, x8)
        xa, h, out = self.new(T, self.r), self.new(T, self.F), self.new(T, self.d)
        g.gemm(x, self.A, xa, transB=True)
        g.gemm(xa, self.B, h, transB=True)
        g.gemm_mx(x, self.W1, h, transB=True, beta=1.0, bias=self.bias)  # h = x W1^T + h + bias
        g.mx_quantize(h, h8, act="gelu", Y=h)  # y over h; h's checkpoint in the same pass
        g.gemm_mx(h, self.W2, out, transB=True)
        return out, (x8, h8, xa)

    def backward(self, dout, saved):
        """Gradients of x, A, B and the bias."""
        x8, h8, xa = saved
        T = dout.shape[0]
        dh, dx = self.new(T, self.F), self.new(T, self.d)
        dA, dB, dha = self.new(self.r, self.d), self.new(self.F, self.r), self.new(T, self.r)
        dbias = torch.empty(self.F, dtype=torch.float32, device="cuda")
        g.gemm_mx(dout, self.W2, dh)                       # dy = dout W2
        g.mx_act_backward(dh, h8, dh, act="gelu", dbias=dbias)
        g.gemm(dh, xa, dB, transA=True)                    # dB = dh^T (x A^T)
        g.gemm(dh, self.B, dha)                            # dh B
        g.gemm_mx(dha, x8, dA, transA=True)                # dA = (dh B)^T x, x from its checkpoint
        g.gemm_mx(dh, self.W1, dx)                         # dx = dh W1 + (dh B) A
        g.gemm(dha, self.A, dx, beta=1.0)
        return dx, dA, dB, dbias

    def forward_4bit(self, x):
        """x W1^T with the activations in W1's 4-bit format too."""
        x4 = g.mx_empty(x.shape[0], self.d, self.W1.fmt)
        g.mx_quantize(x, x4)
        return g.gemm_mx(x4, self.W1, self.new(x.shape[0], self.F))


def main():
    T, d, F = 512, 2048, 5632
    block = Block(d, F)
    x, dout = (torch.randn(T, d, device="cuda").half() for _ in range(2))
    for _ in range(3):
        out, saved = block.forward(x)
        grads = block.backward(dout, saved)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(10):
        out, saved = block.forward(x)
        grads = block.backward(dout, saved)
    end.record()
    torch.cuda.synchronize()
    print(f"step {start.elapsed_time(end) / 10:.3f} ms, "
          f"one token {tuple(block.forward(x[:1])[0].shape)}")
    stored = sum(m.codes.numel() + m.scales.numel() for m in (block.W1, block.W2))
    kept = sum(m.codes.numel() + m.scales.numel() for m in saved[:2])
    print(f"weights {stored / 2**20:.1f} MiB (fp16 {2 * 2 * d * F / 2**20:.1f}), "
          f"checkpoints {kept / 2**20:.1f} MiB (fp16 {2 * T * (d + F) / 2**20:.1f})")
    print("|dA| %.3g  |dB| %.3g  |dbias| %.3g" % tuple(t.float().norm().item() for t in grads[1:]))
    y16 = g.gemm_mx(x, block.W1, block.new(T, F), transB=True).float()
    y4 = block.forward_4bit(x).float()
    print("4-bit activations: relative difference %.3f" % ((y4 - y16).norm() / y16.norm()).item())


if __name__ == "__main__":
    main()
