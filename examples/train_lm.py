"""A training step of a small token model around the FP8 Linear.

Embedding, blocks of (residual add + RMSNorm, FP8 SwiGLU MLP), a last norm and the softmax cross
entropy of the tied head.  What the backward pass needs of the norms and of the MLPs' gate/up
projections is kept in 8 bits; the logits are never stored.  The head writes the shared matrix's
gradient in FP32, the embedding adds its own to it; AdamW keeps its moments in FP8.  (The blocks mix
no tokens: the model predicts a token from the one before it.)

    python examples/train_lm.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_x128_gb300 as fg  # noqa: E402

E, ROW, BLOCK = fg.E4M3, fg.GRAN_1x128, fg.GRAN_128x128


def u8(*shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda")


def f32(*shape):
    return torch.empty(shape, device="cuda")


def bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


class Weight:
    """FP32 master, BF16 working copy, AdamW moments in FP8."""

    decay = 0.01

    def __init__(self, master):
        self.master, n = master, master.numel()
        self.m, self.v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.sm, self.sv = (torch.ones(n // 128, device="cuda") for _ in range(2))
        self.grad, self.bf16 = f32(*master.shape), master.bfloat16()

    def update(self, lr, step):
        h = fg.adamw_hparams(lr, 0.9, 0.95, 1e-8, self.decay, step)
        fg.adamw_step_fp8_states(self.master, self.grad.bfloat16(), self.m, self.sm, self.v, self.sv, h)
        self.bf16.copy_(self.master)


def normal(rows, cols, scale, g):
    return torch.randn((rows, cols), generator=g, device="cuda") * scale


class Linear(Weight):
    """y = x W^T in FP8 (1x128 activations, 128x128 weight blocks); weight [out, in]."""

    def __init__(self, out, inp, g):
        super().__init__(normal(out, inp, inp ** -0.5, g))
        self.q, self.s = u8(out, inp), f32(out // 128, inp // 128)
        self.qT, self.sT = u8(inp, out), f32(inp // 128, out // 128)

    def forward(self, x, y):
        R, (N, K) = x.shape[0], self.master.shape
        fg.quant_128x128(self.bf16, E, self.q, self.s)
        q, s, self.xT, self.sxT = u8(R, K), f32(K // 128, R), u8(K, R), f32(R // 128, K)
        fg.quant_1x128(x, E, q, s, self.xT, self.sxT)
        fg.blockscaled_gemm(q, E, s, ROW, self.q, E, self.s, BLOCK, y)

    def backward(self, dy, dx):
        R, (N, K) = dy.shape[0], self.master.shape
        q, s, qT, sT = u8(R, N), f32(N // 128, R), u8(N, R), f32(R // 128, N)
        fg.quant_1x128(dy, E, q, s, qT, sT)
        fg.transpose_128x128(self.q, self.s, self.qT, self.sT)
        fg.blockscaled_gemm(q, E, s, ROW, self.qT, E, self.sT, BLOCK, dx)
        fg.blockscaled_gemm(qT, E, sT, ROW, self.xT, E, self.sxT, ROW, self.grad)
        del self.xT, self.sxT


class Norm(Weight):
    """Residual add and RMSNorm; keeps the sum in 8 bits."""

    decay = 0.0

    def __init__(self, dim):
        super().__init__(torch.ones(dim, device="cuda"))
        self.w, self.workspace = self.bf16, fg.new_rmsnorm_workspace(dim)

    def forward(self, x, stream, y, total):
        R, C = x.shape
        self.c, self.cs, self.rstd = u8(R, C), f32(C // 128, R), f32(R)
        if stream is None:      # the first block: nothing to add
            fg.rmsnorm_fwd_ckpt(x, self.w, 1e-5, E, y, self.c, self.cs, self.rstd)
            return x
        fg.rmsnorm_fwd_ckpt(x, self.w, 1e-5, E, y, self.c, self.cs, self.rstd, res=stream, sum=total)
        return total

    def backward(self, dy, dstream, dx):
        fg.rmsnorm_bwd_ckpt(self.c, self.cs, self.rstd, self.w, dy, E, dx, self.grad, self.workspace, dsum=dstream)
        return dx


class Block:
    def __init__(self, dim, ffn, g):
        self.norm, self.up, self.down, self.ffn = Norm(dim), Linear(2 * ffn, dim, g), Linear(dim, ffn, g), ffn

    def forward(self, x, stream):
        """x: what the last block adds to the stream; returns what this one adds, and the stream."""
        R, C = x.shape
        y, gu, h, out = bf16(R, C), bf16(R, 2 * self.ffn), bf16(R, self.ffn), bf16(R, C)
        stream = self.norm.forward(x, stream, y, bf16(R, C))
        self.up.forward(y, gu)
        self.c, self.cs = u8(R, 2 * self.ffn), f32(2 * self.ffn // 128, R)
        fg.swiglu_fwd_ckpt(gu, E, h, self.c, self.cs)
        self.down.forward(h, out)
        return out, stream

    def backward(self, dout, dstream):
        """Gradient of the norm's input from those of the block's output and of the stream behind it."""
        R, C = dout.shape
        dh, dgu, dy = bf16(R, self.ffn), bf16(R, 2 * self.ffn), bf16(R, C)
        self.down.backward(dout, dh)
        fg.swiglu_bwd_ckpt(self.c, self.cs, dh, E, dgu)
        self.up.backward(dgu, dy)
        return self.norm.backward(dy, dstream, bf16(R, C))


class Model:
    """Tokens a step: a multiple of 128 (the quantizers' transposed copies)."""

    def __init__(self, vocab, dim, ffn, blocks, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.table = Weight(normal(vocab, dim, dim ** -0.5, g))
        self.blocks = [Block(dim, ffn, g) for _ in range(blocks)]
        self.norm, self.dim = Norm(dim), dim

    def forward(self, ids, target):
        T, V = ids.numel(), self.table.master.shape[0]
        self.ids, self.target = ids, target
        self.x0 = bf16(T, self.dim)
        fg.embedding_fwd(ids, self.table.bf16, self.x0, scale=self.dim ** 0.5)
        x, stream = self.x0, None
        for b in self.blocks:
            x, stream = b.forward(x, stream)
        self.y = bf16(T, self.dim)
        self.norm.forward(x, stream, self.y, bf16(T, self.dim))
        self.loss, self.lse = f32(T), f32(T)
        self.workspace = fg.new_linear_xent_workspace(T, V, self.dim)
        fg.linear_xent_fwd(self.y, self.table.bf16, target, self.loss, self.lse, self.workspace)
        return self.loss

    def backward(self):
        """Gradients of the mean loss over the tokens that count."""
        T, V = self.ids.numel(), self.table.master.shape[0]
        counts = (self.target >= 0).sum()
        dloss = torch.full((T,), 1.0, device="cuda") / counts
        dy = bf16(T, self.dim)
        fg.linear_xent_bwd(self.y, self.table.bf16, self.target, self.loss, self.lse, dloss, dy, self.table.grad, self.workspace)
        # the last norm's sum is the last block's output added to the stream: both get its gradient
        d = self.norm.backward(dy, None, bf16(T, self.dim))
        for b in reversed(self.blocks):
            d = b.backward(d, d)
        fg.embedding_bwd(self.ids, d, self.table.grad, fg.new_embedding_workspace(T, V, self.dim), scale=self.dim ** 0.5, accumulate=True)

    def update(self, lr, step):
        for w in [self.table, self.norm] + [w for b in self.blocks for w in (b.up, b.down, b.norm)]:
            w.update(lr, step)


def main(steps=30):
    torch.manual_seed(2)
    model = Model(vocab=8192, dim=1024, ffn=2816, blocks=2)
    follows = torch.randperm(8192, device="cuda").to(torch.int32)      # each token has one that follows it
    for step in range(1, steps + 1):
        ids = torch.randint(8192, (2048,), device="cuda", dtype=torch.int32)
        target = torch.where(torch.rand(2048, device="cuda") < 0.1, -1, follows[ids.long()])
        loss = model.forward(ids, target)
        model.backward()
        model.update(3e-3, step)
        if step in (1, steps):
            print(f"step {step}: mean loss {float(loss.sum() / (target >= 0).sum()):.3f}")
    status = fg.device_status()
    assert status == fg.OK, fg.status_string(status)


if __name__ == "__main__":
    main()
