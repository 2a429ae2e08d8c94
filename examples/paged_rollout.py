"""One attention layer of a rollout: FP8 projection, paged FP8 cache, prompts and
then single tokens.

The layer's fused QKV projection runs in FP8 (1x128 activations, 128x128 weight
blocks); the prompts' keys and values calibrate the cache's per-tensor scales;
rope_append_kv rotates and appends, paged_attention attends.  A decoding step is
captured once in a CUDA graph and replayed: the lengths and the page table are
read on the device, so the same graph serves every step.

    python examples/paged_rollout.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_x128_gb300 as fg  # noqa: E402


def rope_table(positions, dim, base=500000.0):
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * base ** (
        -torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    return torch.cat([a.cos(), a.sin()], 1).float()


class Layer:
    """QKV projection, cache and attention of one layer (batch rows padded to a multiple of 128)."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, dim=128, page=64, seqs=4, max_len=2048, seed=0):
        self.hidden, self.Hq, self.Hkv, self.D, self.seqs = hidden, q_heads, kv_heads, dim, seqs
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = (q_heads + 2 * kv_heads) * dim
        w = (torch.randn((n, hidden), generator=g, device="cuda") * hidden ** -0.5).bfloat16()
        self.w = torch.empty((n, hidden), dtype=torch.uint8, device="cuda")
        self.sw = torch.empty((n // 128, hidden // 128), device="cuda")
        fg.quant_128x128(w, fg.E4M3, self.w, self.sw)
        per_seq = -(-max_len // page)
        pages = (seqs * per_seq, kv_heads, page, dim)
        self.k = torch.empty(pages, dtype=torch.float8_e4m3fn, device="cuda")
        self.v = torch.empty(pages, dtype=torch.float8_e4m3fn, device="cuda")
        self.k_scale, self.v_scale = torch.ones(1, device="cuda"), torch.ones(1, device="cuda")
        self.cache = fg.PagedKV(self.k, self.v, self.k_scale, self.v_scale)
        self.table = torch.randperm(seqs * per_seq, generator=g, device="cuda").to(torch.int32).view(seqs, per_seq)
        self.kv_lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.rope = rope_table(max_len, dim)
        self.work, self.tensor_work = fg.new_attention_workspace(), fg.new_workspace()

    def buffers(self, rows):
        """What a call of up to `rows` tokens needs, kept between calls."""
        rows = -(-rows // 128) * 128
        b = {"x": torch.zeros((rows, self.hidden), dtype=torch.bfloat16, device="cuda")}
        b["q8"] = torch.empty((rows, self.hidden), dtype=torch.uint8, device="cuda")
        b["s8"] = torch.empty((self.hidden // 128, rows), device="cuda")
        b["qkv"] = torch.empty((rows, self.w.shape[0]), dtype=torch.bfloat16, device="cuda")
        q, k, v = b["qkv"].split([self.Hq * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)
        b["q"], b["k"], b["v"] = (t.unflatten(1, (-1, self.D)) for t in (q, k, v))
        b["codes"] = torch.empty((rows, self.Hkv * self.D), dtype=torch.uint8, device="cuda")
        b["out"] = torch.zeros((rows, self.Hq, self.D), dtype=torch.bfloat16, device="cuda")
        return b

    def project(self, b):
        fg.quant_1x128(b["x"], fg.E4M3, b["q8"], b["s8"])
        fg.blockscaled_gemm(b["q8"], fg.E4M3, b["s8"], fg.GRAN_1x128, self.w, fg.E4M3, self.sw, fg.GRAN_128x128, b["qkv"])

    def calibrate(self, b, tokens):
        """The cache's scales from the prompts' keys and values; a rotation can raise a key by sqrt(2)."""
        for name, scale in (("k", self.k_scale), ("v", self.v_scale)):
            fg.quant_pertensor_current(b[name][:tokens].flatten(1), fg.E4M3, scale, b["codes"], self.tensor_work)
        self.k_scale.mul_(2.0 ** 0.5)

    def attend(self, b, batch):
        fg.rope_append_kv(self.cache, batch, b["k"], b["v"], self.rope, q=b["q"], q_out=b["q"])
        fg.paged_attention(self.cache, batch, b["q"], b["out"], self.work)

    def prompts(self, b, lens):
        """All prompts in one call: b["x"] holds them one after another."""
        offsets = torch.tensor([0, *lens], device="cuda").cumsum(0, dtype=torch.int32)
        self.kv_lens.copy_(offsets[1:] - offsets[:-1])
        self.project(b)
        self.calibrate(b, sum(lens))
        self.attend(b, fg.PagedBatch(offsets, self.kv_lens, self.table, max(lens)))

    def step(self, b):
        """One token of every sequence: b["x"][i] is sequence i's."""
        self.kv_lens.add_(1)
        self.project(b)
        self.attend(b, self.singles)

    def capture_step(self, b):
        self.singles = fg.PagedBatch(torch.arange(self.seqs + 1, dtype=torch.int32, device="cuda"), self.kv_lens, self.table, 1)
        self.step(b)             # first call outside the capture: the kernels' attributes are set
        self.kv_lens.sub_(1)     # (the captured step below writes the same rows again)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step(b)
        return graph


def main(steps=200):
    torch.manual_seed(1)
    lens = [700, 123, 1024, 1]
    layer = Layer(seqs=len(lens))
    b = layer.buffers(sum(lens))
    b["x"][:sum(lens)].normal_()
    layer.prompts(b, lens)
    one = layer.buffers(len(lens))
    one["x"][:len(lens)].normal_()
    graph = layer.capture_step(one)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    status = fg.device_status()
    assert status == fg.OK, fg.status_string(status)
    assert layer.kv_lens.tolist() == [n + steps for n in lens]
    print(f"{len(lens)} sequences, prompts {lens}, {steps} steps: {begin.elapsed_time(end) / steps * 1e3:.1f} us a step")


if __name__ == "__main__":
    main()
