"""A layer's serving step with caches in 4 bits, page tables made on the GPU, and sparse attention.

Requests come, grow by a token a step and end.  Each step is the same few calls, captured once into a CUDA graph
and replayed: ``pages_update`` changes the lengths, takes and gives pages, and finds the new tokens' slots and
positions; ``norm_rotate`` norms queries and keys and rotates them, the indexer's queries to E4M3;
``cache_write`` quantises keys and values to 4 bits and the indexer's keys to E4M3; ``logits_paged`` and ``topk``
select positions, and ``attention_paged`` attends to them.  Prompts enter through the same calls, uncaptured.
Run it on a GB300:

    python examples/serve_4bit.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_mqa_logits_02_gb300 as fm  # noqa: E402

PAGE, KV_HEADS, Q_HEADS, DIM, INDEX_ROTATED = 64, 4, 32, 128, 64
F4, F8 = torch.float4_e2m1fn_x2, torch.float8_e4m3fn


class Layer:
    """One layer's caches, weights and page tables for `requests` requests of up to `longest` tokens."""

    def __init__(self, requests: int, longest: int, pages: int, device, gen):
        def zeros(*shape, dtype):
            return torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype)

        rows = (pages, PAGE, KV_HEADS)
        self.k, self.v = (zeros(*rows, DIM // 2, dtype=F4) for _ in range(2))
        self.k_groups, self.v_groups = (zeros(*rows, DIM // 16, dtype=F8) for _ in range(2))
        self.k_scale, self.v_scale = (torch.zeros(rows, device=device) for _ in range(2))
        self.index = zeros(pages, PAGE, 1, fm.DIM, dtype=F8)
        self.index_scale = torch.zeros((pages, PAGE, 1), device=device)
        self.table = torch.full((requests, -(-longest // PAGE)), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
        self.n_free = torch.full((1,), pages, dtype=torch.int32, device=device)
        self.q_weight, self.k_weight = (torch.exp(0.1 * torch.randn(DIM, generator=gen, device=device)) for _ in range(2))
        self.inv_freq, self.index_freq = (10000.0 ** (-torch.arange(0, n, 2, device=device) / n) for n in (DIM, INDEX_ROTATED))

    def write(self, change, total: int, qkv, index_k):
        """New tokens of all requests: (their step, queries).  qkv: [total, Q_HEADS + 2 KV_HEADS, DIM]."""
        step = fm.pages_update(self.table, self.lens, change, self.free, self.n_free, PAGE, total)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], dim=1)
        q, k = fm.norm_rotate(q, k, step.positions, self.inv_freq, self.q_weight, self.k_weight)
        fm.cache_write(step.slots, k, self.k, self.k_scale, v, self.v, self.v_scale, k_groups=self.k_groups,
                       v_groups=self.v_groups)
        index_k, _ = fm.norm_rotate(index_k, None, step.positions, self.index_freq, interleaved=True)
        fm.cache_write(step.slots, index_k, self.index, self.index_scale)
        return step, q

    def attend(self, positions, q, index_q, w, top: int):
        """Each request's newest token (one each, in order) attends to its `top` best positions."""
        (index_q, by), _ = fm.norm_rotate(index_q, None, positions, self.index_freq, interleaved=True, dtype=F8)
        logits = fm.logits_paged(index_q.unsqueeze(1), self.index, self.index_scale, (w * by).unsqueeze(1), self.table, self.lens)
        picked, _ = fm.topk(logits, top, with_values=False, sorted=False)
        return fm.attention_paged(q, self.k, self.v, self.table, self.lens, k_scale=self.k_scale, v_scale=self.v_scale,
                                  k_groups=self.k_groups, v_groups=self.v_groups, indices=picked)


class Step:
    """A decode step's static buffers and its graph."""

    def __init__(self, layer: Layer, top: int, device):
        B = layer.lens.numel()
        self.change = torch.zeros(B, dtype=torch.int32, device=device)
        self.qkv = torch.zeros((B, Q_HEADS + 2 * KV_HEADS, DIM), dtype=torch.bfloat16, device=device)
        self.index_k = torch.zeros((B, 1, fm.DIM), dtype=torch.bfloat16, device=device)
        self.index_q = torch.zeros((B, fm.HEADS, fm.DIM), dtype=torch.bfloat16, device=device)
        self.w = torch.zeros((B, fm.HEADS), device=device)

        def step():
            new, q = layer.write(self.change, B, self.qkv, self.index_k)
            return new, layer.attend(new.positions, q, self.index_q, self.w, top)

        side = torch.cuda.Stream(device)     # once as it is, with no change: what has to be set up is set up here
        side.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream(device).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.new, self.out = step()

    def run(self, change, qkv, index_k, index_q, w):
        for to, x in ((self.change, change), (self.qkv, qkv), (self.index_k, index_k), (self.index_q, index_q), (self.w, w)):
            to.copy_(x)
        self.graph.replay()
        return self.out


def main(prompt=(700, 65, 130), steps=8, top=128, seed=0):
    """Every request decodes; after half of the steps the first one ends and a new one of its length begins."""
    device = torch.device("cuda:0")
    gen = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=device).to(dtype)

    def tokens(n):
        return randn(n, Q_HEADS + 2 * KV_HEADS, DIM), randn(n, 1, fm.DIM)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    B, longest = len(prompt), max(prompt) + steps
    layer = Layer(B, longest, sum(-(-(n + steps) // PAGE) for n in prompt), device, gen)
    step = Step(layer, top, device)
    layer.write(ints(prompt), sum(prompt), *tokens(sum(prompt)))
    out = None
    for i in range(steps):
        if i == steps // 2:
            layer.write(ints([-longest] + [0] * (B - 1)), 0, *tokens(0))
            layer.write(ints([prompt[0]] + [0] * (B - 1)), prompt[0], *tokens(prompt[0]))
        out = step.run(ints([1] * B), *tokens(B), randn(B, fm.HEADS, fm.DIM), randn(B, fm.HEADS, dtype=torch.float32) / 64)
    if fm.check_error() != 0:
        raise RuntimeError("a step failed")
    return layer, step, out


if __name__ == "__main__":
    layer, step, out = main()
    print(f"lengths {layer.lens.tolist()}, {layer.n_free.item()} pages free, last step's attention {tuple(out.shape)}, "
          f"|out| {out.float().abs().mean():.4f}")
