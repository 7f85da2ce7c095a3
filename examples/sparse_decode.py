"""One sparse-attention layer of a small serving loop, on the library's operators.

Three requests are served from paged e4m3 caches.  ``pages_update`` hands out pages as they grow; the
prompt's rows are quantised into the pages (``cache_write``), packed back and scored as a prompt chunk (``cache_read``, ``fp8_mqa_logits``);
then, token by token, a step writes the new rows, scores every cached position for the newest token
(``logits_paged``), selects the best (``topk``) and attends to those alone (``attention_paged``).
Run it on a GB300:

    python examples/sparse_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_mqa_logits_02_gb300 as fm  # noqa: E402

PAGE, KV_HEADS, Q_HEADS, DIM = 64, 4, 32, 128
F8 = torch.float8_e4m3fn


class Layer:
    """The caches of one layer and their page tables."""

    def __init__(self, requests: int, longest: int, device):
        self.cols = -(-longest // PAGE)
        pages = requests * self.cols
        shape = (pages, PAGE, KV_HEADS, DIM)
        self.k, self.v = (torch.zeros(shape, dtype=F8, device=device) for _ in range(2))
        self.k_scale, self.v_scale = (torch.zeros(shape[:3], device=device) for _ in range(2))
        self.index = torch.zeros((pages, PAGE, 1, fm.DIM), dtype=F8, device=device)
        self.index_scale = torch.zeros((pages, PAGE, 1), device=device)
        self.table = torch.full((requests, self.cols), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(requests, dtype=torch.int32, device=device)
        self.free = torch.randperm(pages).to(device=device, dtype=torch.int32)
        self.n_free = torch.full((1,), pages, dtype=torch.int32, device=device)

    def slots(self, new: list[int]) -> torch.Tensor:
        """Slots for ``new[b]`` further tokens of each request, one request after the other."""
        change = torch.tensor(new, dtype=torch.int32, device=self.lens.device)
        return fm.pages_update(self.table, self.lens, change, self.free, self.n_free, PAGE, sum(new)).slots

    def write(self, slots, k, v, index_keys):
        fm.cache_write(slots, k, self.k, self.k_scale, v, self.v, self.v_scale)
        fm.cache_write(slots, index_keys, self.index, self.index_scale)

    def score_prompt(self, q, w):
        """Causal logits of all cached positions of all requests, as one prompt chunk."""
        starts = torch.nn.functional.pad(self.lens.cumsum(0), (1, 0)).to(torch.int32)
        total = int(starts[-1])
        keys, scale = fm.cache_read(self.index, self.index_scale, self.table, starts, total)
        first = torch.repeat_interleave(starts[:-1], self.lens).to(torch.int32)
        last = torch.arange(1, total + 1, dtype=torch.int32, device=q.device)
        return fm.fp8_mqa_logits(q, keys.squeeze(1), scale.squeeze(1), w, first, last)

    def step(self, q, q_index, w, top: int):
        """The newest token of each request attends to its ``top`` best-scored positions."""
        logits = fm.logits_paged(q_index, self.index, self.index_scale, w, self.table, self.lens)
        picked, _ = fm.topk(logits, top, with_values=False, sorted=False)
        return fm.attention_paged(q, self.k, self.v, self.table, self.lens, k_scale=self.k_scale,
                                  v_scale=self.v_scale, indices=picked)


def main(prompt=(700, 65, 1), steps=8, top=128, seed=0):
    device = torch.device("cuda:0")
    gen = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=device).to(dtype)

    B = len(prompt)
    layer = Layer(B, max(prompt) + steps, device)
    tokens = sum(prompt)
    layer.write(layer.slots(list(prompt)), randn(tokens, KV_HEADS, DIM), randn(tokens, KV_HEADS, DIM),
                randn(tokens, 1, fm.DIM))
    logits = layer.score_prompt(randn(tokens, fm.HEADS, fm.DIM, dtype=F8),
                                randn(tokens, fm.HEADS, dtype=torch.float32) / 64)
    if fm.check_error() != 0:
        raise RuntimeError("the prompt's logits failed")
    out = None
    for _ in range(steps):
        layer.write(layer.slots([1] * B), randn(B, KV_HEADS, DIM), randn(B, KV_HEADS, DIM), randn(B, 1, fm.DIM))
        out = layer.step(randn(B, Q_HEADS, DIM), randn(B, 1, fm.HEADS, fm.DIM, dtype=F8),
                         randn(B, 1, fm.HEADS, dtype=torch.float32) / 64, top)
    if fm.check_error() != 0:
        raise RuntimeError("a step's logits failed")
    return layer, logits, out


if __name__ == "__main__":
    layer, logits, out = main()
    print(f"prompt logits {tuple(logits.shape)}, lengths {layer.lens.tolist()}, "
          f"last step's attention {tuple(out.shape)}, |out| {out.float().abs().mean():.4f}")
