"""One attention layer of a serving loop on the library's calls.

Requests arrive with prompts of different lengths.  Each step takes a piece of
the prompts that are still coming in and one token of every other request,
all in one batch:

    hidden -> W4A4 q|k|v projection -> block tables and slots ->
    keys and values into the E4M3 pages -> attention over the pages ->
    W4A4 output projection

Nothing is read back from the GPU: the scheduler's own lengths are all that
the host needs.  Weights and hidden states are random.

    python examples/paged_serving.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import nvfp4_w4a4_quantized_03_amd as nv  # noqa: E402


class AttentionLayer:
    """W4A4 projections, the paged E4M3 cache and its block table."""

    def __init__(self, hidden, heads, kv_heads, d, pages, page_size, max_requests, max_len,
                 device="cuda:0", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.d, self.page_size = heads, kv_heads, d, page_size

        def weight(n, k):
            w = torch.randn(n, k, generator=gen, device=device) * k ** -0.5
            return nv.quantize(w.to(torch.bfloat16))

        self.qkv = weight((heads + 2 * kv_heads) * d, hidden)
        self.out = weight(hidden, heads * d)
        self.k_cache = torch.empty(pages, kv_heads, page_size, d, dtype=torch.uint8, device=device)
        self.v_cache = torch.empty_like(self.k_cache)
        self.table = torch.full((max_requests, -(-max_len // page_size)), -1, dtype=torch.int32,
                                device=device)
        self.free = torch.randperm(pages, generator=gen, device=device).to(torch.int32)
        # static scales from calibration data, as they come with a checkpoint
        sample = torch.randn(4096, hidden, generator=gen, device=device).to(torch.bfloat16)
        self.x_global = nv.quantize(sample).global_scale
        kv = self.project(sample)
        k, v = (kv[:, a:b].reshape(4096, -1) for a, b in
                ((heads, heads + kv_heads), (heads + kv_heads, heads + 2 * kv_heads)))
        self.k_scale, self.v_scale = nv.fp8_kv_calibrate([k])[0], nv.fp8_kv_calibrate([v])[0]

    def project(self, x):
        y = nv.gemm(nv.quantize(x, self.x_global), self.qkv)
        return y.view(x.shape[0], self.heads + 2 * self.kv_heads, self.d)

    def step(self, x, new, cached):
        """x: hidden states of the new tokens, request by request; new, cached:
        host lists of lengths.  Returns the layer's output, the queries and
        the attention's own output."""
        h, g = self.heads, self.kv_heads
        n = len(new)
        lens = torch.tensor([new, cached], dtype=torch.int32).to(x.device, non_blocking=True)
        qkv = self.project(x)
        pages = nv.kv_page_tables(lens[0], lens[1], self.table[:n], self.free, self.page_size,
                                  x.shape[0])
        nv.kv_page_write(qkv[:, h:h + g], qkv[:, h + g:], self.k_cache, self.v_cache, pages.slots,
                         self.k_scale, self.v_scale)
        o = nv.paged_attention(qkv[:, :h], self.k_cache, self.v_cache, self.table[:n],
                               pages.cu_new, pages.kv_lens, max(new),
                               max(a + b for a, b in zip(new, cached)), k_scale=self.k_scale,
                               v_scale=self.v_scale)
        # the pages just taken leave the front of the free list
        taken = sum(-(-(a + b) // self.page_size) - -(-b // self.page_size)
                    for a, b in zip(new, cached))
        self.free = self.free[taken:]
        y = nv.gemm(nv.quantize(o.view(x.shape[0], -1)), self.out)
        return y, qkv[:, :h], o


def serve(prompts=(700, 33, 1500, 64), chunk=512, decode_steps=8, hidden=5120, heads=40,
          kv_heads=8, d=128, page_size=16, device="cuda:0", seed=0):
    """Brings the prompts in by chunks, then decodes; yields each step's
    (layer, new, cached, output, queries, attention output)."""
    longest = max(prompts) + decode_steps + len(prompts) * (max(prompts) // chunk + 1)
    pages = len(prompts) * -(-longest // page_size)
    layer = AttentionLayer(hidden, heads, kv_heads, d, pages, page_size, len(prompts), longest,
                           device, seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    cached, left, decoded = [0] * len(prompts), list(prompts), 0
    while decoded < decode_steps:
        budget, new = chunk, []
        decoded += not any(left)
        for r in range(len(prompts)):
            if left[r]:
                take = min(left[r], budget)
                left[r] -= take
                budget -= take
            else:
                take = 1
            new.append(take)
        x = torch.randn(sum(new), hidden, generator=gen, device=device).to(torch.bfloat16)
        y, q, o = layer.step(x, new, cached)
        yield layer, new, list(cached), y, q, o
        cached = [a + b for a, b in zip(cached, new)]


if __name__ == "__main__":
    for i, (_, new, cached, y, _, _) in enumerate(serve()):
        torch.cuda.synchronize()
        print("step %2d: %4d new tokens %s over %s cached, output rms %.4f"
              % (i, sum(new), new, cached, float(y.float().square().mean().sqrt())), flush=True)
