"""One attention block of a served model, decoding token by token.

    python examples/decode_attention.py [--steps N] [--cache bf16|int8]

The block's projections are this package's linear layers, and what lies
between them its decode operators:

    int8_linear       x -> q, k, v   (int8 weights, activations quantised)
    qk_norm_rope      norm and rotation of q and k, k and v into a paged cache
    paged_attention   attention of the new token over the cache
    int4_linear       the output projection (4-bit weights)

The step is captured into a graph once and replayed for every token: the
positions, slots and lengths it reads are device tensors that the host
updates between replays.  Weights are random, so the numbers mean nothing;
the time per step does.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_weight_quantized_amd as ck  # noqa: E402


class AttentionBlock:
    def __init__(self, hidden, heads, kv_heads, head_dim, pages, page_size, cache="bf16", rows=32768, device="cuda",
                 seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        n = (heads + 2 * kv_heads) * head_dim
        self.w_qkv = torch.randint(-127, 128, (n, hidden), dtype=torch.int8, device=device, generator=g)
        self.s_qkv = torch.full((n,), 1.0 / (73 * hidden ** 0.5), device=device)
        codes = torch.randint(0, 256, (hidden, heads * head_dim // 2), dtype=torch.uint8, device=device, generator=g)
        scales = torch.full((hidden, -(-heads * head_dim // 128)), 0.2 / (heads * head_dim) ** 0.5,
                            dtype=torch.bfloat16, device=device)
        self.w_out = ck.int4_pack(codes, scales, group=128)
        self.q_norm = torch.ones(head_dim, device=device)
        self.k_norm = torch.ones(head_dim, device=device)
        self.table = ck.rope_table(rows, head_dim, device=device)
        self.cache = ck.KVCache.empty(pages, kv_heads, page_size, head_dim, cache, device)

    def __call__(self, x, positions, slots, table=None, lens=None):
        """x [tokens, hidden].  With a page table, one new token of each
        sequence; without, a prompt's tokens, whose keys and values go into
        the cache (their own attention is not this example's)."""
        h, kvh, d = self.heads, self.kv_heads, self.head_dim
        qkv = ck.int8_linear(x, self.w_qkv, self.s_qkv)
        q, k, v = qkv.split([h * d, kvh * d, kvh * d], 1)
        q, _ = ck.qk_norm_rope(q.view(-1, h, d), k.view(-1, kvh, d), v.view(-1, kvh, d), positions, self.table,
                               self.q_norm, self.k_norm, cache=self.cache, slots=slots)
        if table is None:
            return None
        o = ck.paged_attention(q, self.cache, table, lens)
        return ck.int4_linear(o.view(-1, h * d), self.w_out)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--cache", choices=("bf16", "int8"), default="int8")
    a = ap.parse_args()
    hidden, page = 4096, 16
    per = -(-(a.prompt + a.steps) // page)                   # pages of a sequence
    block = AttentionBlock(hidden, 32, 8, 128, a.batch * per, page, a.cache)
    table = torch.randperm(a.batch * per, device="cuda").int().view(a.batch, per)

    at = torch.arange(a.prompt, device="cuda")
    for b in range(a.batch):                                 # the prompts' keys and values
        x = torch.randn(a.prompt, hidden, device="cuda").bfloat16()
        block(x, at, table[b].long()[at // page] * page + at % page)

    x = torch.randn(a.batch, hidden, device="cuda").bfloat16()
    positions = torch.full((a.batch,), a.prompt, device="cuda")
    slots = torch.empty(a.batch, dtype=torch.int64, device="cuda")
    lens = torch.empty(a.batch, dtype=torch.int32, device="cuda")

    def place():                                             # where this step's token goes
        slots.copy_(table.long().gather(1, (positions // page)[:, None])[:, 0] * page + positions % page)
        lens.copy_(positions + 1)

    place()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, positions, slots, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, positions, slots, table, lens)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    spent = 0.0
    for _ in range(a.steps):
        place()
        begin.record()
        graph.replay()
        end.record()
        x.add_(y)                                            # the residual: the next step's input
        positions.add_(1)
        end.synchronize()
        spent += begin.elapsed_time(end)
    print(f"{a.steps} steps of {a.batch} sequences from {a.prompt} tokens on, {a.cache} cache: "
          f"{1e3 * spent / a.steps:.1f} us a step, finite: {bool(torch.isfinite(x).all())}")


if __name__ == "__main__":
    main()
