"""A prompt, a backup and a decode loop over KV pages held in 4 bits.

One small attention stack (random weights) runs as a serving program would run it
on this library:

  1. a prompt goes through every layer: its angles come from one kv_rotate call,
     each layer appends its keys and values to pool pages (kv_append, which
     also turns the queries) and attends over them (kv_attend);
  2. the prompt's pages go to the pinned host tier (kv_backup), 3.2 times fewer
     bytes over the host link than in 16 bits;
  3. the pages come back somewhere else in the pool (kv_restore), and tokens
     are decoded from them in a captured CUDA graph.

``main()`` decodes the same tokens from the pages as they were and from the
restored ones and returns both, with what the pages hold (kv_fetch).

Run it from the repository's root:  python examples/four_bit_pages.py
"""
from __future__ import annotations

import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from hierarchical_kv_cache_backup_gb300 import kvb  # noqa: E402

LAYERS, HEADS, GROUP, DIM, PAGE = 3, 2, 4, 128, 16
Q_HEADS = HEADS * GROUP
WIDTH = Q_HEADS * DIM


class Stack:
    """Attention layers with a residual stream, their KV pages in a 4-bit pool."""

    def __init__(self, pages: int, max_len: int, seed: int = 0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n = Q_HEADS + 2 * HEADS
        self.w_in = [torch.randn(WIDTH, n * DIM, generator=g, device="cuda").mul(WIDTH ** -0.5).bfloat16() for _ in range(LAYERS)]
        self.w_out = [torch.randn(WIDTH, WIDTH, generator=g, device="cuda").mul(WIDTH ** -0.5).bfloat16() for _ in range(LAYERS)]
        self.pages, self.max_len = pages, max_len
        self.head_bytes = kvb.kv_cache_head_bytes(kvb.KV_CACHE_Q4, DIM)
        self.layout = kvb.make_layout(LAYERS, 2, pages, PAGE, HEADS, self.head_bytes, kvb.KV_PAGE_FIRST, kvb.KV_HND, 1)
        self.page_bytes = kvb.kv_layout_page_bytes(self.layout)
        self.memory = torch.zeros(pages * self.page_bytes, dtype=torch.uint8, device="cuda")
        self.pool = kvb.kv_pool_register(self.layout, self.memory.data_ptr())
        self.rotary = kvb.kv_rotary_create(DIM, kvb.KV_ROTARY_HALF, scaling=kvb.KV_ROTARY_YARN, factor=4.0, original_len=4096,
                                           slow=1.0, fast=32.0)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.steps = {}

    def step(self, tokens: int):
        """Buffers and argument blocks of a step of `tokens` new tokens of one request."""
        if tokens in self.steps:
            return self.steps[tokens]
        s = type("Step", (), {})()
        s.x = torch.empty(tokens, WIDTH, dtype=torch.bfloat16, device="cuda")
        s.positions = torch.empty(tokens, dtype=torch.int64, device="cuda")
        s.slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
        s.length = torch.empty(1, dtype=torch.int32, device="cuda")
        s.q_start = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
        s.table = torch.zeros(1, math.ceil(self.max_len / PAGE), dtype=torch.int32, device="cuda")
        s.rows = torch.empty(tokens, 2, DIM // 2, device="cuda")
        s.qkv = torch.empty(tokens, Q_HEADS + 2 * HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        s.q = torch.empty(tokens, Q_HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        s.out = torch.empty(tokens, Q_HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        q, k, v = s.qkv[:, :Q_HEADS], s.qkv[:, Q_HEADS:Q_HEADS + HEADS], s.qkv[:, Q_HEADS + HEADS:]
        none = kvb.kv_vecs()
        s.angles = kvb.make_rotate_args(none, none, tokens, 0, DIM, kvb.KV_BF16, positions=s.positions.data_ptr(),
                                        rows_out=s.rows.data_ptr())
        s.append, s.attend = [], []
        for layer in range(LAYERS):
            s.append.append(kvb.make_append_args(
                kvb.vecs(k), kvb.vecs(v), kvb.vecs(q), kvb.vecs(s.q), tokens=tokens, q_heads=Q_HEADS, head_dim=DIM,
                dtype=kvb.KV_BF16, format=kvb.KV_CACHE_Q4, layer=layer, rows=s.rows.data_ptr(),
                slots=s.slots.data_ptr(), status=self.status.data_ptr()))
            s.attend.append(kvb.make_attend_args(
                kvb.vecs(s.q), kvb.vecs(s.out), q_start=s.q_start.data_ptr(), lens=s.length.data_ptr(),
                pages=s.table.data_ptr(), pages_stride=s.table.stride(0), requests=1, tokens=tokens, max_q=tokens,
                max_len=self.max_len, q_heads=Q_HEADS, head_dim=DIM, dtype=kvb.KV_BF16, layer=layer,
                scale=DIM ** -0.5, status=self.status.data_ptr()))
        need = kvb.kv_attend_workspace(self.pool, s.attend[0])
        s.workspace = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
        for a in s.attend:
            a.workspace, a.workspace_bytes = s.workspace.data_ptr(), need
        self.steps[tokens] = s
        return s

    def forward(self, s, stream: int | None = None):
        """One pass over the step's x, which is left as the stack's output."""
        kvb.kv_rotate(self.rotary, s.angles, stream)
        for layer in range(LAYERS):
            torch.mm(s.x, self.w_in[layer], out=s.qkv.view(s.x.shape[0], -1))
            kvb.kv_append(self.pool, self.rotary, s.append[layer], stream)
            kvb.kv_attend(self.pool, s.attend[layer], stream)
            s.x.addmm_(s.out.view(s.x.shape[0], -1), self.w_out[layer], beta=0.7, alpha=0.7)

    def close(self):
        torch.cuda.synchronize()
        kvb.kv_rotary_close(self.rotary)
        kvb.kv_pool_close(self.pool)


def main(prompt_tokens: int = 200, decode_tokens: int = 12, seed: int = 0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    n_pages = math.ceil((prompt_tokens + decode_tokens) / PAGE)
    stack = Stack(pages=3 * n_pages + 1, max_len=n_pages * PAGE, seed=seed)
    order = torch.randperm(stack.pages, generator=g, device="cuda").int()
    home, away = order[:n_pages], order[n_pages:2 * n_pages]
    inputs = torch.randn(prompt_tokens + decode_tokens, WIDTH, generator=g, device="cuda").bfloat16()

    def place(s, first: int, table):
        """Where the step's tokens stand and which pages hold them."""
        at = first + torch.arange(s.x.shape[0], device="cuda")
        s.x.copy_(inputs[first:first + s.x.shape[0]])
        s.positions.copy_(at)
        s.slots.copy_(table[at // PAGE].long() * PAGE + at % PAGE)
        s.length.fill_(first + s.x.shape[0])
        s.table[0, :n_pages].copy_(table)

    # 1. the prompt
    s = stack.step(prompt_tokens)
    place(s, 0, home)
    stack.forward(s)

    # 2. its pages to the host tier, and 3. back to other pages
    held = math.ceil(prompt_tokens / PAGE)
    tier = torch.empty(held * stack.page_bytes, dtype=torch.uint8, pin_memory=True)
    host = kvb.kv_host_register(tier.data_ptr(), tier.numel(), held, kvb.KV_NHD, stack.layout)
    torch.cuda.synchronize()
    slots = np.arange(held, dtype=np.int32)
    kvb.kv_fence_wait(kvb.kv_backup(stack.pool, host, home[:held].cpu().numpy(), slots), 10_000_000_000)
    kvb.kv_fence_wait(kvb.kv_restore(stack.pool, host, slots, away[:held].cpu().numpy()), 10_000_000_000)

    # decode in a captured graph, from either set of pages
    d = stack.step(1)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    place(d, prompt_tokens, home)
    stack.forward(d)                      # cuBLAS and the library make ready outside the capture
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        stack.forward(d, side.cuda_stream)
    outputs = []
    for table in (home, away):
        got = []
        for t in range(decode_tokens):
            place(d, prompt_tokens + t, table)
            graph.replay()
            got.append(d.x.clone())
        outputs.append(torch.cat(got))

    # what layer 0's pages hold, as 16-bit values
    k, v = torch.empty(2, prompt_tokens, HEADS, DIM, dtype=torch.bfloat16, device="cuda").unbind(0)
    at = torch.arange(prompt_tokens, device="cuda")
    where = away[at // PAGE].long() * PAGE + at % PAGE
    kvb.kv_fetch(stack.pool, kvb.make_fetch_args(kvb.vecs(k), kvb.vecs(v), tokens=prompt_tokens, head_dim=DIM, dtype=kvb.KV_BF16,
                                                 format=kvb.KV_CACHE_Q4, layer=0, slots=where.data_ptr()))
    torch.cuda.synchronize()
    status = int(stack.status)
    moved = held * stack.page_bytes
    kvb.kv_host_close(host)
    stack.close()
    return {"from_home": outputs[0], "from_restored": outputs[1], "keys": k, "values": v, "status": status,
            "bytes_moved": moved, "bytes_in_16_bits": held * PAGE * LAYERS * 2 * HEADS * DIM * 2}


if __name__ == "__main__":
    r = main()
    same = torch.equal(r["from_home"], r["from_restored"])
    print(f"decoded {r['from_home'].shape[0]} tokens from the pages and from their restored copies: "
          f"{'the same bytes' if same else 'DIFFERENT'}; status {r['status']}")
    print(f"host link: {r['bytes_moved']} bytes each way, {r['bytes_in_16_bits']} in 16 bits")
    sys.exit(0 if same and r["status"] == 0 else 1)
