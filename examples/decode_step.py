"""One decode step of a Kolibri-style decoder on libmoe: every layer is attention over a paged cache and
then the expert layer, on one bf16 residual stream.

    residual -> block_norm -> [q k v projection] -> kv_write -> attn_decode -> [output projection]
             -> block_norm (residual sum, next norm) -> moe_forward -> block_norm (post-norm, sum, next norm) ...

The two projections are plain library products.  Four of five layers see a sliding window of 513
tokens, every fifth the whole context ("We Ported Aleph Alpha's Kolibri to a MacBook. Our Own Gate
Said No.", section "The gate"; it gives no head counts, and the rotation of the windowed layers' queries
and keys is the caller's, between the projection and kv_write).  Weights are random.

    python examples/decode_step.py [--batch 64] [--context 4096] [--layers 5] [--steps 50] [--cache e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routed_expert_layer_fp32_gb300 as moe  # noqa: E402
from routed_expert_layer_fp32_gb300.binding import MOE_BF16, MOE_E4M3  # noqa: E402

WINDOW, FULL_EVERY = 513, 5


class Block:
    """One decoder layer's weights, its cache and its expert layer."""

    def __init__(self, experts: moe.Layer, heads: int, kv_heads: int, dim: int, n_pages: int, page: int, window: int,
                 cache_dtype: int, generator: torch.Generator):
        d = experts.d

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=generator, device="cuda") / rows ** 0.5).bfloat16()

        def gain():
            return 1 + 0.1 * torch.randn(d, generator=generator, device="cuda")

        self.experts, self.window = experts, window
        self.w_qkv, self.w_out = weight(d, (heads + 2 * kv_heads) * dim), weight(heads * dim, d)
        self.attn_norm, self.moe_norm, self.moe_post_norm = gain(), gain(), gain()
        self.cache = moe.KVCache.empty(n_pages, kv_heads, page, dim, cache_dtype)


class Decoder:
    """Fixed buffers for one token of each of `batch` sequences; write the step's embeddings into
    `residual`, then step().  `lens` and `pos` advance on the device, so a captured step replays."""

    def __init__(self, blocks, heads: int, kv_heads: int, dim: int, batch: int, page_table: torch.Tensor, alpha=0.5):
        self.blocks, self.heads, self.kv_heads, self.dim, self.alpha = blocks, heads, kv_heads, dim, alpha
        d = blocks[0].experts.d
        self.page_table = page_table
        self.residual = torch.zeros(batch, d, dtype=torch.bfloat16, device="cuda")
        self.pos = torch.zeros(batch, dtype=torch.int32, device="cuda")   # of the token this step writes
        self.lens = torch.ones(batch, dtype=torch.int32, device="cuda")   # with it
        self.x = torch.empty_like(self.residual)
        self.qkv = torch.empty(batch, (heads + 2 * kv_heads) * dim, dtype=torch.bfloat16, device="cuda")
        self.attn = torch.empty(batch, heads, dim, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(batch, d, dtype=torch.float32, device="cuda")
        self.proj = torch.empty_like(self.residual)
        self.ids = [torch.empty(batch, 6, dtype=torch.int32, device="cuda") for _ in blocks]
        self.wts = torch.empty(batch, 6, device="cuda")
        self.attn_ws = moe.attn_workspace(blocks[0].cache, heads, batch)
        self.moe_ws = moe.workspace(blocks[0].experts, batch)

    def step(self):
        h, hk, dim, batch = self.heads, self.kv_heads, self.dim, self.residual.shape[0]
        rows = self.qkv.view(batch, h + 2 * hk, dim)
        moe.block_norm(self.residual, self.blocks[0].attn_norm, out=self.x)
        for i, b in enumerate(self.blocks):
            torch.mm(self.x, b.w_qkv, out=self.qkv)
            moe.kv_write(rows[:, h:h + hk], rows[:, h + hk:], b.cache, self.pos, self.page_table, self.attn_ws)
            moe.attn_decode(rows[:, :h], b.cache, self.lens, self.page_table, self.attn_ws, window=b.window, out=self.attn)
            torch.mm(self.attn.view(batch, -1), b.w_out, out=self.proj)
            moe.block_norm(self.residual, b.moe_norm, y=self.proj, out=self.x)
            moe.forward(self.x, b.experts, self.moe_ws, out=self.y, ids=self.ids[i], w=self.wts)
            following = self.blocks[i + 1].attn_norm if i + 1 < len(self.blocks) else None
            moe.block_norm(self.residual, following, y=self.y, w_post=b.moe_post_norm, alpha=self.alpha,
                           out=None if following is None else self.x)
        self.pos += 1
        self.lens += 1
        return self.residual


def build(n_layers: int, batch: int, context: int, heads=16, kv_heads=4, dim=128, d=2048, ffn=640, experts=384, page=64,
          cache_dtype=MOE_E4M3, seed=1) -> Decoder:
    from gen import moegen
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-context // page)
    n_pages = batch * width
    table = torch.randperm(n_pages, generator=g, device="cuda").view(batch, width).int()
    # one set of expert weights, a copy at its own addresses for each layer
    layer = moe.Layer.from_host(moegen.make_layer(seed, d, ffn, experts, fp8=True, bias_var=0.5))
    blocks = [Block(layer if i == 0 else layer.clone(), heads, kv_heads, dim, n_pages, page,
                    0 if (i + 1) % FULL_EVERY == 0 else WINDOW, cache_dtype, g) for i in range(n_layers)]
    return Decoder(blocks, heads, kv_heads, dim, batch, table)


SPARE = 8  # positions kept for the warm-up steps


def arguments(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=5)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="e4m3")
    args = ap.parse_args(argv)
    for name in ("batch", "layers", "steps"):
        if getattr(args, name) < 1:
            ap.error(f"--{name} must be 1 at least")
    if args.context <= args.steps + SPARE:  # every timed step attends to a context, and stays in its pages
        ap.error(f"--context must be above --steps + {SPARE} ({args.steps + SPARE})")
    return args


def main():
    args = arguments()
    dec = build(args.layers, args.batch, args.context, cache_dtype=MOE_E4M3 if args.cache == "e4m3" else MOE_BF16)
    for b in dec.blocks:  # a context as if it had been decoded: random keys and values of every position
        g = torch.Generator(device="cuda").manual_seed(7)
        pos = torch.arange(args.context, dtype=torch.int32, device="cuda")
        for s in range(args.batch):
            kv = torch.randn(args.context, 2 * dec.kv_heads, dec.dim, generator=g, device="cuda").bfloat16()
            moe.kv_write(kv[:, :dec.kv_heads], kv[:, dec.kv_heads:], b.cache, pos, dec.page_table, dec.attn_ws,
                         seq=torch.full_like(pos, s))
    start = args.context - args.steps - SPARE
    embed = torch.randn_like(dec.residual)

    def rewind():
        dec.pos.fill_(start)
        dec.lens.fill_(start + 1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        rewind()
        dec.residual.copy_(embed)
        dec.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        dec.residual.copy_(embed)
        dec.step()
    rewind()
    for _ in range(3):
        graph.replay()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 1e3 / args.steps
    for ws in (dec.attn_ws, dec.moe_ws):
        if moe.get_status(ws) != 0:
            raise SystemExit("a device-side error was recorded")
    print(f"{args.layers} layers, batch {args.batch}, context {args.context}, {args.cache} cache: "
          f"{us:.1f} us a step, {args.batch * 1e6 / us:.0f} tokens/s")


if __name__ == "__main__":
    main()
