"""One decode step of a Kolibri-style decoder on libmoe: every layer is attention over a paged cache and
then the expert layer, on one bf16 residual stream.

    residual -> block_norm -> [q k v projection] -> kv_write -> attn_decode -> [output projection]
             -> block_norm (residual sum, next norm) -> moe_forward -> block_norm (post-norm, sum, next norm) ...

The two projections are plain library products.  Four of five layers see a sliding window of 513
tokens, every fifth the whole context ("We Ported Aleph Alpha's Kolibri to a MacBook. Our Own Gate
Said No.", section "The gate"; it gives no head counts, and says nothing of how the windowed layers'
queries and keys are turned).  Weights are random.

With --serve the pages come from a pool that the sequences share: each step plans its tokens' places on the GPU
(page_plan), the windowed layers turn queries and keys on the way into the cache (rope_kv_write), and sequences that
have ended give their pages back (page_release); all of a step is in one CUDA graph, pages that it hands out included.

    python examples/decode_step.py [--batch 64] [--context 4096] [--layers 5] [--steps 50] [--cache e4m3] [--serve]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import routed_expert_layer_fp32_gb300 as moe  # noqa: E402
from routed_expert_layer_fp32_gb300.binding import MOE_BF16, MOE_E4M3, MOE_INT4  # noqa: E402

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

    def place(self, b, q, k, v):
        """k and v of this step's tokens into the block's cache; the queries that attend to it."""
        moe.kv_write(k, v, b.cache, self.pos, self.page_table, self.attn_ws)
        return q

    def step(self):
        h, hk, dim, batch = self.heads, self.kv_heads, self.dim, self.residual.shape[0]
        rows = self.qkv.view(batch, h + 2 * hk, dim)
        moe.block_norm(self.residual, self.blocks[0].attn_norm, out=self.x)
        for i, b in enumerate(self.blocks):
            torch.mm(self.x, b.w_qkv, out=self.qkv)
            q = self.place(b, rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:])
            moe.attn_decode(q, b.cache, self.lens, self.page_table, self.attn_ws, window=b.window, out=self.attn)
            torch.mm(self.attn.view(batch, -1), b.w_out, out=self.proj)
            moe.block_norm(self.residual, b.moe_norm, y=self.proj, out=self.x)
            moe.forward(self.x, b.experts, self.moe_ws, out=self.y, ids=self.ids[i], w=self.wts)
            following = self.blocks[i + 1].attn_norm if i + 1 < len(self.blocks) else None
            moe.block_norm(self.residual, following, y=self.y, w_post=b.moe_post_norm, alpha=self.alpha,
                           out=None if following is None else self.x)
        self.advance()
        return self.residual

    def advance(self):
        self.pos += 1
        self.lens += 1


class Server(Decoder):
    """A Decoder whose sequences share a pool of pages and whose windowed layers turn queries and keys.  `lens` are the
    tokens in the cache, and pos and slot those of the step's tokens, all on the device: admit() and step() plan them.
    A row whose sequence was released is idle until a prompt is admitted to it: it has pos and slot -1, length 0 and no
    pages, and its output means nothing."""

    def __init__(self, blocks, heads, kv_heads, dim, batch, width: int, rope: moe.Rope, alpha=0.5):
        table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        super().__init__(blocks, heads, kv_heads, dim, batch, table, alpha)
        cache = blocks[0].cache
        self.rope, self.page, self.n_pages = rope, cache.page_size, cache.n_pages
        self.lens.zero_()
        self.free = torch.arange(self.n_pages, dtype=torch.int32, device="cuda")
        self.n_free = torch.full((1,), self.n_pages, dtype=torch.int32, device="cuda")
        # a plan's list has the tokens of busy rows one after the other (its parts 16-byte aligned)
        self.places = torch.full((2, -(-batch // 4) * 4), -1, dtype=torch.int32, device="cuda")
        self.rows = torch.full((2, batch), -1, dtype=torch.int32, device="cuda")
        self.pos, self.slot = self.rows
        self.seq = torch.empty(batch, dtype=torch.int32, device="cuda")
        self.starts = torch.empty(batch + 1, dtype=torch.int32, device="cuda")
        self.busy = torch.ones(batch, dtype=torch.int32, device="cuda")  # tokens a step of each row
        self.idle = torch.zeros(batch, dtype=torch.bool, device="cuda")
        self.plan_ws = moe.pages_workspace(batch)

    def admit(self, new_tokens: torch.Tensor, max_tokens: int) -> moe.PagePlan:
        """Places for new_tokens[b] tokens of each sequence (the prompts').  An idle row that gets some is busy."""
        plan = moe.page_plan(self.lens, new_tokens, self.page_table, self.free, self.n_free, self.page, self.n_pages,
                             max_tokens, self.plan_ws)
        self._idle(self.idle & ~((new_tokens > 0) & (self.lens > 0)))  # (one that found no pages has length 0)
        return plan

    def release(self, ended: torch.Tensor):
        moe.page_release(self.lens, ended, self.page_table, self.free, self.n_free, self.page, self.plan_ws)
        self._idle(self.idle | (ended != 0))

    def _idle(self, rows: torch.Tensor):
        self.idle.copy_(rows)
        self.busy.copy_(~rows)

    def place(self, b, q, k, v):
        if b.window == 0:  # the layers of the whole context know no positions
            return super().place(b, q, k, v)
        return moe.rope_kv_write(q, k, v, b.cache, self.rope, self.pos, self.slot, self.attn_ws, q_out=q)

    def step(self):
        batch = self.busy.shape[0]
        moe.page_plan(self.lens, self.busy, self.page_table, self.free, self.n_free, self.page, self.n_pages, batch,
                      self.plan_ws, starts=self.starts, seq=self.seq, pos=self.places[0, :batch], slot=self.places[1, :batch])
        # from the list to the rows (a row without a token begins where the next one does, at its own number at most)
        torch.index_select(self.places, 1, self.starts[:-1], out=self.rows)
        self.rows.masked_fill_(self.idle, -1)
        return super().step()

    def advance(self):
        pass  # the plan has


def build(n_layers: int, batch: int, context: int, heads=16, kv_heads=4, dim=128, d=2048, ffn=640, experts=384, page=64,
          cache_dtype=MOE_E4M3, seed=1, serve=False) -> Decoder:
    from gen import moegen
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = -(-context // page)
    n_pages = batch * width
    table = torch.randperm(n_pages, generator=g, device="cuda").view(batch, width).int()
    # one set of expert weights, a copy at its own addresses for each layer
    layer = moe.Layer.from_host(moegen.make_layer(seed, d, ffn, experts, fp8=True, bias_var=0.5))
    blocks = [Block(layer if i == 0 else layer.clone(), heads, kv_heads, dim, n_pages, page,
                    0 if (i + 1) % FULL_EVERY == 0 else WINDOW, cache_dtype, g) for i in range(n_layers)]
    if serve:
        return Server(blocks, heads, kv_heads, dim, batch, width, moe.Rope(dim))
    return Decoder(blocks, heads, kv_heads, dim, batch, table)


SPARE = 8  # positions kept for the warm-up steps


def arguments(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--layers", type=int, default=5)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--cache", choices=("bf16", "e4m3", "int4"), default="e4m3")
    ap.add_argument("--serve", action="store_true")
    args = ap.parse_args(argv)
    for name in ("batch", "layers", "steps"):
        if getattr(args, name) < 1:
            ap.error(f"--{name} must be 1 at least")
    if args.context <= args.steps + SPARE:  # every timed step attends to a context, and stays in its pages
        ap.error(f"--context must be above --steps + {SPARE} ({args.steps + SPARE})")
    return args


PART = 1 << 16  # tokens that fill() writes at a time (a call of the library takes up to 2^20)


def fill(dec: Decoder, context: int, start: int):
    """A context as if it had been decoded: random keys and values of every position."""
    h, hk, batch = dec.heads, dec.kv_heads, dec.residual.shape[0]
    serving = isinstance(dec, Server)
    generators = [torch.Generator(device="cuda").manual_seed(7) for _ in dec.blocks]
    n = start if serving else context
    for s in range(batch):
        for first in range(0, n, PART):
            pos = torch.arange(first, min(n, first + PART), dtype=torch.int32, device="cuda")
            if serving:
                new = torch.zeros(batch, dtype=torch.int32, device="cuda")
                new[s] = len(pos)
                plan = dec.admit(new, len(pos))
            for b, g in zip(dec.blocks, generators):
                x = torch.randn(len(pos), h + 2 * hk, dec.dim, generator=g, device="cuda").bfloat16()
                q, k, v = x[:, :h], x[:, h:h + hk], x[:, h + hk:]
                if serving and b.window:
                    moe.rope_kv_write(q, k, v, b.cache, dec.rope, plan.pos, plan.slot, dec.attn_ws, q_out=q)
                else:
                    moe.kv_write(k, v, b.cache, pos, dec.page_table, dec.attn_ws, seq=torch.full_like(pos, s))


def main():
    args = arguments()
    dec = build(args.layers, args.batch, args.context, serve=args.serve,
                cache_dtype={"bf16": MOE_BF16, "e4m3": MOE_E4M3, "int4": MOE_INT4}[args.cache])
    start = args.context - args.steps - SPARE
    fill(dec, args.context, start)
    embed = torch.randn_like(dec.residual)

    def rewind():
        if not args.serve:  # (a server's steps go on: their pages are handed out)
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
    for ws in (dec.attn_ws, dec.moe_ws) + ((dec.plan_ws,) if args.serve else ()):
        if moe.get_status(ws) != 0:
            raise SystemExit("a device-side error was recorded")
    print(f"{args.layers} layers, batch {args.batch}, context {args.context}, {args.cache} cache{', serving' * args.serve}: "
          f"{us:.1f} us a step, {args.batch * 1e6 / us:.0f} tokens/s")


if __name__ == "__main__":
    main()
