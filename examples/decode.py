"""A small decoder served with the library: prompts, then one token at a time.

Each layer is attention and a mixture of experts, with random weights.  A prompt's tokens go through
``tl_window_attention`` (every other layer with a sliding window and sinks), their K and V rows
into pages by ``tl_kv_append``; then every step appends one row per sequence and attends to the
pages with ``tl_paged_attention``.  The experts run in ``tl_moe_combine`` for a prompt of more than
128 tokens and in ``tl_moe_tokens`` for the few tokens of a step.  The decoding step is captured
into a CUDA graph once and replayed.  At the end the same tokens are run as prompts, and the logits of
every sequence's last token are compared.

    python examples/decode.py --batch 4 --prompt 200 --steps 16
"""
import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import communication_overlapped_gemm_gb300 as tl  # noqa: E402

BF = torch.bfloat16


class Decoder:
    """Weights, the paged cache of every layer, and the two ways through: prompts and steps."""

    def __init__(self, ctx, layers=2, hidden=512, heads=8, kv_heads=2, d=64, experts=16, ffn=256, topk=2, vocab=1000,
                 window=64, sinks=4, cache_dtype=BF, seed=0):
        self.ctx, self.hidden, self.heads, self.kv, self.d, self.topk = ctx, hidden, heads, kv_heads, d, topk
        self.sinks, self.cache_dtype = sinks, cache_dtype
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") / math.sqrt(shape[-2])).to(BF)

        self.embed = torch.randn((vocab, hidden), generator=gen, device="cuda").to(BF)
        self.head = w(hidden, vocab)
        self.layers = [dict(qkv=w(hidden, (heads + 2 * kv_heads) * d), o=w(heads * d, hidden), router=w(hidden, experts),
                            gate=w(experts, hidden, ffn), up=w(experts, hidden, ffn), down=w(experts, ffn, hidden),
                            window=window if i % 2 else 0) for i in range(layers)]
        self.scale = None if cache_dtype == BF else torch.full((kv_heads,), 0.02, device="cuda")
        few = tl.tl_moe_tokens_workspace_bytes(128, hidden, experts, ffn, topk)
        decode = tl.tl_paged_attention_workspace_bytes(256, heads, kv_heads, d)
        self.work = torch.zeros(max(few, decode), dtype=torch.uint8, device="cuda")  # one for both, in turn
        self.shape = (experts, ffn)

    def open(self, batch, longest, page=16):
        """Pages for `batch` sequences of up to `longest` tokens, in any order."""
        self.page, per = page, -(-longest // page)
        shape = (batch * per, page, self.kv, self.d)
        self.cache = [[torch.zeros(shape, dtype=BF, device="cuda").to(self.cache_dtype) for _ in "kv"] for _ in self.layers]
        self.table = torch.randperm(batch * per, device="cuda").to(torch.int32).view(batch, per)

    def slots(self, seq, pos):
        page = torch.div(pos, self.page, rounding_mode="floor")
        return (self.table[seq, page] * self.page + pos % self.page).to(torch.int32)

    def norm(self, x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(BF)

    def experts(self, layer, x):
        h = self.norm(x)
        logits, out = (h @ layer["router"]).float(), torch.empty(x.shape, dtype=torch.float32, device="cuda")
        args = (self.ctx, h, logits, self.topk, layer["gate"], layer["up"], layer["down"], out)
        if x.shape[0] <= 128:
            tl.tl_moe_tokens(*args, self.work)
        else:
            n = tl.tl_moe_workspace_bytes(x.shape[0], self.hidden, self.shape[0], self.shape[1], self.topk)
            tl.tl_moe_combine(*args, torch.zeros(n, dtype=torch.uint8, device="cuda"))
        return (x.float() + out).to(BF)

    def qkv(self, layer, x):
        rows = (self.norm(x) @ layer["qkv"]).view(-1, self.heads + 2 * self.kv, self.d)
        return rows[:, :self.heads], rows[:, self.heads:self.heads + self.kv], rows[:, self.heads + self.kv:]

    def prompt(self, tokens, cu, slots=None):
        """Packed prompts; their rows go into the cache at `slots`.  Logits of each sequence's last token."""
        x = self.embed[tokens]
        for layer, cache in zip(self.layers, self.cache):
            q, k, v = self.qkv(layer, x)
            if slots is not None:
                tl.tl_kv_append(self.ctx, k, v, *cache, slots, k_scale=self.scale, v_scale=self.scale)
            a = torch.empty((x.shape[0], self.heads, self.d), dtype=BF, device="cuda")
            tl.tl_window_attention(self.ctx, q, k, v, cu, cu, a, window=layer["window"], sinks=self.sinks)
            x = self.experts(layer, (x.float() + (a.flatten(1) @ layer["o"]).float()).to(BF))
        return self.norm(x[cu[1:].long() - 1]) @ self.head

    def step(self, tokens, slots, lengths):
        """One new token of each sequence; `lengths` count it."""
        x = self.embed[tokens]
        for layer, cache in zip(self.layers, self.cache):
            q, k, v = self.qkv(layer, x)
            tl.tl_kv_append(self.ctx, k, v, *cache, slots, k_scale=self.scale, v_scale=self.scale)
            a = torch.empty((x.shape[0], self.heads, self.d), dtype=BF, device="cuda")
            tl.tl_paged_attention(self.ctx, q, *cache, self.table, lengths, a, self.work, window=layer["window"],
                                  sinks=self.sinks, k_scale=self.scale, v_scale=self.scale)
            x = self.experts(layer, (x.float() + (a.flatten(1) @ layer["o"]).float()).to(BF))
        return self.norm(x) @ self.head


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200, help="longest prompt")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = ap.parse_args(argv)
    with tl.Context(0) as ctx:
        m = Decoder(ctx, cache_dtype=torch.float8_e4m3fn if a.e4m3 else BF)
        lens = torch.tensor([max(1, a.prompt - 37 * b) for b in range(a.batch)])
        m.open(a.batch, a.prompt + a.steps + 1)
        text = [torch.randint(0, 1000, (int(n),), device="cuda") for n in lens]

        def packed(seqs):
            cu = torch.zeros(len(seqs) + 1, dtype=torch.int32)
            cu[1:] = torch.tensor([t.numel() for t in seqs]).cumsum(0)
            return torch.cat(seqs), cu.cuda()

        tokens, cu = packed(text)
        seq = torch.repeat_interleave(torch.arange(a.batch), lens).cuda()
        logits = m.prompt(tokens, cu, m.slots(seq, torch.cat([torch.arange(int(n)) for n in lens]).cuda()))

        # the step, captured once
        new, lengths = logits.argmax(-1), (lens + 1).to(torch.int32).cuda()
        slots = m.slots(torch.arange(a.batch, device="cuda"), lengths.long() - 1)
        m.step(new, slots, lengths)  # warm up
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = m.step(new, slots, lengths)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for i in range(a.steps):
            if i:
                new.copy_(out.argmax(-1))
                lengths += 1
                slots.copy_(m.slots(torch.arange(a.batch, device="cuda"), lengths.long() - 1))
            text = [torch.cat([t, n[None]]) for t, n in zip(text, new)]
            graph.replay()
        torch.cuda.synchronize()
        took = (time.perf_counter() - t0) / max(1, a.steps)
        if ctx.check() != tl.TL_OK:
            raise RuntimeError("an index was out of range or a wait ran out")
        again = m.prompt(*packed(text))
        off = float((out.float() - again.float()).norm() / again.float().norm())
        print(f"{a.steps} steps of {a.batch} sequences, {took * 1e6:.0f} us a step; "
              f"last logits against the whole text as a prompt: {off:.4f}")
        return off


if __name__ == "__main__":
    main()
