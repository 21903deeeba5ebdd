"""A small decoder served with the library: prompts, then one token at a time.

Each layer is attention and a mixture of experts, with random weights.  ``tl_cache_plan`` works out where new
tokens go: pages from a list of free ones, slots, positions, bounds.  Queries and keys pass through
``tl_norm_rope`` (a norm of each head and the rotation by position), K and V rows go into pages by
``tl_kv_append``.  A prompt's tokens then attend with ``tl_window_attention`` (every other layer with a sliding window
and sinks) to the rows read back by ``tl_kv_gather``, so that prompts and steps see the same 16-, 8- or 4-bit rows; a
step's tokens attend to the pages with ``tl_paged_attention``.  The experts run in ``tl_moe_combine`` for a prompt of more than
128 tokens and in ``tl_moe_tokens`` for the few tokens of a step, and ``tl_token_logprobs`` picks the next token with its log
probability.  A decoding step, from its plan to its next token, is captured into a CUDA graph once and replayed: lengths,
pages and tokens go on by themselves.  At the end the same tokens are run as prompts, and the logits of
every sequence's last token are compared.  They differ by activations' roundings, some 0.005; where a token's second and third
experts are as good as tied, a rounding can choose the other one, and then it is up to 0.1 (3 or 4 of 100 texts).

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
                 window=64, sinks=4, cache="bf16", seed=0):
        self.ctx, self.hidden, self.heads, self.kv, self.d, self.topk = ctx, hidden, heads, kv_heads, d, topk
        self.sinks, self.format = sinks, cache
        self.gen = gen = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") / math.sqrt(shape[-2])).to(BF)

        self.embed = torch.randn((vocab, hidden), generator=gen, device="cuda").to(BF)
        self.head = w(hidden, vocab)
        self.layers = [dict(qkv=w(hidden, (heads + 2 * kv_heads) * d), o=w(heads * d, hidden), router=w(hidden, experts),
                            gate=w(experts, hidden, ffn), up=w(experts, hidden, ffn), down=w(experts, ffn, hidden),
                            q_norm=1 + w(d, 1)[:, 0], k_norm=1 + w(d, 1)[:, 0],
                            window=window if i % 2 else 0) for i in range(layers)]
        self.freq = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
        # of an 8-bit cache 448 stands for 9, of a 4-bit one 6 times 448: values of rows whose mean square is 1 lie within
        scale = {"bf16": None, "e4m3": 0.02, "e2m1": 0.02 / 6}[cache]
        self.scale = None if scale is None else torch.full((kv_heads,), scale, device="cuda")
        few = tl.tl_moe_tokens_workspace_bytes(128, hidden, experts, ffn, topk)
        decode = tl.tl_paged_attention_workspace_bytes(256, heads, kv_heads, d)
        score = tl.tl_token_logprobs_workspace_bytes(256, vocab, 1)
        self.work = torch.zeros(max(few, decode, score), dtype=torch.uint8, device="cuda")  # one for all, in turn
        self.shape = (experts, ffn)

    def open(self, batch, longest, page=16):
        """Pages for `batch` sequences of up to `longest` tokens, all free, in any order."""
        self.page, per = page, -(-longest // page)
        pages, row = batch * per, (page, self.kv, self.d)
        if self.format == "e2m1":
            row = (page, self.kv, self.d // 2)
            blocks = [torch.zeros((pages, page, self.kv, self.d // 16), device="cuda").to(torch.float8_e4m3fn) for _ in range(2 * len(self.layers))]
        kind = {"bf16": BF, "e4m3": torch.float8_e4m3fn, "e2m1": torch.uint8}[self.format]
        self.cache = [[torch.zeros((pages, *row), device="cuda").to(kind) for _ in "kv"] for _ in self.layers]
        self.kinds = [dict(k_scale=self.scale, v_scale=self.scale) for _ in self.layers]
        if self.format == "e2m1":
            for i, k in enumerate(self.kinds):
                k.update(k_blocks=blocks[2 * i], v_blocks=blocks[2 * i + 1])
        ints = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.lengths, self.taken = ints(batch, per) - 1, ints(batch), ints(1)
        self.free = torch.randperm(pages, generator=self.gen, device="cuda").to(torch.int32)

    def plan(self, tokens, counts=None, rows=0):
        """Where `tokens` new rows go, and the slots of all `rows`; lengths, table and pages taken are brought up to date."""
        batch = self.lengths.numel()
        slots, positions, all_slots = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (tokens, tokens, rows))
        cu_q, cu_k = (torch.empty(batch + 1, dtype=torch.int32, device="cuda") for _ in "qk")
        tl.tl_cache_plan(self.ctx, self.lengths, self.table, self.page, self.free, self.taken, self.taken, self.lengths, cu_q, slots,
                         positions, counts=counts, cu_k=cu_k, kv_slots=all_slots if rows else None)
        return slots, positions, cu_q, cu_k, all_slots

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

    def qkv(self, layer, x, positions):
        rows = (self.norm(x) @ layer["qkv"]).view(-1, self.heads + 2 * self.kv, self.d)
        q, k, v = rows[:, :self.heads], rows[:, self.heads:self.heads + self.kv], rows[:, self.heads + self.kv:]
        tl.tl_norm_rope(self.ctx, q, k, positions, self.freq, q, k, q_weight=layer["q_norm"], k_weight=layer["k_norm"])
        return q, k, v

    def prompt(self, tokens, counts, rows):
        """Packed prompts of `counts` tokens each, after the rows that are there; `rows`: those of all sequences then.
        Logits of each sequence's last token."""
        slots, positions, cu_q, cu_k, all_slots = self.plan(tokens.numel(), counts, rows)
        x = self.embed[tokens]
        for layer, cache, kind in zip(self.layers, self.cache, self.kinds):
            q, k, v = self.qkv(layer, x, positions)
            tl.tl_kv_append(self.ctx, k, v, *cache, slots, **kind)
            keys, values = (torch.empty((rows, self.kv, self.d), dtype=BF, device="cuda") for _ in "kv")
            tl.tl_kv_gather(self.ctx, *cache, all_slots, keys, values, **kind)
            a = torch.empty((x.shape[0], self.heads, self.d), dtype=BF, device="cuda")
            tl.tl_window_attention(self.ctx, q, keys, values, cu_q, cu_k, a, window=layer["window"], sinks=self.sinks)
            x = self.experts(layer, (x.float() + (a.flatten(1) @ layer["o"]).float()).to(BF))
        return self.norm(x[cu_q[1:].long() - 1]) @ self.head

    def step(self, tokens):
        """One new token of each sequence: its logits."""
        slots, positions, *_ = self.plan(tokens.numel())
        x = self.embed[tokens]
        for layer, cache, kind in zip(self.layers, self.cache, self.kinds):
            q, k, v = self.qkv(layer, x, positions)
            tl.tl_kv_append(self.ctx, k, v, *cache, slots, **kind)
            a = torch.empty((x.shape[0], self.heads, self.d), dtype=BF, device="cuda")
            tl.tl_paged_attention(self.ctx, q, *cache, self.table, self.lengths, a, self.work, window=layer["window"],
                                  sinks=self.sinks, **kind)
            x = self.experts(layer, (x.float() + (a.flatten(1) @ layer["o"]).float()).to(BF))
        return self.norm(x) @ self.head

    def choose(self, logits):
        """The most likely token of each row, and its log probability."""
        n = logits.shape[0]
        ids, best = torch.empty((n, 1), dtype=torch.int32, device="cuda"), torch.empty((n, 1), device="cuda")
        tl.tl_token_logprobs(self.ctx, logits, None, None, self.work, top_logprobs=best, top_ids=ids)
        return ids[:, 0].long(), best[:, 0]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200, help="longest prompt")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--seed", type=int, default=0, help="of the prompts")
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    ap.add_argument("--e2m1", action="store_true", help="a 4-bit cache")
    a = ap.parse_args(argv)
    with tl.Context(0) as ctx:
        m = Decoder(ctx, cache="e2m1" if a.e2m1 else "e4m3" if a.e4m3 else "bf16")
        lens = torch.tensor([max(1, a.prompt - 37 * b) for b in range(a.batch)])
        gen = torch.Generator(device="cuda").manual_seed(a.seed)
        text = [torch.randint(0, 1000, (int(n),), generator=gen, device="cuda") for n in lens]

        def prompts(seqs):
            counts = torch.tensor([t.numel() for t in seqs], dtype=torch.int32)
            return m.prompt(torch.cat(seqs), counts.cuda(), int(counts.sum()))

        m.open(a.batch, a.prompt + a.steps + 2)
        new, _ = m.choose(prompts(text))

        # the step, captured once: it takes its tokens from `new` and leaves the next ones there
        state = [t.clone() for t in (m.table, m.lengths, m.taken, new)]
        scores = torch.zeros(a.batch, device="cuda")

        def step():
            logits = m.step(new)
            following, score = m.choose(logits)
            new.copy_(following)
            scores.add_(score)
            return logits

        step()  # warm up, and back
        for t, was in zip((m.table, m.lengths, m.taken, new), state):
            t.copy_(was)
        scores.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        fed = torch.empty((a.steps, a.batch), dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for i in range(a.steps):
            fed[i].copy_(new)
            graph.replay()
        torch.cuda.synchronize()
        took = (time.perf_counter() - t0) / max(1, a.steps)
        if ctx.check() != tl.TL_OK:
            raise RuntimeError("an index was out of range or a wait ran out")
        m.open(a.batch, a.prompt + a.steps + 2)
        again = prompts([torch.cat([t, fed[:, b]]) for b, t in enumerate(text)])
        off = float((out.float() - again.float()).norm() / again.float().norm())
        print(f"{a.steps} steps of {a.batch} sequences, {took * 1e6:.0f} us a step, log probability {float(scores.mean()):.2f} a sequence; "
              f"last logits against the whole text as a prompt: {off:.4f}")
        return off


if __name__ == "__main__":
    main()
