"""What a serving step needs around its attention and experts, with the plain forms: what is timed and compared.

Five operators work on one paged key/value cache and one step's tokens:

  plan    page tables, slots, positions and bounds of a step, from the sequences' lengths
  rope    norms of queries and keys for each head, and the rotation by their positions
  store   new K/V rows written into a cache held in 4 bits, and read back as packed rows
  attend  attention of one new token of each sequence over a cache held in 4 bits
  score   log probabilities of chosen tokens, with the entropy and the most likely alternatives

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits (angles in 64); with
``own`` true it calls the library.

4 bits: a row is held as codes of the values 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (two a byte, the lower half
first), with an e4m3 scale b for every 16 values and one fp32 scale s for each kv head; a code c stands for c b s.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_E4M3 = torch.float8_e4m3fn
_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------- cases
def _case(name, base, kw):
    c = dict(base)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _attend(name, **kw):
    return _case(name, dict(op="attend", batch=1, longest=1, shortest=1, heads=32, kv_heads=8, d=128, page=16, dtype="bf16",
                            window=0, sinks=0, head_major=False), kw)


def _store(name, **kw):
    return _case(name, dict(op="store", tokens=1, kv_heads=8, d=128, page=16, dtype="bf16", head_major=False, padding=0), kw)


def _rope(name, **kw):
    return _case(name, dict(op="rope", tokens=1, farthest=0, heads=32, kv_heads=8, d=128, rotary=128, dtype="bf16", norm=True,
                            interleaved=False, base=10000.0), kw)


def _plan(name, **kw):
    return _case(name, dict(op="plan", batch=1, longest=0, most_new=1, page=16, padding=0, all_rows=False), kw)


def _score(name, **kw):
    return _case(name, dict(op="score", rows=1, vocab=131072, dtype="fp32", top=0, temperature=1.0, masked=0.0, padding=0), kw)


def listed():
    return [
        # one user's chat over a long history
        _attend("attend one sequence 8k", longest=8192, shortest=8192),
        # a large serving batch whose cache takes most of the memory: ragged lengths, larger head-major pages
        _attend("attend batch 128 to 16k", batch=128, longest=16384, heads=64, page=64, head_major=True),
        # a sliding-window layer: an odd group size, odd pages, few visible keys
        _attend("attend window fp16 batch 7", batch=7, longest=33001, shortest=100, heads=28, kv_heads=4, d=64, page=7,
                dtype="fp16", window=1000, sinks=5),
        # one decoding step's new rows, padded to a captured batch size
        _store("store one step of 64", tokens=64, padding=3),
        # a long prompt's rows, and all of them back for the attention of a later turn
        _store("store prompt 8k", tokens=8192, page=64, head_major=True),
        # one decoding step, far into its sequences
        _rope("rope one step of 64", tokens=64, farthest=131072),
        # a long prompt
        _rope("rope prompt 8k", tokens=8192),
        # one decoding step of a batch
        _plan("plan one step of 64", batch=64, longest=8192, padding=3),
        # prompts, some of them later turns, with the slots of all their rows for reading back
        _plan("plan prompts to 4k", batch=37, longest=6001, most_new=4096, all_rows=True),
        # one user's next token with its alternatives, as an API returns them
        _score("score one row", top=20),
        # a decoding batch over 16-bit logits (ties), most of the vocabulary masked out by a grammar
        _score("score 64 rows bf16", rows=64, dtype="bf16", top=5, temperature=0.7, masked=0.6, padding=3),
        # the log probabilities of a prompt, a vocabulary that no vector divides
        _score("score prompt 2k", rows=2048, vocab=50001, top=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "store", "rope", "rope", "plan", "score", "score"))
    dtype = rng.choice(("bf16", "fp16"))
    kv, d = rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
    if op == "attend":
        g, batch = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16)), _log(rng, 1, 128)
        longest = min(_log(rng, 1, 33000), max(1, 128 * 8192 * 8 * 128 // (batch * kv * d)))
        longest = min(longest, max(1, (1 << 33) // (batch * kv * max(g, d))))
        win = _log(rng, 1, 4096) if rng.random() < 0.4 else 0
        return _attend(None, batch=batch, longest=longest, shortest=rng.randint(0, longest), heads=kv * g, kv_heads=kv, d=d,
                       page=rng.choice((1, 5, 8, 16, 32, 64, 100)), dtype=dtype, window=win,
                       sinks=rng.choice((0, 1, 4, 130)) if win else 0, head_major=rng.random() < 0.5)
    if op == "store":
        return _store(None, tokens=_log(rng, 1, 8192), kv_heads=kv, d=d, page=rng.choice((1, 5, 16, 64)), dtype=dtype,
                      head_major=rng.random() < 0.5, padding=rng.choice((0, 2)))
    if op == "rope":
        tokens = _log(rng, 1, 8192)
        return _rope(None, tokens=tokens, farthest=rng.choice((0, 0, _log(rng, 1, 1 << 20))), heads=kv * rng.choice((1, 2, 3, 4, 8)),
                     kv_heads=kv, d=d, rotary=rng.choice((d, d, d // 2, 16)), dtype=dtype, norm=rng.random() < 0.7,
                     interleaved=rng.random() < 0.4, base=rng.choice((10000.0, 500000.0)))
    if op == "plan":
        batch = _log(rng, 1, 1000)
        return _plan(None, batch=batch, longest=_log(rng, 1, 16384), most_new=_log(rng, 1, max(1, 65536 // batch)),
                     page=rng.choice((1, 5, 16, 64, 100)), padding=rng.choice((0, 5)), all_rows=rng.random() < 0.5)
    vocab = _log(rng, 300, 200000)
    return _score(None, rows=_log(rng, 1, min(2048, 2048 * 50001 // vocab)), vocab=vocab, dtype=rng.choice(("fp32", "bf16", "fp16")),
                  top=rng.choice((0, 1, 5, 20, 32)), temperature=rng.choice((1.0, 0.6, 1.3)), masked=rng.choice((0.0, 0.0, 0.9)),
                  padding=rng.choice((0, 1)))


# ---------------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """The lengths of a case's sequences, the longest first: the same for every seed, which only orders them anew."""
    low = case.get("shortest", 0)
    lens = torch.randint(low, case["longest"] + 1, (case["batch"],), generator=torch.Generator().manual_seed(7))
    lens[0] = case["longest"]
    return lens


def _counts(case):
    """New tokens of each sequence of a plan: one in a step, ragged in prompts, none in a padded row."""
    new = torch.randint(1, case["most_new"] + 1, (case["batch"],), generator=torch.Generator().manual_seed(9))
    new[-1] = case["most_new"]
    new[:min(case["padding"], case["batch"] - 1)] = 0
    return new


def _put(t, head_major):
    """A pool [pages, page, kv_heads, n] in memory as it is, or with each page's rows of a head together."""
    return t.transpose(1, 2).contiguous().transpose(1, 2) if head_major else t


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="bf16", std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(_DT[dtype])

    def pools(pages):
        """K and V of so many pages: rows of N(0, 0.5) in 4 bits."""
        kv, p, d = case["kv_heads"], case["page"], case["d"]
        for w in ("k", "v"):
            s[w + "_scale"] = torch.rand(kv, generator=gen, device="cuda") * 0.0005 + 0.001  # about amax / (6 448)
            codes = torch.empty((pages, p, kv, d // 2), dtype=torch.uint8, device="cuda")
            blocks = torch.empty((pages, p, kv, d // 16), dtype=_E4M3, device="cuda")
            step = max(1, (1 << 28) // (p * kv * d))
            for at in range(0, pages, step):
                rows = torch.randn((min(step, pages - at), p, kv, d), generator=gen, device="cuda") * 0.5
                c, b = _to_4_bits(rows, s[w + "_scale"])
                codes[at:at + step], blocks.view(torch.uint8)[at:at + step] = c, b.view(torch.uint8)
            s[w + "_cache"], s[w + "_blocks"] = _put(codes, case["head_major"]), _put(blocks, case["head_major"])

    s = dict(case)
    if case["op"] == "attend":
        lens = _lengths(case)[torch.randperm(case["batch"], generator=host)]
        need = (lens + case["page"] - 1) // case["page"]
        total, most = int(need.sum()), int(need.max())
        order = torch.randperm(total, generator=host).to(torch.int32)  # pages of a used cache come in any order
        table = torch.full((case["batch"], max(most, 1)), -1, dtype=torch.int32)
        table[torch.arange(table.shape[1])[None, :] < need[:, None]] = order
        pools(max(total, 1))
        s["q"] = normal(case["batch"], case["heads"], case["d"], dtype=case["dtype"])
        s["table"], s["lengths"] = table.cuda(), lens.to(torch.int32).cuda()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["batch"], case["heads"]), device="cuda")
    elif case["op"] == "store":
        n = case["tokens"]
        pages = (n + n // 2) // case["page"] + 2
        slots = torch.randperm(pages * case["page"], generator=host)[:n].to(torch.int32)
        if case["padding"]:
            slots[-case["padding"]:] = -1
        s["slots"] = slots.cuda()
        kv = normal(n, 2 * case["kv_heads"], case["d"], dtype=case["dtype"], std=0.5)
        s["k"], s["v"] = kv[:, :case["kv_heads"]], kv[:, case["kv_heads"]:]  # views of one projection's output
        pools(pages)
        s["k_rows"], s["v_rows"] = (torch.zeros(s["k"].shape, dtype=s["k"].dtype, device="cuda") for _ in "kv")
    elif case["op"] == "rope":
        n, hq, hk, d, r = case["tokens"], case["heads"], case["kv_heads"], case["d"], case["rotary"]
        qkv = normal(n, hq + 2 * hk, d, dtype=case["dtype"], std=1.5)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"], s["k_weight"] = (normal(d, dtype=case["dtype"], std=0.2) + 1 if case["norm"] else None for _ in "qk")
        at = torch.randint(0, case["farthest"] + 1, (n,), generator=host) if case["farthest"] else torch.arange(n)
        s["positions"] = at.to(torch.int32).cuda()
        s["inv_freq"] = (1.0 / case["base"] ** (torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
        s["q_out"] = torch.empty((n, hq, d), dtype=_DT[case["dtype"]], device="cuda")
        s["k_out"] = torch.empty((n, hk, d), dtype=_DT[case["dtype"]], device="cuda")
    elif case["op"] == "plan":
        order, p = torch.randperm(case["batch"], generator=host), case["page"]
        lens, new = _lengths(case)[order], _counts(case)[order]
        has, needs = (lens + p - 1) // p, (lens + new + p - 1) // p
        pages = torch.randperm(int(needs.sum()) + 16, generator=host).to(torch.int32)
        used = int(has.sum())
        table = torch.full((case["batch"], int(needs.max()) + 2), -1, dtype=torch.int32)
        table[torch.arange(table.shape[1])[None, :] < has[:, None]] = pages[:used]
        s["table"], s["lengths"], s["counts"] = table.cuda(), lens.to(torch.int32).cuda(), new.to(torch.int32).cuda()
        # pages that were given out before lie ahead of the free ones
        s["free_pages"] = torch.cat([pages[:3].clone().fill_(-1), pages[used:]]).cuda()
        s["taken"] = torch.tensor([3], dtype=torch.int32, device="cuda")
        ints = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        n = int(new.sum()) + case["padding"]
        s["slots"], s["positions"], s["cu_q"], s["cu_k"] = ints(n), ints(n), ints(case["batch"] + 1), ints(case["batch"] + 1)
        s["new_lengths"], s["taken_out"] = ints(case["batch"]), ints(1)
        s["kv_slots"] = ints(int((lens + new).sum()) + case["padding"]) if case["all_rows"] else None
    else:
        n, v = case["rows"], case["vocab"]
        x = torch.randn((n, v), generator=gen, device="cuda") * 2.0
        likely = torch.randint(0, v, (n, 12), generator=gen, device="cuda")  # a model's few good tokens
        x.scatter_add_(1, likely, torch.rand((n, 12), generator=gen, device="cuda") * 12.0)
        if case["masked"]:
            x[:, torch.rand(v, generator=gen, device="cuda") < case["masked"]] = -math.inf
        x[torch.arange(n, device="cuda"), likely[:, 0]] = 9.0  # the target is never masked
        s["logits"] = x.to(_DT[case["dtype"]])
        t = likely[:, 0].to(torch.int32)
        if case["padding"] and n > 1:
            t[-case["padding"]:] = -1
        s["targets"] = t
        for w in ("logprob", "entropy"):
            s[w] = torch.zeros(n, device="cuda")
        s["top_logprobs"] = torch.zeros((n, case["top"]), device="cuda")
        s["top_ids"] = torch.zeros((n, case["top"]), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _to_4_bits(x, scale):
    """Rows [..., kv_heads, d] in 32 bits as codes [..., kv_heads, d / 2] and e4m3 scales [..., kv_heads, d / 16]."""
    x, s = x.unflatten(-1, (-1, 16)), scale[:, None]
    b = (x.abs().amax(-1) / (6.0 * s)).clamp(max=448.0).to(_E4M3)
    t = (b.float() * s)[..., None]
    q = torch.where(t == 0.0, 0.0, x / t)
    a = q.abs()  # ties go to the even code
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    c = (c + 8 * torch.signbit(q)).to(torch.uint8).flatten(-2)
    return c[..., ::2] | (c[..., 1::2] << 4), b


def _from_4_bits(codes, blocks):
    """What codes and block scales stand for, before the head's scale, in 32 bits."""
    c = torch.tensor(_CODES + tuple(-x for x in _CODES), device="cuda")
    pairs = torch.stack([c.repeat(16), c.repeat_interleave(16)], -1)  # of each byte
    x = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (x * blocks.float()[..., None]).flatten(-2)


def _pages_of(s, w):
    """[batch, places, kv_heads, d] in 32 bits: the rows of each sequence in order."""
    t = s["table"].clamp(min=0).long()
    x = _from_4_bits(s[w + "_cache"][t].flatten(1, 2), s[w + "_blocks"].view(torch.uint8)[t].view(_E4M3).flatten(1, 2))
    return x * s[w + "_scale"][:, None]


def _plain_attend(s):
    b, hq, d = s["q"].shape
    hk = s["kv_heads"]
    k, v = _pages_of(s, "k"), _pages_of(s, "v")
    at = torch.arange(k.shape[1], device="cuda")[None, :]
    n = s["lengths"].long()[:, None]
    seen = at < n
    v = torch.where(seen[:, :, None, None], v, 0.0)
    if s["window"]:
        seen = seen & ((at >= n - s["window"]) | (at < s["sinks"]))
    q = s["q"].float().reshape(b, hk, hq // hk, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    scores = torch.where(seen[:, None, None, :], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = (scores - top).exp()
    total = w.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    out = torch.matmul(w / torch.where(total == 0, 1.0, total), v.transpose(1, 2)).reshape(b, hq, d)
    return {"out": out.to(s["q"].dtype), "lse": lse.reshape(b, hq)}


def _plain_store(s):
    return {**_stored(s, "k"), **_stored(s, "v")}


def _stored(s, w):
    cache, blocks, out = s[w + "_cache"], s[w + "_blocks"].view(torch.uint8), s[w + "_rows"]
    live = s["slots"] >= 0
    keep = live.nonzero().squeeze(1)  # (a padded token writes nothing)
    at = s["slots"][keep].long()
    page, row = at // s["page"], at % s["page"]
    c, b = _to_4_bits(s[w][keep].float(), s[w + "_scale"])
    cache[page, row], blocks[page, row] = c, b.view(torch.uint8)
    x = _from_4_bits(cache[page, row], blocks[page, row].view(_E4M3)) * s[w + "_scale"][:, None]
    out[keep] = x.to(out.dtype)
    return {w + "_rows": out, w + "_blocks": s[w + "_blocks"]}


def _plain_rope(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    c, n = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return {"q": _turned(s, s["q"], s["q_weight"], c, n), "k": _turned(s, s["k"], s["k_weight"], c, n)}


def _turned(s, rows, weight, c, n):
    x, r = rows.float(), s["rotary"]
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    if s["interleaved"]:
        a, b = x[..., :r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * n, a * n + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * n, a * n + b * c], -1)
    return torch.cat([y, x[..., r:]], -1).to(rows.dtype)


def _plain_plan(s):
    p, lens, new = s["page"], s["lengths"].long(), s["counts"].long()
    has, needs = (lens + p - 1) // p, (lens + new + p - 1) // p
    start = (needs - has).cumsum(0) - (needs - has) + s["taken"].long()
    col = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (col >= has[:, None]) & (col < needs[:, None])
    at = (start[:, None] + col - has[:, None]).clamp(0, s["free_pages"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free_pages"][at], s["table"]))
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu_q, cu_k = torch.cat([zero, new.cumsum(0)]), torch.cat([zero, (lens + new).cumsum(0)])

    def places(cu, first, n):
        """Of each of n packed tokens: its slot and its position (past the last one: -1 and 0)."""
        t = torch.arange(n, device="cuda")
        b = torch.searchsorted(cu[1:], t, right=True).clamp(max=cu.numel() - 2)
        pos = torch.where(t < cu[-1], first[b] + t - cu[b], 0)
        slot = s["table"][b, pos // p].long() * p + pos % p
        return torch.where(t < cu[-1], slot, -1).int(), pos.int()

    slots, positions = places(cu_q, lens, s["slots"].numel())
    got = {"table": s["table"], "slots": slots, "positions": positions, "cu_q": cu_q.int(), "cu_k": cu_k.int(),
           "lengths": (lens + new).int(), "taken": (s["taken"] + (needs - has).sum()).int()}
    if s["kv_slots"] is not None:
        got["kv_slots"] = places(cu_k, torch.zeros_like(lens), s["kv_slots"].numel())[0]
    return got


def _plain_score(s):
    x = s["logits"].float() * (1.0 / s["temperature"])
    m = x.amax(-1, keepdim=True)
    y = x - m
    w = y.exp()
    total = w.sum(-1, keepdim=True)
    lse = total.log()
    seen = w > 0
    entropy = lse.squeeze(1) - (torch.where(seen, w, 0.0) * torch.where(seen, y, 0.0)).sum(-1) / total.squeeze(1)
    live = s["targets"] >= 0
    chosen = torch.gather(y - lse, 1, s["targets"].clamp(min=0).long()[:, None]).squeeze(1)
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :s["top"]]  # ties: the lower index
    best = torch.gather(y - lse, 1, ids)
    return {"logprob": torch.where(live, chosen, s["logprob"]), "entropy": torch.where(live, entropy, s["entropy"]),
            "top_logprobs": torch.where(live[:, None], best, s["top_logprobs"]),
            "top_ids": torch.where(live[:, None], ids.int(), s["top_ids"])}


# ---------------------------------------------------------------------------------------------- the library's calls
_held = {}


def _workspace(nbytes):
    """One zeroed workspace for every call of this program (they run in order on one stream)."""
    if "ws" not in _held or _held["ws"].numel() < nbytes:
        _held["ws"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    return _held["ws"]


def _library():
    if "tl" not in _held:
        import communication_overlapped_gemm_gb300 as tl
        _held["tl"], _held["ctx"] = tl, tl.Context(0)
    return _held["tl"], _held["ctx"]


def _own(s):
    tl, ctx = _library()
    if s["op"] == "attend":
        ws = _workspace(tl.tl_paged_attention_workspace_bytes(s["batch"], s["heads"], s["kv_heads"], s["d"]))
        tl.tl_paged_attention(ctx, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["out"], ws, lse=s["lse"],
                              window=s["window"], sinks=s["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                              k_blocks=s["k_blocks"], v_blocks=s["v_blocks"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "store":
        kw = dict(k_scale=s["k_scale"], v_scale=s["v_scale"], k_blocks=s["k_blocks"], v_blocks=s["v_blocks"])
        tl.tl_kv_append(ctx, s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], **kw)
        tl.tl_kv_gather(ctx, s["k_cache"], s["v_cache"], s["slots"], s["k_rows"], s["v_rows"], **kw)
        return {w: s[w] for w in ("k_rows", "k_blocks", "v_rows", "v_blocks")}
    if s["op"] == "rope":
        tl.tl_norm_rope(ctx, s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                        k_weight=s["k_weight"], eps=1e-6, interleaved=s["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "plan":
        tl.tl_cache_plan(ctx, s["lengths"], s["table"], s["page"], s["free_pages"], s["taken"], s["taken_out"],
                         s["new_lengths"], s["cu_q"], s["slots"], s["positions"], counts=s["counts"], cu_k=s["cu_k"],
                         kv_slots=s["kv_slots"])
        got = {"table": s["table"], "slots": s["slots"], "positions": s["positions"], "cu_q": s["cu_q"], "cu_k": s["cu_k"],
               "lengths": s["new_lengths"], "taken": s["taken_out"]}
        return got if s["kv_slots"] is None else {**got, "kv_slots": s["kv_slots"]}
    ws = _workspace(tl.tl_token_logprobs_workspace_bytes(s["rows"], s["vocab"], s["top"]))
    tl.tl_token_logprobs(ctx, s["logits"], s["targets"], s["logprob"], ws, entropy=s["entropy"], top_logprobs=s["top_logprobs"],
                         top_ids=s["top_ids"], scale=1.0 / s["temperature"])
    return {w: s[w] for w in ("logprob", "entropy", "top_logprobs", "top_ids")}


def run(state):
    if own:
        return _own(state)
    return {"attend": _plain_attend, "store": _plain_store, "rope": _plain_rope, "plan": _plain_plan,
            "score": _plain_score}[state["op"]](state)


# ---------------------------------------------------------------------------------------------- work
def _visible(n, window, sinks):
    """Keys that the newest of n tokens sees."""
    return n if not window else min(n, window + min(sinks, max(0, n - window)))


def work(case):
    if case["op"] == "attend":
        keys = sum(_visible(n, case["window"], case["sinks"]) for n in _lengths(case).tolist())
        io = 2 * case["batch"] * case["heads"] * case["d"] * 2 + 4 * case["batch"] * case["heads"]
        return {"bytes": 2 * keys * case["kv_heads"] * case["d"] * 9 // 16 + io, "flops": 4 * keys * case["heads"] * case["d"]}
    if case["op"] == "store":
        n = (case["tokens"] - min(case["tokens"], case["padding"])) * 2 * case["kv_heads"] * case["d"]
        return {"bytes": 2 * n * (2 + 9 / 16) + 8 * case["tokens"], "flops": 4 * n}
    if case["op"] == "rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["d"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 8 * n}
    if case["op"] == "plan":
        lens, new, p = _lengths(case), _counts(case), case["page"]
        n, k = int(new.sum()), int((lens + new).sum()) if case["all_rows"] else 0
        pages = int(((lens + new + p - 1) // p - (lens + p - 1) // p).sum())
        return {"bytes": 4 * (5 * case["batch"] + 2 * pages + 2 * n + k + k // p), "flops": 4 * (n + k)}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * _BYTES[case["dtype"]] + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    cuda = dict(dtype=torch.float64, device="cuda")
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], **cuda)

    def e4m3(x):
        """Nearest value of the 8-bit format with 4 exponent and 3 mantissa bits (ties to even), saturating."""
        _, e = torch.frexp(x.abs())
        step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
        return (torch.round(x / step) * step).clamp(-448.0, 448.0)

    def e2m1(x):
        """Nearest value of the 4-bit format (steps of 1/2 to 2, 1 to 4, 2 to 6, ties to even), saturating."""
        a = x.abs().clamp(max=6.0)
        step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).double()
        return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), x)

    def held(cache, blocks, scale, page, row, h):
        """Rows of one kv head that a cache holds, [n, d]."""
        byte = cache[page, row, h].long()
        both = torch.stack([byte % 16, torch.div(byte, 16, rounding_mode="floor")], -1).flatten(-2)
        x = half[both % 8] * torch.where(both >= 8, -1.0, 1.0)
        b = blocks.view(torch.uint8)[page, row, h].view(_E4M3).double()
        return x * b.repeat_interleave(16, -1) * scale[h].double()

    def attend(s):
        out = torch.zeros(s["q"].shape, **cuda)
        lse = torch.full(s["q"].shape[:2], -math.inf, **cuda)
        g = s["heads"] // s["kv_heads"]
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            pos = torch.arange(n, device="cuda")
            if s["window"]:
                pos = pos[(pos >= n - s["window"]) | (pos < s["sinks"])]
            page, row = s["table"][b, torch.div(pos, s["page"], rounding_mode="floor")].long(), pos % s["page"]
            for h in range(s["kv_heads"]):
                k, v = (held(s[w + "_cache"], s[w + "_blocks"], s[w + "_scale"], page, row, h) for w in "kv")
                scores = s["q"][b, h * g:(h + 1) * g].double() @ k.T / math.sqrt(s["d"])
                out[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = torch.softmax(scores, -1) @ v, torch.logsumexp(scores, -1)
        return {"out": out, "lse": lse}

    def store(s):
        got = {}
        slots = s["slots"].tolist()
        kept = torch.tensor([i for i, at in enumerate(slots) if at >= 0], dtype=torch.int64, device="cuda")
        at = s["slots"][kept].long()
        for w in "kv":
            scale = s[w + "_scale"].double()[:, None]
            x = s[w][kept].double().unflatten(-1, (-1, 16))
            b = e4m3(x.abs().amax(-1) / (6.0 * scale))
            t = (b * scale)[..., None]
            y = torch.where(t > 0, e2m1(x / t), 0.0) * t
            rows, blocks = s[w + "_rows"].double(), s[w + "_blocks"].double()
            rows[kept] = y.flatten(-2)
            blocks[torch.div(at, s["page"], rounding_mode="floor"), at % s["page"]] = b
            got[w + "_rows"], got[w + "_blocks"] = rows, blocks
        return got

    def rope(s):
        turn = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
        unit = torch.polar(torch.ones_like(turn), turn)[:, None, :]
        got = {}
        for w in "qk":
            x, r = s[w].double(), s["rotary"]
            if s[w + "_weight"] is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s[w + "_weight"].double()
            first, second = (slice(0, r, 2), slice(1, r, 2)) if s["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            got[w] = y
        return got

    def score(s):
        x = s["logits"].double() / s["temperature"]
        live = s["targets"] >= 0
        y = torch.log_softmax(x, -1)
        entropy = torch.special.entr(y.exp()).sum(-1)
        chosen = y[torch.arange(s["rows"], device="cuda"), s["targets"].clamp(min=0).long()]
        best = torch.topk(y, s["top"], -1).values
        keep = lambda new, old: torch.where(live if new.dim() == 1 else live[:, None], new, old.double())  # noqa: E731
        return {"logprob": keep(chosen, s["logprob"]), "entropy": keep(entropy, s["entropy"]),
                "top_logprobs": keep(best, s["top_logprobs"]), "top_ids": None}

    if case["op"] == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"attend": attend, "store": store, "rope": rope, "score": score}[case["op"]](s)
