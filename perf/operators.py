"""The operators of a decoder's serving step, with their plain forms: what is timed and compared.

Four operators work on one paged key/value cache and one mixture-of-experts layer:

  append  new K/V rows are written into the pages of a cache (bf16, fp16 or e4m3 with a scale per head)
  paged   attention of one new token of each sequence over the cache (with a sliding window and sinks)
  window  causal attention of prompts of ragged lengths (with a sliding window and sinks)
  moe     a whole mixture-of-experts layer for a few tokens

With ``own`` false ``run`` computes them with elementary torch operations in 32 bits; with ``own`` true
it calls the library.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------------------------- cases
def _paged(name, **kw):
    c = dict(op="paged", batch=1, longest=1, shortest=1, heads=32, kv_heads=8, d=128, page=16, dtype="bf16",
             cache="bf16", window=0, sinks=0, head_major=False)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _window(name, **kw):
    c = dict(op="window", batch=1, longest=1, shortest=1, prior=0, heads=32, kv_heads=8, d=128, dtype="bf16", window=0,
             sinks=0)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _append(name, **kw):
    c = dict(op="append", tokens=1, kv_heads=8, d=128, page=16, dtype="bf16", cache="bf16", head_major=False,
             padding=0)
    c.update(kw)
    return dict(name=name, **c) if name else c


def _moe(name, **kw):
    c = dict(op="moe", tokens=1, hidden=2048, experts=64, ffn=1408, topk=2)
    c.update(kw)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one user's chat: a single sequence, where the latency of the split and the join counts
        _paged("paged one sequence 4k", longest=4096, shortest=4096),
        # an ordinary serving batch: ragged lengths
        _paged("paged batch 32 to 8k", batch=32, longest=8192),
        # a large batch over an 8-bit cache, the pages larger
        _paged("paged e4m3 batch 128 to 16k", batch=128, longest=16384, heads=64, cache="e4m3", page=64),
        # a sliding-window layer: long sequences, few visible keys, an odd group size, odd pages, head-major pages
        _paged("paged window fp16 batch 7", batch=7, longest=33001, shortest=100, heads=28, kv_heads=4, d=64, page=7,
               dtype="fp16", cache="fp16", window=1000, sinks=5, head_major=True),
        # short prompts (chat turns) packed in one call
        _window("window short prompts", batch=6, longest=200),
        # a long prompt through a sliding-window layer
        _window("window prompt 8k", longest=8192, shortest=8192, window=1024, sinks=4),
        # turns that continue a conversation whose keys are there already: full causal attention
        _window("causal continued fp16 d64", batch=2, longest=4097, shortest=2999, prior=513, heads=16, kv_heads=2,
                d=64, dtype="fp16"),
        # one decoding step's new rows, padded to a captured batch size
        _append("append one step of 64", tokens=64, padding=3),
        # a long prompt's rows into an 8-bit cache
        _append("append prompt 8k to e4m3", tokens=8192, cache="e4m3", page=64, head_major=True),
        # one token: latency
        _moe("moe one token"),
        # sizes that no tile divides
        _moe("moe odd sizes", tokens=13, hidden=1000, experts=24, ffn=712, topk=3),
        # a decoding batch that touches nearly every expert
        _moe("moe 64 tokens", tokens=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("paged", "paged", "window", "window", "append", "moe", "moe"))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "paged":
        kv, g, d = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16)), rng.choice((64, 128))
        batch = _log(rng, 1, 128)
        longest = _log(rng, 1, max(1, min(33000, 128 * 16384 * 8 * 128 // (batch * kv * d))))
        longest = min(longest, max(1, (1 << 34) // (batch * kv * max(g, d))))
        win = _log(rng, 1, 4096) if rng.random() < 0.4 else 0
        return _paged(None, batch=batch, longest=longest, shortest=rng.randint(0, longest), heads=kv * g, kv_heads=kv,
                      d=d, page=rng.choice((1, 5, 8, 16, 32, 64, 100)), dtype=dtype,
                      cache=rng.choice((dtype, dtype, "e4m3")), window=win, sinks=rng.choice((0, 1, 4, 130)) if win else 0,
                      head_major=rng.random() < 0.5)
    if op == "window":
        kv, g, d = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 6, 8, 16)), rng.choice((64, 128))
        batch = _log(rng, 1, 8)
        # batch * heads * longest^2 scores at most (the plain form holds them)
        longest = _log(rng, 1, max(1, min(8192, int(math.sqrt(2 ** 31 / (batch * kv * g))))))
        win = _log(rng, 1, 4096) if rng.random() < 0.6 else 0
        return _window(None, batch=batch, longest=longest, shortest=rng.randint(1, longest),
                       prior=rng.choice((0, 0, rng.randint(1, longest))) if batch * kv * g * longest ** 2 < 2 ** 30 else 0,
                       heads=kv * g,
                       kv_heads=kv, d=d, dtype=dtype, window=win, sinks=rng.choice((0, 1, 4, 130)) if win else 0)
    if op == "append":
        return _append(None, tokens=_log(rng, 1, 8192), kv_heads=rng.choice((1, 2, 4, 8)), d=rng.choice((64, 128)),
                       page=rng.choice((1, 5, 16, 64)), dtype=dtype, cache=rng.choice((dtype, "e4m3")),
                       head_major=rng.random() < 0.5, padding=rng.choice((0, 2)))
    experts = rng.choice((4, 8, 24, 60, 64))
    return _moe(None, tokens=_log(rng, 1, 64), hidden=8 * _log(rng, 16, 256), experts=experts,
                ffn=8 * _log(rng, 8, 176), topk=rng.randint(1, min(experts, 6)))


# ---------------------------------------------------------------------------------------------- inputs
def _lengths(case):
    """The lengths of a case's sequences, the longest first: the same for every seed, which only orders them anew."""
    lens = torch.randint(case["shortest"], case["longest"] + 1, (case["batch"],), generator=torch.Generator().manual_seed(7))
    lens[0] = case["longest"]
    return lens


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype="bf16", std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(_DT[dtype])

    def cache(pages):
        kv, p, d = case["kv_heads"], case["page"], case["d"]
        shape = (pages, kv, p, d) if case["head_major"] else (pages, p, kv, d)
        c = normal(*shape, dtype=case["cache"], std=0.5 if case["cache"] != "e4m3" else 32.0)
        return c.transpose(1, 2) if case["head_major"] else c

    s = dict(case)
    if case["op"] in ("paged", "append") and case["cache"] == "e4m3":  # about amax / 448 of N(0, 0.5) rows
        for w in ("k_scale", "v_scale"):
            s[w] = torch.rand(case["kv_heads"], generator=gen, device="cuda") * 0.005 + 0.0125
    else:
        s["k_scale"] = s["v_scale"] = None
    if case["op"] == "paged":
        lens = _lengths(case)[torch.randperm(case["batch"], generator=host)]
        need = (lens + case["page"] - 1) // case["page"]
        total, most = int(need.sum()), int(need.max())
        order = torch.randperm(total, generator=host).to(torch.int32)  # pages of a used cache come in any order
        table = torch.full((case["batch"], max(most, 1)), -1, dtype=torch.int32)
        table[torch.arange(table.shape[1])[None, :] < need[:, None]] = order
        s["k_cache"], s["v_cache"] = cache(max(total, 1)), cache(max(total, 1))
        s["q"] = normal(case["batch"], case["heads"], case["d"], dtype=case["dtype"])
        s["table"], s["lengths"] = table.cuda(), lens.to(torch.int32).cuda()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["batch"], case["heads"]), device="cuda")
    elif case["op"] == "window":
        lens = _lengths(case)[torch.randperm(case["batch"], generator=host)]
        cu_q = torch.zeros(case["batch"] + 1, dtype=torch.int32)
        cu_q[1:] = lens.cumsum(0)
        cu_k = torch.zeros(case["batch"] + 1, dtype=torch.int32)
        cu_k[1:] = (lens + case["prior"]).cumsum(0)
        nq, nk, hq, hk, d = int(cu_q[-1]), int(cu_k[-1]), case["heads"], case["kv_heads"], case["d"]
        if case["prior"]:
            s["q"], kv = normal(nq, hq, d, dtype=case["dtype"]), normal(nk, 2 * hk, d, dtype=case["dtype"])
            s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
        else:  # views of one projection's output
            qkv = normal(nq, hq + 2 * hk, d, dtype=case["dtype"])
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["cu_q"], s["cu_k"] = cu_q.cuda(), cu_k.cuda()
        s["out"] = torch.empty((nq, hq, d), dtype=_DT[case["dtype"]], device="cuda")
        s["lse"] = torch.empty((nq, hq), device="cuda")
    elif case["op"] == "append":
        n = case["tokens"]
        pages = (n + n // 2) // case["page"] + 2
        slots = torch.randperm(pages * case["page"], generator=host)[:n].to(torch.int32)
        if case["padding"]:
            slots[-case["padding"]:] = -1
        s["slots"] = slots.cuda()
        kv = normal(n, 2 * case["kv_heads"], case["d"], dtype=case["dtype"], std=0.5)
        s["k"], s["v"] = kv[:, :case["kv_heads"]], kv[:, case["kv_heads"]:]
        s["k_cache"], s["v_cache"] = cache(pages), cache(pages)
    else:
        t, h, e, f = case["tokens"], case["hidden"], case["experts"], case["ffn"]
        s["x"] = normal(t, h)
        s["logits"] = torch.randn((t, e), generator=gen, device="cuda")
        s["w_gate"], s["w_up"], s["w_down"] = normal(e, h, f, std=0.02), normal(e, h, f, std=0.02), normal(e, f, h, std=0.02)
        s["out"] = torch.empty((t, h), device="cuda")
        s["experts_out"] = torch.empty((t, case["topk"]), dtype=torch.int32, device="cuda")
        s["gates_out"] = torch.empty((t, case["topk"]), device="cuda")
    return s


# ---------------------------------------------------------------------------------------------- plain forms
def _softmax_rows(scores, seen):
    """Weights of the visible places of each row (none visible: all zero), and the log of their sum."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    w = (scores - top).exp()
    total = w.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    return w / torch.where(total == 0, 1.0, total), lse


def _pages_of(cache, table):
    """[batch, places, kv_heads, d] in 32 bits: the rows of each sequence in order."""
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    got = raw[table.clamp(min=0).long()].flatten(1, 2)
    return got.view(cache.dtype).float() if raw is not cache else got.float()


def _plain_paged(s):
    b, hq, d = s["q"].shape
    hk = s["kv_heads"]
    k, v = _pages_of(s["k_cache"], s["table"]), _pages_of(s["v_cache"], s["table"])
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][:, None], v * s["v_scale"][:, None]
    at = torch.arange(k.shape[1], device="cuda")[None, :]
    n = s["lengths"].long()[:, None]
    seen = at < n
    v = torch.where(seen[:, :, None, None], v, 0.0)
    if s["window"]:
        seen = seen & ((at >= n - s["window"]) | (at < s["sinks"]))
    q = s["q"].float().reshape(b, hk, hq // hk, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    w, lse = _softmax_rows(scores, seen[:, None, None, :])
    out = torch.matmul(w, v.transpose(1, 2)).reshape(b, hq, d)
    return {"out": out.to(s["q"].dtype), "lse": lse.reshape(b, hq)}


def _plain_window(s):
    hq, hk, d, batch = s["heads"], s["kv_heads"], s["d"], s["batch"]
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    nq, nk, mq = s["q"].shape[0], s["k"].shape[0], s["longest"]
    mk = mq + s["prior"]
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    q = s["q"].float()[(cu_q[:-1, None] + iq).clamp(max=nq - 1)]  # [batch, mq, hq, d]
    rows = (cu_k[:-1, None] + ik).clamp(max=nk - 1)
    k, v = s["k"].float()[rows], s["v"].float()[rows]
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    p = (lk - lq)[:, None, None] + iq[None, :, None]
    seen = (ik <= p) & (ik < lk[:, None, None])
    if s["window"]:
        seen = seen & ((ik > p - s["window"]) | (ik < s["sinks"]))
    q = q.reshape(batch, mq, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * (1.0 / math.sqrt(d))
    w, lse = _softmax_rows(scores, seen[:, None, None])
    out = torch.matmul(w, v.transpose(1, 2)[:, :, None])  # [batch, hk, g, mq, d]
    seq = torch.searchsorted(cu_q[1:], torch.arange(nq, device="cuda"), right=True)
    i = torch.arange(nq, device="cuda") - cu_q[seq]
    out = out.permute(0, 3, 1, 2, 4)[seq, i].reshape(nq, hq, d)
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[seq, i].reshape(nq, hq)}


def _put(cache, rows, scale, page, slots):
    if scale is not None:
        rows = (rows.float() / scale[:, None]).clamp(-448.0, 448.0).to(cache.dtype)
        cache, rows = cache.view(torch.uint8), rows.view(torch.uint8)
    keep = slots >= 0
    at = slots[keep].long()
    cache[at // page, at % page] = rows[keep]


def _plain_append(s):
    _put(s["k_cache"], s["k"], s["k_scale"], s["page"], s["slots"])
    _put(s["v_cache"], s["v"], s["v_scale"], s["page"], s["slots"])
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _plain_moe(s):
    t, k = s["tokens"], s["topk"]
    order = torch.sort(s["logits"], dim=-1, descending=True, stable=True).indices[:, :k]  # ties: the lower index
    w = (s["logits"] - s["logits"].amax(-1, keepdim=True)).exp()
    gates = torch.gather(w / w.sum(-1, keepdim=True), 1, order)
    at = order.reshape(-1)
    x = s["x"].float().repeat_interleave(k, 0)[:, None]
    a, b = torch.bmm(x, s["w_gate"][at].float()), torch.bmm(x, s["w_up"][at].float())
    y = torch.bmm(a / (1.0 + (-a).exp()) * b, s["w_down"][at].float()).reshape(t, k, -1)
    return {"out": (gates[:, :, None] * y).sum(1), "experts": order.to(torch.int32), "gates": gates}


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
    if s["op"] == "paged":
        ws = _workspace(tl.tl_paged_attention_workspace_bytes(s["batch"], s["heads"], s["kv_heads"], s["d"]))
        tl.tl_paged_attention(ctx, s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["out"], ws,
                              lse=s["lse"], window=s["window"], sinks=s["sinks"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "window":
        tl.tl_window_attention(ctx, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["out"], lse=s["lse"],
                               window=s["window"], sinks=s["sinks"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "append":
        tl.tl_kv_append(ctx, s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], k_scale=s["k_scale"],
                        v_scale=s["v_scale"])
        return {"k": s["k_cache"], "v": s["v_cache"]}
    ws = _workspace(tl.tl_moe_tokens_workspace_bytes(s["tokens"], s["hidden"], s["experts"], s["ffn"], s["topk"]))
    tl.tl_moe_tokens(ctx, s["x"], s["logits"], s["topk"], s["w_gate"], s["w_up"], s["w_down"], s["out"], ws,
                     experts_out=s["experts_out"], gates_out=s["gates_out"])
    return {"out": s["out"], "experts": s["experts_out"], "gates": s["gates_out"]}


def run(state):
    if own:
        return _own(state)
    return {"paged": _plain_paged, "window": _plain_window, "append": _plain_append, "moe": _plain_moe}[state["op"]](state)


# ---------------------------------------------------------------------------------------------- work
def _visible(n, window, sinks):
    """Keys that the newest of n tokens sees."""
    return n if not window else min(n, window + min(sinks, max(0, n - window)))


def work(case):
    if case["op"] == "paged":
        lens = _lengths(case).tolist()
        keys = sum(_visible(n, case["window"], case["sinks"]) for n in lens)
        io = 2 * case["batch"] * case["heads"] * case["d"] * 2 + 4 * case["batch"] * case["heads"]
        return {"bytes": 2 * keys * case["kv_heads"] * case["d"] * _BYTES[case["cache"]] + io,
                "flops": 4 * keys * case["heads"] * case["d"]}
    if case["op"] == "window":
        lens = _lengths(case).tolist()
        pairs = sum(_visible(case["prior"] + i + 1, case["window"], case["sinks"]) for n in lens for i in range(n))
        nq, nk = sum(lens), sum(lens) + case["batch"] * case["prior"]
        return {"bytes": 2 * nq * case["heads"] * case["d"] * 2 + 2 * nk * case["kv_heads"] * case["d"] * 2 + 4 * nq * case["heads"],
                "flops": 4 * pairs * case["heads"] * case["d"]}
    if case["op"] == "append":
        n = (case["tokens"] - min(case["tokens"], case["padding"])) * 2 * case["kv_heads"] * case["d"]
        return {"bytes": n * (2 + _BYTES[case["cache"]]) + 4 * case["tokens"], "flops": n}
    a = case["tokens"] * case["topk"]
    # distinct experts that the tokens touch (each token's topk are distinct), the logits being even
    hit = case["experts"] * (1.0 - (1.0 - case["topk"] / case["experts"]) ** case["tokens"])
    return {"bytes": hit * 6 * case["hidden"] * case["ffn"] + case["tokens"] * (6 * case["hidden"] + 4 * case["experts"]),
            "flops": 6.0 * a * case["hidden"] * case["ffn"]}


# ---------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    def rows_of(q, k, v, seen, scale):
        """One kv head: q [g, n, d], k and v [m, d], seen [n, m], all float64."""
        scores = (q @ k.T) * scale
        scores = scores.masked_fill(~seen, -math.inf)
        lse = torch.logsumexp(scores, -1)
        w = torch.where(seen.any(-1, keepdim=True), torch.softmax(scores, -1), torch.zeros((), dtype=torch.float64, device="cuda"))
        return w @ v, lse

    def paged(s):
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        g = s["heads"] // s["kv_heads"]
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            pos = torch.arange(n, device="cuda")
            if s["window"]:
                pos = pos[(pos >= n - s["window"]) | (pos < s["sinks"])]
            page, row = s["table"][b, torch.div(pos, s["page"], rounding_mode="floor")].long(), pos % s["page"]
            seen = torch.ones((1, pos.numel()), dtype=torch.bool, device="cuda")
            for h in range(s["kv_heads"]):
                k, v = (c.select(2, h).view(torch.uint8)[page, row].view(c.dtype).double() if c.dtype == torch.float8_e4m3fn
                        else c.select(2, h)[page, row].double() for c in (s["k_cache"], s["v_cache"]))
                if s["k_scale"] is not None:
                    k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
                o, e = rows_of(s["q"][b, h * g:(h + 1) * g, None].double(), k, v, seen, s["d"] ** -0.5)
                out[b, h * g:(h + 1) * g], lse[b, h * g:(h + 1) * g] = o[:, 0], e[:, 0]
        return {"out": out, "lse": lse}

    def window(s):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
        g = s["heads"] // s["kv_heads"]
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for b in range(s["batch"]):
            q, k, v = s["q"][cq[b]:cq[b + 1]].double(), s["k"][ck[b]:ck[b + 1]].double(), s["v"][ck[b]:ck[b + 1]].double()
            n, m = q.shape[0], k.shape[0]
            p, j = torch.arange(n, device="cuda")[:, None] + (m - n), torch.arange(m, device="cuda")[None, :]
            seen = j <= p
            if s["window"]:
                seen &= (p - j < s["window"]) | (j < s["sinks"])
            for h in range(s["heads"]):
                o, e = rows_of(q[None, :, h], k[:, h // g], v[:, h // g], seen, s["d"] ** -0.5)
                out[cq[b]:cq[b + 1], h], lse[cq[b]:cq[b + 1], h] = o[0], e[0]
        return {"out": out, "lse": lse}

    def e4m3(x):
        """Nearest value of the 8-bit format with 4 exponent and 3 mantissa bits (ties to even), saturating."""
        _, e = torch.frexp(x.abs())
        step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
        return (torch.round(x / step) * step).clamp(-448.0, 448.0)

    def append(s):
        got = {}
        slots = s["slots"].tolist()
        kept = [i for i, at in enumerate(slots) if at >= 0]
        at = torch.tensor([slots[i] for i in kept], device="cuda")
        for name, scale in (("k", s["k_scale"]), ("v", s["v_scale"])):
            cache, rows = s[name + "_cache"].double(), s[name][torch.tensor(kept, device="cuda")].double()
            cache[torch.div(at, s["page"], rounding_mode="floor"), at % s["page"]] = \
                rows if scale is None else e4m3(rows / scale.double()[:, None])
            got[name] = cache
        return got

    def moe(s):
        logits = s["logits"].double()
        w = torch.softmax(logits, -1)
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        gates = torch.zeros((s["tokens"], s["topk"]), dtype=torch.float64, device="cuda")
        for t, row in enumerate(logits.tolist()):
            for j, e in enumerate(sorted(range(len(row)), key=lambda i: (-row[i], i))[:s["topk"]]):
                x = s["x"][t].double()
                h = torch.nn.functional.silu(x @ s["w_gate"][e].double()) * (x @ s["w_up"][e].double())
                gates[t, j] = w[t, e]
                out[t] += w[t, e] * (h @ s["w_down"][e].double())
        return {"out": out, "experts": None, "gates": gates}

    s = prepare(case, seed)
    return {"paged": paged, "window": window, "append": append, "moe": moe}[case["op"]](s)
