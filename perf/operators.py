"""Cases of the verify-step operators: the 8-bit paged cache (write, read back,
attend) and the scoring of given tokens.

``run`` makes one pass through one operator, in its plain form (elementary
torch operations in 32 bits) or, with ``own`` set, through the library's
entry point.  ``exact`` gives the same outputs from the definitions in 64
bits.  Sizes follow the repository's own workloads where it has them: 32
query heads over 8 key/value heads of 128 (a [Q|K|V] row of 4096 + 1024 +
1024), 64 decode rows, 4 sequences x 9 draft tokens, 8 segments x 512 prompt
tokens, a vocabulary of 32000; the rest are generic.

A sequence's rows are its last tokens: with ``kv_len`` tokens cached after the
call and n_i rows, row j holds position kv_len - n_i + j.  The cache keeps
e4m3 codes in pages of P tokens and one power-of-two scale for each page and
head, an exponent byte e standing for 2^(e - 127).  Within a page's head,
K lies as [P/16][4][D/16][4][16] (16-token group, quad, 16-dim chunk, token
of the quad, dim) and V as [P/16][D][16] (16-token group, dim, token).
"""
import math

import torch

own = False

E_MIN, E_MAX = 10, 247  # exponent bytes a page's scale may take: 2^-117 .. 2^120
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token a sequence joins its page: a decode step's cache write
        {"name": "write_step", "op": "write", "dtype": "bf16", "seqs": 64, "rows": 1, "ctx": 1000, "ragged": True,
         "kv_heads": 8, "dim": 128, "page": 16},
        # the prompts of the prefill workload, 8 x 512 tokens, into fresh pages
        {"name": "write_prompt", "op": "write", "dtype": "bf16", "seqs": 8, "rows": 512, "ctx": 0, "ragged": False,
         "kv_heads": 8, "dim": 128, "page": 64},
        # cached prefixes brought back to rows, to be moved or attended elsewhere
        {"name": "read_prefix", "op": "read", "dtype": "bf16", "seqs": 4, "rows": 4096, "ctx": 0, "ragged": False,
         "kv_heads": 8, "dim": 128, "page": 64},
        # ragged tails of three sequences in f32, odd head count, rows that begin inside a page
        {"name": "read_odd", "op": "read", "dtype": "f32", "seqs": 3, "rows": 777, "ctx": 1234, "ragged": True,
         "kv_heads": 5, "dim": 64, "page": 32},
        # one short conversation: launch and latency
        {"name": "attend_one", "op": "attend", "dtype": "bf16", "seqs": 1, "rows": 1, "ctx": 700, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0},
        # a full decode batch of unlike lengths
        {"name": "attend_batch", "op": "attend", "dtype": "bf16", "seqs": 64, "rows": 1, "ctx": 8191, "ragged": True,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0},
        # the speculative-verify batch: 4 sequences x 9 draft tokens
        {"name": "attend_verify", "op": "attend", "dtype": "bf16", "seqs": 4, "rows": 9, "ctx": 6000, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 16, "window": 0},
        # one very long context in f32, wide heads, five query heads to a key/value head
        {"name": "attend_long", "op": "attend", "dtype": "f32", "seqs": 1, "rows": 1, "ctx": 131071, "ragged": False,
         "heads": 10, "kv_heads": 2, "dim": 256, "page": 128, "window": 0},
        # the prefill workload's 8 x 512 prompt tokens attending to themselves
        {"name": "attend_prompt", "op": "attend", "dtype": "bf16", "seqs": 8, "rows": 512, "ctx": 0, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # a chunk of a long prompt: many rows over a long cache
        {"name": "attend_chunk", "op": "attend", "dtype": "bf16", "seqs": 2, "rows": 1024, "ctx": 15000, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0},
        # draft tokens of the verify batch scored over a large odd vocabulary, with 20 alternatives
        {"name": "score_verify", "op": "score", "dtype": "f32", "n": 36, "vocab": 131071, "top": 20},
        # every prompt token's log probability (the vocabulary of the embedding workload)
        {"name": "score_prompt", "op": "score", "dtype": "bf16", "n": 4096, "vocab": 32000, "top": 5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "score", "score"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "score":
        c |= {"vocab": _log(rng, 300, 200000), "top": rng.choice([0, 1, rng.randint(2, 32)])}
        c["n"] = _log(rng, 1, max(1, min(4096, 60_000_000 // c["vocab"])))
        return c
    c |= {"dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.7}
    if op != "attend":
        c |= {"kv_heads": rng.randint(1, 12), "seqs": _log(rng, 1, 64), "ctx": rng.choice([0, _log(rng, 1, 3000)])}
        c["rows"] = _log(rng, 1, min(16384 // c["seqs"], 12_000_000 // (c["kv_heads"] * c["dim"] * c["seqs"]) + 1))
        return c
    c["kv_heads"] = rng.randint(1, 8)
    c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
    many = rng.random() < 0.4  # rows of prompts, or of decode and verify steps
    c["seqs"] = _log(rng, 1, 8) if many else _log(rng, 1, 128)
    wide = c["heads"] * c["dim"] * c["seqs"]
    c["rows"] = _log(rng, 17, min(1500, int(math.sqrt(1.5e11 / wide)))) if many else rng.choice([1, 1, rng.randint(2, 16)])
    most = 1.0e11 / (wide * c["rows"]) - c["rows"] / 2 if many else 1.5e8 / wide
    c["ctx"] = rng.choice([0, 1, 1, 1]) * _log(rng, 1, max(2, min(100000, most)))
    c["window"] = rng.choice([0, 0, _log(rng, 1, 8192)])
    return c


# ---------------------------------------------------------------- lengths of a case
def _share(i):
    return (0.37 + 0.6180339887 * i) % 1.0


def _lengths(case):
    """(rows, tokens cached after the call) of each sequence."""
    got = []
    for i in range(case["seqs"]):
        f = _share(i) if case["ragged"] else 1.0
        rows = 1 + int((case["rows"] - 1) * f)
        got.append((rows, rows + int(case["ctx"] * f)))
    return got


def _visible(rows, length, window):
    """Tokens that each row of a sequence sees."""
    return [min(length - rows + j + 1, window) if window else length - rows + j + 1 for j in range(rows)]


def work(case):
    if case["op"] == "score":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["n"] * (case["vocab"] * size + 16 + 8 * case["top"]), "flops": 4 * case["n"] * case["vocab"]}
    size = 2 if case["dtype"] == "bf16" else 4
    lens = _lengths(case)
    row = case["kv_heads"] * case["dim"]
    n = sum(r for r, _ in lens)
    if case["op"] != "attend":
        pages = sum((t - 1) // case["page"] - (t - r) // case["page"] + 1 for r, t in lens)
        return {"bytes": 2 * n * row * (size + 1) + 2 * pages * case["kv_heads"] + 4 * pages + 8 * len(lens), "flops": 2 * n * row}
    seen, pairs = 0, 0
    for r, t in lens:
        v = _visible(r, t, case["window"])
        seen += min(t, v[0] + r - 1)
        pairs += sum(v)
    pages = seen / case["page"]
    wide = case["heads"] * case["dim"]
    return {"bytes": 2 * seen * row + 2 * pages * case["kv_heads"] + 4 * pages + 2 * n * wide * size + 4 * n * case["heads"],
            "flops": 4 * pairs * wide}


# ---------------------------------------------------------------- inputs
def _tile(k, v):
    """[..., P, D] codes of K and of V in the cache's order, each [..., P D]."""
    *lead, P, D = k.shape
    kt = k.reshape(*lead, P // 16, 4, 4, D // 16, 16).transpose(-3, -2)
    vt = v.reshape(*lead, P // 16, 16, D).transpose(-2, -1)
    return kt.reshape(*lead, P * D), vt.reshape(*lead, P * D)


def _untile_k(k, P, D):
    *lead, _ = k.shape
    return k.reshape(*lead, P // 16, 4, D // 16, 4, 16).transpose(-3, -2).reshape(*lead, P, D)


def _untile_v(v, P, D):
    *lead, _ = v.shape
    return v.reshape(*lead, P // 16, D, 16).transpose(-2, -1).reshape(*lead, P, D)


def _need(amax):
    """The exponent byte of the smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    return torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype) + 127, E_MIN).clamp(E_MIN, E_MAX)


def _power(e):
    """2^(e - 127) of whole exponent bytes."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.to(torch.int32) - 127)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "score":
        n, V = case["n"], case["vocab"]
        # a few likely tokens over a broad tail; a part of the vocabulary ruled out, as a grammar does
        x = normal(n, V) * 2.5 + 2.0 * normal(1, V)
        out = torch.rand(V, generator=g, device="cuda") < 0.03
        out[0] = False
        logits = x.masked_fill(out, -math.inf).to(dt)
        likely = x.masked_fill(out, -math.inf).argmax(1)
        other = (torch.rand(n, generator=g, device="cuda") * V).long().clamp(max=V - 1)
        ids = torch.where(torch.rand(n, generator=g, device="cuda") < 0.6, likely, other).int()
        k = case["top"]
        s = {"case": case, "logits": logits, "ids": ids, "logp": torch.empty(n, device="cuda"),
             "entropy": torch.empty(n, device="cuda"), "rank": torch.empty(n, dtype=torch.int32, device="cuda"),
             "top_ids": torch.empty(n, k, dtype=torch.int32, device="cuda"), "top_logp": torch.empty(n, k, device="cuda")}
        if own:
            from adapter_lora_bgmv_amd import binding as B
            s["code"] = B.LORA_BF16 if case["dtype"] == "bf16" else B.LORA_F32
            s["ws_bytes"] = B.lora_token_logprobs_workspace_bytes(s["code"], V, n, k)
            s["ws"] = torch.zeros(max(s["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
        return s

    H, D, P, S = case["kv_heads"], case["dim"], case["page"], case["seqs"]
    lens = _lengths(case)
    per = max((t + P - 1) // P for _, t in lens)
    used = [(t + P - 1) // P for _, t in lens]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    starts = torch.tensor([0] + used, device="cuda").cumsum(0)
    at = torch.arange(per, device="cuda")[None] + starts[:-1, None]
    ok = torch.arange(per, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]
    table = torch.where(ok, order[at.clamp(max=n_pages - 1)], -1).int().contiguous()
    # keys with a few strong channels, values of unlike size from page to page
    k = normal(n_pages, H, P, D) * torch.where(torch.arange(D, device="cuda") % 37 == 5, 4.0, 1.0)
    v = normal(n_pages, H, P, D) * torch.exp2(normal(n_pages, H, 1, 1))
    ke, ve = _need(k.abs().amax((2, 3))), _need(v.abs().amax((2, 3)))
    k = (k / _power(ke)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    v = (v / _power(ve)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    kc, vc = _tile(k, v)
    del k, v
    n = sum(r for r, _ in lens)
    s = {"case": case, "k": kc.contiguous(), "v": vc.contiguous(), "ke": ke.to(torch.uint8), "ve": ve.to(torch.uint8),
         "table": table, "indptr": torch.tensor([0] + [r for r, _ in lens], device="cuda").cumsum(0).int(),
         "kv_len": torch.tensor([t for _, t in lens], device="cuda").int(), "n": n, "most_rows": max(r for r, _ in lens),
         "per": per}
    if case["op"] == "write":
        # the K and V parts of interleaved rows
        s["rows"] = (normal(n, 2 * H * D) * torch.exp2(normal(n, 1))).to(dt)
    elif case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty(n, H * D, dtype=dt, device="cuda") for _ in range(2))
    else:
        s["q"] = normal(n, case["heads"] * D).to(dt)
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(n, case["heads"], device="cuda")
        s["scale"] = D ** -0.5
    if own:
        from adapter_lora_bgmv_amd import binding as B
        s["code"] = B.LORA_BF16 if case["dtype"] == "bf16" else B.LORA_F32
        s["cache"] = B.KVCache(s["k"], s["v"], s["ke"], s["ve"], page_tokens=P, head_dim=D)
        s["seqs"] = B.KVSeqs(table, s["indptr"], s["kv_len"], max_rows=s["most_rows"])
        if case["op"] == "attend":
            s["ws_bytes"] = B.lora_kv_attend_workspace_bytes(s["cache"], s["seqs"], s["code"], case["heads"], n)
            s["ws"] = torch.zeros(max(s["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return globals()[("own_" if own else "plain_") + s["case"]["op"]](s)


def own_write(s):
    from adapter_lora_bgmv_amd import binding as B
    row = s["rows"].shape[1]
    B.lora_kv_write(s["cache"], s["seqs"], s["code"], s["rows"], row, s["rows"][:, row // 2:], row, s["n"])
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_exp": s["ke"], "v_exp": s["ve"]}


def own_read(s):
    from adapter_lora_bgmv_amd import binding as B
    row = s["k_out"].shape[1]
    B.lora_kv_read(s["cache"], s["seqs"], s["code"], s["k_out"], row, s["v_out"], row, s["n"])
    return {"k": s["k_out"], "v": s["v_out"]}


def own_attend(s):
    from adapter_lora_bgmv_amd import binding as B
    c, row = s["case"], s["q"].shape[1]
    B.lora_kv_attend(s["cache"], s["seqs"], s["code"], c["heads"], s["q"], row, s["scale"], c["window"], s["n"], s["out"], row,
                     s["lse"], s["ws"], s["ws_bytes"])
    return {"out": s["out"], "lse": s["lse"]}


def own_score(s):
    from adapter_lora_bgmv_amd import binding as B
    c = s["case"]
    B.lora_token_logprobs(s["code"], c["vocab"], s["logits"], c["vocab"], s["ids"], c["n"], c["top"], s["logp"], s["entropy"],
                          s["rank"], s["top_ids"], s["top_logp"], s["ws"], s["ws_bytes"])
    return {"logp": s["logp"], "entropy": s["entropy"], "rank": s["rank"], "top_ids": s["top_ids"], "top_logp": s["top_logp"]}


def _rows(s):
    """Sequence, position, page and place in the page of every row."""
    P = s["case"]["page"]
    r = torch.arange(s["n"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["indptr"][1:].contiguous(), r, right=True)
    pos = s["kv_len"][seq] - s["indptr"][seq + 1] + r
    return seq, pos, s["table"][seq, pos // P].long(), (pos % P).long()


def plain_write(s):
    c = s["case"]
    H, D, P = c["kv_heads"], c["dim"], c["page"]
    _, _, page, at = _rows(s)
    x = s["rows"].float().reshape(s["n"], 2, H, D)
    start = s["kv_len"] - (s["indptr"][1:] - s["indptr"][:-1])
    first = s["table"][torch.arange(c["seqs"], device="cuda"), start // P].long()  # the page that each sequence's rows begin in
    kept = torch.arange(P, device="cuda")[None, :] < (start % P)[:, None]           # its tokens from before
    a = torch.arange(D, device="cuda")
    t, h = at[:, None, None], torch.arange(H, device="cuda")[None, :, None]
    place_k = (t // 16) * (16 * D) + (t % 16 // 4) * (4 * D) + (a // 16) * 64 + (t % 4) * 16 + a % 16
    place_v = (t // 16) * (16 * D) + a * 16 + t % 16
    _write_one(s["k"], s["ke"], x[:, 0], page, first, kept, place_k, h, _untile_k, P, D, lambda o: _tile(o, o)[0])
    _write_one(s["v"], s["ve"], x[:, 1], page, first, kept, place_v, h, _untile_v, P, D, lambda o: _tile(o, o)[1])
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_exp": s["ke"], "v_exp": s["ve"]}


def _write_one(pool, exps, x, page, first, kept, place, h, untile, P, D, tile):
    size = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(2)
    most = torch.zeros(exps.shape, device="cuda").scatter_reduce(0, page[:, None].expand_as(size), size, "amax")
    need = _need(most)
    before = exps[first].to(need.dtype)
    old = kept.any(1)[:, None]
    # a page with tokens from before keeps at least their scale, and they follow it where it grows
    after = torch.where(old, torch.maximum(before, need[first]), need[first])
    codes = untile(pool[first], P, D)
    moved = (codes.view(torch.float8_e4m3fn).float() * torch.ldexp(torch.ones_like(after, dtype=torch.float32), before - after)[..., None, None])
    codes = torch.where(kept[:, None, :, None], moved.to(torch.float8_e4m3fn).view(torch.uint8), codes)
    pool[first] = tile(codes)
    need[first] = after
    exps[page] = need[page].to(torch.uint8)
    y = x / _power(need[page])[..., None]
    pool[page[:, None, None], h, place] = torch.where(torch.isfinite(y), y, math.nan).to(torch.float8_e4m3fn).view(torch.uint8)


def plain_read(s):
    c = s["case"]
    H, D, P = c["kv_heads"], c["dim"], c["page"]
    _, _, page, at = _rows(s)
    a = torch.arange(D, device="cuda")
    t, h = at[:, None, None], torch.arange(H, device="cuda")[None, :, None]
    place_k = (t // 16) * (16 * D) + (t % 16 // 4) * (4 * D) + (a // 16) * 64 + (t % 4) * 16 + a % 16
    place_v = (t // 16) * (16 * D) + a * 16 + t % 16
    got = {}
    got["k"] = s["k"][page[:, None, None], h, place_k].view(torch.float8_e4m3fn).float() * _power(s["ke"][page])[..., None]
    got["v"] = s["v"][page[:, None, None], h, place_v].view(torch.float8_e4m3fn).float() * _power(s["ve"][page])[..., None]
    return {m: y.reshape(s["n"], H * D).to(s["k_out"].dtype) for m, y in got.items()}


def plain_attend(s):
    c = s["case"]
    H, D, P, S, R = c["kv_heads"], c["dim"], c["page"], c["seqs"], s["most_rows"]
    G, L = c["heads"] // H, s["per"] * P
    page = s["table"].clamp(min=0).long()
    k = _untile_k(s["k"][page], P, D).view(torch.float8_e4m3fn).float() * _power(s["ke"][page])[..., None, None]
    v = _untile_v(s["v"][page], P, D).view(torch.float8_e4m3fn).float() * _power(s["ve"][page])[..., None, None]
    k = k.transpose(1, 2).reshape(S, H, L, D)  # [S, pages, H, P, D] -> [S, H, tokens, D]
    v = v.transpose(1, 2).reshape(S, H, L, D)
    t = torch.arange(L, device="cuda")
    v = torch.where((t < s["kv_len"][:, None])[:, None, :, None], v, 0.0)
    rows = s["indptr"][1:] - s["indptr"][:-1]
    j = torch.arange(R, device="cuda")
    live = j < rows[:, None]
    at = (s["indptr"][:-1, None] + j).clamp(max=s["n"] - 1).long()
    q = s["q"][at].float().reshape(S, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, R * G, D)
    w = (q @ k.transpose(2, 3)).reshape(S, H, R, G, L) * s["scale"]
    pos = s["kv_len"][:, None] - rows[:, None] + j  # [S, R]
    seen = t <= pos[..., None]
    if c["window"]:
        seen = seen & (t > pos[..., None] - c["window"])
    w = w.masked_fill(~seen[:, None, :, None, :], -math.inf)
    top = w.amax(-1, keepdim=True)
    w = torch.exp(w - torch.where(top == -math.inf, 0.0, top))
    total = w.sum(-1, keepdim=True)
    o = ((w / total).reshape(S, H, R * G, L) @ v).reshape(S, H, R, G, D)
    o = torch.where(total > 0, o, 0.0).permute(0, 2, 1, 3, 4).reshape(S * R, H * G * D)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 2, 1, 3).reshape(S * R, H * G)
    put = torch.where(live, at, s["n"]).reshape(-1)
    out = torch.empty(s["n"] + 1, H * G * D, device="cuda").index_copy(0, put, o)[:-1]
    lse = torch.empty(s["n"] + 1, H * G, device="cuda").index_copy(0, put, lse)[:-1]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def plain_score(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    d = x - top
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = (log_total - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total).squeeze(1)
    there = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
    mine = x.gather(1, s["ids"].clamp(0, c["vocab"] - 1).long()[:, None])
    logp = torch.where(there, (mine - top - log_total).squeeze(1), -math.inf)
    rank = torch.where(there, 1 + (x > mine).sum(1), 0).int()
    best, at = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    return {"logp": logp, "entropy": entropy, "rank": rank, "top_ids": at[:, : c["top"]].int(),
            "top_logp": best[:, : c["top"]].float() - top - log_total}


# ---------------------------------------------------------------- the definitions in 64 bits
def _decoded(codes):
    """e4m3 codes as the numbers they stand for: sign, four bits of exponent (bias 7), three of mantissa."""
    b = codes.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    x = torch.where((b & 127) == 127, math.nan, x)
    return torch.where(b >= 128, -x, x)


def _token_order(P, D):
    """For every (token, dim) of a page's head, the byte that holds it: K's and V's."""
    t, d = torch.arange(P, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    return ((((t // 16 * 4 + t % 16 // 4) * (D // 16) + d // 16) * 4 + t % 4) * 16 + d % 16,
            (t // 16 * D + d) * 16 + t % 16)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "score":
        got = {"logp": [], "entropy": [], "top_logp": []}
        for part, ids in zip(s["logits"].split(256), s["ids"].split(256)):
            x = part.double()
            lse = torch.logsumexp(x, 1, keepdim=True)
            lp = x - lse
            p = torch.exp(lp)
            got["entropy"].append(-(p * lp.clamp(min=-1e9)).sum(1))
            got["logp"].append(lp.gather(1, ids.long()[:, None]).squeeze(1))
            got["top_logp"].append(lp.sort(1, descending=True).values[:, : case["top"]].contiguous())
        got = {m: torch.cat(y) for m, y in got.items()}
        return {**got, "rank": None, "top_ids": None}
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    at_k, at_v = _token_order(P, D)
    lens, b = _lengths(case), 0
    if case["op"] == "write":
        n = s["n"]
        x = s["rows"].double().reshape(n, 2, H, D)
        k, v = _decoded(s["k"]), _decoded(s["v"])
        for i, (rows, length) in enumerate(lens):
            for p in range((length - rows) // P, (length - 1) // P + 1):
                lo, hi = max(p * P, length - rows), min((p + 1) * P, length)
                page = int(s["table"][i, p])
                for w, (pool, exps, at) in enumerate(((k, s["ke"], at_k), (v, s["ve"], at_v))):
                    part = x[b + lo - (length - rows): b + hi - (length - rows), w]  # [tokens, H, D]
                    big = part.abs().amax((0, 2)).clamp(min=1e-300)
                    e = torch.ceil(torch.log2(big / 448)).clamp(E_MIN - 127, E_MAX - 127)
                    e = torch.where(448 * torch.exp2(e) < big, e + 1, e)
                    if lo > p * P:
                        was = exps[page].double() - 127
                        e = torch.maximum(e, was)
                        for t in range(lo - p * P):
                            pool[page][:, at[t]] = pool[page][:, at[t]] * torch.exp2(was - e)[:, None]
                    for t in range(lo, hi):
                        pool[page][:, at[t - p * P]] = part[t - lo] * torch.exp2(-e)[:, None]
            b += rows
        return {"k": k, "v": v, "k_exp": None, "v_exp": None}
    got = {"k": [], "v": []} if case["op"] == "read" else {"out": [], "lse": []}
    for i, (rows, length) in enumerate(lens):
        page = s["table"][i, : (length + P - 1) // P].long()
        k, v = (_decoded(pool[page][:, :, at]) * torch.exp2(exps[page].double() - 127)[..., None, None]
                for pool, exps, at in ((s["k"], s["ke"], at_k), (s["v"], s["ve"], at_v)))
        k, v = (y.transpose(1, 2).reshape(-1, H, D)[:length] for y in (k, v))
        if case["op"] == "read":
            got["k"].append(k[length - rows:].reshape(rows, H * D))
            got["v"].append(v[length - rows:].reshape(rows, H * D))
            continue
        q = s["q"][b: b + rows].double().reshape(rows, H, -1, D)
        pos = torch.arange(length - rows, length, device="cuda")[:, None]
        t = torch.arange(length, device="cuda")[None]
        out = (t > pos) | ((t <= pos - case["window"]) if case["window"] else torch.zeros_like(t > pos))
        o, l = [], []
        for h in range(H):
            w = torch.matmul(q[:, h], k[:, h].t().contiguous()) * s["scale"]  # [rows, G, tokens]
            w = w.masked_fill(out[:, None], -math.inf)
            o.append(torch.matmul(torch.softmax(w, -1), v[:, h].contiguous()))
            l.append(torch.logsumexp(w, -1))
        got["out"].append(torch.stack(o, 1).reshape(rows, -1))
        got["lse"].append(torch.stack(l, 1).reshape(rows, -1))
        b += rows
    return {m: torch.cat(y) for m, y in got.items()}
