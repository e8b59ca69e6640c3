"""Cases of a decode step's further operators: the product in 8-bit floating
point with a scale for each block of 128 and the quantisation in front of it,
keys and values appended to the 8-bit paged cache with the position rotation on
the way, and the sampling of the next tokens.

``run`` makes one pass through one operator, in its plain form (elementary
torch operations) or, with ``own`` set, through the library's entry point.
``exact`` gives the same outputs from the definitions in 64 bits.  Sizes
follow the repository's own workloads where it has them: 64 decode rows, 4
sequences x 9 draft tokens, 8 segments x 512 prompt tokens, a [Q|K|V] row of
4096 + 1024 + 1024 over 4096, gate and up of 2 x 11008, a vocabulary of 32000;
the rest are generic.

8-bit product: codes are e4m3, activations have a scale for each row and 128
columns, weights one for each 128 x 128 block.  Quantisation takes the smallest
power of two s with |x| <= 448 s, within 2^-117 .. 2^120.

Rotation: pair i of a head's first `rot` dims turns by position * inv_freq[i];
pairs are (i, i + rot/2) or, interleaved, (2i, 2i + 1).  The cache is that of
perf/operators.py: pages of P tokens, one exponent byte for each page and head,
K as [P/16][4][D/16][4][16] and V as [P/16][D][16].

Sampling: token t has the weight rint(2^43 exp((x_t - max x) / T)), a whole
number.  In the order by value, equal values by the lower index first, the
first top_k tokens stay, of those the fewest whose weights reach top_p of
theirs, of those the ones of at least min_p of the largest weight; the first
always stays.  The token is the first, by index, at which the running sum of
the weights that stayed exceeds floor(u * their sum).  T = 0 takes the first.
"""
import math

import torch

own = False

E_MIN, E_MAX = 10, 247  # exponent bytes a scale may take: 2^-117 .. 2^120
UNIT = 2.0 ** 43        # the largest weight of a row's tokens
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode batch's hidden rows on their way into an 8-bit projection: launch and latency
        {"name": "quantize_step", "op": "quantize", "dtype": "bf16", "rows": 64, "k": 4096, "block": 1, "pad": 0},
        # a layer's gate and up weights brought to 8 bits when a model is loaded
        {"name": "quantize_weight", "op": "quantize", "dtype": "bf16", "rows": 22016, "k": 4096, "block": 128, "pad": 0},
        # one user's next token: the [Q|K|V] projection of one row, weights streamed once
        {"name": "matmul_one", "op": "matmul", "dtype": "bf16", "n": 1, "n_out": 6144, "k": 4096, "pad": 0},
        # a full decode batch through the vocabulary projection
        {"name": "matmul_step", "op": "matmul", "dtype": "bf16", "n": 64, "n_out": 32000, "k": 4096, "pad": 0},
        # the prompts of the prefill workload, 8 x 512 rows, through gate and up
        {"name": "matmul_prompt", "op": "matmul", "dtype": "bf16", "n": 4096, "n_out": 22016, "k": 4096, "pad": 0},
        # f32 results, sizes off every tile, the last blocks cut, rows inside wider ones
        {"name": "matmul_odd", "op": "matmul", "dtype": "f32", "n": 301, "n_out": 2056, "k": 1424, "pad": 16},
        # one token a sequence turned and appended: a decode step
        {"name": "rotate_step", "op": "rotate", "dtype": "bf16", "seqs": 64, "rows": 1, "ctx": 1000, "ragged": True,
         "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "inter": False, "theta": 10000.0, "page": 16},
        # the prompts of the prefill workload, 8 x 512 tokens, into fresh pages
        {"name": "rotate_prompt", "op": "rotate", "dtype": "bf16", "seqs": 8, "rows": 512, "ctx": 0, "ragged": False,
         "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "inter": False, "theta": 10000.0, "page": 64},
        # ragged chunks late in long contexts, f32, interleaved pairs over a part of the head, an odd head count
        {"name": "rotate_far", "op": "rotate", "dtype": "f32", "seqs": 3, "rows": 333, "ctx": 131071, "ragged": True,
         "heads": 15, "kv_heads": 5, "dim": 64, "rot": 32, "inter": True, "theta": 500000.0, "page": 32},
        # one user's next token from a large odd vocabulary
        {"name": "sample_one", "op": "sample", "dtype": "f32", "n": 1, "vocab": 131071, "mix": "nucleus"},
        # a decode batch, every user with settings of their own
        {"name": "sample_step", "op": "sample", "dtype": "bf16", "n": 64, "vocab": 32000, "mix": "all"},
        # a large batch of completions drawn in step, settings of all kinds
        {"name": "sample_many", "op": "sample", "dtype": "bf16", "n": 4096, "vocab": 32000, "mix": "all"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "rotate", "rotate", "sample", "sample"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "quantize":
        c |= {"block": rng.choice([1, 1, 128]), "k": 16 * _log(rng, 1, 1024), "pad": 16 * rng.choice([0, 0, 1, 5])}
        c["rows"] = _log(rng, 1, min(40000, 80_000_000 // c["k"]))
    elif op == "matmul":
        c |= {"n_out": 8 * _log(rng, 8, 4000), "k": 16 * _log(rng, 8, 1024), "pad": 16 * rng.choice([0, 0, 1, 5])}
        c["n_out"] = min(c["n_out"], 8 * (130_000_000 // (8 * c["k"])))
        most = int((3.5e11 if c["dtype"] == "bf16" else 0.9e11) / (c["n_out"] * c["k"]))
        c["n"] = _log(rng, 1, max(1, min(16384, most)))
    elif op == "sample":
        c |= {"vocab": _log(rng, 300, 200000), "mix": rng.choice(["all", "all", "plain", "nucleus", "top"])}
        c["n"] = _log(rng, 1, max(1, min(4096, 60_000_000 // c["vocab"])))
    else:
        c |= {"dim": rng.choice([64, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.7,
              "inter": rng.random() < 0.4, "theta": rng.choice([10000.0, 500000.0]), "kv_heads": rng.randint(1, 8)}
        c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, 16 * rng.randint(1, c["dim"] // 16)])
        c["heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 5, 7, 8])
        c["seqs"] = _log(rng, 1, 64)
        wide = (c["heads"] + 2 * c["kv_heads"]) * c["dim"] * c["seqs"]
        c["rows"] = _log(rng, 1, max(1, min(16384 // c["seqs"], 25_000_000 // wide)))
        c["ctx"] = rng.choice([0, 1, 1]) * _log(rng, 1, max(2, min(200000, 200_000_000 // (c["kv_heads"] * c["dim"] * c["seqs"]))))
    return c


# ---------------------------------------------------------------- lengths of a case
def _lengths(case):
    """(rows, tokens cached after the call) of each sequence."""
    got = []
    for i in range(case["seqs"]):
        f = (0.37 + 0.6180339887 * i) % 1.0 if case["ragged"] else 1.0
        rows = 1 + int((case["rows"] - 1) * f)
        got.append((rows, rows + int(case["ctx"] * f)))
    return got


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "quantize":
        n, k, b = case["rows"], case["k"], case["block"]
        return {"bytes": n * k * (size + 1) + 4 * -(-n // b) * -(-k // 128), "flops": 2 * n * k}
    if case["op"] == "matmul":
        n, o, k = case["n"], case["n_out"], case["k"]
        blocks = -(-k // 128)
        return {"bytes": (n + o) * k + 4 * blocks * (n + -(-o // 128)) + n * o * size, "flops": 2 * n * o * k}
    if case["op"] == "sample":
        return {"bytes": case["n"] * (case["vocab"] * size + 28), "flops": 4 * case["n"] * case["vocab"]}
    lens = _lengths(case)
    n, H, D = sum(r for r, _ in lens), case["kv_heads"], case["dim"]
    pages = sum((t - 1) // case["page"] - (t - r) // case["page"] + 1 for r, t in lens)
    return {"bytes": n * D * (2 * case["heads"] * size + 2 * H * (size + 1)) + 2 * pages * H + 4 * pages + 8 * len(lens),
            "flops": 3 * n * (case["heads"] + H) * case["rot"] + 2 * n * H * D}


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


def _blocks(x, rows, cols):
    """[ceil(n / rows), rows, ceil(k / cols), cols], zeros where the last blocks are cut."""
    n, k = x.shape
    x = torch.nn.functional.pad(x, (0, -k % cols, 0, -n % rows))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // cols, cols)


def _code(case):
    from adapter_lora_bgmv_amd import binding as B
    return B.LORA_BF16 if case["dtype"] == "bf16" else B.LORA_F32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return globals()["prepare_" + case["op"]](case, g, TYPES[case["dtype"]])


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare_quantize(case, g, dt):
    n, k, pad = case["rows"], case["k"], case["pad"]
    if case["block"] == 1:  # hidden rows: a few strong channels, rows of unlike size
        x = _normal(g, n, k) * torch.where(torch.arange(k, device="cuda") % 61 == 7, 12.0, 1.0) * torch.exp2(_normal(g, n, 1))
    else:
        x = _normal(g, n, k) * 0.02
    wide = torch.zeros(n, k + pad, dtype=dt, device="cuda")
    wide[:, :k] = x.to(dt)
    s = {"case": case, "x": wide, "codes": torch.zeros(n, k + pad, dtype=torch.uint8, device="cuda"),
         "scale": torch.zeros(-(-n // case["block"]), -(-k // 128), device="cuda")}
    if own:
        s["code"] = _code(case)
    return s


def prepare_matmul(case, g, dt):
    n, o, k, pad = case["n"], case["n_out"], case["k"], case["pad"]
    x = _normal(g, n, k) * torch.where(torch.arange(k, device="cuda") % 61 == 7, 12.0, 1.0) * torch.exp2(_normal(g, n, 1))
    w = _normal(g, o, k) * 0.02 * torch.exp2(0.5 * _normal(g, o, 1))
    s = {"case": case}
    for name, t, b in (("x", x, 1), ("w", w, 128)):
        t4 = _blocks(t, b, 128)
        # scales as checkpoints hold them: the largest magnitude over 448, no power of two
        scale = t4.abs().amax((1, 3)).clamp(min=1e-12) / 448.0
        codes = (t4 / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        codes = codes.reshape(t4.shape[0] * b, -1)[: t.shape[0], :k]
        wide = torch.zeros(t.shape[0], k + pad, dtype=torch.uint8, device="cuda")
        wide[:, :k] = codes
        s[name], s[name + "_scale"] = wide, scale.contiguous()
    s["y"] = torch.zeros(n, o + pad, dtype=dt, device="cuda")
    if own:
        from adapter_lora_bgmv_amd import binding as B
        s["code"] = _code(case)
        s["ws_bytes"] = B.lora_matmul_fp8_workspace_bytes(s["code"], o, k, n)
        s["ws"] = torch.zeros(max(s["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    return s


def prepare_rotate(case, g, dt):
    H, D, P, heads = case["kv_heads"], case["dim"], case["page"], case["heads"]
    lens = _lengths(case)
    used = [(t + P - 1) // P for _, t in lens]
    per, n_pages, n = max(used), sum(used) + 3, sum(r for r, _ in lens)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    starts = torch.tensor([0] + used, device="cuda").cumsum(0)
    at = torch.arange(per, device="cuda")[None] + starts[:-1, None]
    ok = torch.arange(per, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]
    s = {"case": case, "n": n, "table": torch.where(ok, order[at.clamp(max=n_pages - 1)], -1).int().contiguous(),
         "indptr": torch.tensor([0] + [r for r, _ in lens], device="cuda").cumsum(0).int(),
         "kv_len": torch.tensor([t for _, t in lens], device="cuda").int(), "most_rows": max(r for r, _ in lens)}
    # what the pages hold from before: codes of ordinary size, either sign
    for m in "kv":
        s[m] = torch.randint(0, 254, (n_pages, H, P * D), generator=g, device="cuda", dtype=torch.uint8)
        s[m] += (s[m] >= 127).to(torch.uint8)  # 0x7f is NaN, and 0xff out of range
        s[m + "e"] = torch.randint(118, 121, (n_pages, H), generator=g, device="cuda", dtype=torch.uint8)
    s["qkv"] = (_normal(g, n, (heads + 2 * H) * D) * torch.exp2(0.7 * _normal(g, n, 1))).to(dt)
    s["q_out"] = torch.zeros(n, heads * D, dtype=dt, device="cuda")
    i = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
    s["inv_freq"] = (case["theta"] ** (-i / case["rot"])).float()
    if own:
        from adapter_lora_bgmv_amd import binding as B
        s["code"] = _code(case)
        s["cache"] = B.KVCache(s["k"], s["v"], s["ke"], s["ve"], page_tokens=P, head_dim=D)
        s["seqs"] = B.KVSeqs(s["table"], s["indptr"], s["kv_len"], max_rows=s["most_rows"])
        s["rotary"] = B.Rotary(s["inv_freq"], interleaved=case["inter"])
    return s


def prepare_sample(case, g, dt):
    n, V = case["n"], case["vocab"]

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    # a few likely tokens over a broad tail; a part of the vocabulary ruled out, as a grammar does
    x = _normal(g, n, V) * 2.5 + 2.0 * _normal(g, 1, V)
    out = uniform(V) < 0.03
    out[0] = False
    s = {"case": case, "logits": x.masked_fill(out, -math.inf).to(dt), "u": uniform(n)}
    # temperatures of 0 (one row in ten), 0.5 .. 1.3 and 1; what a row's user set beside it
    t = torch.where(uniform(n) < 0.3, 1.0, 0.5 + 0.8 * uniform(n))
    k = (5 * torch.exp2(5 * uniform(n))).int()  # 5 .. 160
    p, m = 0.8 + 0.19 * uniform(n), 0.02 + 0.1 * uniform(n)
    mix = case["mix"]
    if mix == "all":
        t = torch.where(uniform(n) < 0.1, 0.0, t)
    s["temperature"] = t
    s["top_k"] = torch.where(uniform(n) < {"all": 0.4, "top": 1.1}.get(mix, 0.0), k, 0).int()
    s["top_p"] = torch.where(uniform(n) < {"all": 0.5, "nucleus": 1.1}.get(mix, 0.0), p, 1.0)
    s["min_p"] = torch.where(uniform(n) < {"all": 0.2}.get(mix, 0.0), m, 0.0)
    s["ids"], s["logp"] = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda")
    if own:
        from adapter_lora_bgmv_amd import binding as B
        s["code"] = _code(case)
        s["ws_bytes"] = B.lora_token_sample_workspace_bytes(s["code"], V, n)
        s["ws"] = torch.zeros(max(s["ws_bytes"], 256), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return globals()[("own_" if own else "plain_") + s["case"]["op"]](s)


def own_quantize(s):
    from adapter_lora_bgmv_amd import binding as B
    c, wide = s["case"], s["x"].shape[1]
    B.lora_quantize_fp8(s["code"], c["rows"], c["k"], s["x"], wide, c["block"], s["codes"], wide, s["scale"], s["scale"].shape[1])
    return {"codes": s["codes"][:, : c["k"]].view(torch.float8_e4m3fn), "scale": s["scale"]}


def own_matmul(s):
    from adapter_lora_bgmv_amd import binding as B
    c, wide = s["case"], s["x"].shape[1]
    B.lora_matmul_fp8(s["code"], c["n_out"], c["k"], s["w"], wide, s["w_scale"], s["w_scale"].shape[1], s["x"], wide, s["x_scale"],
                      s["x_scale"].shape[1], c["n"], s["y"], s["y"].shape[1], s["ws"], s["ws_bytes"])
    return {"y": s["y"][:, : c["n_out"]]}


def own_rotate(s):
    from adapter_lora_bgmv_amd import binding as B
    c, wide = s["case"], s["qkv"].shape[1]
    q, kv = c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
    B.lora_kv_write_rotary(s["cache"], s["seqs"], s["rotary"], s["code"], c["heads"], s["qkv"], wide, s["q_out"], q,
                           s["qkv"][:, q:], wide, s["qkv"][:, q + kv:], wide, s["n"])
    return {"q": s["q_out"], "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_exp": s["ke"],
            "v_exp": s["ve"]}


def own_sample(s):
    from adapter_lora_bgmv_amd import binding as B
    c = s["case"]
    B.lora_token_sample(s["code"], c["vocab"], s["logits"], c["vocab"], s["temperature"], s["top_k"], s["top_p"], s["min_p"],
                        s["u"], c["n"], s["ids"], s["logp"], s["ws"], s["ws_bytes"])
    return {"ids": s["ids"], "logp": s["logp"]}


def plain_quantize(s):
    c = s["case"]
    n, k, b = c["rows"], c["k"], c["block"]
    x = _blocks(s["x"][:, :k].float(), b, 128)
    scale = _power(_need(x.abs().amax((1, 3))))
    codes = (x / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(x.shape[0] * b, -1)
    s["codes"][:, :k] = codes[:n, :k]
    s["scale"].copy_(scale)
    return {"codes": s["codes"][:, :k].view(torch.float8_e4m3fn), "scale": s["scale"]}


def plain_matmul(s):
    c = s["case"]
    n, o, k = c["n"], c["n_out"], c["k"]
    x = s["x"][:, :k].view(torch.float8_e4m3fn).float() * s["x_scale"].repeat_interleave(128, 1)[:, :k]
    w = s["w"][:, :k].view(torch.float8_e4m3fn).float() * s["w_scale"].repeat_interleave(128, 0)[:o].repeat_interleave(128, 1)[:, :k]
    s["y"][:, :o] = (x @ w.t()).to(s["y"].dtype)
    return {"y": s["y"][:, :o]}


def _angles(s, pos):
    """cos and sin [n, 1, rot / 2] in 64 bits: far positions times frequencies."""
    a = pos.double()[:, None] * s["inv_freq"].double()
    return torch.cos(a)[:, None], torch.sin(a)[:, None]


def _turned(x, cos, sin, rot, inter):
    """Heads [n, heads, D] with their first `rot` dims turned."""
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def plain_rotate(s):
    c, n = s["case"], s["n"]
    H, D, P, heads = c["kv_heads"], c["dim"], c["page"], c["heads"]
    r = torch.arange(n, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["indptr"][1:].contiguous(), r, right=True)
    pos = s["kv_len"][seq] - s["indptr"][seq + 1] + r
    page, at = s["table"][seq, pos // P].long(), (pos % P).long()
    x = s["qkv"].reshape(n, heads + 2 * H, D)
    cos, sin = _angles(s, pos)
    s["q_out"].copy_(_turned(x[:, :heads].float(), cos.float(), sin.float(), c["rot"], c["inter"]).reshape(n, heads * D))
    # in 64 bits: which code and which scale a key next to a border takes
    k = _turned(x[:, heads: heads + H].double(), cos, sin, c["rot"], c["inter"]).float()
    v = x[:, heads + H:].float()
    start = s["kv_len"] - (s["indptr"][1:] - s["indptr"][:-1])
    first = s["table"][torch.arange(c["seqs"], device="cuda"), start // P].long()  # the page that each sequence's rows begin in
    kept = torch.arange(P, device="cuda")[None, :] < (start % P)[:, None]           # its tokens from before
    a = torch.arange(D, device="cuda")
    t, h = at[:, None, None], torch.arange(H, device="cuda")[None, :, None]
    place_k = (t // 16) * (16 * D) + (t % 16 // 4) * (4 * D) + (a // 16) * 64 + (t % 4) * 16 + a % 16
    place_v = (t // 16) * (16 * D) + a * 16 + t % 16
    _write_one(s["k"], s["ke"], k, page, first, kept, place_k, h, _untile_k, P, D, lambda o: _tile(o, o)[0])
    _write_one(s["v"], s["ve"], v, page, first, kept, place_v, h, _untile_v, P, D, lambda o: _tile(o, o)[1])
    return {"q": s["q_out"], "k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_exp": s["ke"],
            "v_exp": s["ve"]}


def _write_one(pool, exps, x, page, first, kept, place, h, untile, P, D, tile):
    most = torch.zeros(exps.shape, device="cuda").scatter_reduce(0, page[:, None].expand(x.shape[:2]), x.abs().amax(2), "amax")
    need = _need(most)
    # a page with tokens from before keeps at least their scale, and they follow it where it grows
    before = exps[first].to(need.dtype)
    after = torch.where(kept.any(1)[:, None], torch.maximum(before, need[first]), need[first])
    codes = untile(pool[first], P, D)
    moved = codes.view(torch.float8_e4m3fn).float() * torch.ldexp(torch.ones_like(after, dtype=torch.float32), before - after)[..., None, None]
    codes = torch.where(kept[:, None, :, None], moved.to(torch.float8_e4m3fn).view(torch.uint8), codes)
    pool[first] = tile(codes)
    need[first] = after
    exps[page] = need[page].to(torch.uint8)
    pool[page[:, None, None], h, place] = (x / _power(need[page])[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def plain_sample(s):
    # in 64 bits and whole numbers: a running sum next to the number drawn
    V = s["case"]["vocab"]
    x = s["logits"].double()
    top = x.amax(1, keepdim=True)
    greedy = s["temperature"][:, None] == 0
    t = torch.where(greedy, 1.0, s["temperature"][:, None].double())
    w = torch.round(torch.exp((x - top) / t) * UNIT).long()
    best, order = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    at = torch.arange(V, device="cuda")[None]
    k = torch.where(greedy, 1, torch.where(s["top_k"][:, None] > 0, s["top_k"][:, None].long(), V))
    ws = w.gather(1, order)
    kept = at < k
    run_sum = ws.cumsum(1)
    mass = torch.where(kept, ws, 0).sum(1, keepdim=True)
    p = s["top_p"][:, None].double()
    kept &= (p >= 1) | (run_sum - ws < torch.ceil(p * mass.double()).long())
    kept &= ws >= torch.ceil(s["min_p"][:, None].double() * UNIT).long()
    kept |= at == 0
    w = torch.where(torch.zeros_like(kept).scatter(1, order, kept), w, 0)
    run_sum = w.cumsum(1)
    total = run_sum[:, -1:]
    goal = torch.minimum(torch.floor(s["u"][:, None].double() * total.double()).long(), total - 1)
    at = (run_sum <= goal).sum(1, keepdim=True)
    logp = (x.gather(1, at) - top) / t - torch.log(total.double() / UNIT)
    s["ids"].copy_(at.squeeze(1))
    s["logp"].copy_(torch.where(greedy, 0.0, logp).squeeze(1))
    return {"ids": s["ids"], "logp": s["logp"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def _decoded(codes):
    """e4m3 codes as the numbers they stand for: sign, four bits of exponent (bias 7), three of mantissa."""
    b = codes.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    x = torch.where((b & 127) == 127, math.nan, x)
    return torch.where(b >= 128, -x, x)


def _smallest_power(big):
    """log2 of the smallest power of two s with big <= 448 s, within the range of scales."""
    e = torch.ceil(torch.log2(big.clamp(min=1e-300) / 448)).clamp(E_MIN - 127, E_MAX - 127)
    return torch.where(448 * torch.exp2(e) < big, e + 1, e)


def exact(case, seed):
    return globals()["exact_" + case["op"]](case, prepare(case, seed))


def exact_quantize(case, s):
    n, k, b = case["rows"], case["k"], case["block"]
    x = s["x"][:, :k].double()
    scale = torch.zeros_like(s["scale"], dtype=torch.float64)
    y = torch.zeros_like(x)
    for j in range(scale.shape[1]):
        part = x[:, 128 * j: 128 * (j + 1)]
        big = torch.nn.functional.pad(part.abs().amax(1), (0, -n % b)).reshape(-1, b).amax(1)
        scale[:, j] = torch.exp2(_smallest_power(big))
        y[:, 128 * j: 128 * (j + 1)] = part / scale[:, j].repeat_interleave(b)[:n, None]
    return {"codes": y, "scale": scale}


def exact_matmul(case, s):
    n, o, k = case["n"], case["n_out"], case["k"]
    y = torch.zeros(n, o, dtype=torch.float64, device="cuda")
    for j in range(s["x_scale"].shape[1]):
        x = _decoded(s["x"][:, 128 * j: min(k, 128 * (j + 1))]) * s["x_scale"][:, j: j + 1].double()
        w = _decoded(s["w"][:, 128 * j: min(k, 128 * (j + 1))])
        for b in range(s["w_scale"].shape[0]):
            w[128 * b: 128 * (b + 1)] *= s["w_scale"][b, j].double()
        y += torch.matmul(x, w.t().contiguous())
    return {"y": y}


def exact_rotate(case, s):
    H, D, P, heads, rot = case["kv_heads"], case["dim"], case["page"], case["heads"], case["rot"]
    t, d = torch.arange(P, device="cuda")[:, None], torch.arange(D, device="cuda")[None]
    at_k = (((t // 16 * 4 + t % 16 // 4) * (D // 16) + d // 16) * 4 + t % 4) * 16 + d % 16
    at_v = (t // 16 * D + d) * 16 + t % 16
    lens, b = _lengths(case), 0
    if sum((r + P - 1) // P + 1 for r, _ in lens) > 3000:
        return None
    x = s["qkv"].double().reshape(s["n"], heads + 2 * H, D)
    i = torch.arange(rot // 2, device="cuda")
    one, two = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
    pos = torch.cat([torch.arange(length - rows, length, device="cuda") for rows, length in lens]).double()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos[:, None] * s["inv_freq"].double())[:, None]
    z = torch.complex(x[:, : heads + H, one], x[:, : heads + H, two]) * turn
    x[:, : heads + H, one], x[:, : heads + H, two] = z.real, z.imag
    k, v = _decoded(s["k"]), _decoded(s["v"])
    for n, (rows, length) in enumerate(lens):
        for p in range((length - rows) // P, (length - 1) // P + 1):
            lo, hi = max(p * P, length - rows), min((p + 1) * P, length)
            page = int(s["table"][n, p])
            for pool, exps, at, h0 in ((k, s["ke"], at_k, heads), (v, s["ve"], at_v, heads + H)):
                part = x[b + lo - (length - rows): b + hi - (length - rows), h0: h0 + H]  # [tokens, H, D]
                e = _smallest_power(part.abs().amax((0, 2)))
                if lo > p * P:
                    was = exps[page].double() - 127
                    e = torch.maximum(e, was)
                    old = at[: lo - p * P].reshape(-1)
                    pool[page][:, old] = pool[page][:, old] * torch.exp2(was - e)[:, None]
                new = at[lo - p * P: hi - p * P].reshape(-1)
                pool[page][:, new] = (part * torch.exp2(-e)[:, None]).transpose(0, 1).reshape(H, -1)
        b += rows
    return {"q": x[:, :heads].reshape(s["n"], heads * D), "k": k, "v": v, "k_exp": None, "v_exp": None}


def exact_sample(case, s):
    got = []
    for a in range(0, case["n"], 128):
        x = s["logits"][a: a + 128].double()
        t, k, p, m, u = (s[name][a: a + 128, None].double() for name in ("temperature", "top_k", "top_p", "min_p", "u"))
        y = x / torch.where(t == 0, 1.0, t)
        prob = torch.softmax(y, 1)
        value, order = torch.sort(x, dim=1, descending=True, stable=True)
        q = prob.gather(1, order)
        place = torch.arange(case["vocab"], device="cuda")[None].double()
        q = torch.where((k > 0) & (place >= k), 0.0, q)
        q = q / q.sum(1, keepdim=True)
        q = torch.where((p < 1) & (q.cumsum(1) - q >= p) & (place > 0), 0.0, q)
        q = torch.where(q < m * q[:, :1], 0.0, q)
        q = torch.where((t == 0) & (place > 0), 0.0, q)
        q = q / q.sum(1, keepdim=True)
        back = torch.zeros_like(q).scatter(1, order, q)
        pick = (back.cumsum(1) <= u).sum(1, keepdim=True).clamp(max=case["vocab"] - 1)
        got.append(torch.log(back.gather(1, pick)).squeeze(1))
    return {"ids": None, "logp": torch.cat(got)}
