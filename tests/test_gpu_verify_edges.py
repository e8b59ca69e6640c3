"""Edges of the verify-step operators' contracts: row ranges that decrease or
leave the call, the ends of the size ranges, unusual numbers, other streams."""
import numpy as np
import pytest

import verify_ref as R
from adapter_lora_bgmv_amd import binding as B
from test_gpu_verify import DT, Setup, check_scores, dev, host
from test_gpu_verify_forms import set_codes

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lora_init()


# ---------------------------------------------------------------- row ranges
RANGES = [
    # row_indptr (repeated to the sequences), n
    ("falls", lambda S: [0, 16] * (S // 2) + [0], 16),
    ("falls once, long ones overlapping", lambda S: [0] * (S - 3) + [16, 0, 16, 0], 16),
    ("leaves [0, n)", lambda S: [-7] + list(range(-3, S - 4)) + [2 ** 31 - 1], 20),
    ("falls outside [0, n)", lambda S: [-3, -9] * (S // 2) + [2 ** 31 - 1], 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name,make,n", RANGES)
def test_row_ranges_that_fall_or_leave_the_call(name, make, n, dtype):
    """Sequences short and long, some of them split: whatever the ranges, nothing
    outside the operands changes, and a workspace full of a larger call's leavings is
    no way out of them.  Ranges that only leave [0, n) serve the rows inside it."""
    S, H, G, D, P = 64, 2, 2, 64, 16
    heads = H * G
    s = Setup(400, [(1, 60)] * (S - 2) + [(1, 6000)] * 2, H, D, P)
    code = DT[dtype][0]
    tdt = getattr(torch, DT[dtype][1])
    # the larger call that the workspace remembers
    big = Setup(401, [(200, 5000), (190, 3000), (3, 8000)], H, D, P)
    for max_rows in (1, 0):
        seqs = B.KVSeqs(dev(s.seqs["table"]), dev(np.array(make(S), np.int32)), dev(s.seqs["kv_len"]), max_rows=max_rows)
        need = B.lora_kv_attend_workspace_bytes(s.cache, seqs, code, heads, n)
        ws = torch.zeros(max(need, B.lora_kv_attend_workspace_bytes(big.cache, big.dseqs, code, heads, big.n)), dtype=torch.uint8,
                         device="cuda")
        big.attend(dtype, heads, ws=ws)
        row, pad = heads * D, 64
        q = torch.randn(n, row, device="cuda").to(tdt)
        box = torch.full((pad + n + pad, row), 33.0, dtype=tdt, device="cuda")
        lbox = torch.full((pad + n + pad, heads), 33.0, device="cuda")
        B.lora_kv_attend(s.cache, seqs, code, heads, q, row, 0.125, 0, n, box[pad:], row, lbox[pad:], ws, ws.numel())
        torch.cuda.synchronize()
        for t in (box, lbox):
            assert bool((t[:pad] == 33).all()) and bool((t[pad + n:] == 33).all())
        if name == "leaves [0, n)":  # a row a sequence
            want, wl, mag, big_, toks = R.attend(s.host, {**s.seqs, "indptr": np.clip(make(S), 0, n)},
                                                 host(q).reshape(n, heads, D), 0.125, 0)
            bo, bl = R.attend_bounds(dtype, want, wl, mag, big_, toks, D)
            assert (np.abs(host(box[pad:pad + n]).reshape(want.shape) - want) <= bo).all()
            assert (np.abs(host(lbox[pad:pad + n]) - wl) <= bl).all()
        # reads stay inside their rows, writes inside the pool
        kbox, vbox = (torch.full((pad + n + pad, H * D), 33.0, dtype=tdt, device="cuda") for _ in range(2))
        B.lora_kv_read(s.cache, seqs, code, kbox[pad:], H * D, vbox[pad:], H * D, n)
        pool = torch.full((s.cache.k.numel() + 2 * 4096,), 99, dtype=torch.uint8, device="cuda")
        shape = s.cache.k.shape
        kp = pool[4096:-4096].view(shape)
        other = B.KVCache(kp, kp.clone(), s.cache.k_scale.clone(), s.cache.v_scale.clone(), page_tokens=P, head_dim=D)
        B.lora_kv_write(other, seqs, code, q, row, q[:, H * D:], row, n)
        torch.cuda.synchronize()
        for t in (kbox, vbox):
            assert bool((t[:pad] == 33).all()) and bool((t[pad + n:] == 33).all())
        assert bool((pool[:4096] == 99).all()) and bool((pool[-4096:] == 99).all())
    s.check(dtype, heads)  # and the next call is served as ever


# ---------------------------------------------------------------- cache
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_numbers_read_back(dtype):
    """Under the largest scale, 2^120, codes up to 240 are read exactly, and what
    is rounded to 256 or more as infinity; a page's smaller values stay exact."""
    H, D, P = 1, 64, 16
    top = 2.0 ** 120
    s = Setup(430, [(7, 7)], H, D, P)
    x = np.zeros((7, 2 * D))
    # 248 is the tie between 240 and 256; bf16 has the numbers used here
    for t, v in enumerate([255.0, 248.0, 247.0, 240.0, 224.5, 2.0, 0.0]):
        x[t] = v * top * np.where(np.arange(2 * D) % 3 == 1, -1.0, 1.0)
    x[6, 9] = 2.0 ** 111
    dx = dev(x, dtype)
    B.lora_kv_write(s.cache, s.dseqs, DT[dtype][0], dx, 2 * D, dx[:, D:], 2 * D, s.n)
    o = torch.zeros_like(dx)
    B.lora_kv_read(s.cache, s.dseqs, DT[dtype][0], o, 2 * D, o[:, D:], 2 * D, s.n)
    torch.cuda.synchronize()
    assert host(s.cache.k_scale)[s.seqs["table"][0, 0], 0] == 247
    want = np.sign(x) * np.array([np.inf, np.inf, 240 * top, 240 * top, 224 * top, 2 * top, 1.0])[:, None]
    want[6] = 0.0
    want[6, 9] = 2.0 ** 111
    assert np.array_equal(host(o), want)

# ---------------------------------------------------------------- windows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 31 - 60, 5000])
def test_windows_wider_than_the_sequences_hide_nothing(window, D, dtype):
    """Up to the largest, also where a sequence has more rows than tokens, and
    so rows at negative positions."""
    s = Setup(410, [(6, 3), (40, 3), (70, 64), (3, 1), (5, 700)], 1, D, 16)
    s.check(dtype, 4, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 50, 2 ** 31 - 1, 2 ** 31 - 30])
def test_lengths_far_past_the_page_table(window, dtype):
    """Up to the largest int: the rows stand past every page and see what the table
    holds, or the part that a window of nearly that size leaves."""
    s = Setup(411, [(5, 64), (40, 64), (1, 50), (2, 33)], 1, 64, 16)
    s.seqs["kv_len"][:] = [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 1, 33]
    s.upload()
    s.check(dtype, 4, window)
    x = torch.randn(s.n, 128, device="cuda")
    before = host(s.cache.k).copy()
    s.seqs["kv_len"][3] = 0
    s.upload()
    B.lora_kv_write(s.cache, s.dseqs, B.LORA_F32, x, 128, x[:, 64:], 128, s.n)
    o = torch.full_like(x, 5.0)
    B.lora_kv_read(s.cache, s.dseqs, B.LORA_F32, o, 128, o[:, 64:], 128, s.n)
    torch.cuda.synchronize()
    assert np.array_equal(host(s.cache.k), before) and bool((o == 5).all())


def test_a_cache_past_four_gibibytes():
    """The last pages of a pool of 5 GiB a side give what the same pages give in a small one."""
    H, D, P, heads = 8, 128, 128, 16
    s = Setup(440, [(1, 900), (3, 300), (40, 500)], H, D, P)
    few, many = s.host.ke.shape[0], 40960
    shift = many - few
    pools = [torch.empty(many, H, P * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.empty(many, H, dtype=torch.uint8, device="cuda") for _ in range(2)]
    size = pools[0].numel()
    assert size >= 5 << 30
    for big, small in zip(pools + exps, (s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale)):
        big[shift:] = small
    large = B.KVCache(*pools, *exps, page_tokens=P, head_dim=D)
    table = s.seqs["table"]
    seqs = B.KVSeqs(dev(np.where(table >= 0, table + shift, table).astype(np.int32)), s.dseqs.row_indptr, s.dseqs.kv_len)
    x = torch.randn(s.n, 2 * H * D, device="cuda").bfloat16()
    q = torch.randn(s.n, heads * D, device="cuda").bfloat16()
    got = []
    for cache, sq in ((s.cache, s.dseqs), (large, seqs)):
        B.lora_kv_write(cache, sq, B.LORA_BF16, x, 2 * H * D, x[:, H * D:], 2 * H * D, s.n)
        o = torch.zeros_like(x)
        B.lora_kv_read(cache, sq, B.LORA_BF16, o, 2 * H * D, o[:, H * D:], 2 * H * D, s.n)
        need = B.lora_kv_attend_workspace_bytes(cache, sq, B.LORA_BF16, heads, s.n)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(q)
        B.lora_kv_attend(cache, sq, B.LORA_BF16, heads, q, heads * D, D ** -0.5, 0, s.n, out, heads * D, None, ws, need)
        torch.cuda.synchronize()
        got.append([host(o), host(out)] + [host(t[-few:]) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)])
    for a, b in zip(*got):
        assert np.array_equal(a, b, equal_nan=a.dtype.kind == "f")
    assert np.abs(got[0][1]).max() > 0.1

# ---------------------------------------------------------------- values near the end of f32's range
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 20000)], [(20, 20000), (3, 500)]])
@pytest.mark.parametrize("power", [57, 70, 106, 116])
def test_sums_over_many_large_values(power, lens, dtype):
    """Values of 2^power in every page, then in every third of them: the output is
    a mean of them and as finite as they are."""
    s = Setup(420, lens, 1, 64, 128)
    place = {int(p): i for i, p in enumerate(s.seqs["table"][0])}
    set_codes(s, "v", lambda p, x: (2.0 + np.clip(x, -1.0, 2.0)) * 2.0 ** power)
    s.check(dtype, 2, scale=2.0 ** -20)  # nearly equal weights
    s.check(dtype, 2)
    set_codes(s, "v", lambda p, x: x if place.get(p, 0) % 3 else x * 2.0 ** -power)
    s.check(dtype, 2)

# ---------------------------------------------------------------- weights far below the largest
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 300)], [(9, 300)], [(40, 300)]])
@pytest.mark.parametrize("gap", [10, 20, 26, 31, 36, 60])
def test_small_weights_where_the_largest_meet_zeros(gap, lens, dtype):
    """One token outweighs all others by 2^gap and is zero in half of the dims,
    where the outputs are the others': as exact as any down to 2^-22, from
    there on within half a step, 2^-33 of the largest weight, a token."""
    D, pos = 64, 5
    s = Setup(450, lens, 1, D, 16, spread=0.0)
    page = int(s.seqs["table"][0, pos // 16])

    def keys(p, x):
        y = np.zeros_like(x)
        y[:, 0] = x[:, 0] * 0.01
        if p == page:
            y[pos, 0] = gap * np.log(2.0)
        return y

    def values(p, x):
        if p == page:
            x[pos, ::2] = 0.0
        return x

    set_codes(s, "k", keys)
    set_codes(s, "v", values)
    q = np.zeros((s.n, 2, D))
    q[:, :, 0] = 1.0
    q, out, lse = s.attend(dtype, 2, scale=1.0, q=q)
    want, wl, mag, big, toks = R.attend(s.host, s.seqs, q, 1.0, 0)
    bo, bl = R.attend_bounds(dtype, want, wl, mag, big, toks, D)
    if dtype == "bf16" and gap > 21:  # keys' rounding moves the gap by a part in 16
        pages = s.seqs["table"][0, :-(-lens[0][1] // 16)]
        v = R.TABLE[s.host.v[pages, 0]] * np.exp2(s.host.ve[pages, 0].astype(float) - 127)[:, None, None]
        bo = bo + 2.0 ** -33 * np.abs(v.reshape(-1, D)[:lens[0][1]]).sum(0)
    assert (np.abs(out - want) <= bo).all() and (np.abs(lse - wl) <= bl).all()
    assert np.abs(out[..., ::2]).max() < 300 * 2.0 ** -(gap * 15 / 16) * 300

# ---------------------------------------------------------------- streams
def small_step(seed=5):
    from adapter_lora_bgmv_amd import verify_step as V
    z = V.Sizes(hidden=512, heads=8, kv_heads=2, head_dim=64, vocab=1000, page_tokens=16, slots=3, rank=16)
    step = V.VerifyStep(z, n_seqs=3, draft=4, max_tokens=208, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(7)
    for t in (step.cache.k, step.cache.v):
        t.copy_(torch.randint(0, 126, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    step.cache.k_scale.fill_(120)
    step.cache.v_scale.fill_(118)
    torch.cuda.synchronize()
    return step


@pytest.mark.parametrize("raw", [False, True])  # a torch stream, a raw handle
def test_verify_steps_on_a_side_stream(raw):
    """Steps one after the other on another stream give what they give on the
    current one, though the stream is kept busy while the next inputs come."""
    rng = np.random.default_rng(8)
    lens = [[50 + 4 * i, 7 + 4 * i, 150 + 4 * i] for i in range(6)]
    ids = [rng.integers(0, 1000, 12) for _ in lens]
    xs = [torch.from_numpy(rng.standard_normal((12, 512))).cuda().bfloat16() for _ in lens]
    outs = []
    for side in (False, True):
        step, got = small_step(), []
        stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
        busy = torch.zeros(1 << 26, device="cuda")
        torch.cuda.synchronize()
        for x, l, i in zip(xs, lens, ids):
            with torch.cuda.stream(stream):
                for _ in range(10):
                    busy.add_(1.0)
            step.run(x, l, i, (stream.cuda_stream if raw else stream) if side else None)
            with torch.cuda.stream(stream):
                got += [t.clone() for t in step.scores.values()] + [step.out.clone()]
        torch.cuda.synchronize()
        outs.append([host(t) for t in got] + [host(step.cache.k), host(step.cache.v)])
    for a, b in zip(*outs):
        assert np.array_equal(a, b)


# ---------------------------------------------------------------- scores
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,short,top", [(1, 0, 32), (2, 0, 32), (3, 1, 31), (2, 2, 32), (3, 6, 32), (2, 7, 30)])
def test_scores_at_the_end_of_the_vocabulary_range(n, short, top, dtype):
    """Rows of 2^20 logits or a few less that begin at every place of a 16-byte
    vector, their largest logits at the very end."""
    V = (1 << 20) - short
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((n, V))
    x[:, V - 9:] = 8.0 + np.arange(9)
    x[:, 3] = 7.0
    for skew, extra in ((1, 1), (3, 2), (7, 3)):
        check_scores(x, [V - 1] * n, top, dtype, skew, V + extra)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,top", [(4, 40, 32), (4, 900, 32), (4, 70001, 32), (1100, 900, 5)])
def test_alternatives_of_rows_with_nan_lie_in_the_vocabulary(n, V, top, dtype):
    """NaN of either sign, in all of a row, most of it or half of it: NaN scores and different ids in range."""
    rng = np.random.default_rng(V)
    x = torch.from_numpy(rng.standard_normal((n, V)).astype(np.float32)).cuda()
    share = torch.tensor([1.0, 0.97, 0.5, 1.0], device="cuda").repeat(n // 4)[:, None]
    nan = torch.from_numpy(rng.random((n, V)).astype(np.float32)).cuda() < share
    nan[:, 0] = True
    bits, ty = (x.to(torch.bfloat16), torch.int16) if dtype == "bf16" else (x, torch.int32)
    quiet = 0x7FC0 << (0 if dtype == "bf16" else 16)
    sign = torch.from_numpy(rng.random((n, V))).cuda() < torch.tensor([1.0, 1.0, 0.5, 0.0], device="cuda").repeat(n // 4)[:, None]
    lowest = -(1 << 15) if dtype == "bf16" else -(1 << 31)
    filled = torch.where(sign, torch.tensor(quiet + lowest, dtype=ty, device="cuda"), torch.tensor(quiet, dtype=ty, device="cuda"))
    logits = torch.where(nan, filled, bits.view(ty)).view(bits.dtype)
    assert torch.isnan(logits[0]).all() and bool(torch.signbit(logits[0]).all())
    code = DT[dtype][0]
    need = B.lora_token_logprobs_workspace_bytes(code, V, n, top)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    lp, en, tl = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, top, device="cuda")
    ti = torch.full((n, top), -9, dtype=torch.int32, device="cuda")
    for _ in range(2):
        B.lora_token_logprobs(code, V, logits, V, torch.zeros(n, dtype=torch.int32, device="cuda"), n, top, lp, en, None, ti, tl,
                              ws, need)
    torch.cuda.synchronize()
    for t in (lp, en, tl):
        assert bool(torch.isnan(t).all())
    assert bool(((ti >= 0) & (ti < V)).all())
    assert bool((ti.sort(1).values.diff(dim=1) > 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,top", [(3, 40, 32), (3, 900, 20), (3, 70001, 32), (1100, 900, 5)])
def test_zeros_of_either_sign_are_equal(n, V, top, dtype):
    """Rows whose largest logits are 0 and -0, many of them or a few."""
    rng = np.random.default_rng(V + 1)
    for share in (1.0, 0.3, 6.0 / V):
        x = -np.abs(rng.standard_normal((n, V))) - 1.0
        zero = rng.random((n, V)) < share
        x[zero] = 0.0
        x[zero & (rng.random((n, V)) < 0.5)] = -0.0
        check_scores(x, rng.integers(0, V, n), top, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,top", [(513, 100001, 20), (512, 200000, 0), (130, 1 << 20, 7)])
def test_scores_of_many_rows_over_a_large_vocabulary(n, V, top, dtype):
    """A workgroup to a row, or a few: hundreds of terms to a thread's running sums."""
    code, name = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(n, V, generator=g, device="cuda") * 3.0).to(getattr(torch, name))
    ids = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)
    lp, en, tl = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, top, device="cuda")
    rk, ti = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, top, dtype=torch.int32, device="cuda")
    need = B.lora_token_logprobs_workspace_bytes(code, V, n, top)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    B.lora_token_logprobs(code, V, x, V, ids, n, top, lp, en, rk, ti, tl, ws, need)
    torch.cuda.synchronize()
    some = list(range(0, n, max(n // 9, 1))) + [n - 1]
    want = R.score(host(x[some]), host(ids[some]), top)
    assert np.array_equal(host(rk[some]), want[2]) and np.array_equal(host(ti[some]), want[3])
    # V / 256 terms a thread at most, then trees; exponents and exp2, log2 as for shorter rows
    u = 2.0 ** -24
    off = (V / 256 + 128) * u
    for got, w, slack in ((lp, want[0], off), (tl, want[4], off), (en, want[1], off * (2 + np.log(V)))):
        assert (np.abs(host(got[some]) - w) <= slack + 4 * u * np.abs(w)).all()
