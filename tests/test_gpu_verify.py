"""The verify-step operators on the GPU against plain 64-bit forms
(verify_ref.py): the 8-bit paged cache bit for bit, the attention and the
token scores within bounds derived from their roundings."""
import numpy as np
import pytest

import verify_ref as R
from adapter_lora_bgmv_amd import binding as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": (B.LORA_BF16, "bfloat16"), "f32": (B.LORA_F32, "float32")}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lora_init()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(getattr(torch, DT[dtype][1]))


def host(t):
    return t.double().cpu().numpy() if t.dtype.is_floating_point else t.cpu().numpy()


class Setup:
    """A pool of random pages (every byte that no token holds is NaN), and
    sequences of (rows, length) over shuffled pages."""

    def __init__(self, seed, lens, H, D, P, spare_pages=2, bad=(), stale=0x7F, spread=3.0, table_pad=0):
        rng = self.rng = np.random.default_rng(seed)
        self.H, self.D, self.P, self.lens = H, D, P, lens
        used = [max(-(-t // P), 0) for _, t in lens]
        n_pages = sum(used) + spare_pages
        order = rng.permutation(n_pages)
        per = max(used + [1])
        table = np.full((len(lens), per + table_pad), -1, np.int32)
        at = 0
        for i, u in enumerate(used):
            table[i, :u] = order[at:at + u]
            at += u
        k = rng.standard_normal((n_pages, H, P, D))
        v = rng.standard_normal((n_pages, H, P, D)) * np.exp2(rng.standard_normal((n_pages, H, 1, 1)) * spread)
        ke = np.array([[R.scale_byte(np.abs(x).max()) for x in p] for p in k], np.uint8)
        ve = np.array([[R.scale_byte(np.abs(x).max()) for x in p] for p in v], np.uint8)
        kc = R.encode(k * np.exp2(127 - ke.astype(float))[..., None, None])
        vc = R.encode(v * np.exp2(127 - ve.astype(float))[..., None, None])
        live = np.zeros((n_pages, P), bool)
        for i, (_, t) in enumerate(lens):
            for p in range(max(t, 0)):
                live[table[i, p // P], p % P] = True
        kc[~live[:, None, :].repeat(H, 1)] = stale
        vc[~live[:, None, :].repeat(H, 1)] = stale
        for i, p in bad:  # entries that name no page
            table[i, p] = [-1, n_pages, -2 ** 31, 2 ** 31 - 1][(i + p) % 4]
        self.seqs = {"table": table, "kv_len": np.array([t for _, t in lens], np.int32),
                     "indptr": np.cumsum([0] + [r for r, _ in lens]).astype(np.int32)}
        self.n = int(self.seqs["indptr"][-1])
        c = R.Cache(np.zeros((n_pages, H, P * D), np.uint8), np.zeros((n_pages, H, P * D), np.uint8), ke, ve, P, D)
        c.k, c.v = kc, vc
        self.host = c
        self.upload()

    def upload(self, max_rows=0):
        k, v = self.host.raw()
        self.cache = B.KVCache(dev(k), dev(v), dev(self.host.ke), dev(self.host.ve), page_tokens=self.P, head_dim=self.D)
        self.dseqs = B.KVSeqs(dev(self.seqs["table"]), dev(self.seqs["indptr"]), dev(self.seqs["kv_len"]), max_rows=max_rows)

    def downloaded(self):
        c = self.cache
        return R.Cache(host(c.k), host(c.v), host(c.k_scale), host(c.v_scale), self.P, self.D)

    def attend(self, dtype, heads, window=0, scale=None, q=None, pad=0, stream=None, ws=None, lse=True):
        code, name = DT[dtype]
        D, n = self.D, self.n
        if q is None:
            q = self.rng.standard_normal((n, heads, D)) * 1.5
        wide = heads * D + pad
        dq = torch.zeros(n, wide, dtype=getattr(torch, name), device="cuda")
        dq[:, :heads * D] = dev(q.reshape(n, -1), dtype)
        out = torch.full((n, wide), 77.0, dtype=dq.dtype, device="cuda")
        dl = torch.full((n, heads), 77.0, device="cuda") if lse else None
        need = B.lora_kv_attend_workspace_bytes(self.cache, self.dseqs, code, heads, n)
        if ws is None:
            ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        scale = D ** -0.5 if scale is None else scale
        call = lambda st=stream: B.lora_kv_attend(self.cache, self.dseqs, code, heads, dq, wide, scale, window, n, out, wide,
                                                  dl, ws, need, st)
        call()
        torch.cuda.synchronize()
        self.call, self.out, self.lse, self.ws = call, out, dl, ws
        assert bool((out[:, heads * D:] == 77).all())  # the columns beside are left alone
        return host(dq)[:, :heads * D].reshape(n, heads, D), host(out)[:, :heads * D].reshape(n, heads, D), \
            host(dl) if lse else None

    def check(self, dtype, heads, window=0, **kw):
        q, out, lse = self.attend(dtype, heads, window, **kw)
        scale = float(np.float32(kw.get("scale") or self.D ** -0.5))
        want, wl, mag, big, toks = R.attend(self.host, self.seqs, q, scale, window)
        bo, bl = R.attend_bounds(dtype, want, wl, mag, big, toks, self.D)
        rows = [r for _, r, _ in R.rows_of(self.seqs)]
        with np.errstate(invalid="ignore"):
            for r in rows:
                assert np.array_equal(np.isnan(out[r]), np.isnan(want[r])), f"row {r}: NaN"
                bad = np.abs(out[r] - want[r]) > bo[r]
                assert not bad.any(), f"row {r}: {np.abs(out[r] - want[r])[bad].max()} over {bo[r][bad].max()}"
                if lse is not None:
                    both = np.isfinite(wl[r])
                    assert np.array_equal(lse[r][~both], wl[r][~both], equal_nan=True), f"row {r}: lse {lse[r]} {wl[r]}"
                    assert (np.abs(lse[r] - wl[r])[both] <= bl[r][both]).all(), f"row {r}: lse"
        return out


# ---------------------------------------------------------------- cache
WRITES = [
    # lens, H, P
    ([(1, 1)], 1, 16),
    ([(1, 17), (1, 16), (1, 31)], 3, 16),
    ([(5, 18), (40, 40), (0, 9), (33, 70)], 2, 32),
    ([(130, 130), (1, 64), (2, 65), (63, 127)], 1, 64),
    ([(9, 200), (300, 421)], 2, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(WRITES)))
def test_write_then_read(case, D, dtype):
    """Every byte of the pool after a write, then the rows read back."""
    lens, H, P = WRITES[case]
    s = Setup(case * 7 + D, lens, H, D, P)
    wide = (3 + 2 * H) * D
    x = s.rng.standard_normal((s.n, wide)) * np.exp2(s.rng.integers(-12, 13, (s.n, 1)))
    dx = dev(x, dtype)
    hx = host(dx)
    k, v = (hx[:, o * D:(o + H) * D].reshape(s.n, H, D) for o in (3, 3 + H))
    B.lora_kv_write(s.cache, s.dseqs, DT[dtype][0], dx[:, 3 * D:], wide, dx[:, (3 + H) * D:], wide, s.n)
    torch.cuda.synchronize()
    R.write(s.host, s.seqs, k, v)
    got = s.downloaded()
    for name in ("ke", "ve", "k", "v"):
        a, b = getattr(got, name), getattr(s.host, name)
        if name in "kv":
            a, b = np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b)
        assert np.array_equal(a, b), f"{name}: {int((a != b).sum())} of {a.size} differ"
    row = H * D + 8
    ok, ov = (torch.full((s.n, row), 55.0, dtype=dx.dtype, device="cuda") for _ in range(2))
    B.lora_kv_read(s.cache, s.dseqs, DT[dtype][0], ok, row, ov, row, s.n)
    torch.cuda.synchronize()
    wk, wv = (np.full((s.n, H, D), 55.0) for _ in range(2))
    R.read(s.host, s.seqs, wk, wv)
    for o, w in ((ok, wk), (ov, wv)):
        o = host(o)
        assert np.array_equal(o[:, :H * D].reshape(s.n, H, D), w)
        assert (o[:, H * D:] == 55).all()


def test_write_special_values():
    """Zeros, subnormals, infinities, NaN, the largest numbers; a page that
    grows from the smallest scale to the largest."""
    P, D = 16, 64
    for dtype in ("bf16", "f32"):
        s = Setup(1, [(1, t) for t in (1, 5, 9)] + [(3, 7)], 1, D, P)
        x = np.zeros((s.n, 2 * D))
        x[1, :] = 3.3e38
        x[2, 3], x[2, 9], x[2, 10], x[2, D + 1] = np.inf, np.nan, 2.0, -np.inf
        x[3, :] = 1.5 * 2.0 ** -127 * np.arange(2 * D)
        x[4, 5], x[5, 6] = -448.0, 449.0
        dx = dev(x, dtype)
        hx = host(dx)
        B.lora_kv_write(s.cache, s.dseqs, DT[dtype][0], dx, 2 * D, dx[:, D:], 2 * D, s.n)
        torch.cuda.synchronize()
        R.write(s.host, s.seqs, hx[:, None, :D], hx[:, None, D:])
        got = s.downloaded()
        assert np.array_equal(got.ke, s.host.ke) and np.array_equal(got.ve, s.host.ve)
        for a, b in ((got.k, s.host.k), (got.v, s.host.v)):
            assert np.array_equal(R.TABLE[a], R.TABLE[b], equal_nan=True)


def test_write_token_by_token_equals_the_reference():
    """A page filled one token a call while its values grow: the scale follows."""
    P, D, H = 16, 128, 2
    s = Setup(5, [(1, 1)], H, D, P)
    for t in range(20):
        s.seqs["kv_len"][:] = t + 1
        s.seqs["table"] = np.array([[0, 1]], np.int32)
        if t == 0:
            s.upload()
        d = B.KVSeqs(dev(s.seqs["table"]), dev(s.seqs["indptr"]), dev(s.seqs["kv_len"]))
        x = s.rng.standard_normal((1, 2 * H * D)) * 1.5 ** t
        dx = dev(x, "bf16")
        hx = host(dx).reshape(1, 2, H, D)
        B.lora_kv_write(s.cache, d, B.LORA_BF16, dx, 2 * H * D, dx[:, H * D:], 2 * H * D, 1)
        R.write(s.host, s.seqs, hx[:, 0], hx[:, 1])
        got = s.downloaded()
        assert np.array_equal(got.ke, s.host.ke) and np.array_equal(got.ve, s.host.ve), t
        assert np.array_equal(R.TABLE[got.k], R.TABLE[s.host.k], equal_nan=True), t
        assert np.array_equal(R.TABLE[got.v], R.TABLE[s.host.v], equal_nan=True), t


def test_tokens_without_a_page_are_not_touched():
    """Bad page entries, lengths below the rows and past the table: those
    tokens are neither written nor read, everything else is."""
    H, D, P = 2, 64, 16
    s = Setup(9, [(20, 50), (6, 4), (3, 0), (4, 40), (2, -5)], H, D, P, bad=[(0, 2), (3, 1)])
    s.seqs["kv_len"][3] = 50  # past the row's table (4 pages of 16 hold it, the entries are -1)
    s.upload()
    x = s.rng.standard_normal((s.n, 2 * H * D))
    dx = dev(x, "f32")
    hx = host(dx).reshape(s.n, 2, H, D)
    B.lora_kv_write(s.cache, s.dseqs, B.LORA_F32, dx, 2 * H * D, dx[:, H * D:], 2 * H * D, s.n)
    R.write(s.host, s.seqs, hx[:, 0], hx[:, 1])
    got = s.downloaded()
    assert np.array_equal(got.k, s.host.k) and np.array_equal(got.v, s.host.v)
    o = torch.full((s.n, 2 * H * D), 55.0, device="cuda")
    B.lora_kv_read(s.cache, s.dseqs, B.LORA_F32, o, 2 * H * D, o[:, H * D:], 2 * H * D, s.n)
    want = np.full((s.n, 2, H, D), 55.0)
    R.read(s.host, s.seqs, want[:, 0], want[:, 1])
    assert (want == 55).any() and np.array_equal(host(o).reshape(want.shape), want)


# ---------------------------------------------------------------- attention
ATTENDS = [
    # lens, H, G, D, P, window
    ([(1, 1)], 1, 1, 64, 16, 0),
    ([(1, 63), (1, 64), (1, 65)], 2, 4, 128, 16, 0),
    ([(1, 700)], 8, 4, 128, 16, 0),
    ([(9, 300), (9, 9), (9, 129), (9, 1000)], 2, 4, 128, 16, 0),
    ([(3, 100), (1, 5), (7, 7), (0, 20), (2, 350)], 3, 5, 64, 32, 0),
    ([(2, 333), (1, 17)], 1, 7, 256, 64, 0),
    ([(1, 130), (16, 400)], 2, 3, 256, 128, 0),
    ([(5, 300), (1, 299), (12, 40)], 2, 2, 128, 32, 33),
    ([(4, 90), (1, 200)], 2, 8, 64, 16, 1),
    ([(40, 40)], 1, 4, 128, 64, 0),
    ([(150, 200), (33, 300), (1, 77), (4, 64)], 2, 4, 128, 64, 0),
    ([(100, 230), (65, 65)], 1, 2, 64, 16, 50),
    ([(70, 70), (90, 111)], 1, 3, 256, 32, 0),
    ([(1, 5000)], 1, 8, 128, 16, 0),
    ([(2, 3000), (1, 40)], 2, 1, 64, 128, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTENDS)))
def test_attend(case, dtype):
    lens, H, G, D, P, window = ATTENDS[case]
    s = Setup(100 + case, lens, H, D, P)
    s.check(dtype, H * G, window, pad=0 if case % 2 else 24)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_rows", [1, 9, 150, 1000])
def test_attend_any_bound_on_rows(max_rows, dtype):
    """max_rows chooses kernels only, wrong bounds too."""
    s = Setup(31, [(150, 200), (1, 90), (9, 70)], 2, 64, 32)
    s.upload(max_rows)
    s.check(dtype, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_rows_that_see_nothing(dtype):
    """No tokens, lengths below the rows, pages that name nothing, a window
    over such a page: zeros and -inf, whatever the pool holds."""
    s = Setup(12, [(2, 0), (6, 4), (1, 16), (3, 40), (1, -3), (5, 70)], 2, 128, 16,
              bad=[(2, 0), (3, 1), (5, 0), (5, 3)], stale=0xFF)
    s.check(dtype, 4)
    out = s.check(dtype, 4, window=2)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(9, 75)], [(80, 150)]])
def test_attend_nan_reaches_only_the_rows_that_see_it(lens, dtype):
    """NaN in keys and in values of tokens that only the later rows see."""
    for which in ("k", "v"):
        s = Setup(13, lens, 1, 128, 16)
        m, t = lens[0]
        pos = t - m // 2
        page = s.seqs["table"][0, pos // 16]
        getattr(s.host, which)[page, 0, pos % 16, 5] = 0x7F
        s.upload()
        out = s.check(dtype, 4)
        early = m - m // 2
        assert np.isfinite(out[:early]).all() and np.isnan(out[early:]).any()


def test_attend_page_scales_far_apart():
    """Values of 2^-60 and of 2^60 in one sequence, and keys whose scores decide for the small ones."""
    s = Setup(14, [(1, 64), (20, 64)], 1, 64, 16, spread=20.0)
    for dtype in ("bf16", "f32"):
        s.check(dtype, 1)
        s.check(dtype, 1, scale=4.0)


def test_attend_strided_table_and_no_lse():
    s = Setup(15, [(1, 100), (3, 50)], 2, 64, 16, table_pad=5)
    s.check("bf16", 4, lse=False)


def test_attend_repeats_bit_for_bit_and_leaves_the_workspace_ready():
    for lens in ([(1, 5000), (2, 900)], [(200, 3000)]):
        s = Setup(16, lens, 2, 128, 16)
        s.attend("bf16", 8)
        first = host(s.out).copy()
        for _ in range(3):
            s.out.fill_(3.0)
            s.call()
            torch.cuda.synchronize()
            assert np.array_equal(host(s.out), first)


def test_verify_calls_in_a_graph_and_on_another_stream():
    """Write, attend and score captured once; lengths, pages and logits rewritten between replays."""
    H, G, D, P, n, V = 2, 4, 128, 16, 6, 1000
    s = Setup(17, [(3, 40), (3, 99)], H, D, P, spare_pages=12)
    s.seqs["table"] = np.concatenate([s.seqs["table"], np.arange(2)[:, None] + s.host.ke.shape[0] - 2], 1).astype(np.int32)
    s.upload()
    x = torch.randn(n, 2 * H * D, device="cuda").bfloat16()
    q = torch.randn(n, H * G * D, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(n, H * G, device="cuda")
    logits = torch.randn(n, V, device="cuda")
    ids = torch.randint(0, V, (n,), device="cuda", dtype=torch.int32)
    lp, en = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    rk, ti, tl = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, 4, dtype=torch.int32, device="cuda"), \
        torch.empty(n, 4, device="cuda")
    need = B.lora_kv_attend_workspace_bytes(s.cache, s.dseqs, B.LORA_BF16, H * G, n)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    need2 = B.lora_token_logprobs_workspace_bytes(B.LORA_F32, V, n, 4)
    ws2 = torch.zeros(max(need2, 256), dtype=torch.uint8, device="cuda")

    def step():
        B.lora_kv_write(s.cache, s.dseqs, B.LORA_BF16, x, 2 * H * D, x[:, H * D:], 2 * H * D, n)
        B.lora_kv_attend(s.cache, s.dseqs, B.LORA_BF16, H * G, q, H * G * D, D ** -0.5, 0, n, out, H * G * D, lse, ws, need)
        B.lora_token_logprobs(B.LORA_F32, V, logits, V, ids, n, 4, lp, en, rk, ti, tl, ws2, need2)

    outs = (out, lse, lp, en, rk, ti, tl, s.cache.k, s.cache.v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        step()
        torch.cuda.synchronize()
        want = [host(t).copy() for t in outs]
        for t in outs[:7]:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert np.array_equal(host(t), w, equal_nan=t.dtype.is_floating_point), i
        s.dseqs.kv_len.add_(3)
        x.normal_()
        q.normal_()
        logits.normal_()


# ---------------------------------------------------------------- scores
def check_scores(x, ids, top, dtype, skew=0, stride=None):
    n, V = x.shape
    stride = stride or V
    code, name = DT[dtype]
    flat = torch.full((skew + n * stride,), float("nan"), dtype=getattr(torch, name), device="cuda")
    rows = flat[skew:].view(n, stride)
    rows[:, :V] = dev(x, dtype)
    hx = host(rows)[:, :V]
    lp, en = (torch.full((n,), 9.0, device="cuda") for _ in range(2))
    rk = torch.full((n,), 9, dtype=torch.int32, device="cuda")
    ti, tl = torch.full((n, top), 9, dtype=torch.int32, device="cuda"), torch.full((n, top), 9.0, device="cuda")
    need = B.lora_token_logprobs_workspace_bytes(code, V, n, top)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    for _ in range(2):  # the second on the workspace as the first left it
        B.lora_token_logprobs(code, V, rows, stride, dev(np.asarray(ids, np.int32)), n, top, lp, en, rk, ti, tl, ws, need)
    torch.cuda.synchronize()
    wlp, wen, wrk, wti, wtl = R.score(hx, ids, top)
    assert np.array_equal(host(rk), wrk)
    assert np.array_equal(host(ti), wti)
    # at most 128 terms a thread, then trees; t = (x - m) log2 e of at most 40 where it counts; exp2 and log2 an ulp each
    u = 2.0 ** -24
    off = (128 + 128) * u
    for got, want, slack in ((host(lp), wlp, off), (host(tl), wtl, off), (host(en), wen, off * (2 + np.log(V)))):
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf])
        assert (np.abs(got - want)[~inf] <= slack + 4 * u * np.abs(want[~inf])).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,top", [(1, 1, 1), (3, 5, 5), (2, 7, 0), (5, 300, 32), (4, 4097, 20), (36, 32000, 5),
                                     (1, 131071, 20), (1100, 1000, 3), (2, 70001, 32), (1030, 9001, 1), (1, 1 << 20, 7)])
def test_scores(n, V, top, dtype):
    rng = np.random.default_rng(n * 31 + V)
    x = rng.standard_normal((n, V)) * 4
    x[rng.random((n, V)) < 0.05] = -np.inf
    x[:, V // 2] = 1.0
    ids = rng.integers(0, V, n)
    ids[rng.random(n) < 0.3] = V // 2
    ids[-1] = [-1, V, 2 ** 31 - 1][V % 3]
    check_scores(x, ids, top, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("skew,extra", [(1, 1), (3, 6), (5, 3)])
def test_scores_of_rows_at_any_alignment(skew, extra, dtype):
    rng = np.random.default_rng(skew)
    for V in (3, 2048, 50001):
        check_scores(rng.standard_normal((7, V)) * 3, rng.integers(0, V, 7), min(V, 9), dtype, skew, V + extra)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 1100])
def test_scores_of_unlikely_rows(n, dtype):
    """Equal, rising, falling and crowded rows, rows of -inf and of the type's lowest value."""
    for V in (40000, 5000):
        x = np.zeros((n, V))
        i = np.arange(V)
        low = float(torch.finfo(getattr(torch, DT[dtype][1])).min)
        kinds = [np.zeros(V), i / 512.0, -i / 512.0, np.where(i % 4096 < 8, 50.0 + i % 64, 0.0), np.full(V, -np.inf),
                 np.full(V, low), np.where(i == 77, 3.0, low), np.where(i % 2 == 0, -np.inf, 1.0), np.full(V, 3e38)]
        for r in range(n):
            x[r] = kinds[r % len(kinds)]
        if n == 2:
            for a in range(0, len(kinds) - 1, 2):
                check_scores(np.stack(kinds[a:a + 2]), [V - 1, 77], 32, dtype)
            continue
        check_scores(x[:1036], [77] * 1036, 20, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_of_rows_with_nan_or_infinity(dtype):
    for n, V in ((3, 30000), (1100, 900)):
        x = np.random.default_rng(2).standard_normal((n, V))
        x[0, 5], x[1, V - 1] = np.nan, np.inf
        code, name = DT[dtype]
        dx = dev(x, dtype)
        lp, en, tl = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), torch.zeros(n, 3, device="cuda")
        ti = torch.full((n, 3), -1, dtype=torch.int32, device="cuda")
        need = B.lora_token_logprobs_workspace_bytes(code, V, n, 3)
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
        B.lora_token_logprobs(code, V, dx, V, torch.zeros(n, dtype=torch.int32, device="cuda"), n, 3, lp, en, None, ti, tl, ws, need)
        torch.cuda.synchronize()
        for t in (lp, en, tl):
            assert torch.isnan(t[:2]).all() and torch.isfinite(t[2:]).all()
        assert bool(((ti >= 0) & (ti < V)).all())
