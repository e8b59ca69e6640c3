"""Sampling on the GPU against the definition in 64 bits and whole numbers."""
import numpy as np
import pytest

import decode_ops_ref as D
from adapter_lora_bgmv_amd import binding as B

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"bf16": (B.LORA_BF16, "bfloat16"), "f32": (B.LORA_F32, "float32")}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lora_init()


class Draw:
    """Rows of logits and their settings; `skew` elements before the first row."""

    def __init__(self, x, dtype, t=None, k=None, p=None, m=None, u=None, pad=0, skew=0):
        n, V = x.shape
        self.n, self.V, self.dtype = n, V, dtype
        flat = torch.full((skew + n * (V + pad),), float("nan"), dtype=getattr(torch, DT[dtype][1]), device="cuda")
        self.x = flat[skew:].view(n, V + pad)
        self.x[:, :V] = torch.from_numpy(np.ascontiguousarray(x)).cuda().to(flat.dtype)
        self.hx = self.x[:, :V].double().cpu().numpy()
        f = lambda v, d, kind: None if v is None else np.broadcast_to(np.asarray(v, kind), (n,)).copy()
        self.set = {"t": f(t, 1, np.float32), "k": f(k, 0, np.int32), "p": f(p, 1, np.float32), "m": f(m, 0, np.float32),
                    "u": f(0.5 if u is None else u, 0, np.float32)}
        self.dev = {a: None if v is None else torch.from_numpy(v).cuda() for a, v in self.set.items()}
        self.ids = torch.full((n + 2,), 77, dtype=torch.int32, device="cuda")
        self.logp = torch.full((n + 2,), 77.0, device="cuda")
        self.need = B.lora_token_sample_workspace_bytes(DT[dtype][0], V, n)
        self.ws = torch.zeros(max(self.need, 256), dtype=torch.uint8, device="cuda")

    def run(self, stream=None, logp=True):
        d = self.dev
        B.lora_token_sample(DT[self.dtype][0], self.V, self.x, self.x.shape[1], d["t"], d["k"], d["p"], d["m"], d["u"], self.n,
                            self.ids, self.logp if logp else None, self.ws, self.need, stream)

    def result(self):
        torch.cuda.synchronize()
        assert bool((self.ids[self.n:] == 77).all()) and bool((self.logp[self.n:] == 77).all())
        return self.ids[:self.n].cpu().numpy(), self.logp[:self.n].double().cpu().numpy()

    def check(self):
        self.run()
        ids, logp = self.result()
        for i in range(self.n):
            kw = {a: v[i].item() for a, v in self.set.items() if v is not None}
            ok, lp = D.sample(self.hx[i], **kw)
            assert ids[i] in ok, f"row {i} {kw}: {ids[i]}, want {ok}"
            want = lp[ok.index(ids[i])]
            # one rounding of logp, and of the row's weights 2^-43 each in the logarithm
            assert (np.isnan(want) and np.isnan(logp[i])) or abs(logp[i] - want) <= 2.0 ** -24 * abs(want) + 1e-12, f"row {i}"
        return ids


def settings(rng, n, V):
    """Settings of all kinds, one row's beside another's."""
    pick = lambda *v: np.array([v[j](rng) for j in rng.integers(0, len(v), n)])
    return {"t": pick(lambda r: 1.0, lambda r: 0.0, lambda r: r.uniform(0.3, 1.5), lambda r: 0.05, lambda r: 8.0),
            "k": pick(lambda r: 0, lambda r: 1, lambda r: r.integers(2, 60), lambda r: r.integers(1, 2 * V), lambda r: -3),
            "p": pick(lambda r: 1.0, lambda r: r.uniform(0.05, 0.99), lambda r: 0.9, lambda r: 0.0, lambda r: 1.5),
            "m": pick(lambda r: 0.0, lambda r: 0.0, lambda r: r.uniform(0.0, 0.3), lambda r: 1.0, lambda r: -1.0),
            "u": rng.random(n).astype(np.float32)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n,pad,skew", [(1, 4, 0, 0), (2, 9, 1, 1), (7, 33, 0, 3), (63, 20, 2, 0), (256, 30, 0, 1), (1000, 60, 3, 0),
                                          (2049, 40, 0, 7), (4096, 30, 0, 0), (32000, 20, 0, 0), (131071, 6, 0, 1)])
def test_sample(V, n, pad, skew, dtype):
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((n, V)) * 3 + 2 * rng.standard_normal(V)
    x[rng.random((n, V)) < 0.05] = -np.inf
    x[:, V // 2] = np.where(np.isinf(x[:, V // 2]), 0.0, x[:, V // 2])
    Draw(x, dtype, pad=pad, skew=skew, **settings(rng, n, V)).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_equal_logits(V, dtype):
    """Rows of one value, of two, of whole numbers: cuts among equals go by the index."""
    rng = np.random.default_rng(V)
    n = 24
    x = np.zeros((n, V))
    x[8:16] = rng.integers(0, 2, (8, V))
    x[16:] = rng.integers(-3, 4, (8, V))
    x[3:5] = -0.0
    x[4, ::3] = 0.0
    kw = settings(rng, n, V)
    kw["k"][::3] = rng.integers(1, V, len(kw["k"][::3]))
    kw["p"][1::3] = rng.uniform(0.1, 0.9, len(kw["p"][1::3]))
    kw["t"][:] = np.where(kw["t"] < 0.1, 1.0, kw["t"])
    Draw(x, dtype, **kw).check()


def test_rising_and_falling_rows():
    V = 20000
    x = np.stack([np.linspace(-9, 9, V), np.linspace(9, -9, V), np.sin(np.arange(V)) * 5, np.full(V, -np.inf)])
    x[3, V - 1] = -1e30
    for k, p in ((0, 1.0), (200, 0.95), (1500, 1.0), (0, 0.5)):
        for u in (0.0, 0.3, 0.99999994):
            Draw(x, "f32", k=k, p=p, u=u).check()


def test_rows_without_a_distribution():
    """NaN, +infinity, nothing but -infinity; settings that are none."""
    x = np.random.default_rng(0).standard_normal((16, 500))
    x[0, 3], x[1, 499], x[2], x[3, 1:] = np.nan, np.inf, -np.inf, -np.inf
    x[4, 10] = -np.nan
    t, p, m, u = (np.full(16, v) for v in (0.9, 0.8, 0.01, 0.4))
    t[5], t[6], t[7], p[8], m[9], u[10] = -1, np.inf, np.nan, np.nan, np.nan, np.nan
    u[11], u[12], u[13], m[14], t[15] = -3.0, 1.0, np.inf, 7.0, 1e-40
    ids = Draw(x, "f32", t=t, p=p, m=m, u=u).check()
    assert (ids[[0, 1, 2, 4, 5, 6, 7, 8, 9, 10]] == -1).all() and (np.delete(ids, [0, 1, 2, 4, 5, 6, 7, 8, 9, 10]) >= 0).all()


def test_extreme_logits():
    """The types' ends, and temperatures that take every difference to 0 or to nothing."""
    big = 3.38e38
    x = np.array([[big, -big, 0, big], [-big, -big, -big, -big], [1e-40, -1e-40, 0, 1e-38], [88, 87, -1e4, 3]])
    for t in (1e-30, 1e-3, 1.0, 1e30, 3e38):
        for u in (0.0, 0.26, 0.5, 0.76, 0.99):
            Draw(x, "f32", t=t, u=u).check()
    ids, _ = Draw(x, "f32", t=0.0).result()
    assert Draw(x, "f32", t=0.0).check().tolist() == [0, 0, 3, 0]


def test_settings_that_are_not_given():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((10, 3000)) * 2
    Draw(x, "bf16", u=rng.random(10)).check()
    d = Draw(x, "bf16", k=5, u=rng.random(10))
    d.check()
    want, _ = d.result()
    d.logp.fill_(77.0)
    d.ids.fill_(77)
    d.run(logp=False)
    assert np.array_equal(d.result()[0], want) and bool((d.logp == 77).all())


def test_even_numbers_draw_every_token_by_its_share():
    """4096 numbers spread evenly over [0, 1): a token of share p comes up between
    4096 p - 1 and 4096 p + 1 times."""
    V, N = 60, 4096
    x = np.tile(np.random.default_rng(1).standard_normal(V) * 1.5, (N, 1))
    d = Draw(x, "f32", t=0.7, u=(np.arange(N) + 0.5) / N)
    d.run()
    count = np.bincount(d.result()[0], minlength=V)
    p = np.exp((d.hx[0] - d.hx[0].max()) / np.float64(np.float32(0.7)))
    assert (np.abs(count - N * p / p.sum()) <= 1 + 1e-6).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_row_does_not_depend_on_its_batch(dtype):
    """Alone, in a small batch and in a large one: the same token and logp, bit for bit."""
    rng = np.random.default_rng(6)
    n, V = 700, 5003
    x = rng.standard_normal((n, V)) * 3
    kw = settings(rng, n, V)
    d = Draw(x, dtype, **kw)
    d.run()
    ids, logp = d.result()
    for rows in ([0], [5, 6, 7], list(range(100, 170))):
        e = Draw(x[rows], dtype, **{a: v[rows] for a, v in kw.items()})
        e.run()
        got = e.result()
        assert np.array_equal(got[0], ids[rows]) and np.array_equal(got[1], logp[rows], equal_nan=True)


@pytest.mark.parametrize("n,V", [(1, 131071), (64, 32000)])
def test_captured_and_on_another_stream(n, V):
    rng = np.random.default_rng(8)
    d = Draw(rng.standard_normal((n, V)) * 3, "bf16", **settings(rng, n, V))
    d.run()
    want = d.result()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        d.run(s)
    other = Draw(rng.standard_normal((3, 999)), "f32", k=9, u=0.3)
    for _ in range(3):
        d.ids.fill_(77)
        d.logp.fill_(77.0)
        g.replay()
        got = d.result()
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1], equal_nan=True)
        other.check()
    d.ids.fill_(77)
    torch.cuda.synchronize()
    d.run(s)
    s.synchronize()
    assert np.array_equal(d.result()[0], want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n,skew", [(1 << 20, 4, 3), ((1 << 20) - 5, 3, 0), (9001, 520, 1), (33000, 130, 5)])
def test_large_vocabularies_and_many_rows(V, n, skew, dtype):
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((n, V)) * 3
    Draw(x, dtype, skew=skew, pad=3, **settings(rng, n, V)).check()


@pytest.mark.parametrize("n", [12, 900])
def test_bad_logits_in_any_part_of_a_long_row(n):
    """One NaN or infinity at the row's ends and between them; a row whose only
    finite logit lies there; the rows beside draw as ever."""
    V = 20011
    rng = np.random.default_rng(n)
    x = rng.standard_normal((n, V))
    for i, at in enumerate((0, 2047, 2048, V - 1)):
        x[i, at] = np.nan
        x[4 + i, at] = np.inf
        x[8 + i] = -np.inf
        x[8 + i, at] = -3.0
    d = Draw(x[:12], "f32", skew=1, k=[0, 7] * 6, p=[1.0, 1.0, 0.9] * 4, u=rng.random(12))
    ids = d.check()
    assert (ids[:8] == -1).all() and ids[8:].tolist() == [0, 2047, 2048, V - 1]
    e = Draw(x, "f32", skew=1, k=5, u=0.5)
    e.run()
    ids, logp = e.result()
    assert (ids[:8] == -1).all() and np.isnan(logp[:8]).all() and ids[8:12].tolist() == [0, 2047, 2048, V - 1]
    assert (ids[12:] >= 0).all()


def test_a_workspace_used_again_and_calls_at_once():
    """A workspace that a larger call left full, and two streams with one each."""
    rng = np.random.default_rng(12)
    big = Draw(rng.standard_normal((80, 32000)) * 3, "bf16", **settings(rng, 80, 32000))
    small = Draw(rng.standard_normal((3, 9000)) * 3, "f32", **settings(rng, 3, 9000))
    many = Draw(rng.standard_normal((600, 700)) * 3, "f32", **settings(rng, 600, 700))
    want = [d.check() for d in (big, small, many)]
    small.ws = many.ws = big.ws
    for d, w in ((big, want[0]), (small, want[1]), (many, want[2]), (big, want[0])):
        if B.lora_token_sample_workspace_bytes(DT[d.dtype][0], d.V, d.n) > big.need:
            continue
        assert np.array_equal(d.check(), w)
    small.ws = torch.full_like(big.ws, 255)
    assert np.array_equal(small.check(), want[1])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        big.run(a)
        small.run(b)
    assert np.array_equal(big.result()[0], want[0]) and np.array_equal(small.result()[0], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(131071, 4), (32000, 70), (16000, 600)])
def test_flat_rows(V, n, dtype):
    """Rows whose tokens lie within few powers of two, by any cut."""
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((n, V)) * rng.choice([0.01, 0.1, 0.2, 0.5, 1.0, 1.5], (n, 1))
    kw = settings(rng, n, V)
    rows = np.arange(n) if n < 100 else rng.integers(0, n, 80)
    d = Draw(x, dtype, **kw)
    d.run()
    ids, logp = d.result()
    e = Draw(x[rows], dtype, **{a: v[rows] for a, v in kw.items()})
    assert np.array_equal(e.check(), ids[rows]) and np.array_equal(e.result()[1], logp[rows], equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(9001, 1), (70001, 5), (131071, 1), (32000, 33), (5000, 700)])
def test_top_p_alone_among_more_equal_logits_than_a_list_holds(V, n, dtype):
    """Top-p without top-k where its bin holds every logit, on rows of several
    workgroups and of one: equal weights, so the cut is at ceil(p V) and the
    number picks among those, draw after draw the same."""
    rng = np.random.default_rng(V)
    p, u = rng.uniform(0.2, 0.95, n).astype(np.float32), rng.random(n).astype(np.float32)
    d = Draw(np.full((n, V), -1.25), dtype, p=p, u=u)
    stay = np.ceil(p.astype(np.float64) * V)
    want = np.floor(u.astype(np.float64) * stay)
    other = Draw(rng.standard_normal((n, V)) * 3, dtype, p=0.9, u=u)  # other weights in LDS and workspace
    for _ in range(5):
        other.run()
        d.ids.fill_(77)
        d.logp.fill_(77.0)
        d.run()
        ids, logp = d.result()
        assert np.array_equal(ids, want)
        # log of 1/stay, rounded once
        assert (np.abs(logp + np.log(stay)) <= 2.0 ** -24 * np.log(stay) + 1e-12).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(1, 6), (2, 6), (500, 18), (9001, 18), (131071, 6), (5003, 600)])
def test_settings_that_are_nan_beside_ones_that_need_no_draw(V, n, dtype):
    """A NaN among top_p, min_p and uniform leaves a row without a token also
    where T = 0, top_k = 1 or min_p above 1 take the first one anyway."""
    rng = np.random.default_rng(V + n)
    x = rng.standard_normal((n, V)) * 3
    kind, bad = np.arange(n) % 6, np.arange(n) // 6 % 3
    t, k, p, m, u = np.full(n, 0.9), np.zeros(n, int), np.full(n, 0.8), np.zeros(n), rng.random(n)
    t[kind == 0] = 0.0
    k[kind == 1] = 1
    m[kind == 2] = 7.0
    k[kind == 3], m[kind == 3] = 1, 7.0
    t[kind == 4], k[kind == 4] = 0.0, 40
    hurt = kind < 5  # the sixth kind draws
    p[hurt & (bad == 0)], m[hurt & (bad == 1)], u[hurt & (bad == 2)] = np.nan, np.nan, np.nan
    rows = np.arange(n) if n < 100 else np.arange(36)
    d = Draw(x, dtype, t=t, k=k, p=p, m=m, u=u)
    d.run()
    ids, logp = d.result()
    assert (ids[hurt] == -1).all() and np.isnan(logp[hurt]).all(), np.flatnonzero(hurt & (ids >= 0))
    assert (ids[~hurt] >= 0).all()
    e = Draw(x[rows], dtype, t=t[rows], k=k[rows], p=p[rows], m=m[rows], u=u[rows])
    assert np.array_equal(e.check(), ids[rows])
