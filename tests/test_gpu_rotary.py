"""The cache write with the position rotation on the GPU against plain 64-bit
forms: the cache byte for byte, the queries within their roundings."""
import numpy as np
import pytest

import decode_ops_ref as D
import verify_ref as R
from adapter_lora_bgmv_amd import binding as B
from test_gpu_verify import DT, Setup, dev, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lora_init()


def freqs(rot, theta=10000.0):
    return (theta ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def positions(seqs, n):
    pos = np.full(n, -(2 ** 31))
    for _, r, p in R.rows_of(seqs):
        pos[r] = p
    return pos


class Call:
    """[Q|K|V] rows of a setup through the operator."""

    def __init__(self, s, dtype, heads, rot, interleaved=False, inv=None, place=False, x=None):
        self.s, self.dtype, self.heads = s, dtype, heads
        H, Dm, n = s.H, s.D, s.n
        self.wide = (heads + 2 * H) * Dm + 8
        if x is None:
            x = s.rng.standard_normal((n, self.wide)) * np.exp2(s.rng.integers(-6, 7, (n, 1)))
        self.dx = dev(x, dtype)
        self.x = host(self.dx)
        self.inv = freqs(rot) if inv is None else inv
        self.interleaved = interleaved
        self.rotary = B.Rotary(dev(self.inv), interleaved=interleaved)
        self.out = self.dx if place else torch.full((n, heads * Dm + 16), 55.0, dtype=self.dx.dtype, device="cuda")

    def run(self, stream=None):
        s, q, kv = self.s, self.heads * self.s.D, self.s.H * self.s.D
        B.lora_kv_write_rotary(s.cache, s.dseqs, self.rotary, DT[self.dtype][0], self.heads, self.dx, self.wide, self.out,
                               self.out.shape[1], self.dx[:, q:], self.wide, self.dx[:, q + kv:], self.wide, s.n, stream)

    def check(self):
        s, H, Dm, n, heads = self.s, self.s.H, self.s.D, self.s.n, self.heads
        self.run()
        torch.cuda.synchronize()
        x = self.x[:, :(heads + 2 * H) * Dm].reshape(n, heads + 2 * H, Dm)
        pos = positions(s.seqs, n)
        live = pos > -(2 ** 31)
        turned = D.turn(x[:, :heads + H], np.where(live, pos, 0), self.inv, self.interleaved)
        with np.errstate(over="ignore", invalid="ignore"):
            R.write(s.host, s.seqs, turned[:, heads:].astype(np.float32).astype(np.float64), x[:, heads + H:])
        got = s.downloaded()
        for name in ("ke", "ve", "k", "v"):
            a, b = getattr(got, name), getattr(s.host, name)
            if name in "kv":
                a, b = np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b)
            assert np.array_equal(a, b), f"{name}: {int((a != b).sum())} of {a.size} differ"
        if not heads:
            return
        out = host(self.out)
        q = out[:, :heads * Dm].reshape(n, heads, Dm)
        want = turned[:, :heads]
        bound = D.turn_bound(self.dtype, x[:, :heads], want, len(self.inv), self.interleaved)
        with np.errstate(invalid="ignore"):
            bad = ~(np.abs(q - want) <= bound)[live]
        assert not bad.any(), f"{int(bad.sum())} queries off: {np.nanmax((np.abs(q - want) / bound)[live])} of the bound"
        rest = out[:, heads * Dm:]
        if self.out is self.dx:
            assert np.array_equal(rest, self.x[:, heads * Dm:], equal_nan=True)
            assert np.array_equal(out[~live], self.x[~live])
        else:
            assert (rest == 55).all() and (out[~live] == 55).all()


CASES = [
    # lens, H, P, heads, rot of D (None: all), interleaved
    ([(1, 1)], 1, 16, 1, None, False),
    ([(1, 17), (1, 16), (1, 31)], 3, 16, 6, None, True),
    ([(5, 18), (40, 40), (0, 9), (33, 70)], 2, 32, 8, 16, False),
    ([(130, 130), (1, 64), (2, 65), (63, 127)], 1, 64, 7, 48, True),
    ([(9, 200), (300, 421)], 2, 128, 2, 48, False),
    ([(1, t) for t in range(1, 70)], 1, 16, 3, 32, False),
    ([(7, 30)], 2, 32, 0, None, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D_", [64, 128, 256])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rotary_write(case, D_, dtype):
    lens, H, P, heads, rot, inter = CASES[case]
    s = Setup(case * 11 + D_, lens, H, D_, P)
    Call(s, dtype, heads, rot or D_, inter).check()


@pytest.mark.parametrize("interleaved", [False, True])
def test_queries_in_place(interleaved):
    s = Setup(3, [(20, 50), (0, 3), (9, 9)], 2, 128, 16)
    Call(s, "bf16", 8, 96, interleaved, place=True).check()
    s = Setup(4, [(20, 50), (0, 3), (9, 9)], 2, 64, 16)
    Call(s, "f32", 4, 64, interleaved, place=True).check()


def test_far_positions():
    """Lengths up to the largest int: what 32-bit angles would lose.  Only the
    last pages are there."""
    P, D_ = 128, 64
    for dtype in ("bf16", "f32"):
        s = Setup(8, [(5, 5), (3, 3)], 1, D_, P)
        far = [1_000_003, 131_071]
        pages = [-(-t // P) for t in far]
        table = np.full((2, max(pages)), -1, np.int32)
        for i, t in enumerate(far):
            table[i, pages[i] - 1] = i
        s.seqs["table"], s.seqs["kv_len"] = table, np.array(far, np.int32)
        s.upload()
        Call(s, dtype, 4, 64, inv=freqs(64, 500000.0)).check()
        s.seqs["kv_len"] = np.array([2 ** 31 - 1, 2 ** 30], np.int32)  # past the table: queries turn, keys have no page
        s.upload()
        Call(s, dtype, 4, 64, inv=freqs(64)).check()


def test_rows_without_a_page_or_a_sequence():
    """Bad page entries, lengths below the rows and past the table: those keys
    are not written, their queries turn; rows outside every sequence stay."""
    s = Setup(9, [(20, 50), (6, 4), (3, 0), (4, 40), (2, -5)], 2, 64, 16, bad=[(0, 2), (3, 1)])
    s.seqs["kv_len"][3] = 50
    s.upload()
    Call(s, "f32", 4, 64).check()
    s = Setup(10, [(4, 10), (5, 20)], 2, 64, 16)
    s.seqs["indptr"] = np.array([3, 7, 12], np.int32)
    s.n = 15
    s.upload()
    Call(s, "bf16", 4, 32, True).check()


def test_zero_frequencies_leave_rows_and_special_values():
    """Frequencies of 0 leave everything as lora_kv_write has it; infinities and
    NaN make their pair NaN in the cache; large values overflow to NaN codes."""
    s = Setup(12, [(30, 41), (3, 3)], 2, 128, 16)
    c = Call(s, "bf16", 4, 128, inv=np.zeros(64, np.float32))
    c.check()
    s = Setup(13, [(12, 12)], 1, 64, 16)
    x = s.rng.standard_normal((12, 4 * 64 + 8))
    x[0, 128 + 3], x[5, 128 + 40], x[6, 128 + 8] = np.inf, np.nan, -np.inf
    x[7, 128:192] = 3e38
    Call(s, "f32", 2, 64, x=x).check()
    s = Setup(14, [(12, 12)], 1, 64, 16)
    c = Call(s, "f32", 2, 64, inv=np.full(32, 1e30, np.float32))  # angles of 2^50 and more count as 0
    c.inv = np.zeros(32, np.float32)
    c.check()
    s = Setup(17, [(12, 12)], 1, 64, 16)
    c = Call(s, "f32", 2, 64, inv=np.array([np.inf, np.nan] + [2.0 ** -7] * 30, np.float32))
    c.run()
    torch.cuda.synchronize()
    bad = np.isnan(host(c.out)[:, :128].reshape(12, 2, 64)).any((0, 1))
    assert np.array_equal(np.flatnonzero(bad), [0, 1, 32, 33])


def test_turns_keep_lengths_and_relative_angles():
    """The invariants of the rotation: norms stay, and q . k depends on the distance alone."""
    D_, P = 128, 16
    s = Setup(15, [(1, 1)], 1, D_, P)
    x = s.rng.standard_normal((1, 3 * D_ + 8))
    got = []
    for at in (1, 900):
        q = []
        for length in (at, at + 37):
            table = np.full((1, -(-length // P)), -1, np.int32)
            s.seqs["table"], s.seqs["kv_len"] = table, np.array([length], np.int32)
            s.upload()
            c = Call(s, "f32", 1, D_, x=x)
            c.run()
            torch.cuda.synchronize()
            q.append(host(c.out)[0, :D_])
        got.append(q[0] @ q[1])
        # 128 products of values that are off by 4 2^-24 of |a| + |b|
        assert abs(np.linalg.norm(q[0]) - np.linalg.norm(c.x[0, :D_])) <= 8 * 2.0 ** -24 * np.linalg.norm(c.x[0, :D_])
    assert abs(got[0] - got[1]) <= 4 * 8 * 2.0 ** -24 * (c.x[0, :D_] ** 2).sum()


def test_captured_and_on_another_stream():
    s = Setup(16, [(9, 300), (9, 9), (1, 129)], 2, 128, 16)
    c = Call(s, "bf16", 8, 128)
    c.check()
    want, pages = host(c.out), s.downloaded()
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        c.run(st)
    for _ in range(3):
        c.out.fill_(55.0)
        g.replay()
        torch.cuda.synchronize()
        got = s.downloaded()
        assert np.array_equal(host(c.out), want)
        for name in ("ke", "ve", "k", "v"):
            assert np.array_equal(getattr(got, name), getattr(pages, name))


def test_more_workgroups_than_one_dimension_of_a_grid_holds():
    """2^24 workgroups of pages and heads, and the queries' behind them: a call
    that lora_kv_write takes, too, and whose angles of 0 leave its codes the same."""
    n_seqs, rows, H, D_, P, heads = 1024, 8, 4500, 64, 16, 3
    n, row = n_seqs * rows, H * D_
    assert min(n, n // P + 2 * n_seqs) * (H + (H + 1) // 2) > 2 ** 24
    owners = [0, 1, 511, 1023]  # the sequences that have a page; the others' tokens are not written
    table = torch.full((n_seqs, 1), -1, dtype=torch.int32, device="cuda")
    table[owners, 0] = torch.tensor([2, 0, 3, 1], dtype=torch.int32, device="cuda")
    seqs = B.KVSeqs(table, torch.arange(0, n + 1, rows, dtype=torch.int32, device="cuda"),
                    torch.full((n_seqs,), rows, dtype=torch.int32, device="cuda"), max_rows=rows)
    x = torch.zeros(n, row, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(5)
    for i in owners:
        x[i * rows:(i + 1) * rows].normal_(generator=g)
    q = torch.randn(n, heads * D_, generator=g, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    a, b = (B.KVCache.empty(4, H, D_, P, "cuda") for _ in range(2))
    for c in (a, b):
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            t.zero_()
    torch.cuda.synchronize()
    B.lora_kv_write(a, seqs, B.LORA_BF16, x, row, x, row, n)
    rotary = B.Rotary(torch.zeros(D_ // 2, device="cuda"))
    B.lora_kv_write_rotary(b, seqs, rotary, B.LORA_BF16, heads, q, heads * D_, out, heads * D_, x, row, x, row, n)
    torch.cuda.synchronize()
    assert torch.equal(out, q)
    assert bool((a.k_scale > 0).all()) and bool((a.k != 0).any())
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name
