"""The 8-bit product and its quantisation on the GPU against plain 64-bit
forms (decode_ops_ref.py): codes and scales bit for bit, products within
bounds derived from their roundings."""
import numpy as np
import pytest

import decode_ops_ref as D
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def padded(a, stride, fill):
    t = torch.full((len(a), stride), fill, dtype=torch.from_numpy(a[:0]).dtype, device="cuda")
    t[:, :a.shape[1]] = dev(a)
    return t


def quantized(x, dtype, block, pad=0):
    """(codes, scale) of the library for host rows x, as host arrays."""
    n, k = x.shape
    t = torch.full((n, k + pad), 9.0, dtype=getattr(torch, DT[dtype][1]), device="cuda")
    t[:, :k] = dev(x).to(t.dtype)
    nb, kb = -(-n // block), -(-k // 128)
    codes = torch.full((n + 1, k + pad + (-pad) % 16), 77, dtype=torch.uint8, device="cuda")
    scale = torch.full((nb + 1, kb + 2), 55.0, device="cuda")
    B.lora_quantize_fp8(DT[dtype][0], n, k, t, t.shape[1], block, codes, codes.shape[1], scale, kb + 2)
    torch.cuda.synchronize()
    assert bool((codes[n:] == 77).all()) and bool((codes[:, k:] == 77).all())  # what lies beside is left alone
    assert bool((scale[nb:] == 55).all()) and bool((scale[:, kb:] == 55).all())
    return t[:, :k].double().cpu().numpy(), codes[:n, :k].cpu().numpy(), scale[:nb, :kb].double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,block,pad", [(1, 16, 1, 0), (3, 128, 1, 8), (5, 400, 1, 16), (64, 4096, 1, 0), (300, 1040, 1, 24),
                                           (1, 16, 128, 0), (128, 128, 128, 0), (129, 144, 128, 8), (300, 1040, 128, 0)])
def test_quantize(n, k, block, pad, dtype):
    rng = np.random.default_rng(n * k + block)
    x = rng.standard_normal((n, k)) * np.exp2(rng.integers(-20, 20, (n, 1)))
    x[:, 3 % k::61] *= 300
    hx, codes, scale = quantized(x, dtype, block, pad)
    want, ws = D.quantize(hx, block)
    assert np.array_equal(scale, ws)
    assert np.array_equal(codes, want), f"{int((codes != want).sum())} of {codes.size} differ"


@pytest.mark.parametrize("block", [1, 128])
def test_quantize_special_values(block):
    """Zeros, subnormals, the largest numbers, infinities and NaN, halfway values."""
    x = np.zeros((8, 272))
    x[1, :128] = 1e-40
    x[2, :] = 3.3e38
    x[3, 5], x[3, 9], x[3, 130], x[3, 200] = np.inf, 2.0, -np.inf, np.nan
    x[4, :] = np.linspace(-448, 448, 272)
    x[5, :254] = np.concatenate([(R.TABLE[:127] + R.TABLE[1:128])[:127] / 2, R.TABLE[:127]])[:254]
    x[5] = np.nan_to_num(x[5])
    x[6, 0], x[6, 200] = 448.0, 448.5
    x[7, :] = -2.0 ** -126
    hx, codes, scale = quantized(x, "f32", block)
    want, ws = D.quantize(hx, block)
    assert np.array_equal(scale, ws)
    assert np.array_equal(R.TABLE[codes], R.TABLE[want], equal_nan=True)


def codes_of(rng, n, k):
    """Codes of ordinary size with a few of the largest and zeros, no NaN."""
    x = rng.standard_normal((n, k)) * 40
    x[rng.random((n, k)) < 0.01] = 448
    x[rng.random((n, k)) < 0.05] = 0
    return R.encode(np.clip(x, -448, 448))


class Product:
    def __init__(self, seed, n, n_out, k, pad=16, dtype="bf16"):
        rng = np.random.default_rng(seed)
        kb = -(-k // 128)
        self.n, self.n_out, self.k, self.dtype = n, n_out, k, dtype
        self.x, self.w = codes_of(rng, n, k), codes_of(rng, n_out, k)
        self.xs = np.exp2(rng.standard_normal((n, kb))).astype(np.float32)
        self.ws = (0.01 * rng.standard_normal((-(-n_out // 128), kb))).astype(np.float32)
        self.pad = pad

    def upload(self):
        # what lies beside the codes and scales is NaN
        self.dx, self.dw = padded(self.x, self.k + self.pad, 127), padded(self.w, self.k + self.pad, 127)
        self.dxs, self.dws = padded(self.xs, self.xs.shape[1] + 3, float("nan")), padded(self.ws, self.ws.shape[1] + 1, float("nan"))
        self.y = torch.full((self.n + 2, self.n_out + 8), 55.0, dtype=getattr(torch, DT[self.dtype][1]), device="cuda")
        self.need = B.lora_matmul_fp8_workspace_bytes(DT[self.dtype][0], self.n_out, self.k, self.n)
        self.work = torch.zeros(max(self.need, 256), dtype=torch.uint8, device="cuda")

    def call(self, stream=None):
        B.lora_matmul_fp8(DT[self.dtype][0], self.n_out, self.k, self.dw, self.dw.shape[1], self.dws, self.dws.shape[1], self.dx,
                          self.dx.shape[1], self.dxs, self.dxs.shape[1], self.n, self.y, self.y.shape[1], self.work, self.need, stream)

    def result(self):
        torch.cuda.synchronize()
        assert bool((self.y[self.n:] == 55).all()) and bool((self.y[:, self.n_out:] == 55).all())
        return self.y[:self.n, :self.n_out].double().cpu().numpy()

    def check(self):
        self.upload()
        self.call()
        got = self.result()
        want, mag = D.matmul(self.x, self.xs.astype(float), self.w, self.ws.astype(float))
        bound = D.matmul_bound(self.dtype, want, mag, self.k)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        live = np.isfinite(want)
        bad = np.abs(got - want)[live] > bound[live]
        assert not bad.any(), f"{int(bad.sum())} of {bad.size}: {(np.abs(got - want)[live] / bound[live]).max()} of the bound"
        return got


SIZES = [(1, 8, 16), (1, 64, 128), (2, 1000, 400), (3, 40, 144), (16, 128, 256), (17, 264, 1040), (33, 136, 2064), (48, 96, 4096),
         (64, 512, 4112), (1, 264, 16384), (65, 200, 400), (100, 1000, 272), (129, 264, 1424), (300, 2056, 640), (257, 520, 128), (70, 8, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_out,k", SIZES)
def test_matmul(n, n_out, k, dtype):
    Product(n + n_out, n, n_out, k, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_out,k", [(2100, 2056, 272), (4200, 4360, 144), (16384, 1032, 128)])
def test_matmul_of_many_rows(n, n_out, k, dtype):
    """The forms with the largest tiles, the last ones cut."""
    Product(7, n, n_out, k, dtype=dtype, pad=0).check()


@pytest.mark.parametrize("n", [1, 20, 64, 65, 400])
def test_matmul_keeps_nan_to_its_rows_and_columns(n):
    """A NaN code of x reaches its row, one of W its column, a scale its block;
    infinite scales and scales of 0 and below."""
    p = Product(3, n, 264, 528)
    p.x[n // 2, 500] = 0xFF
    p.w[130, 17] = 0x7F
    p.ws[0, 1], p.ws[1, 2] = 0.0, -1.0
    p.xs[n - 1, 0] = 0.0
    got = p.check()
    assert np.isnan(got[n // 2]).all() and np.isnan(got[:, 130]).all()
    assert np.isfinite(np.delete(np.delete(got, n // 2, 0), 130, 1)).all()


def test_matmul_rows_do_not_depend_on_their_place():
    """A row's results are the same bits wherever it stands in a batch of the same form."""
    for n, other in ((64, 40), (400, 390)):
        a = Product(11, n, 520, 1040)
        b = Product(11, n, 520, 1040)
        first = a.check()
        b.x, b.xs = b.x[::-1][:other].copy(), b.xs[::-1][:other].copy()
        b.n = other
        assert np.array_equal(b.check(), first[::-1][:other])


@pytest.mark.parametrize("n", [5, 64, 333])
def test_matmul_captured_and_on_another_stream(n):
    p = Product(5, n, 1032, 656)
    want = p.check()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        p.call(s)
    other = Product(6, n, 264, 400)
    for _ in range(3):
        p.y.fill_(55.0)
        g.replay()
        assert np.array_equal(p.result(), want)
        other.check()
    p.y.fill_(55.0)
    torch.cuda.synchronize()
    p.call(s)
    s.synchronize()
    assert np.array_equal(p.result(), want)


def test_quantize_then_multiply():
    """Hidden rows and weights through both operators: within the codes' own rounding of the product."""
    rng = np.random.default_rng(2)
    n, o, k = 30, 264, 656
    x, w = rng.standard_normal((n, k)), rng.standard_normal((o, k)) * 0.05
    hx, xc, xs = quantized(x, "bf16", 1)
    hw, wc, wsc = quantized(w, "bf16", 128)
    p = Product(0, n, o, k)
    p.x, p.xs, p.w, p.ws = xc, xs.astype(np.float32), wc, wsc.astype(np.float32)
    got = p.check()
    # codes are off by 2^-4 of a value, or half of the smallest step 2^-9 times the scale
    ex = 2.0 ** -4 * np.abs(hx) + 2.0 ** -10 * np.repeat(xs, 128, 1)[:, :k]
    ew = 2.0 ** -4 * np.abs(hw) + 2.0 ** -10 * np.repeat(np.repeat(wsc, 128, 0)[:o], 128, 1)[:, :k]
    off = ex @ np.abs(hw).T + np.abs(hx) @ ew.T + ex @ ew.T
    y, mag = D.matmul(xc, xs, wc, wsc)
    assert (np.abs(got - hx @ hw.T) <= off + D.matmul_bound("bf16", y, mag, k)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_out,k", [(20, 22016, 144), (33, 32000, 128), (60, 11008, 272), (100, 22016, 16), (128, 32000, 144), (128, 8192, 1040),
                                       (1, 40, 16384), (1, 32000, 144), (9, 32000, 1040), (16, 11008, 400), (16, 136, 8336), (300, 11008, 144), (40, 136, 8336), (128, 264, 16384), (200, 136, 8336), (2000, 2056, 1168)])
def test_matmul_of_wide_and_deep_weights(n, n_out, k, dtype):
    Product(n + n_out + k, n, n_out, k, dtype=dtype).check()


@pytest.mark.parametrize("n", [2, 40, 150, 1000])
def test_products_at_once(n):
    """Calls on two streams that share weights and rows."""
    p, q = (Product(n, n, 1032, 400) for _ in range(2))
    p.upload()
    q.upload()
    q.dw, q.dws, q.dx, q.dxs = p.dw, p.dws, p.dx, p.dxs
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        p.call(a)
        q.call(b)
    y, mag = D.matmul(p.x, p.xs, p.w, p.ws)
    for c in (p, q):
        assert (np.abs(c.result() - y) <= D.matmul_bound("bf16", y, mag, 400)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_out,k", [(65, 64, 144), (66, 72, 16), (130, 1032, 400), (1030, 1032, 240), (1030, 4104, 272), (4100, 4104, 144), (4100, 4104, 112)])
def test_matmul_of_rows_that_end_with_their_storage(n, n_out, k, dtype):
    """Rows side by side, the last one's codes the storage's last, and a last block that is cut."""
    p = Product(n + n_out, n, n_out, k, pad=0, dtype=dtype)
    p.check()
    assert p.dw.untyped_storage().nbytes() == n_out * k and p.dx.untyped_storage().nbytes() == n * k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_out,k", [(4000, 4040, 272), (4090, 4096, 16), (3900, 4088, 1424)])
def test_matmul_by_the_largest_tiles(n, n_out, k, dtype):
    """256 tiles of 256 x 256 or a few more: one round of them is less than what smaller ones take."""
    Product(n + k, n, n_out, k, dtype=dtype, pad=16 * (k % 32 == 0)).check()


def code(v):
    return int(R.encode(np.array([float(v)]))[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,n_out", [(8, 264), (8, 32000), (20, 264), (64, 264), (64, 11008), (70, 264), (1030, 2056), (4000, 4040)])
def test_matmul_of_scales_whose_product_f32_does_not_hold(n, n_out, dtype):
    """Two scales of a block whose product is beyond f32, over sums that bring
    the result back into its range or leave it beyond, or is below its normal
    numbers."""
    p = Product(n, n, n_out, 784, dtype=dtype)
    p.ws[0, :6] = 2.0 ** 30, 2.0 ** 40, 1.37 * 2.0 ** -60, 2.0 ** 30, 1.0, 0.0
    ordinary = p.x[:8].copy(), p.xs[:8].copy()
    at = lambda b: np.s_[b * 128:(b + 1) * 128]
    p.x[:8] = 0
    p.xs[0, 0] = 2.0 ** 120                        # a sum of 0
    p.xs[1, 1] = 2.0 ** 100                        # one of 2^-18
    p.x[1, 128 + 9], p.w[:128, 128 + 9] = code(2.0 ** -9), code(2.0 ** -9)
    p.w[:16, at(2)] = code(448.0)
    p.x[2:4, at(2)] = code(448.0)                  # ones of up to 2^24.6
    p.xs[2, 2], p.xs[3, 2] = 1.21 * 2.0 ** -85, 1.21 * 2.0 ** -93
    p.x[4, at(3)], p.xs[4, 3] = code(1.0), 2.0 ** 120  # beyond f32 in the end
    p.x[5, at(4)], p.xs[5, 4] = code(3.0), np.inf
    p.x[6, at(5)], p.xs[6, 5] = code(448.0), 2.0 ** 127  # by a scale of 0
    p.xs[7] = 0.0
    p.upload()
    p.call()
    got = p.result()
    with np.errstate(over="ignore"):
        want, mag = D.matmul(p.x, p.xs.astype(float), p.w, p.ws.astype(float))
        # matmul_bound's, with half a step of the type's smallest numbers in the place of its absolute term, and
        # half a step of 2^-149 of the scales' product by sums of up to 128 448^2 in each of the blocks
        bound = D.matmul_bound(dtype, want, mag, p.k) - 1e-37 + (2.0 ** -134 if dtype == "bf16" else 2.0 ** -150)
        bound += 2.0 ** -150 * 128 * 448.0 ** 2 * 7
    beyond = np.abs(want) > 3.4e38
    assert beyond[4].any() and np.isinf(want[5]).any() and (want[6, :128] == 0).all()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[beyond], np.sign(want[beyond]) * np.inf)
    live = np.isfinite(want) & ~beyond
    bad = np.abs(got[live] - want[live]) > bound[live]
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} in rows {sorted(set(np.argwhere(live)[bad][:, 0].tolist()))[:9]}"
    # the rows beside are the same bits where none of these rows is there
    p.x[:8], p.xs[:8] = ordinary
    p.upload()
    p.call()
    assert np.array_equal(p.result()[8:], got[8:])
