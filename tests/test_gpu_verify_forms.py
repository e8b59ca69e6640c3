"""The attention's forms and rare paths: column counts at every border between
forms, maxima that keep moving, value scales out of the operand's range, pages
of zeros, many sequences, and the verify step run as one."""
import numpy as np
import pytest

import verify_ref as R
from adapter_lora_bgmv_amd import binding as B
from test_gpu_verify import Setup, host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lora_init()


def set_codes(s, which, f):
    """Rewrites every page's codes of K or V from f(page, values) -> values, with their scales."""
    codes, exps = (s.host.k, s.host.ke) if which == "k" else (s.host.v, s.host.ve)
    for p in range(codes.shape[0]):
        for h in range(codes.shape[1]):
            x = R.TABLE[codes[p, h]] * 2.0 ** (int(exps[p, h]) - 127)
            nan = np.isnan(x)
            y = f(p, np.where(nan, 0.0, x))
            exps[p, h] = R.scale_byte(np.abs(y).max())
            codes[p, h] = np.where(nan, codes[p, h], R.encode(y * 2.0 ** (127 - int(exps[p, h]))))
    s.upload()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [4, 5, 16, 17, 32, 33, 65])
def test_columns_at_the_forms_borders(rows, D, dtype):
    """4 query heads to a key/value head: 16, 20, 64, 68, 128, 132 and 260 columns, and a single row beside them."""
    s = Setup(200 + rows, [(rows, 70 + rows), (1, 65), (rows, rows)], 1, D, 16)
    s.check(dtype, 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 700)], [(9, 700)], [(40, 700)]])
@pytest.mark.parametrize("step", [4.0, -4.0, 40.0])
def test_scores_that_keep_rising_or_falling(lens, step, dtype):
    """The largest score moves by more than the lag from tile to tile, up and down."""
    D = 64
    s = Setup(210, lens, 1, D, 64)
    order = {int(p): i for i, p in enumerate(s.seqs["table"][0])}
    q = np.zeros((s.n, 2, D))
    q[:, :, 0] = 1.0
    q[:, :, 1:] = s.rng.standard_normal((s.n, 2, D - 1)) * 0.1
    set_codes(s, "k", lambda p, x: np.concatenate([np.full_like(x[:, :1], 8 + order.get(p, 0) * step), x[:, 1:]], 1))
    got = s.attend(dtype, 2, scale=1.0, q=q)
    want, wl, mag, big, toks = R.attend(s.host, s.seqs, got[0], 1.0, 0)
    bo, bl = R.attend_bounds(dtype, want, wl, mag, big, toks, D)
    assert (np.abs(got[1] - want) <= bo).all() and (np.abs(got[2] - wl) <= bl).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 400)], [(9, 400)], [(40, 400)]])
@pytest.mark.parametrize("kind", ["zeros", "tiny", "large", "mixed"])
def test_value_scales_of_every_size(lens, kind, dtype):
    """Pages whose values are all zero (the smallest scale), 1e-9, 1e6, and all of
    these side by side: denominators and sums lose nothing."""
    s = Setup(220, lens, 2, 128, 16)
    first = s.seqs["table"][0]
    place = {int(p): i for i, p in enumerate(first)}

    def f(p, x):
        i = place.get(p, 0)
        if kind == "zeros":
            return x * 0.0 if i % 3 else x * 300.0
        if kind == "tiny":
            return x * 1e-9
        if kind == "large":
            return x * 1e6
        return x * [0.0, 1e-9, 1.0, 1e6][i % 4]

    set_codes(s, "v", f)
    s.check(dtype, 4)
    s.check(dtype, 4, window=37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_a_page_of_huge_values_do_not_feel_it(dtype):
    """Values of 1e30 in tokens that only the last rows see leave the others exact."""
    s = Setup(230, [(60, 130)], 1, 64, 16)
    last = int(s.seqs["table"][0, 129 // 16])
    set_codes(s, "v", lambda p, x: x * 1e30 if p == last else x * 1e-3)
    out = s.check(dtype, 2)
    assert np.abs(out[:50]).max() < 1.0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_lanes(dtype):
    """150 sequences, empty ones among them: several to a lane of the search."""
    rng = np.random.default_rng(3)
    lens = [(int(r), int(r + t)) for r, t in zip(rng.integers(0, 4, 150), rng.integers(0, 90, 150))]
    lens[70] = (30, 300)
    Setup(240, lens, 1, 64, 16).check(dtype, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 256])
def test_units_cut_into_many_pieces(D, dtype):
    """One long sequence beside short ones, few heads: the join of many pieces."""
    s = Setup(250, [(1, 9000), (1, 3), (2, 640)], 1, D, 128)
    s.check(dtype, 3)
    s.check(dtype, 3, window=5000)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_keys_and_values_in_whole_and_cut_tiles(dtype):
    """NaN that every row sees, that some see, and that none does, in one call of both many and few rows."""
    s = Setup(260, [(70, 300), (1, 100), (3, 90)], 1, 128, 16)
    for which, seq, pos in (("v", 0, 10), ("v", 0, 260), ("k", 1, 20), ("v", 2, 88)):
        getattr(s.host, which)[s.seqs["table"][seq, pos // 16], 0, pos % 16, 3] = 0x7F
    s.upload()
    s.check(dtype, 2)
    s.check(dtype, 2, window=64)


def test_a_workspace_of_any_content_serves():
    """What the workspace held before does not matter to the attention."""
    for lens in ([(1, 3000)], [(50, 2000), (1, 30)]):
        s = Setup(270, lens, 1, 64, 16)
        need = B.lora_kv_attend_workspace_bytes(s.cache, s.dseqs, B.LORA_BF16, 2, s.n)
        q = s.rng.standard_normal((s.n, 2, 64))
        first = s.attend("bf16", 2, q=q, ws=torch.zeros(need, dtype=torch.uint8, device="cuda"))[1]
        again = s.attend("bf16", 2, q=q, ws=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))[1]
        assert np.array_equal(first, again)


def test_verify_step_example():
    """The example's step, stage by stage from its own inputs, over two steps of drafts."""
    from adapter_lora_bgmv_amd import verify_step as V
    z = V.Sizes(hidden=512, heads=8, kv_heads=2, head_dim=64, vocab=1000, page_tokens=16, slots=3, rank=16)
    step = V.VerifyStep(z, n_seqs=3, draft=4, max_tokens=208, seed=5)
    rng = np.random.default_rng(6)
    n, Q, K = step.n, step.q_dim, step.kv_dim
    kc, vc, ke, ve = (host(t) for t in (step.cache.k.random_(0, 126), step.cache.v.random_(0, 126),
                                        step.cache.k_scale.fill_(120), step.cache.v_scale.fill_(118)))
    cache = R.Cache(kc, vc, ke, ve, 16, 64)
    for lens in ([50, 7, 190], [54, 11, 194]):
        ids = rng.integers(0, 1000, n)
        x = torch.from_numpy(rng.standard_normal((n, 512))).cuda().bfloat16()
        got = {m: host(t) for m, t in step.run(x, lens, ids).items()}
        torch.cuda.synchronize()
        qkv, hx, slot = host(step.qkv), host(x), host(step.seq_slot)
        # one bf16 rounding of the fused projection: 2^-9 of the value, f32 sums of 512 products and the rank-16 delta
        w, a, b = host(step.w_qkv), host(step.a), host(step.b)
        want = hx @ w.T + 2.0 * np.stack([b[s] @ (a[s] @ r) for s, r in zip(slot, hx)])
        size = np.abs(hx) @ np.abs(w).T + 2.0 * np.stack([np.abs(b[s]) @ (np.abs(a[s]) @ np.abs(r)) for s, r in zip(slot, hx)])
        assert (np.abs(qkv - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size).all()
        seqs = {"table": host(step.seqs.page_table), "kv_len": np.array(lens), "indptr": host(step.seqs.row_indptr)}
        R.write(cache, seqs, qkv[:, Q:Q + K].reshape(n, 2, 64), qkv[:, Q + K:].reshape(n, 2, 64))
        out, lse, mag, big, toks = R.attend(cache, seqs, qkv[:, :Q].reshape(n, 8, 64), 0.125, 0)
        bo, bl = R.attend_bounds("bf16", out, lse, mag, big, toks, 64)
        mine = host(step.out)
        assert (np.abs(mine.reshape(out.shape) - out) <= bo).all() and (np.abs(host(step.lse) - lse) <= bl).all()
        wv, logits = host(step.w_vocab), host(step.logits)
        assert (np.abs(logits - mine @ wv.T) <= 2.0 ** -8 * np.abs(logits) + 2.0 ** -14 * (np.abs(mine) @ np.abs(wv).T)).all()
        lp, en, rk, ti, tl = R.score(logits, ids, z.top)
        assert np.array_equal(got["rank"], rk) and np.array_equal(got["top_ids"], ti)
        for m, t in (("logp", lp), ("entropy", en), ("top_logp", tl)):
            assert (np.abs(got[m] - t) <= 1e-4).all(), m
