"""Refusals of the verify-step entry points, before any launch and without a
GPU, and the plain forms that the GPU tests compare with."""
import ctypes as C

import numpy as np
import pytest

import verify_ref as R
from adapter_lora_bgmv_amd import binding as B

FAKE = 4096  # an aligned non-NULL address; validation fails before it is used
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return B.lib()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, n_pages=64, n_kv_heads=8, head_dim=128, page_tokens=16)
    a.update(kw)
    return B.lora_kv_cache(*[a[f] for f, _ in B.lora_kv_cache._fields_])


def seqs(**kw):
    a = dict(page_table=FAKE, row_indptr=FAKE, kv_len=FAKE, n_seqs=4, max_pages=16, table_stride=16, max_rows=1)
    a.update(kw)
    return B.lora_kv_seqs(*[a[f] for f, _ in B.lora_kv_seqs._fields_])


def rows_call(L, fn, c=None, s=None, dtype=B.LORA_BF16, k=FAKE, ks=1024, v=FAKE, vs=1024, n=4):
    c, s = c or cache(), s or seqs()
    rc = getattr(L, fn)(C.byref(c), C.byref(s), dtype, k, ks, v, vs, n, None)
    return rc, L.lora_last_error().decode()


def attend(L, c=None, s=None, dtype=B.LORA_BF16, heads=32, q=FAKE, qs=4096, scale=0.1, window=0, n=4, out=FAKE, os=4096,
           ws=FAKE, ws_bytes=BIG):
    c, s = c or cache(), s or seqs()
    rc = L.lora_kv_attend(C.byref(c), C.byref(s), dtype, heads, q, qs, scale, window, n, out, os, None, ws, ws_bytes, None)
    return rc, L.lora_last_error().decode()


def score(L, dtype=B.LORA_BF16, V=1000, logits=FAKE, stride=1000, ids=FAKE, n=4, top=3, logp=FAKE, ti=FAKE, tl=FAKE, ws=FAKE,
          ws_bytes=BIG):
    rc = L.lora_token_logprobs(dtype, V, logits, stride, ids, n, top, logp, None, None, ti, tl, ws, ws_bytes, None)
    return rc, L.lora_last_error().decode()


KV_REFUSALS = [
    (dict(dtype=5), -4, "dtype 5"),
    (dict(c=dict(n_pages=0)), -1, "n_pages 0"),
    (dict(c=dict(n_kv_heads=0)), -1, "n_kv_heads 0"),
    (dict(c=dict(head_dim=96)), -5, "head_dim 96"),
    (dict(c=dict(page_tokens=48)), -5, "page_tokens 48"),
    (dict(c=dict(page_tokens=256)), -5, "page_tokens 256"),
    (dict(c=dict(n_pages=2 ** 31, page_tokens=128)), -1, "groups"),
    (dict(c=dict(k=None)), -2, "k"),
    (dict(c=dict(v_scale=None)), -2, "v_scale"),
    (dict(c=dict(v=FAKE + 8)), -5, "aligned"),
    (dict(s=dict(n_seqs=0)), -1, "n_seqs 0"),
    (dict(s=dict(n_seqs=20000)), -1, "n_seqs 20000"),
    (dict(s=dict(max_pages=0)), -1, "max_pages 0"),
    (dict(s=dict(max_pages=2 ** 28, table_stride=2 ** 28)), -1, "max_pages"),
    (dict(s=dict(table_stride=15)), -3, "table_stride 15 < max_pages 16"),
    (dict(s=dict(kv_len=None)), -2, "kv_len"),
    (dict(n=16385), -1, "16385"),
]


def unpack(kw):
    kw = dict(kw)
    for key, make in (("c", cache), ("s", seqs)):
        if key in kw:
            kw[key] = make(**kw[key])
    return kw


@pytest.mark.parametrize("kw,code,text", KV_REFUSALS)
@pytest.mark.parametrize("fn", ["lora_kv_write", "lora_kv_read", "lora_kv_attend"])
def test_cache_and_sequence_refusals(L, fn, kw, code, text):
    kw = unpack(kw)
    rc, msg = attend(L, **kw) if fn == "lora_kv_attend" else rows_call(L, fn, **kw)
    assert rc == code and text in msg and msg.startswith(fn), (rc, msg)


@pytest.mark.parametrize("fn", ["lora_kv_write", "lora_kv_read"])
def test_row_refusals(L, fn):
    for kw, code, text in [(dict(ks=1023), -3, "k row stride 1023"), (dict(vs=8), -3, "v row stride 8"),
                           (dict(ks=1028), -5, "multiple of 8"), (dict(vs=1026, dtype=B.LORA_F32), -5, "multiple of 4"),
                           (dict(k=None), -2, "k must"), (dict(v=FAKE + 4), -5, "aligned"),
                           (dict(ks=2 ** 31), -3, "exceeds")]:
        rc, msg = rows_call(L, fn, **kw)
        assert rc == code and text in msg, (rc, msg)
    assert rows_call(L, fn, n=0, k=None, v=None)[0] == 0
    for c, s in ((None, C.byref(seqs())), (C.byref(cache()), None)):
        assert getattr(L, fn)(c, s, 1, FAKE, 1024, FAKE, 1024, 4, None) == -2


def test_attend_refusals(L):
    for kw, code, text in [(dict(heads=0), -1, "n_heads 0"), (dict(heads=12), -1, "multiple of n_kv_heads 8"),
                           (dict(scale=0.0), -1, "scale"), (dict(scale=-1.0), -1, "scale"),
                           (dict(scale=float("inf")), -1, "scale"), (dict(scale=float("nan")), -1, "scale"),
                           (dict(window=2 ** 31), -1, "window"), (dict(qs=4095), -3, "q row stride"),
                           (dict(os=4100), -5, "out row stride"), (dict(q=None), -2, "q must"),
                           (dict(out=FAKE + 2), -5, "out"), (dict(ws=None), -7, "workspace"),
                           (dict(ws_bytes=1000), -7, "1000 bytes"), (dict(ws=FAKE + 8), -5, "workspace")]:
        rc, msg = attend(L, **kw)
        assert rc == code and text in msg, (rc, msg)
    assert attend(L, n=0, q=None, out=None, ws=None)[0] == 0
    assert B.lib().lora_kv_attend_workspace_bytes(None, None, 1, 8, 4) == 0


def test_attend_workspace_needs_no_device(L):
    c = cache()
    one = L.lora_kv_attend_workspace_bytes(C.byref(c), C.byref(seqs()), B.LORA_BF16, 32, 4)
    many = L.lora_kv_attend_workspace_bytes(C.byref(c), C.byref(seqs(max_rows=0)), B.LORA_BF16, 32, 4000)
    assert 0 < one <= many
    assert L.lora_kv_attend_workspace_bytes(C.byref(c), C.byref(seqs()), B.LORA_BF16, 32, 0) == 0


def test_score_refusals(L):
    for kw, code, text in [(dict(dtype=-1), -4, "dtype -1"), (dict(V=0), -1, "n_vocab 0"),
                           (dict(V=(1 << 20) + 1, stride=1 << 21), -1, "n_vocab 1048577"), (dict(n=16385), -1, "16385"),
                           (dict(top=33), -1, "top 33"), (dict(V=2, top=3), -1, "n_vocab 2"), (dict(stride=999), -3, "999"),
                           (dict(logits=None), -2, "logits"), (dict(ids=None), -2, "token_ids"), (dict(logp=None), -2, "logp"),
                           (dict(ti=None), -2, "top_ids"), (dict(tl=None), -2, "top_logp"),
                           (dict(logits=FAKE + 1), -5, "aligned"), (dict(logits=FAKE + 2, dtype=B.LORA_F32), -5, "aligned"),
                           (dict(V=100000, stride=100000, ws=None), -7, "workspace"),
                           (dict(V=100000, stride=100000, ws_bytes=64), -7, "64 bytes"),
                           (dict(V=100000, stride=100000, ws=FAKE + 4), -5, "workspace")]:
        rc, msg = score(L, **kw)
        assert rc == code and text in msg, (rc, msg)
    assert score(L, n=0, logits=None)[0] == 0
    assert B.lora_token_logprobs_workspace_bytes(B.LORA_BF16, 32000, 16000, 5) == 0  # rows enough: a workgroup each
    assert B.lora_token_logprobs_workspace_bytes(B.LORA_BF16, 32000, 1, 5) > 0


def test_no_gpu_is_a_loud_error(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc, msg in (rows_call(L, "lora_kv_write"), attend(L), score(L)):
        assert rc == -6 and msg


def test_bindings_refuse_other_arrays():
    import torch
    k = torch.zeros(2, 1, 16 * 64, dtype=torch.uint8)
    e = torch.zeros(2, 1, dtype=torch.uint8)
    B.KVCache(k, k.clone(), e, e.clone(), page_tokens=16, head_dim=64)
    for bad in ((k.int(), k, e, e), (k, k[:1], e, e), (k, k, e.t(), e), (k, k, e, e.float())):
        with pytest.raises(ValueError):
            B.KVCache(*bad, page_tokens=16, head_dim=64)
    table, ptr, lens = (torch.zeros(*s, dtype=torch.int32) for s in ((3, 4), (4,), (3,)))
    assert B.KVSeqs(table[:, :2], ptr, lens).c.table_stride == 4
    for bad in ((table.long(), ptr, lens), (table, ptr[:3], lens), (table, ptr, lens[:2]), (table.t()[:3], ptr, lens)):
        with pytest.raises(ValueError):
            B.KVSeqs(*bad)


# ---------------------------------------------------------------- the plain forms themselves
def test_reference_codes_round_to_nearest_even():
    import torch
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * np.exp2(rng.integers(-14, 9, 20000))).astype(np.float32)
    x = np.concatenate([x[np.abs(x) <= 448], (R.TABLE[:126] + R.TABLE[1:127]) / 2]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.encode(x), want)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(R.TABLE, every, equal_nan=True)


def test_reference_scale_is_the_smallest_power_that_holds():
    for a in (448.0, 448.0001, 447.9, 1e-30, 3e38, 2.0 ** -140, 0.875, 1.75, 1.7500001):
        e = R.scale_byte(a)
        assert a <= 448 * 2.0 ** (e - 127) and (e == R.E_MIN or a > 448 * 2.0 ** (e - 128))


def test_reference_orders_are_permutations():
    for P in (16, 32, 64, 128):
        for D in (64, 128, 256):
            for o in (R.k_order(P, D), R.v_order(P, D)):
                assert np.array_equal(np.sort(o.reshape(-1)), np.arange(P * D))
