"""Refusals of the 8-bit product, the cache write with rotation and the
sampling, before any launch and without a GPU."""
import ctypes as C

import pytest

from adapter_lora_bgmv_amd import binding as B
from test_verify_abi_cpu import BIG, FAKE, KV_REFUSALS, cache, seqs, unpack


@pytest.fixture(scope="module")
def L():
    return B.lib()


def quantize(L, dtype=B.LORA_BF16, n=4, k=256, x=FAKE, xs=256, block=1, codes=FAKE, cs=256, scale=FAKE, ss=2):
    rc = L.lora_quantize_fp8(dtype, n, k, x, xs, block, codes, cs, scale, ss, None)
    return rc, L.lora_last_error().decode()


def matmul(L, dtype=B.LORA_BF16, n_out=64, k=256, W=FAKE, wst=256, wsc=FAKE, wss=2, x=FAKE, xst=256, xsc=FAKE, xss=2, n=4, y=FAKE,
           yst=64, ws=FAKE, ws_bytes=BIG):
    rc = L.lora_matmul_fp8(dtype, n_out, k, W, wst, wsc, wss, x, xst, xsc, xss, n, y, yst, ws, ws_bytes, None)
    return rc, L.lora_last_error().decode()


def rotary(**kw):
    a = dict(inv_freq=FAKE, rot_dim=128, interleaved=0)
    a.update(kw)
    return B.lora_rotary(*[a[f] for f, _ in B.lora_rotary._fields_])


def rotate(L, c=None, s=None, r=None, dtype=B.LORA_BF16, heads=32, q=FAKE, qs=6144, out=FAKE, os=4096, k=FAKE, ks=6144, v=FAKE,
           vs=6144, n=4):
    c, s, r = c or cache(), s or seqs(), r or rotary()
    rc = L.lora_kv_write_rotary(C.byref(c), C.byref(s), C.byref(r), dtype, heads, q, qs, out, os, k, ks, v, vs, n, None)
    return rc, L.lora_last_error().decode()


def sample(L, dtype=B.LORA_BF16, V=1000, logits=FAKE, stride=1000, t=FAKE, k=FAKE, p=FAKE, m=FAKE, u=FAKE, n=4, ids=FAKE, logp=FAKE,
           ws=FAKE, ws_bytes=BIG):
    rc = L.lora_token_sample(dtype, V, logits, stride, t, k, p, m, u, n, ids, logp, ws, ws_bytes, None)
    return rc, L.lora_last_error().decode()


def test_quantize_refusals(L):
    for kw, code, text in [(dict(dtype=7), -4, "dtype 7"), (dict(block=64), -5, "block_rows 64"), (dict(block=0), -5, "block_rows 0"),
                           (dict(k=0), -1, "k 0"), (dict(k=24), -5, "k 24"), (dict(k=2 ** 31), -1, "k 2147483648"),
                           (dict(n=2 ** 31, k=16, xs=16, cs=16), -1, "n_rows 2147483648"), (dict(xs=248), -3, "x row stride 248"),
                           (dict(xs=260), -5, "multiple of 8"), (dict(xs=258, dtype=B.LORA_F32), -5, "multiple of 4"),
                           (dict(x=None), -2, "x must"), (dict(x=FAKE + 8), -5, "aligned"), (dict(cs=240), -3, "codes row stride 240"),
                           (dict(cs=264), -5, "multiple of 16"), (dict(codes=None), -2, "codes"), (dict(codes=FAKE + 4), -5, "aligned"),
                           (dict(ss=1), -3, "scale stride 1"), (dict(scale=None), -2, "scales"), (dict(scale=FAKE + 2), -5, "aligned")]:
        rc, msg = quantize(L, **kw)
        assert rc == code and text in msg and msg.startswith("lora_quantize_fp8"), (kw, rc, msg)
    assert quantize(L, n=0, x=None, codes=None, scale=None)[0] == 0


def test_matmul_refusals(L):
    for kw, code, text in [(dict(dtype=2), -4, "dtype 2"), (dict(n_out=0), -1, "n_out 0"), (dict(n_out=60), -5, "n_out 60"),
                           (dict(n_out=2 ** 26 + 8, yst=2 ** 27), -1, "n_out 67108872"), (dict(k=0), -1, "k_in 0"),
                           (dict(k=65552, wst=65552, xst=65552), -1, "k_in 65552"), (dict(k=250), -5, "k_in 250"),
                           (dict(n=16385), -1, "16385"), (dict(wst=240), -3, "W row stride 240"), (dict(xst=264), -5, "x row stride 264"),
                           (dict(W=None), -2, "W codes"), (dict(wsc=None), -2, "W codes"), (dict(x=None), -2, "x codes"),
                           (dict(xsc=None), -2, "x codes"), (dict(wss=1), -3, "W scale stride 1"), (dict(xss=1), -3, "x scale stride 1"),
                           (dict(W=FAKE + 8), -5, "W"), (dict(x=FAKE + 1), -5, "x"), (dict(wsc=FAKE + 2), -5, "aligned"),
                           (dict(yst=56), -3, "y row stride 56"), (dict(yst=68), -5, "multiple of 8"),
                           (dict(yst=66, dtype=B.LORA_F32), -5, "multiple of 4"), (dict(y=None), -2, "y must"),
                           (dict(y=FAKE + 4), -5, "aligned"), (dict(wst=2 ** 22 + 16), -3, "W 4194320"),
                           (dict(xst=2 ** 22 + 16), -3, "x 4194320"), (dict(xss=2 ** 22 + 1), -3, "scales 4194305")]:
        rc, msg = matmul(L, **kw)
        assert rc == code and text in msg and msg.startswith("lora_matmul_fp8"), (kw, rc, msg)
    assert matmul(L, n=0, W=None, wsc=None, x=None, xsc=None, y=None, ws=None, ws_bytes=0)[0] == 0


@pytest.mark.parametrize("kw,code,text", KV_REFUSALS)
def test_rotary_refuses_what_the_write_refuses(L, kw, code, text):
    rc, msg = rotate(L, **unpack(kw))
    assert rc == code and text in msg and msg.startswith("lora_kv_write_rotary"), (rc, msg)


def test_rotary_refusals(L):
    for kw, code, text in [(dict(r=rotary(inv_freq=None)), -2, "inv_freq"), (dict(r=rotary(inv_freq=FAKE + 2)), -5, "inv_freq"),
                           (dict(r=rotary(rot_dim=0)), -5, "rot_dim 0"), (dict(r=rotary(rot_dim=24)), -5, "rot_dim 24"),
                           (dict(r=rotary(rot_dim=144)), -5, "rot_dim 144"), (dict(r=rotary(interleaved=2)), -5, "interleaved 2"),
                           (dict(r=rotary(interleaved=-1)), -5, "interleaved -1"), (dict(heads=65536, qs=2 ** 24, os=2 ** 24), -1, "n_heads 65536"),
                           (dict(q=None), -2, "q must"), (dict(out=None), -2, "q_out must"), (dict(q=FAKE + 8), -5, "q "),
                           (dict(qs=4088), -3, "q row stride 4088"), (dict(os=4088), -3, "q_out row stride 4088"),
                           (dict(os=4100), -5, "q_out row stride 4100"), (dict(q=FAKE, out=FAKE), -3, "in place"),
                           (dict(ks=1016), -3, "k row stride"), (dict(vs=1028), -5, "v row stride"), (dict(k=None), -2, "k must"),
                           (dict(v=FAKE + 2), -5, "v ")]:
        if "in place" not in text:
            kw = {"out": 2 * FAKE, **kw}
        rc, msg = rotate(L, **kw)
        assert rc == code and text in msg, (kw, rc, msg)
    assert rotate(L, n=0, q=None, out=None, k=None, v=None)[0] == 0
    assert L.lora_kv_write_rotary(C.byref(cache()), C.byref(seqs()), None, 1, 0, None, 0, None, 0, FAKE, 1024, FAKE, 1024, 4, None) == -2
    # more workgroups than a grid has
    c, s = cache(n_kv_heads=65535, n_pages=1000), seqs(n_seqs=16384, max_pages=16, table_stride=16)
    wide = 65535 * 128
    rc, msg = rotate(L, c=c, s=s, heads=65535, qs=wide, out=2 * FAKE, os=wide, ks=wide, vs=wide, n=16384)
    assert rc == -1 and "workgroups" in msg, (rc, msg)


def test_sample_refusals(L):
    for kw, code, text in [(dict(dtype=3), -4, "dtype 3"), (dict(V=0), -1, "n_vocab 0"),
                           (dict(V=(1 << 20) + 1, stride=1 << 21), -1, "n_vocab 1048577"), (dict(n=16385), -1, "16385"),
                           (dict(stride=999), -3, "row_stride 999"), (dict(logits=None), -2, "logits"), (dict(u=None), -2, "uniform"),
                           (dict(ids=None), -2, "ids"), (dict(logits=FAKE + 1), -5, "aligned"),
                           (dict(logits=FAKE + 2, dtype=B.LORA_F32), -5, "aligned")]:
        rc, msg = sample(L, **kw)
        assert rc == code and text in msg and msg.startswith("lora_token_sample"), (kw, rc, msg)
    assert sample(L, n=0, logits=None, u=None, ids=None, ws=None)[0] == 0


def test_workspaces_need_no_device(L):
    assert L.lora_matmul_fp8_workspace_bytes(B.LORA_BF16, 64, 256, 0) == 0
    assert L.lora_token_sample_workspace_bytes(B.LORA_BF16, 1000, 0) == 0
    for n in (1, 64, 4096, 16384):
        assert L.lora_matmul_fp8_workspace_bytes(B.LORA_BF16, 4096, 4096, n) < 1 << 30
        assert L.lora_token_sample_workspace_bytes(B.LORA_F32, 131071, n) < 1 << 30


def test_no_gpu_is_a_loud_error(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for rc, msg in (quantize(L), matmul(L), rotate(L, out=2 * FAKE), sample(L)):
        assert rc == -6 and msg


def test_rotary_binding_refuses_other_arrays():
    import torch
    f = torch.zeros(32)
    assert B.Rotary(f).rot_dim == 64
    for bad in (f.double(), f[::2], f.reshape(2, 16)):
        with pytest.raises(ValueError):
            B.Rotary(bad)
