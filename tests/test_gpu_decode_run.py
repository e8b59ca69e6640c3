"""The step with 8-bit base weights, rotation and next tokens, run as a serving
loop runs it: every part against the plain 64-bit form of what it was handed,
and the whole from a graph."""
import numpy as np
import pytest

import decode_ops_ref as D
import verify_ref as R
from adapter_lora_bgmv_amd import binding as B
from adapter_lora_bgmv_amd.verify_step import Sizes, VerifyStep
from test_gpu_verify import host

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
SMALL = dict(hidden=272, heads=4, kv_heads=2, head_dim=64, vocab=1000, page_tokens=16, slots=3, rank=16, top=4)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    B.lora_init()


def step_of(**options):
    step = VerifyStep(Sizes(**SMALL, **options), n_seqs=5, draft=3, max_tokens=64)
    for a in (step.cache.k, step.cache.v):
        a.fill_(0x7F)
    for a in (step.cache.k_scale, step.cache.v_scale):
        a.fill_(127)
    rng = np.random.default_rng(0)
    if options.get("sample"):
        for name, v in (("temperature", rng.choice([0.0, 0.7, 1.0], step.n)), ("top_p", rng.choice([0.8, 1.0], step.n)),
                        ("min_p", rng.choice([0.0, 0.05], step.n)), ("top_k", rng.choice([0, 20], step.n))):
            t = getattr(step, name)
            t.copy_(torch.as_tensor(v.astype(np.float32 if t.dtype == torch.float32 else np.int32)))
    return step, rng


def mirror(step):
    c = step.cache
    return R.Cache(host(c.k), host(c.v), host(c.k_scale), host(c.v_scale), step.s.page_tokens, step.s.head_dim)


def test_every_part_of_a_step():
    step, rng = step_of(base8=True, theta=10000.0, sample=True)
    s, n = step.s, step.n
    for t in (3, 6, 16, 19, 41):  # the drafts reach past a page's end, and a length jumps over pages that hold NaN
        x = (torch.randn(n, s.hidden, device="cuda", generator=torch.Generator("cuda").manual_seed(t))).bfloat16()
        step.seqs.kv_len.fill_(t)
        step.ids.random_(0, s.vocab)
        step.uniform.copy_(torch.as_tensor(rng.random(n).astype(np.float32)))
        seqs = {"table": host(step.seqs.page_table), "kv_len": np.full(5, t), "indptr": np.arange(0, n + 1, 3)}
        parts = step.parts(x)
        parts["qkv"]()
        torch.cuda.synchronize()
        codes, scale = D.quantize(host(x), 1)
        assert np.array_equal(host(step.x8[0]), codes) and np.array_equal(host(step.x8[1]), scale)
        y, mag = D.matmul(codes, scale, host(step.w_qkv8[0]), host(step.w_qkv8[1]))
        low = np.stack([host(step.a[i]) @ v for i, v in zip(host(step.seq_slot), host(x))])
        delta = np.stack([2.0 * host(step.b[i]) @ v for i, v in zip(host(step.seq_slot), low)])
        size = np.stack([2.0 * np.abs(host(step.b[i])) @ (np.abs(host(step.a[i])) @ np.abs(v)) for i, v in zip(host(step.seq_slot), host(x))])
        # a rounding of the product, one of the sum, and the delta's f32 sums over hidden + rank terms
        bound = D.matmul_bound("bf16", y, mag, s.hidden) + 2.0 ** -8 * (np.abs(y + delta) + 2.0 ** -8 * np.abs(y)) + (s.hidden + s.rank) * 2.0 ** -24 * size
        qkv = host(step.qkv)
        assert (np.abs(qkv - (y + delta)) <= bound).all()
        before = mirror(step)
        parts["write"]()
        torch.cuda.synchronize()
        heads = qkv.reshape(n, -1, s.head_dim)
        pos = np.concatenate([np.arange(t - 3, t)] * 5)
        turned = D.turn(heads[:, :s.heads + s.kv_heads], pos, host(step.rotary.inv_freq), False)
        R.write(before, seqs, turned[:, s.heads:].astype(np.float32).astype(float), heads[:, s.heads + s.kv_heads:])
        after = mirror(step)
        for name in ("ke", "ve", "k", "v"):
            a, b = getattr(after, name), getattr(before, name)
            if name in "kv":  # a code's NaN has two forms, 0x7F and 0xFF
                a, b = np.where((a & 127) == 127, 127, a), np.where((b & 127) == 127, 127, b)
            at = np.argwhere(a != b)
            assert not len(at), f"{name} at {t} tokens: {len(at)} differ, first {at[:4].tolist()}, {a[a != b][:4]} for {b[a != b][:4]}"
        q = host(step.qkv)[:, :step.q_dim].reshape(n, s.heads, -1)
        assert (np.abs(q - turned[:, :s.heads]) <= D.turn_bound("bf16", heads[:, :s.heads], turned[:, :s.heads], s.head_dim // 2, False)).all()
        parts["attend"]()
        torch.cuda.synchronize()
        want, lse, m, big, toks = R.attend(after, seqs, q, float(np.float32(s.head_dim ** -0.5)), 0)
        bo, _ = R.attend_bounds("bf16", want, lse, m, big, toks, s.head_dim)
        out = host(step.out).reshape(want.shape)
        live = np.isfinite(want)
        assert np.array_equal(np.isfinite(out), live) and (np.abs(out - want)[live] <= bo[live]).all()
        parts["vocabulary"]()
        torch.cuda.synchronize()
        codes, scale = D.quantize(host(step.out), 1)
        assert np.array_equal(R.TABLE[host(step.out8[0])], R.TABLE[codes], equal_nan=True) and np.array_equal(host(step.out8[1]), scale)
        y, mag = D.matmul(codes, scale, host(step.w_vocab8[0]), host(step.w_vocab8[1]))
        logits = host(step.logits)
        fine = np.isfinite(y)
        assert np.array_equal(np.isfinite(logits), fine)
        assert (np.abs(logits - y)[fine] <= D.matmul_bound("bf16", y, mag, step.q_dim)[fine]).all()
        parts["scores"]()
        parts["sample"]()
        torch.cuda.synchronize()
        for i in range(n):
            kw = {a: getattr(step, f)[i].item() for a, f in zip("tkpmu", ("temperature", "top_k", "top_p", "min_p", "uniform"))}
            ids, logp = D.sample(logits[i], **kw)
            got = step.scores["token"][i].item()
            assert got in ids
            if got >= 0:
                assert abs(step.scores["token_logp"][i].item() - logp[ids.index(got)]) <= 2.0 ** -24 * abs(logp[ids.index(got)]) + 1e-12


def test_the_step_as_a_whole_and_from_a_graph():
    step, rng = step_of(base8=True, theta=10000.0, sample=True)
    n, results = step.n, []
    xs = [torch.randn(n, step.s.hidden, device="cuda").bfloat16() for _ in range(4)]
    us = rng.random((4, n)).astype(np.float32)
    for i in range(4):
        got = step.run(xs[i], [3 * (i + 1)] * 5, np.arange(n), uniform=us[i])
        results.append({k: host(v).copy() for k, v in got.items()} | {"qkv": host(step.qkv).copy()})
    cache = mirror(step)
    fresh, _ = step_of(base8=True, theta=10000.0, sample=True)
    x = xs[0].clone()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for call in fresh.parts(x, stream).values():
            call()
    for i in range(4):
        x.copy_(xs[i])
        fresh.seqs.kv_len.fill_(3 * (i + 1))
        fresh.ids.copy_(torch.arange(n, dtype=torch.int32))
        fresh.uniform.copy_(torch.as_tensor(us[i]))
        graph.replay()
        torch.cuda.synchronize()
        for k, v in results[i].items():
            got = host(fresh.qkv if k == "qkv" else fresh.scores[k])
            assert np.array_equal(got, v, equal_nan=v.dtype.kind == "f"), (i, k)
    again = mirror(fresh)
    for name in ("ke", "ve", "k", "v"):
        assert np.array_equal(getattr(again, name), getattr(cache, name))


def test_options_leave_the_rest_of_the_step_as_it_was():
    """Without options the same calls as ever, and next tokens change no score."""
    base, _ = step_of()
    more, _ = step_of(sample=True)
    assert list(base.parts(None)) == ["qkv", "write", "attend", "vocabulary", "scores"]
    assert list(more.parts(None)) == ["qkv", "write", "attend", "vocabulary", "scores", "sample"]
    x = torch.randn(base.n, base.s.hidden, device="cuda").bfloat16()
    a = base.run(x, [3] * 5, np.arange(base.n))
    b = more.run(x, [3] * 5, np.arange(base.n), uniform=np.zeros(base.n))
    for k in a:
        assert torch.equal(a[k], b[k])
