"""One layer's speculative-verify step through the library, as a serving loop runs it.

    python -m adapter_lora_bgmv_amd.verify_step

``VerifyStep.run`` takes the hidden rows of every sequence's draft tokens and
    projects them to [Q|K|V] rows, each row with its sequence's adapter (lora_apply),
    writes their keys and values into the 8-bit paged cache (lora_kv_write),
    attends over the cache (lora_kv_attend),
    projects to the vocabulary, base weights only (lora_apply), and
    scores the draft tokens (lora_token_logprobs).
With Sizes' options it also
    keeps its base weights in 8 bits (lora_quantize_fp8 in front of each projection,
        lora_matmul_fp8, the adapters' delta by lora_shrink and lora_expand_fold, so
        that a row with an adapter is rounded twice),
    turns queries and keys by their positions on the way into the cache
        (lora_kv_write_rotary in the place of lora_kv_write), and
    draws every row's next token (lora_token_sample), by the settings that the
        step's arrays temperature, top_k, top_p and min_p hold and the numbers
        handed to run.
Everything stays on the device and on one stream; pages, lengths, adapters and
token ids are device arrays whose contents change from step to step, so the
calls can be captured into a graph once.  The command runs a step of the
sizes below and prints the time of each part.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass

import numpy as np

from . import binding as B


@dataclass
class Sizes:
    """A 4096-wide layer of 32 query heads over 8 key/value heads of 128, 16 adapters of rank 16."""
    hidden: int = 4096
    heads: int = 32
    kv_heads: int = 8
    head_dim: int = 128
    vocab: int = 32000
    page_tokens: int = 16
    slots: int = 16
    rank: int = 16
    top: int = 5
    base8: bool = False   # base weights as 8-bit codes
    theta: float = 0.0    # of the position rotation; 0: none
    sample: bool = False  # next tokens


class VerifyStep:
    uniform = None  # the numbers that next tokens are drawn with: an array where Sizes asks for them

    def __init__(self, sizes: Sizes, n_seqs: int, draft: int, max_tokens: int, seed: int = 0, device="cuda"):
        import torch
        self.s, self.n_seqs, self.draft = sizes, n_seqs, draft
        self.n = n_seqs * draft
        s, rng = sizes, np.random.default_rng(seed)
        self.q_dim, self.kv_dim = s.heads * s.head_dim, s.kv_heads * s.head_dim
        self.row = self.q_dim + 2 * self.kv_dim
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

        def zeros(*shape, dtype=torch.bfloat16):
            return torch.zeros(*shape, dtype=dtype, device=device)

        self.w_qkv, self.w_vocab = weights(self.row, s.hidden), weights(s.vocab, self.q_dim)
        self.a, self.b = weights(s.slots, s.rank, s.hidden), weights(s.slots, self.row, s.rank)
        self.scales = np.full(s.slots, 2.0, np.float32)
        self.route = B.DeviceRoute(self.a, self.b, self.scales)
        slot = rng.integers(0, s.slots, n_seqs)
        self.seq_slot = torch.from_numpy(np.repeat(slot, draft).astype(np.int32)).to(device)
        # every sequence owns its pages; a pool hands them out in any order
        per = -(-max_tokens // s.page_tokens)
        self.cache = B.KVCache.empty(n_seqs * per, s.kv_heads, s.head_dim, s.page_tokens, device)
        table = rng.permutation(n_seqs * per).reshape(n_seqs, per).astype(np.int32)
        self.seqs = B.KVSeqs(torch.from_numpy(table).to(device),
                             torch.arange(0, self.n + 1, draft, dtype=torch.int32, device=device),
                             zeros(n_seqs, dtype=torch.int32), max_rows=draft)
        self.qkv, self.out = zeros(self.n, self.row), zeros(self.n, self.q_dim)
        self.lse = zeros(self.n, s.heads, dtype=torch.float32)
        self.logits = zeros(self.n, s.vocab)
        self.ids = zeros(self.n, dtype=torch.int32)
        self.scores = {"logp": zeros(self.n, dtype=torch.float32), "entropy": zeros(self.n, dtype=torch.float32),
                       "rank": zeros(self.n, dtype=torch.int32), "top_ids": zeros(self.n, s.top, dtype=torch.int32),
                       "top_logp": zeros(self.n, s.top, dtype=torch.float32)}
        need = [B.lora_workspace_bytes(B.LORA_OP_APPLY, B.LORA_BF16, self.n, self.row, s.hidden, s.rank),
                B.lora_kv_attend_workspace_bytes(self.cache, self.seqs, B.LORA_BF16, s.heads, self.n),
                B.lora_workspace_bytes(B.LORA_OP_APPLY, B.LORA_BF16, self.n, s.vocab, self.q_dim, 0),
                B.lora_token_logprobs_workspace_bytes(B.LORA_BF16, s.vocab, self.n, s.top)]
        if s.base8:
            need[0] = B.lora_matmul_fp8_workspace_bytes(B.LORA_BF16, self.row, s.hidden, self.n)
            need[2] = B.lora_matmul_fp8_workspace_bytes(B.LORA_BF16, s.vocab, self.q_dim, self.n)
            self.w_qkv8, self.w_vocab8 = (self._codes(w, 128) for w in (self.w_qkv, self.w_vocab))
            self.w_qkv = self.w_vocab = None  # the codes take their place
            self.x8, self.out8 = (self._room(self.n, k, 1, device) for k in (s.hidden, self.q_dim))
            self.t = zeros(self.n, s.rank, dtype=torch.float32)
        if s.theta:
            i = torch.arange(0, s.head_dim, 2, dtype=torch.float64, device=device)
            self.rotary = B.Rotary((s.theta ** (-i / s.head_dim)).float())
        if s.sample:
            need.append(B.lora_token_sample_workspace_bytes(B.LORA_BF16, s.vocab, self.n))
            self.temperature, self.top_p = (torch.ones(self.n, device=device) for _ in range(2))
            self.min_p, self.uniform = (zeros(self.n, dtype=torch.float32) for _ in range(2))
            self.top_k = zeros(self.n, dtype=torch.int32)
            self.scores |= {"token": zeros(self.n, dtype=torch.int32), "token_logp": zeros(self.n, dtype=torch.float32)}
        self.ws = [(zeros(max(b, 256), dtype=torch.uint8), b) for b in need]
        if self.out.is_cuda:  # all of the above is there whatever stream the first step runs on
            torch.cuda.current_stream(self.out.device).synchronize()

    @staticmethod
    def _room(n, k, block, device):
        """Codes and scales of n rows of k columns, not filled."""
        import torch
        return (torch.zeros(n, k, dtype=torch.uint8, device=device),
                torch.zeros(-(-n // block), -(-k // 128), device=device))

    @classmethod
    def _codes(cls, w, block):
        import torch
        codes, scale = cls._room(*w.shape, block, w.device)
        with torch.cuda.device(w.device) if w.is_cuda else contextlib.nullcontext():
            cls._quantize(w, w.shape[1], block, (codes, scale), w.shape[0])
        return codes, scale

    @staticmethod
    def _quantize(x, k, block, to, n, stream=None):
        B.lora_quantize_fp8(B.LORA_BF16, n, k, x, k, block, to[0], k, to[1], to[1].shape[1], stream)

    def _product(self, w, x, y, ws, stream):
        n_out, k = w[0].shape
        B.lora_matmul_fp8(B.LORA_BF16, n_out, k, w[0], k, w[1], w[1].shape[1], x[0], k, x[1], x[1].shape[1], self.n, y, n_out, *ws, stream)

    def parts(self, x, stream=None):
        """The step's calls on hidden rows x, in order."""
        calls = self._base_parts(x, stream)
        s, code, c = self.s, B.LORA_BF16, self.scores
        k, v = self.qkv[:, self.q_dim:], self.qkv[:, self.q_dim + self.kv_dim:]
        if s.base8:
            def qkv():
                self._quantize(x, s.hidden, 1, self.x8, self.n, stream)
                self._product(self.w_qkv8, self.x8, self.qkv, self.ws[0], stream)
                B.lora_shrink(self.route, x, s.hidden, self.seq_slot, self.n, self.t, stream)
                B.lora_expand_fold(self.route, self.t, self.seq_slot, self.n, self.qkv, self.row, stream)

            def vocabulary():
                self._quantize(self.out, self.q_dim, 1, self.out8, self.n, stream)
                self._product(self.w_vocab8, self.out8, self.logits, self.ws[2], stream)
            calls |= {"qkv": qkv, "vocabulary": vocabulary}
        if s.theta:
            calls["write"] = lambda: B.lora_kv_write_rotary(self.cache, self.seqs, self.rotary, code, s.heads, self.qkv, self.row, self.qkv,
                                                            self.row, k, self.row, v, self.row, self.n, stream)
        if s.sample:
            calls["sample"] = lambda: B.lora_token_sample(code, s.vocab, self.logits, s.vocab, self.temperature, self.top_k, self.top_p,
                                                          self.min_p, self.uniform, self.n, c["token"], c["token_logp"], *self.ws[4], stream)
        return calls

    def _base_parts(self, x, stream):
        s, code = self.s, B.LORA_BF16
        k, v = self.qkv[:, self.q_dim:], self.qkv[:, self.q_dim + self.kv_dim:]
        c = self.scores
        return {
            "qkv": lambda: B.lora_apply(code, self.row, s.hidden, self.w_qkv, s.hidden, self.route, x, s.hidden, self.seq_slot,
                                        self.n, self.qkv, self.row, *self.ws[0], stream),
            "write": lambda: B.lora_kv_write(self.cache, self.seqs, code, k, self.row, v, self.row, self.n, stream),
            "attend": lambda: B.lora_kv_attend(self.cache, self.seqs, code, s.heads, self.qkv, self.row, s.head_dim ** -0.5, 0,
                                               self.n, self.out, self.q_dim, self.lse, *self.ws[1], stream),
            "vocabulary": lambda: B.lora_apply(code, s.vocab, self.q_dim, self.w_vocab, self.q_dim, None, self.out, self.q_dim,
                                               None, self.n, self.logits, s.vocab, *self.ws[2], stream),
            "scores": lambda: B.lora_token_logprobs(code, s.vocab, self.logits, s.vocab, self.ids, self.n, s.top, c["logp"],
                                                    c["entropy"], c["rank"], c["top_ids"], c["top_logp"], *self.ws[3], stream),
        }

    def run(self, x, lengths, ids, stream=None, uniform=None):
        """Scores of the draft tokens `ids` [n]; `lengths` are the sequences' tokens, these drafts included.
        `uniform` [n]: the numbers in [0, 1) that next tokens are drawn with, given with
        Sizes' sample and only with it; new ones for every step.

        The step's inputs are copied on the stream that its kernels run on (a
        torch stream or a raw handle; None: the current one), so that they wait
        for the step before.  x has to be ready on it, and the scores are.
        """
        import torch
        if uniform is None and self.uniform is not None:
            raise ValueError("a step that draws next tokens needs uniform, a number for each row")
        if uniform is not None and self.uniform is None:
            raise ValueError("uniform was given to a step that draws no tokens: Sizes(sample=True) does")
        if stream is None:
            stream = torch.cuda.current_stream()
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            self.seqs.kv_len.copy_(torch.as_tensor(np.asarray(lengths, np.int32)))
            self.ids.copy_(torch.as_tensor(np.asarray(ids, np.int32)))
            if uniform is not None:
                self.uniform.copy_(torch.as_tensor(np.asarray(uniform, np.float32)))
            for call in self.parts(x, stream).values():
                call()
        return self.scores


def main():
    import time

    import torch
    for sizes in (Sizes(), Sizes(base8=True, theta=10000.0, sample=True)):
        step = VerifyStep(sizes, n_seqs=4, draft=9, max_tokens=6144)
        x = torch.randn(step.n, step.s.hidden, device="cuda").bfloat16()
        # a prompt's worth of cached tokens: random codes with a scale of 2^-7
        step.cache.k.random_(0, 126)
        step.cache.v.random_(0, 126)
        step.cache.k_scale.fill_(120)
        step.cache.v_scale.fill_(120)
        uniform = np.random.default_rng(1).random(step.n) if sizes.sample else None
        got = step.run(x, [6009] * 4, np.arange(step.n), uniform=uniform)
        if sizes.sample:
            print("8-bit base weights, rotation, next tokens")
            print("tokens drawn behind the first sequence's drafts:", got["token"][:9].tolist())
        print("log probabilities of the first sequence's drafts:", [round(p, 3) for p in got["logp"][:9].tolist()])
        for name, call in step.parts(x).items():
            torch.cuda.synchronize()
            t = time.perf_counter()
            for _ in range(200):
                call()
            torch.cuda.synchronize()
            print(f"{name:12s} {(time.perf_counter() - t) / 200 * 1e6:8.1f} us")


if __name__ == "__main__":
    main()
