"""One layer's speculative-verify step through the library, as a serving loop runs it.

    python -m adapter_lora_bgmv_amd.verify_step

``VerifyStep.run`` takes the hidden rows of every sequence's draft tokens and
    projects them to [Q|K|V] rows, each row with its sequence's adapter (lora_apply),
    writes their keys and values into the 8-bit paged cache (lora_kv_write),
    attends over the cache (lora_kv_attend),
    projects to the vocabulary, base weights only (lora_apply), and
    scores the draft tokens (lora_token_logprobs).
A model's position encoding, which the step leaves out, would turn queries and
keys between the projection and the write.
Everything stays on the device and on one stream; pages, lengths, adapters and
token ids are device arrays whose contents change from step to step, so the
calls can be captured into a graph once.  The command runs a step of the
sizes below and prints the time of each part.
"""
from __future__ import annotations

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


class VerifyStep:
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
        self.ws = [(zeros(max(b, 256), dtype=torch.uint8), b) for b in need]
        if self.out.is_cuda:  # all of the above is there whatever stream the first step runs on
            torch.cuda.current_stream().synchronize()

    def parts(self, x, stream=None):
        """The step's calls on hidden rows x, in order."""
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

    def run(self, x, lengths, ids, stream=None):
        """Scores of the draft tokens `ids` [n]; `lengths` are the sequences' tokens, these drafts included.

        The step's inputs are copied on the stream that its kernels run on (a
        torch stream or a raw handle; None: the current one), so that they wait
        for the step before.  x has to be ready on it, and the scores are.
        """
        import torch
        if stream is None:
            stream = torch.cuda.current_stream()
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            self.seqs.kv_len.copy_(torch.as_tensor(np.asarray(lengths, np.int32)))
            self.ids.copy_(torch.as_tensor(np.asarray(ids, np.int32)))
            for call in self.parts(x, stream).values():
                call()
        return self.scores


def main():
    import time

    import torch
    step = VerifyStep(Sizes(), n_seqs=4, draft=9, max_tokens=6144)
    x = torch.randn(step.n, step.s.hidden, device="cuda").bfloat16()
    # a prompt's worth of cached tokens: random codes with a scale of 2^-7
    step.cache.k.random_(0, 126)
    step.cache.v.random_(0, 126)
    step.cache.k_scale.fill_(120)
    step.cache.v_scale.fill_(120)
    got = step.run(x, [6009] * 4, np.arange(step.n))
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
