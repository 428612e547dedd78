"""Speculative decoding of a small hybrid model: one KDA layer and one softmax-attention layer, random weights.

Every step drafts a few tokens per sequence, runs them through both layers without touching the committed
states (the KDA layer's recurrent states, the attention layer's paged cache), verifies them against the model's own
probabilities, and commits the accepted ones to both: ``kda_replay`` and ``kda_cache_append``.

    python examples/spec_step.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_linear_attention_chunk_gb300 as kda  # noqa: E402


class HybridModel:
    """x -> x + KDA(x) -> x + attention(x) -> logits, for N sequences decoded side by side."""

    def __init__(self, N=4, vocab=512, width=256, kda_heads=2, q_heads=8, kv_heads=2, d=64, page=16, max_ctx=512, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s, scale: (scale * torch.randn(*s, generator=gen, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.N, self.vocab, self.H, self.Hq, self.Hkv, self.d, self.gen = N, vocab, kda_heads, q_heads, kv_heads, d, gen
        self.embed, self.unembed = rand(vocab, width, scale=1.0), rand(width, vocab, scale=3 * width ** -0.5)
        self.w_kda = rand(width, kda_heads * (4 * d + 1), scale=width ** -0.5)     # q | k | v | gate | beta
        self.w_kda_out = rand(kda_heads * d, width, scale=(kda_heads * d) ** -0.5)
        self.w_attn = rand(width, (q_heads + 2 * kv_heads) * d, scale=width ** -0.5)  # q | k | v
        self.w_attn_out = rand(q_heads * d, width, scale=(q_heads * d) ** -0.5)
        self.inv_freq, self.mscale = kda.rope_frequencies(d)
        # committed: recurrent states, pages with their table and lengths, and the next token (not yet committed)
        pages = -(-max_ctx // page)
        self.states = torch.zeros(N, kda_heads, d, d, device="cuda")
        self.k_pages, self.v_pages = (torch.zeros(N * pages, page, kv_heads, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.table = torch.randperm(N * pages, generator=gen, device="cuda").int().view(N, pages)
        self.ctx_len = torch.zeros(N, dtype=torch.int32, device="cuda")
        self.root = torch.randint(0, vocab, (N,), generator=gen, device="cuda", dtype=torch.int32)
        self.flags = kda.KDA_PREP_L2NORM_Q | kda.KDA_PREP_L2NORM_K | kda.KDA_PREP_SIGMOID_GATE | kda.KDA_PREP_SIGMOID_BETA

    def draft(self, count):
        """`count` drafted tokens after each root: (tokens, the draft's distributions), packed by sequence; the draft is
        the model without its layers."""
        tokens, probs = [self.root], []
        for _ in range(count + 1):
            p = torch.softmax((self.embed[tokens[-1].long()] @ self.unembed).float(), -1)
            probs.append(p)
            tokens.append(torch.multinomial(p, 1, generator=self.gen)[:, 0].int())
        return torch.stack(tokens[:-1], 1).flatten(), torch.stack(probs, 1).flatten(0, 1)

    def forward(self, tokens, cu):
        """Target distributions after every drafted token, and what a commit needs of them."""
        T, H, d = tokens.shape[0], self.H, self.d
        x = self.embed[tokens.long()]
        y = x @ self.w_kda
        q, k, v, g = (z.view(T, H, d).contiguous() for z in y[:, :4 * H * d].split(H * d, 1))
        beta = y[:, 4 * H * d:].contiguous()
        o, _ = kda.kda_chunk_fwd_prep(q, k, v, g, beta, self.flags, cu_seqlens=cu, init_state=self.states, scale=d ** -0.5,
                                      output_final_state=False)
        x = x + o.view(T, H * d) @ self.w_kda_out
        fused = (x @ self.w_attn).view(T, self.Hq + 2 * self.Hkv, d)
        qa, ka, va = fused.split((self.Hq, self.Hkv, self.Hkv), 1)  # slices: no copies
        seq = torch.repeat_interleave(torch.arange(self.N, device="cuda"), (cu[1:] - cu[:-1]).long(), output_size=T)
        positions = (self.ctx_len[seq] + torch.arange(T, device="cuda") - cu[seq]).int()
        qa, ka = kda.kda_rope(qa, ka, positions, self.inv_freq, mscale=self.mscale)
        a, _ = kda.kda_tree_attn(qa, ka, va, self.k_pages, self.v_pages, self.table, self.ctx_len, cu, return_lse=False,
                                 max_nodes=min(T // self.N, kda.KDA_MAX_TREE_NODES))
        x = x + a.view(T, -1) @ self.w_attn_out
        return torch.softmax((x @ self.unembed).float(), -1), (k, v, g, beta), (ka, va)

    def step(self, drafts=3):
        """One speculative step.  Returns the number of tokens committed per sequence."""
        tokens, draft_probs = self.draft(drafts)
        T = tokens.shape[0]
        cu = torch.arange(0, T + 1, drafts + 1, dtype=torch.int32, device="cuda")
        target, kda_rows, (ka, va) = self.forward(tokens, cu)
        u = torch.rand(T + self.N, generator=self.gen, device="cuda")
        cu_accept, rows, self.root = kda.kda_draft_verify(tokens, cu, target, u[:T], u[T:], draft_probs=draft_probs)
        counts = (cu_accept[1:] - cu_accept[:-1]).tolist()  # (the step's only wait for the GPU)
        picked = rows[:sum(counts)].long()
        kda.kda_replay_prep(self.states, *(z[picked] for z in kda_rows), cu_accept, self.flags)
        self.ctx_len = kda.kda_cache_append(ka, va, self.k_pages, self.v_pages, self.table, self.ctx_len, cu_accept, rows=rows)
        self.last = dict(tokens=tokens[picked], counts=counts)
        return counts


def main(steps=8):
    model = HybridModel()
    committed = 0
    for i in range(steps):
        counts = model.step()
        committed += sum(counts)
        print(f"step {i}: committed {counts}, context {model.ctx_len.tolist()}")
    print(f"{committed / (steps * model.N):.2f} tokens per sequence and step")


if __name__ == "__main__":
    main(*(int(x) for x in sys.argv[1:]))
