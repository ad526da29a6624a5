"""Speculative decoding steps end to end on the library's calls: a prompt shared by all
sequences, draft trees, an 8-bit KV cache.

    python examples/decode_step.py [--steps 4] [--batch 8] [--prompt 700]

The "model" is one attention layer of random weights between an embedding and a
vocabulary projection (there are no trained weights here), and the draft tree of a step
is drawn at random around the layer's own favourites, so some of it is accepted.  Every
step does what a serving loop does around the model's matrix products:

    spec_kv_append          keys and values of the tree's nodes into the cache
    spec_prefix_attention   the nodes' attention: prompt + own history + ancestors
    spec_verify_tree        which root path of the tree the target keeps
    spec_token_logprobs     log probabilities, entropy and alternatives of what is emitted
    spec_kv_compact_tree    the kept path's entries move up behind the history
    spec_rollback_lengths   the committed length

With check=True, main() recomputes each step's attention for the kept path from the cache
as spec_kv_read gives it back, and compares.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_32_gb300 as sv  # noqa: E402

HEADS, KV_HEADS, DIM, VOCAB, NODES = 16, 4, 64, 2000, 10


class Layer:
    def __init__(self, g):
        def w(*s):
            return (torch.randn(*s, generator=g, device="cuda") / s[0] ** 0.5).bfloat16()
        width = HEADS * DIM
        self.embed = torch.randn(VOCAB, width, generator=g, device="cuda").bfloat16()
        self.wq, self.wk, self.wv = w(width, width), w(width, KV_HEADS * DIM), w(width, KV_HEADS * DIM)
        self.out = w(width, VOCAB)

    def qkv(self, tokens):
        x = self.embed[tokens.long()]
        return (x @ self.wq).unflatten(-1, (HEADS, DIM)), (x @ self.wk).unflatten(-1, (KV_HEADS, DIM)), \
            (x @ self.wv).unflatten(-1, (KV_HEADS, DIM))

    def logits(self, tokens, attended):
        return (self.embed[tokens.long()] + attended.flatten(-2)) @ self.out


def draft_tree(g, layer, last):
    """A random tree of NODES nodes per row (node 0: the last token), whose tokens are often what the
    layer would say without attention."""
    B = last.shape[0]
    parent = torch.full((B, NODES), -1, dtype=torch.int32, device="cuda")
    tokens = torch.empty(B, NODES, dtype=torch.int32, device="cuda")
    tokens[:, 0] = last
    for i in range(1, NODES):
        p = torch.randint(max(0, i - 3), i, (B,), generator=g, device="cuda")
        parent[:, i] = p.int()
        before = tokens.gather(1, p[:, None].long())[:, 0]
        guess = (layer.embed[before.long()] @ layer.out).argmax(-1)
        luck = torch.randint(0, VOCAB, (B,), generator=g, device="cuda")
        tokens[:, i] = torch.where(torch.rand(B, generator=g, device="cuda") < 0.8, guess, luck).int()
    return parent, tokens


def main(steps=4, batch=8, prompt=700, seed=0, check=False, out=print):
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(g)
    entry = sv.spec_kv_entry_bytes(KV_HEADS, DIM)
    prefix = torch.zeros(2, 1, prompt, entry, dtype=torch.uint8, device="cuda")
    cache = torch.zeros(2, batch, steps * NODES + NODES, entry, dtype=torch.uint8, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, k, v = layer.qkv(torch.randint(0, VOCAB, (1, prompt), generator=g, device="cuda"))
    sv.spec_kv_append(prefix, k, v, zero)
    kv_len = torch.zeros(batch, dtype=torch.int32, device="cuda")
    last = torch.randint(0, VOCAB, (batch,), generator=g, device="cuda", dtype=torch.int32)
    emitted_total = 0
    for step in range(steps):
        parent, tokens = draft_tree(g, layer, last)
        q, k, v = layer.qkv(tokens)
        status = sv.spec_kv_append(cache, k, v, kv_len)
        attended, lse, st = sv.spec_prefix_attention(q, cache, kv_len, prefix=prefix, parent=parent, kv_heads=KV_HEADS)
        logits = layer.logits(tokens, attended).contiguous()
        kept = sv.spec_verify_tree(logits, parent, tokens, margin_kappa=0.3)
        # the target rows that said the emitted tokens: the root's and the kept nodes'
        path = kept["path_nodes"]
        rows = torch.cat((torch.zeros(batch, 1, dtype=torch.int64, device="cuda"), path[:, :-1].clamp_min(0).long()), 1)
        said = torch.gather(logits, 1, rows[..., None].expand(-1, -1, VOCAB))
        lp = sv.spec_token_logprobs(said, kept["out_tokens"], m=5)
        moved = sv.spec_kv_compact_tree(cache, kv_len, kept["accepted_len"], path)
        new_len, n = sv.spec_rollback_lengths(kv_len, kept["accepted_len"], kept["num_emitted"], kept["out_tokens"])
        if check:
            assert status.tolist() == st.tolist() == moved.tolist() == [0] * batch
            check_step(q, attended, cache, prefix, kv_len, kept)
            given = lp["logprob"][torch.arange(NODES, device="cuda") < kept["num_emitted"][:, None]]
            assert bool((given <= 0).all()) and not bool(torch.isnan(given).any())
        emitted_total += int(n.sum())
        last = kept["out_tokens"].gather(1, (kept["num_emitted"] - 1)[:, None].long())[:, 0]
        kv_len = new_len
        out(f"step {step}: emitted {n.tolist()}, cache lengths {kv_len.tolist()}, "
            f"mean log probability {float(lp['logprob'].nanmean()):.3f}")
    return emitted_total


def check_step(q, attended, cache, prefix, kv_len, kept):
    """The kept path, after compaction, is a chain behind the history: its attention, from the cache as
    it reads back."""
    depth = int(kept["accepted_len"].max())
    k, v, _ = sv.spec_kv_read(cache, kv_len + kept["accepted_len"] + 1, cache.shape[2], heads=KV_HEADS, head_dim=DIM,
                              dtype=torch.float32)
    one = torch.full((1,), prefix.shape[2], dtype=torch.int32, device="cuda")
    pk, pv, _ = sv.spec_kv_read(prefix, one, prefix.shape[2], heads=KV_HEADS, head_dim=DIM, dtype=torch.float32)
    for b in range(q.shape[0]):
        n = int(kv_len[b])
        for d in range(int(kept["accepted_len"][b]) + 1):
            node = 0 if d == 0 else int(kept["path_nodes"][b, d - 1])
            kk = torch.cat((pk[0], k[b, :n + d + 1])).repeat_interleave(HEADS // KV_HEADS, 1)
            vv = torch.cat((pv[0], v[b, :n + d + 1])).repeat_interleave(HEADS // KV_HEADS, 1)
            p = torch.softmax(torch.einsum("hd,thd->ht", q[b, node].float(), kk) / DIM ** 0.5, -1)
            want = torch.einsum("ht,thd->hd", p, vv)
            torch.testing.assert_close(attended[b, node].float(), want, rtol=2e-2, atol=2e-3)
    return depth


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--steps", type=int, default=4)
    a.add_argument("--batch", type=int, default=8)
    a.add_argument("--prompt", type=int, default=700)
    a = a.parse_args()
    main(a.steps, a.batch, a.prompt, check=True)
