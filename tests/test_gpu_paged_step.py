"""Decoding steps over a paged cache with a sliding window: page plan, append through its slots, tree
attention, verification, compaction, committed lengths and the next drafts' sampling, each step held
against a contiguous cache that goes through the same (needs a GB300)."""
import numpy as np
import pytest

from tests.test_gpu_attention import check_row, random_tree
from tests.test_gpu_paged_attention import visible

pytestmark = pytest.mark.gpu

B, N, HQ, H, D, V = 5, 12, 8, 2, 64, 200
PAGE, COLUMNS, PAGES, WINDOW, SINKS, STEPS = 16, 20, 32, 40, 3, 24


class State:
    """A paged cache and its bookkeeping, and the step's inputs in buffers that stay where they are."""

    def __init__(self, sv, kind):
        import torch
        i32 = dict(dtype=torch.int32, device="cuda")
        self.sv = sv
        self.table = torch.full((B, COLUMNS), -1, **i32)
        self.free = torch.randperm(PAGES, generator=torch.Generator().manual_seed(4)).int().cuda()
        self.ring = torch.tensor([5, PAGES], **i32)
        self.n = torch.zeros(B, **i32)
        ct = getattr(torch, kind)
        self.entry = (sv.spec_kv_entry_bytes(H, D),) if kind == "uint8" else (H, D)
        self.pool = torch.empty(2, PAGES, PAGE, *self.entry, dtype=ct, device="cuda")
        self.pool.fill_(255 if kind == "uint8" else float("nan"))
        self.k, self.v = (torch.zeros(B, N, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.q = torch.zeros(B, N, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.parent, self.tokens = (torch.zeros(B, N, **i32) for _ in range(2))
        self.parent[:, 0] = -1
        self.logits = torch.zeros(B, N, V, device="cuda")
        self.u = torch.zeros(B * N, device="cuda")
        self.min_p = torch.full((B * N,), 0.05, device="cuda")

    def step(self):
        sv = self.sv
        slots, planned = sv.spec_page_plan(self.table, self.free, self.ring, self.n, N, PAGE, window=WINDOW, sinks=SINKS)
        flat = self.pool.view(2, 1, PAGES * PAGE, *self.entry).expand(2, B * N, PAGES * PAGE, *self.entry)
        sv.spec_kv_append(flat, self.k.view(B * N, 1, H, D), self.v.view(B * N, 1, H, D), slots.view(-1))
        out, lse, seen = sv.spec_paged_attention(self.q, self.pool, self.table, self.n, parent=self.parent, window=WINDOW,
                                                 sinks=SINKS, kv_heads=H)
        r = sv.spec_verify_tree(self.logits, self.parent, self.tokens)
        moved = sv.spec_kv_compact_pages(self.pool, self.table, self.n, r["accepted_len"], r["path_nodes"])
        after, _ = sv.spec_rollback_lengths(self.n, r["accepted_len"], r["num_emitted"], r["out_tokens"])
        drafts = sv.spec_sample(self.logits.view(B * N, V), self.u, min_p=self.min_p)
        return dict(out=out, lse=lse, accepted=r["accepted_len"], path=r["path_nodes"], after=after, drafts=drafts["token"],
                    status=(planned, seen, r["row_status"], moved, drafts["row_status"]))


@pytest.mark.parametrize("how", ["eager", "stream", "captured"])
@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
def test_steps(kind, how):
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    g = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    s = State(sv, kind)
    line = torch.zeros(2, B, COLUMNS * PAGE, *s.entry, dtype=s.pool.dtype, device="cuda")
    side = torch.cuda.Stream()
    graph = None
    if how == "captured":
        spare = State(sv, kind)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            spare.step()  # everything is loaded
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                r = s.step()
        torch.cuda.current_stream().wait_stream(side)
    kept = 0
    for step in range(STEPS):
        for x in (s.k, s.v, s.q):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        s.u.copy_(torch.rand(s.u.shape, generator=g, device="cuda"))
        parent = np.stack([random_tree(rng, N, 4) for _ in range(B)])
        tokens = rng.permuted(np.tile(np.arange(V), (B, 1)), axis=1)[:, :N]
        logits = rng.standard_normal((B, N, V)).astype(np.float32)
        for b in range(B):
            for i in range(1, N):  # a node's last child is what the target wants behind it, mostly
                if rng.random() < 0.8:
                    logits[b, parent[b, i], tokens[b, i]] = 10 + i
        s.parent.copy_(torch.from_numpy(parent))
        s.tokens.copy_(torch.from_numpy(tokens))
        s.logits.copy_(torch.from_numpy(logits))
        if how == "captured":
            graph.replay()
        elif how == "stream":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                r = s.step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            r = s.step()
        for status in r["status"]:
            assert not status.any()
        # the same on the contiguous cache
        sv.spec_kv_append(line, s.k, s.v, s.n)
        total = s.n + N
        T = int(total.max())
        kx, vx, _ = sv.spec_kv_read(line, total, T, heads=H, head_dim=D, dtype=torch.float32)
        kx, vx, qx = (x.cpu().double().numpy() for x in (kx, vx, s.q))
        o, z = r["out"].cpu().double().numpy(), r["lse"].cpu().double().numpy()
        rounded = "bfloat16" if N * HQ // H > 32 else kind
        for b in range(B):
            n = int(s.n[b])
            check_row(o[b], z[b], qx[b], kx[b, :n + N], vx[b, :n + N], visible(n, N, WINDOW, SINKS, parent[b]), D**-0.5, rounded,
                      2.0**-8)
        sv.spec_kv_compact_tree(line, s.n, r["accepted"], r["path"])
        assert torch.equal(r["after"], s.n + 1 + r["accepted"])
        kept += int(r["accepted"].sum())
        s.n.copy_(r["after"])
        # the entries that a later step can see, where the table says they are
        table = s.table.cpu().numpy()
        used = table[table >= 0]
        assert len(set(used.tolist())) == len(used) and int(s.ring[1]) == PAGES - len(used)
        for b in range(B):
            n = int(s.n[b])
            for t in range(n):
                if t < SINKS or t > n - WINDOW:
                    p = table[b, t // PAGE]
                    assert p >= 0 and torch.equal(s.pool[:, p, t % PAGE], line[:, b, t])
        x = s.logits.view(B * N, V).double()
        drawn = torch.gather(x, 1, r["drafts"].long()[:, None])[:, 0]
        assert (drawn >= x.amax(1) + np.log(0.05) - 1e-4).all()
    assert kept > STEPS * B // 2 and int(s.n.min()) > WINDOW
