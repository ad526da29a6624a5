"""spec_paged_attention against a plain 64-bit restatement (needs a GB300).

The tolerance of an output element is derived in test_gpu_attention.py (check_row): the rounding of
the weights to the product's 16-bit type, of the scores and sums in fp32, of fp16 weights on their
grid, and of the output.  The product's type is the cache's; over e4m3 codes bf16 for bf16 queries of
more than 32 rows per KV head (scaled codes are bf16 numbers exactly), else fp16 (as there)."""
import numpy as np
import pytest

from tests.test_gpu_attention import check_row, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def visible(n, c, window, sinks, parent):
    """[c, n + c] bool: which tokens each query sees; and the queries' positions."""
    pos = np.arange(n, n + c)
    up = np.tril(np.ones((c, c), bool))
    if parent is not None:
        up = np.zeros((c, c), bool)
        for i in range(c):
            up[i, i] = True
            if i:
                up[i] |= up[parent[i]]
                pos[i] = pos[parent[i]] + 1
    where = np.concatenate((np.arange(n), pos))
    see = np.concatenate((np.ones((c, n), bool), up), 1)
    if window:
        see &= (where[None, :] < sinks) | (pos[:, None] - where[None, :] < window)
    return see


class Problem:
    """Inputs in a pool of pages in random order; NaN in every slot that no token was written to, pages
    that no query of a row sees taken away."""

    def __init__(self, sv, B, N, Hq, H, D, lens, page=16, window=0, sinks=0, kind="bfloat16", qt="bfloat16", tree=False,
                 count=None, seed=0, qsize=2.0, vsize=1.0, spare=2, layout="dense"):
        import torch
        self.sv, self.kind, self.bf16 = sv, kind, torch.bfloat16
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        qd = getattr(torch, qt)
        self.out_u = 2.0**-8 if qt == "bfloat16" else 2.0**-11
        self.B, self.N, self.Hq, self.H, self.D, self.page = B, N, Hq, H, D, page
        self.window, self.sinks = window, sinks
        self.lens = np.asarray(lens, np.int64)
        self.count = None if count is None else np.asarray(count, np.int32)
        self.c = np.full(B, N) if count is None else self.count
        self.parent = np.stack([random_tree(rng, N, 4) for _ in range(B)]) if tree else None
        q = (qsize * torch.randn(B, N, Hq, D, generator=g)).to(qd)
        self.qx = q.double().numpy()
        if layout == "dense":
            self.q = q.cuda()
        else:  # a slice of a wider projection, at an odd offset
            wide = torch.zeros(B, N, Hq, D + 3, dtype=qd)
            wide[..., 1:D + 1] = q
            self.q = wide.cuda()[..., 1:D + 1]
        columns = int(-(-(self.lens.max() + N) // page)) + spare
        pages = B * columns + 3
        self.table = rng.permutation(pages)[: B * columns].reshape(B, columns).astype(np.int32)
        shape = (2, pages, page, sv.spec_kv_entry_bytes(H, D)) if kind == "uint8" else (2, pages, page, H, D)
        ct = getattr(torch, kind)
        if layout == "dense":
            self.cache = torch.empty(shape, dtype=ct, device="cuda")
        else:  # pages inside a larger pool, tokens apart
            self.cache = torch.empty(2, pages, 2 * page + 1, *shape[3:], dtype=ct, device="cuda")[:, :, 1:2 * page + 1:2]
        self.cache.fill_(255 if kind == "uint8" else float("nan"))
        T = int((self.lens + self.c).max())
        k, v = (torch.randn(B, T, H, D, generator=g) for _ in range(2))
        v = v * vsize * (torch.exp2(torch.randint(-3, 4, (B, T, H, 1), generator=g).float()) if kind == "uint8" else 1.0)
        # every row through a contiguous cache, to have the entries' numbers
        line = torch.zeros((2, B, T) + shape[3:], dtype=ct, device="cuda")
        total = i32(self.lens + self.c)
        sv.spec_kv_append(line, k.cuda(), v.cuda(), i32(np.zeros(B)), count=total)
        kx, vx, _ = sv.spec_kv_read(line, total, T, heads=H, head_dim=D, dtype=torch.float32)
        self.kx, self.vx = kx.cpu().double().numpy(), vx.cpu().double().numpy()
        self.see = [visible(int(n), int(c), window, sinks, None if self.parent is None else self.parent[b])
                    for b, (n, c) in enumerate(zip(self.lens, self.c))]
        for b in range(B):
            n = int(self.lens[b] + self.c[b])
            for t0 in range(0, n, page):
                m = min(page, n - t0)
                self.cache[:, self.table[b, t0 // page], :m] = line[:, b, t0:t0 + m]
            # a page none of whose tokens is seen need not be there
            for j in range(columns):
                seen = self.see[b][:, j * page:(j + 1) * page] if self.see[b].size else np.zeros((0, 0))
                if not seen.any():
                    self.table[b, j] = [-1, pages, 2**31 - 1][(b + j) % 3]
        self.dt = i32(self.table)

    def run(self, **kw):
        return self.sv.spec_paged_attention(self.q, self.cache, self.dt, i32(self.lens), parent=None if self.parent is None else i32(self.parent),
                                            count=None if self.count is None else i32(self.count), window=self.window,
                                            sinks=self.sinks, kv_heads=self.H, **kw)

    def check(self, scale=None, rows=None, **kw):
        out, lse, status = self.run(scale=scale, **kw)
        assert status.tolist() == [0] * self.B
        o, z = out.cpu().double().numpy(), lse.cpu().double().numpy()
        scale = self.D ** -0.5 if scale is None else scale
        kind = "bfloat16" if self.kind == "uint8" and self.q.dtype == self.bf16 and self.N * self.Hq // self.H > 32 else self.kind
        for b in range(self.B) if rows is None else rows:
            c, n = int(self.c[b]), int(self.lens[b])
            assert not o[b, c:].any() and np.isneginf(z[b, c:]).all()
            if c:
                check_row(o[b, :c], z[b, :c], self.qx[b, :c], self.kx[b, :n + c], self.vx[b, :n + c], self.see[b], scale,
                          kind, self.out_u)
        return out, lse, status


KINDS = [("bfloat16", "bfloat16"), ("float16", "float16"), ("uint8", "bfloat16"), ("uint8", "float16")]


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("B,N,Hq,H,D,lens,page,window,sinks", [
    (1, 1, 1, 1, 64, [0], 16, 0, 0), (1, 1, 8, 2, 128, [700], 16, 0, 0), (3, 1, 4, 4, 80, [5, 100, 33], 16, 50, 4),
    (2, 1, 32, 4, 128, [1000, 2100], 16, 300, 4), (2, 6, 8, 2, 128, [300, 77], 32, 64, 1), (3, 5, 28, 4, 64, [0, 1, 200], 48, 7, 0),
    (1, 9, 8, 1, 96, [513], 128, 200, 70), (2, 3, 6, 3, 16, [40, 500], 1024, 1, 0), (4, 2, 16, 2, 112, [15, 16, 17, 31], 16, 16, 16),
    (1, 1, 8, 8, 128, [3000], 64, 1000, 999), (2, 4, 8, 2, 128, [0, 3], 16, 2, 100), (2, 1, 40, 20, 64, [300, 90], 16, 100, 4),
    (2, 3, 33, 11, 48, [200, 31], 32, 0, 0), (1, 8, 36, 9, 128, [260], 16, 0, 0), (150, 1, 4, 2, 64, list(range(0, 450, 3)), 16, 60, 4)])
def test_chains(sv, kind, qt, B, N, Hq, H, D, lens, page, window, sinks):
    Problem(sv, B, N, Hq, H, D, lens, page, window, sinks, kind, qt).check()


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("N,Hq,H,D,lens,page,window,sinks", [
    (40, 4, 4, 64, [0, 25], 16, 0, 0), (130, 8, 2, 128, [0, 300], 16, 100, 4), (300, 4, 1, 128, [0, 17], 32, 64, 20),
    (257, 7, 1, 80, [3, 90], 64, 1, 0), (600, 4, 2, 64, [0, 1000], 16, 333, 1), (513, 2, 2, 128, [0, 40], 128, 5000, 4)])
def test_prompts(sv, kind, qt, N, Hq, H, D, lens, page, window, sinks):
    """Many queries per row, over several blocks of them."""
    Problem(sv, 2, N, Hq, H, D, lens, page, window, sinks, kind, qt).check()


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "uint8"])
@pytest.mark.parametrize("B,N,Hq,H,D,window,sinks", [(48, 130, 8, 4, 64, 0, 0), (80, 40, 32, 8, 128, 200, 4), (60, 65, 8, 4, 80, 30, 20)])
def test_uneven_items(sv, B, N, Hq, H, D, window, sinks, kind):
    """Items of one row tile and of two take turns on an SM, with one block of keys and with several."""
    p = Problem(sv, B, N, Hq, H, D, [(97 * b * b) % (20 if b % 3 else 700) for b in range(B)], 16, window, sinks, kind,
                "float16" if kind == "float16" else "bfloat16")
    out, lse, _ = p.check(rows=range(0, B, 7))
    for _ in range(5):
        again = p.run()
        assert (again[0] == out).all() and (again[1] == lse).all()
    # a row by itself, whose keys may be cut in another way
    for b in range(3, B, 11):
        q = Problem.__new__(Problem)
        q.__dict__.update(p.__dict__)
        q.B, q.q, q.dt, q.lens, q.c = 1, p.q[b:b + 1], p.dt[b:b + 1], p.lens[b:b + 1], p.c[b:b + 1]
        o, z, _ = q.run()
        n = int(p.lens[b]) + N
        check_row(o[0].cpu().double().numpy(), z[0].cpu().double().numpy(), p.qx[b], p.kx[b, :n], p.vx[b, :n], p.see[b], D**-0.5,
                  "bfloat16" if kind == "uint8" else kind, p.out_u)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
def test_many_items(sv, kind, tree):
    """More items than SMs: blocks of two row tiles, of one and of none follow one another, with few keys and
    with many; what is not finite in one row is not another's."""
    import torch
    B = 44
    p = Problem(sv, B, 130, 8, 4, 64, [(53 * b) % 400 for b in range(B)], 16, 90, 4, kind, tree=tree,
                count=[0 if b % 11 == 3 else 1 + (37 * b) % 130 for b in range(B)])
    clean = p.check()
    b, t = next((b, t) for b in range(5, B) for t in range(p.lens[b]) if p.c[b] > 60 and p.see[b][0, t] and not p.see[b][:, t].all())
    g = p.table[b, t // 16]
    if kind == "uint8":
        p.cache[1, g, t % 16, 64 + 5] = 0x7f  # head 1: one code
    else:
        p.cache[1, g, t % 16, 1, 5] = float("inf")
    out, lse, status = p.run()
    assert not status.any() and torch.equal(lse, clean[1])
    want = clean[0].clone()
    sees = torch.from_numpy(p.see[b][:, t].copy()).cuda().nonzero()[:, 0]
    for h in (2, 3):
        want[b, sees, h, 5] = float("nan") if kind == "uint8" else float("inf")
    assert torch.equal(out.nan_to_num(nan=7e4), want.nan_to_num(nan=7e4))


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("N,Hq,H,D,lens,window,sinks", [
    (10, 16, 4, 64, [0, 40, 333], 0, 0), (60, 8, 2, 128, [500, 0, 64], 100, 4), (33, 4, 4, 128, [20, 31, 700], 3, 0),
    (2, 4, 1, 96, [9, 100, 1], 1, 1), (64, 32, 8, 64, [5, 90, 200], 8, 300), (300, 2, 1, 64, [30, 3, 0], 20, 0)])
def test_trees(sv, kind, qt, N, Hq, H, D, lens, window, sinks):
    Problem(sv, 3, N, Hq, H, D, lens, 16, window, sinks, kind, qt, tree=True).check()


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
def test_counts(sv, tree, kind):
    """Rows with fewer queries, none among them; what lies behind is left out."""
    Problem(sv, 5, 7, 8, 2, 64, [100, 0, 31, 64, 10], 16, 40, 3, kind, count=[7, 0, 1, 3, 0], tree=tree).check()
    Problem(sv, 3, 90, 8, 2, 128, [100, 0, 31], 16, 40, 3, kind, count=[90, 5, 33], tree=tree).check()


@pytest.mark.parametrize("kind", ["bfloat16", "float16", "uint8"])
@pytest.mark.parametrize("N", [2, 100])
def test_layouts(sv, kind, N):
    """Strided queries, tokens and pages."""
    Problem(sv, 2, N, 8, 2, 64, [50, 200], 16, 70, 4, kind, "float16" if kind == "float16" else "bfloat16", layout="wide").check()


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("N,tree", [(1, False), (3, False), (20, True), (150, False)])
def test_large_numbers(sv, kind, qt, N, tree):
    """Scores of many hundreds, large and small values; a negative scale, and a scale of zero."""
    p = Problem(sv, 2, N, 8, 2, 64, [200, 37], 16, 90, 4, kind, qt, qsize=30.0, vsize=100.0, tree=tree)
    p.check()
    p.check(scale=-0.05)
    p.check(scale=0.0)


@pytest.mark.parametrize("N,tree", [(1, False), (6, False), (60, True), (200, False)])
@pytest.mark.parametrize("kind", ["bfloat16", "float16", "uint8"])
def test_numbers_that_nobody_may_see(sv, N, tree, kind):
    """Infinities and NaN in keys and values of tokens behind the window: queries that do not see a token
    are not touched by it, those that do get what the formula gives."""
    import torch
    p = Problem(sv, 2, N, 4, 2, 64, [150, 61], 16, 30, 2, kind, "float16" if kind == "float16" else "bfloat16", tree=tree)
    clean = p.run()
    hit = []
    for b, t in ((0, 100), (0, 119), (0, 126), (1, 3), (1, 35), (1, 50)):
        g = p.table[b, t // 16]
        if not 0 <= g < p.cache.shape[1]:
            continue
        if kind == "uint8":
            p.cache[1, g, t % 16, 2 * 64] = 255  # head 0: no scale
            p.cache[1, g, t % 16, 64 + 5] = 0x7f  # head 1: one code
        else:
            p.cache[1, g, t % 16, 0, 3] = float("nan")
            p.cache[1, g, t % 16, 1, 5] = float("inf")
        hit.append((b, t))
    assert hit
    out, lse, status = p.run()
    assert status.tolist() == [0, 0]
    assert torch.equal(lse, clean[1])
    o, want = out.float().cpu().numpy(), clean[0].float().cpu().numpy().copy()
    for b, t in hit:
        for i in range(N):
            if p.see[b][i, t]:
                for h in range(4):
                    if h // 2 == 0:
                        want[b, i, h, slice(None) if kind == "uint8" else 3] = np.nan
                    elif kind == "uint8":
                        want[b, i, h, 5] = np.nan
                    else:
                        want[b, i, h, 5] = np.inf
    assert np.array_equal(o, want, equal_nan=True)
    # a key that is no number: it is in the scores of those that see it alone
    b, t = hit[0]
    p2 = Problem(sv, 2, N, 4, 2, 64, [150, 61], 16, 30, 2, kind, "float16" if kind == "float16" else "bfloat16", tree=tree)
    if kind == "uint8":
        p2.cache[0, p2.table[b, t // 16], t % 16, 2 * 64] = 255
    else:
        p2.cache[0, p2.table[b, t // 16], t % 16, 0, 7] = float("nan")
    out, lse, _ = p2.run()
    bad = torch.isnan(lse).cpu().numpy()
    want = np.zeros_like(bad)
    want[b, :, :2] = p.see[b][:, t][:, None]
    assert np.array_equal(bad, want)
    assert np.array_equal(torch.isnan(out).any(-1).cpu().numpy(), want)


@pytest.mark.parametrize("N", [2, 90])
@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
def test_bad_rows(sv, N, kind):
    """Flagged rows are zeros and -inf; the rows between them are right."""
    p = Problem(sv, 6, N, 8, 2, 64, [100, 20, 64, 300, 5, 50], 16, 60, 4, kind)
    good = p.run()
    lens, count = p.lens.copy(), np.full(6, N)
    table = p.table.copy()
    lens[1] = -1
    count[2] = N + 1
    table[3, (300 - 20) // 16] = -1  # in the window
    table[4, 0] = 10**6
    p.lens, p.count, p.dt = lens, count, i32(table)
    out, lse, status = p.run()
    assert status.tolist() == [0, 8, 8, 8, 8, 0]
    import torch
    for b in range(6):
        if status[b]:
            assert not out[b].any() and torch.isneginf(lse[b]).all()
        else:
            assert torch.equal(out[b], good[0][b]) and torch.equal(lse[b], good[1][b])


def test_bad_parents(sv):
    import torch
    p = Problem(sv, 4, 30, 8, 2, 64, [100, 20, 64, 30], 16, 60, 4, tree=True)
    good = p.run()
    p.parent[1, 0] = 0
    p.parent[2, 7] = 7
    out, lse, status = p.run()
    assert status.tolist() == [0, 4, 4, 0]
    for b in range(4):
        if status[b]:
            assert not out[b].any() and torch.isneginf(lse[b]).all()
        else:
            assert torch.equal(out[b], good[0][b])


def test_long_row(sv):
    """One long row without a window and with one, in parts; 70000 tokens back in the cache."""
    Problem(sv, 1, 1, 8, 2, 64, [70000], 64, 0, 0, "uint8").check()
    Problem(sv, 1, 3, 4, 1, 128, [40000], 16, 30000, 8).check()


def test_offsets_past_32_bits(sv):
    """Pages and planes of a pool of over 4 GB."""
    import torch
    H, D, page, N = 8, 128, 16, 2
    entry = H * D
    pages = (5 << 30) // (page * entry * 2)
    cache = torch.empty(2, pages, page, H, D, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    n = 60
    table = np.concatenate((rng.choice(np.arange(pages - 50, pages), 4, replace=False), [pages // 2]))[None].astype(np.int32)
    k, v = torch.randn(2, n + N, H, D, device="cuda").bfloat16()
    for t in range(n + N):
        cache[0, table[0, t // page], t % page] = k[t]
        cache[1, table[0, t // page], t % page] = v[t]
    q = torch.randn(1, N, H, D, device="cuda").bfloat16()
    out, lse, status = sv.spec_paged_attention(q, cache, i32(table), i32([n]))
    assert status.tolist() == [0]
    check_row(out[0].cpu().double().numpy(), lse[0].cpu().double().numpy(), q[0].cpu().double().numpy(), k.cpu().double().numpy(),
              v.cpu().double().numpy(), visible(n, N, 0, 0, None), D ** -0.5, "bfloat16", 2.0**-8)


def test_one_page_table_as_rows(sv):
    """Without a window, over pages in order, the answers are those of spec_prefix_attention."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    B, N, Hq, H, D, S = 3, 5, 8, 2, 64, 96
    cache = torch.randn(2, B, S, H, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(B, N, Hq, D, generator=g, device="cuda").bfloat16()
    n = i32([80, 3, 40])
    a, za, _ = sv.spec_prefix_attention(q, cache, n)
    table = torch.arange(B * S // 16, dtype=torch.int32, device="cuda").view(B, -1)
    b, zb, _ = sv.spec_paged_attention(q, cache.view(2, B * S // 16, 16, H, D), table, n)
    assert torch.allclose(a.float(), b.float(), rtol=2**-6, atol=2**-8) and torch.allclose(za, zb, atol=1e-5)


def test_repeats_and_captures(sv):
    """The same bits every time, from a graph as well, while other sizes run on the same stream."""
    import torch
    p = Problem(sv, 4, 6, 16, 4, 64, [500, 20, 64, 300], 16, 100, 4, "uint8")
    other = Problem(sv, 8, 1, 16, 4, 64, [500, 20, 64, 300] * 2, 16, 0, 0, "uint8", seed=3)
    want = p.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lens = i32(p.lens)
    with torch.cuda.stream(s):
        call = lambda: sv.spec_paged_attention(p.q, p.cache, p.dt, lens, window=100, sinks=4, kv_heads=4)  # noqa: E731
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = call()
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for x in got:
            x.zero_()
        g.replay()
        o = other.run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(o, other.run()))


@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
@pytest.mark.parametrize("B,N,tree", [(3, 60, True), (40, 40, False), (1, 700, False)])
def test_waits_that_run_out(sv, kind, B, N, tree):
    """A bounded wait that nothing ends: what the part belonged to is empty and its row flagged, everything else
    is as ever, and so is the next call."""
    import torch
    p = Problem(sv, B, N, 8, 2, 64, [(37 * b) % 300 for b in range(B)], 16, 100, 4, kind, tree=tree, count=[N - b % 3 for b in range(B)])
    good = p.run()
    limit = sv.get_wait_timeout_ns()
    try:
        sv.set_wait_timeout_ns(2_000_000)
        for force in (1, 2, 3):
            sv.debug_force_wait_timeout(force)
            out, lse, status = p.run()
            torch.cuda.synchronize()
            assert set(status.tolist()) <= {0, 6} and 6 in status.tolist()
            empty = torch.isneginf(lse)
            assert not out[empty].any()
            assert torch.equal(out[~empty], good[0][~empty]) and torch.equal(lse[~empty], good[1][~empty])
            lost = (empty & ~torch.isneginf(good[1])).flatten(1).any(1)
            assert torch.equal(lost, status == 6)
            heads = [0, 1] if force == 1 else [force - 2]
            for g in heads:
                assert bool(empty[:, :, 4 * g:4 * g + 4].all())
    finally:
        sv.debug_force_wait_timeout(False)
        sv.set_wait_timeout_ns(limit)
    again = p.run()
    assert all(torch.equal(a, b) for a, b in zip(again, good))
