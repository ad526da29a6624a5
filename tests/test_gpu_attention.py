"""spec_prefix_attention against a plain 64-bit restatement (needs a GB300).

Tolerance of an output element, with p the exact softmax weights, A = sum p |v|
and T the keys seen:
  - the weights are rounded to the 16-bit type of the product (u = 2^-8 for
    bf16, 2^-11 for fp16 and e4m3 caches): u A;
  - a score is a sum of D products in fp32 (the tensor cores may truncate):
    its error is at most delta = 2^-23 (D + 8) max_t scale sum_d |q_d k_td| + 2^-20,
    and moves every weight by that, relative, twice (weight and sum): 2 delta A;
  - sums over T keys in fp32: 2^-23 T A;
  - fp16 weights below 2^-14 of the largest (of p 2^e, in an e4m3 cache whose
    values are 2^e c) round on a fixed grid: 2^-25 max_t(p_t 2^e_t) sum_t |c_t|;
  - the output's own rounding: u_out |out| (2^-8 or 2^-11), fp16 also 2^-25.
lse: delta + 2^-23 T + 2^-20 |lse|."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def seen(N, parent):
    """[N, N] bool: which of the pass's own tokens each query sees."""
    a = np.zeros((N, N), bool)
    for i in range(N):
        j = i
        while j >= 0:
            a[i, j] = True
            j = j - 1 if parent is None else int(parent[j])
    return a


def exponents(x):
    """Scale exponents of head vectors [..., D] (float64) as the e4m3 cache picks them."""
    amax = np.abs(x).max(-1)
    f, e = np.frexp(np.where(amax == 0, 1.0, amax) / 448.0)
    return np.clip(np.where(amax == 0, -126, np.where(f == 0.5, e - 1, e)), -126, None)


def check_row(got, lse, q, k, v, vis, scale, kind, out_u):
    """One row: q [N, Hq, D], k, v [T, H, D], vis [N, T], float64 (v: values; kind: cache type)."""
    N, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    u = 2.0**-8 if kind == "bfloat16" else 2.0**-11
    for h in range(Hq):
        g = h // G
        kk, vv = k[:, g], v[:, g]
        any_seen = vis.any(0)
        kk, vv = np.where(any_seen[:, None], kk, 0.0), np.where(any_seen[:, None], vv, 0.0)
        x = scale * (q[:, h] @ kk.T)
        mag = abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T)
        x = np.where(vis, x, -np.inf)
        M = x.max(-1, keepdims=True)
        w = np.exp(x - M)
        tot = w.sum(-1, keepdims=True)
        p = w / tot
        want = p @ vv
        A = p @ np.abs(vv)
        T = vis.sum(-1)[:, None]
        delta = 2.0**-23 * (D + 8) * np.where(vis, mag, 0).max(-1, keepdims=True) + 2.0**-20
        tol = (u + 2 * delta + 2.0**-23 * T) * A + out_u * np.abs(want) + 2.0**-40
        if kind != "bfloat16":
            e = exponents(vv) if kind == "uint8" else np.zeros(vv.shape[0])
            c = np.abs(vv) * np.exp2(-e)[:, None]
            tol += 2.0**-25 * (p * np.exp2(e)).max(-1, keepdims=True) * (np.where(vis, 1.0, 0.0) @ c)
        gh = got[:, h]
        if out_u == 2.0**-11:
            tol += 2.0**-25
            # past fp16's range the output is an infinity (either within tol of the border)
            over = np.isinf(gh) & (np.abs(want) + tol >= 65520.0) & (np.sign(gh) == np.sign(want))
            assert np.all(np.abs(want[~over]) - tol[~over] < 65520.0)
            gh = np.where(over, want, gh)
        err = np.abs(gh - want)
        assert np.all(err <= tol), (h, float((err / tol).max()), float(err.max()))
        wl = (M + np.log(tot))[:, 0]
        tl = delta[:, 0] + 2.0**-23 * T[:, 0] + 2.0**-20 * np.abs(wl)
        assert np.all(np.abs(lse[:, h] - wl) <= tl), (h, np.abs(lse[:, h] - wl).max(), tl.min())


def random_tree(rng, N, wide):
    p = np.full(N, -1, np.int32)
    for i in range(1, N):
        p[i] = rng.integers(max(0, i - wide), i)
    return p


class Problem:
    """Inputs, with NaN in every slot no token was written to."""

    def __init__(self, sv, B, N, Hq, H, D, P, lens, kind="bfloat16", qt="bfloat16", tree=False, count=None, seed=0,
                 qsize=2.0, vsize=1.0, slack=3, layout="dense", extra_prefix=0):
        import torch
        self.sv, self.kind = sv, kind
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        qd = getattr(torch, qt)
        self.out_u = 2.0**-8 if qt == "bfloat16" else 2.0**-11
        self.B, self.N, self.Hq, self.H, self.D, self.P = B, N, Hq, H, D, P
        self.lens = np.asarray(lens, np.int32)
        self.count = None if count is None else np.asarray(count, np.int32)
        self.n = self.count if count is not None else np.full(B, N, np.int32)
        q = (qsize * torch.randn(B, N, Hq, D, generator=g)).to(qd)
        self.qx = q.double().numpy()
        if layout == "dense":
            self.q = q.cuda()
        else:  # a slice of a wider projection, at an odd offset
            wide = torch.zeros(B, N, Hq, D + 3, dtype=qd)
            wide[..., 1:D + 1] = q
            self.q = wide.cuda()[..., 1:D + 1]
        S = int(self.lens.max()) + N + slack
        self.S = S
        shape = (2, B, S, sv.spec_kv_entry_bytes(H, D)) if kind == "uint8" else (2, B, S, H, D)
        ct = getattr(torch, kind)
        if layout == "dense":
            self.cache = torch.empty(shape, dtype=ct, device="cuda")
        else:  # rows and planes inside a larger pool of slots
            self.cache = torch.empty(2, B, 2 * S + 1, *shape[3:], dtype=ct, device="cuda")[:, :, 1:2 * S + 1:2]
        self.cache.fill_(255 if kind == "uint8" else float("nan"))
        k, v = (torch.randn(B, S, H, D, generator=g) for _ in range(2))
        v = v * vsize * (torch.exp2(torch.randint(-3, 4, (B, S, H, 1), generator=g).float()) if kind == "uint8" else 1.0)
        i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
        total = i32(self.lens + self.n)
        assert sv.spec_kv_append(self.cache, k.cuda(), v.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"),
                                 count=total).tolist() == [0] * B
        kx, vx, _ = sv.spec_kv_read(self.cache, total, S, heads=H, head_dim=D, dtype=torch.float32)
        self.kx, self.vx = kx.cpu().double().numpy(), vx.cpu().double().numpy()
        self.prefix = None
        if P:
            PS = P + extra_prefix
            pshape = (2, 1, PS) + shape[3:]
            self.prefix = torch.empty(pshape, dtype=ct, device="cuda")
            self.prefix.fill_(255 if kind == "uint8" else float("nan"))
            pk, pv = (torch.randn(1, P, H, D, generator=g).cuda() for _ in range(2))
            z = torch.zeros(1, dtype=torch.int32, device="cuda")
            sv.spec_kv_append(self.prefix, pk, pv * vsize, z)
            a, b, _ = sv.spec_kv_read(self.prefix, i32([P]), P, heads=H, head_dim=D, dtype=torch.float32)
            self.pk, self.pv = a[0].cpu().double().numpy(), b[0].cpu().double().numpy()
        self.parent = np.stack([random_tree(rng, N, 7) for _ in range(B)]) if tree else None
        self.scale = D ** -0.5

    def call(self, **kw):
        import torch
        i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        return self.sv.spec_prefix_attention(self.q, self.cache, i32(self.lens), prefix=self.prefix, prefix_len=self.P or None,
                                             parent=i32(self.parent), count=i32(self.count), kv_heads=self.H, **kw)

    def check(self, rows=None, status=None):
        out, lse, st = self.call()
        assert st.tolist() == (status or [0] * self.B)
        got, lg = out.cpu().double().numpy(), lse.cpu().double().numpy()
        again, lse2, _ = self.call()
        assert np.array_equal(got, again.cpu().double().numpy(), equal_nan=True)
        assert np.array_equal(lg, lse2.cpu().double().numpy(), equal_nan=True)
        for b in range(self.B) if rows is None else rows:
            n, L = int(self.n[b]), int(self.lens[b])
            assert np.all(got[b, n:] == 0) and np.all(np.isneginf(lg[b, n:]))
            if n == 0:
                continue
            k, v = self.kx[b, :L + n], self.vx[b, :L + n]
            vis = np.concatenate([np.ones((n, L), bool), seen(n, None if self.parent is None else self.parent[b])], 1)
            if self.P:
                k, v = np.concatenate([self.pk, k]), np.concatenate([self.pv, v])
                vis = np.concatenate([np.ones((n, self.P), bool), vis], 1)
            check_row(got[b, :n], lg[b, :n], self.qx[b, :n], k, v, vis, self.scale, self.kind, self.out_u)
        return out, lse


KINDS = [("bfloat16", "bfloat16"), ("float16", "float16"), ("uint8", "bfloat16"), ("uint8", "float16")]


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("B,N,Hq,H,D,P,lens,tree", [
    (1, 1, 1, 1, 128, 0, [0], False),                       # one token that sees itself
    (1, 1, 8, 2, 64, 1, [0], False),
    (2, 1, 32, 8, 128, 100, [15, 40], False),
    (3, 1, 7, 1, 80, 63, [0, 16, 17], False),               # 7 query heads a KV head
    (4, 6, 8, 2, 128, 200, [0, 1, 63, 64], False),
    (2, 5, 12, 3, 96, 0, [65, 127], False),
    (3, 9, 16, 2, 64, 257, [300, 5, 31], False),            # more than 32 query rows a KV head
    (2, 17, 4, 4, 128, 129, [48, 200], True),
    (1, 60, 8, 2, 128, 64, [33], True),
    (2, 70, 4, 1, 64, 31, [10, 3], True),                   # more than 64 nodes
    (5, 2, 2, 1, 16, 1000, [7, 0, 100, 64, 30], False),
    (33, 4, 8, 1, 112, 300, list(range(0, 330, 10)), False),  # many rows behind one prefix
])
def test_against_plain(sv, kind, qt, B, N, Hq, H, D, P, lens, tree):
    Problem(sv, B, N, Hq, H, D, P, lens, kind, qt, tree, seed=B * N + D).check()


@pytest.mark.parametrize("kind,qt", KINDS)
def test_views_of_larger_pools(sv, kind, qt):
    """Strided queries at odd offsets, strided slots, a prefix longer than the part that is used."""
    Problem(sv, 3, 5, 8, 2, 128, 150, [20, 0, 77], kind, qt, seed=5, layout="views", extra_prefix=9).check()
    Problem(sv, 2, 30, 8, 2, 64, 70, [20, 100], kind, qt, tree=True, seed=6, layout="views", extra_prefix=1).check()


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("N,tree", [(4, False), (40, True)])
def test_counts_and_bad_rows(sv, kind, qt, N, tree):
    """Rows with fewer queries or none; rows that cannot be used leave the others right."""
    p = Problem(sv, 6, N, 8, 2, 64, 90, [9, 30, 0, 64, 12, 50], kind, qt, tree, count=[N, 0, 1, N - 1, 2, N], seed=8)
    p.check()
    out0, lse0, _ = p.call()
    lens, count, parent = p.lens.copy(), p.count.copy(), None if p.parent is None else p.parent.copy()
    p.lens[0], p.lens[3], p.count[4] = -1, p.S - 1, N + 1
    want = [8, 0, 0, 8, 8, 0]
    if tree:
        p.parent[5, 3], want[5] = 3, 4
        p.parent[0, 0], want[0] = 0, 4  # two faults: the smaller code
    out, lse, st = p.call()
    assert st.tolist() == want
    for b in range(6):
        if want[b]:
            assert float(out[b].abs().max()) == 0.0 and bool((lse[b] == float("-inf")).all())
        else:
            assert bool((out[b] == out0[b]).all()) and bool((lse[b] == lse0[b]).all())
    p.lens, p.count, p.parent = lens, count, parent


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("N,tree", [(5, False), (50, True)])
def test_what_a_query_does_not_see_may_hold_anything(sv, kind, qt, N, tree):
    """NaN and infinities in a token of the pass reach the queries that see it and no others."""
    import torch
    p = Problem(sv, 2, N, 8, 2, 64, 40, [13, 30], kind, qt, tree, seed=11)
    out0, lse0 = p.check()
    bad = N - 2
    for plane in (0, 1):
        c0 = p.cache.clone()
        for b in range(2):
            at = int(p.lens[b]) + bad
            if kind == "uint8":
                p.cache[plane, b, at, 0:2] = 127 + 128 * b  # codes that stand for NaN in head 0 ...
                p.cache[plane, b, at, 128 + 1] = 255          # ... and a NaN scale in head 1
            else:
                p.cache[plane, b, at] = float("inf") if b else float("nan")
        out, lse, st = p.call()
        assert st.tolist() == [0, 0]
        for b in range(2):
            sees = torch.from_numpy(seen(N, None if p.parent is None else p.parent[b])[:, bad]).cuda()
            assert torch.equal(out[b][~sees], out0[b][~sees]) and torch.equal(lse[b][~sees], lse0[b][~sees])
            hit = (out[b][sees] != out0[b][sees]) | torch.isnan(out[b][sees])
            assert bool(hit.any())
            if kind == "uint8":
                assert bool(torch.isnan(out[b][sees][:, 4:]).all())  # head 1's queries
        p.cache.copy_(c0)


@pytest.mark.parametrize("qt", ["bfloat16", "float16"])
def test_e4m3_scales_far_apart(sv, qt):
    """Zero vectors, tiny and huge values next to each other in one cache, tiny and huge queries."""
    import torch
    p = Problem(sv, 1, 3, 4, 2, 64, 0, [100], "uint8", qt, seed=3)
    S = int(p.lens[0]) + 3
    g = torch.Generator().manual_seed(9)
    k = torch.randn(1, S, 2, 64, generator=g)
    v = torch.randn(1, S, 2, 64, generator=g)
    v[0, 10:20] = 0.0
    v[0, 20:30] *= 1e-30
    v[0, 30:32] *= 1e6
    k[0, 30:32] *= -4.0
    k[0, 40] *= 1e-20
    k[0, 50] = 0.0
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    for scale_v in (1.0, 1e-25, 1e20):
        p.sv.spec_kv_append(p.cache, k.cuda(), (v * scale_v).cuda(), z)
        n = torch.tensor([S], dtype=torch.int32, device="cuda")
        kx, vx, _ = p.sv.spec_kv_read(p.cache, n, p.S, heads=2, head_dim=64, dtype=torch.float32)
        p.kx, p.vx = kx.cpu().double().numpy(), vx.cpu().double().numpy()
        if qt == "bfloat16" or scale_v == 1.0:  # what the output type can hold
            p.check()
    p.sv.spec_kv_append(p.cache, k.cuda(), v.cuda(), z)
    if qt == "bfloat16":
        p.kx, p.vx = [t.cpu().double().numpy() for t in p.sv.spec_kv_read(p.cache, n, p.S, heads=2, head_dim=64, dtype=torch.float32)[:2]]
        for f in (1e-20, 1e12):  # queries outside fp16's range, some rows only
            q = p.qx.copy()
            q[0, 1] *= f
            qc = torch.from_numpy(q).to(torch.bfloat16)
            p.q = qc.cuda()
            keep, p.qx = p.qx, qc.double().numpy()
            p.check()
            p.qx = keep


@pytest.mark.parametrize("kind,qt", KINDS)
def test_long_caches(sv, kind, qt):
    """Many parts, uneven lengths; weights concentrated on one far token."""
    p = Problem(sv, 2, 2, 8, 2, 128, 20001, [5000, 64], kind, qt, seed=21, qsize=6.0)
    p.check()
    Problem(sv, 1, 1, 4, 1, 128, 0, [30011], kind, qt, seed=22).check()


@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
def test_offsets_past_32_bits(sv, kind):
    """A cache whose last row lies more than 2^32 bytes in, a prefix of more than 2^31."""
    import torch
    H, D, N = 8, 128, 2
    E = sv.spec_kv_entry_bytes(H, D, getattr(torch, kind))
    S = (1 << 32) // E + 10
    shape = (2, 2, S, E) if kind == "uint8" else (2, 2, S, H, D)
    p = Problem(sv, 2, N, 16, H, D, 40, [6, 9], kind, "bfloat16", seed=4)
    big = torch.zeros(shape, dtype=p.cache.dtype, device="cuda")
    big[:, :, :p.S] = p.cache
    p.cache, old = big, p.cache
    p.check()
    del old


def test_no_keys_and_empty_calls(sv):
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2, 3, 4, 64, device="cuda", dtype=torch.bfloat16)
    c = torch.zeros(2, 2, 5, 2, 64, device="cuda", dtype=torch.bfloat16)
    out, lse, st = sv.spec_prefix_attention(q, c, i(2), count=i(2))  # no query at all
    assert float(out.abs().max()) == 0 and bool((lse == float("-inf")).all()) and st.tolist() == [0, 0]
    out, lse, st = sv.spec_prefix_attention(q[:0], c[:, :0], i(0))
    assert out.shape == (0, 3, 4, 64) and st.shape == (0,)
    out, lse, st = sv.spec_prefix_attention(q[:, :0], c, i(2))
    assert out.shape == (2, 0, 4, 64) and st.tolist() == [0, 0]


def test_on_another_stream_and_in_a_graph(sv):
    import torch
    p = Problem(sv, 3, 4, 8, 2, 128, 500, [20, 0, 77], "uint8", "bfloat16", seed=30)
    out0, lse0 = p.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse, _ = p.call(stream=s)
    s.synchronize()
    assert torch.equal(out, out0) and torch.equal(lse, lse0)
    lens = torch.from_numpy(p.lens).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, _ = sv.spec_prefix_attention(p.q, p.cache, lens, prefix=p.prefix, kv_heads=2)
    p.q.copy_(p.q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    p.qx = p.q.cpu().double().numpy()
    want, _ = p.check()
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("B,N,Hq,H,D,P,lens,tree", [
    (43, 3, 8, 2, 128, 1000, list(range(0, 129, 3)), False),   # three blocks of 256 rows, a ragged last one
    (16, 2, 8, 1, 64, 4097, [0] * 16, False),                  # exactly one block; one token in the last block of tokens
    (2, 33, 16, 2, 128, 128, [127, 128], True),                # trees over block borders
    (1, 200, 8, 1, 64, 0, [300], True),                        # 1600 rows of one tree
    (2, 64, 8, 2, 96, 500, [64, 1], False),
    (40, 1, 16, 2, 48, 256, [5] * 40, False),
])
def test_many_query_rows(sv, kind, qt, B, N, Hq, H, D, P, lens, tree):
    Problem(sv, B, N, Hq, H, D, P, lens, kind, qt, tree, seed=B + N).check(rows=sorted({0, B // 2, B - 1}))


@pytest.mark.parametrize("kind,qt", KINDS)
def test_prefix_weights_far_apart(sv, kind, qt):
    """Scores that grow along the prefix (the sums have to follow) and large queries; a negative and a zero scale."""
    p = Problem(sv, 24, 2, 8, 2, 128, 3000, [10] * 24, kind, qt, seed=77, qsize=8.0)
    p.check(rows=[0, 23])
    for scale in (-0.05, 0.0):
        p.scale = scale
        call = p.call
        p.call = lambda **kw: call(scale=scale, **kw)
        p.check(rows=[3])
        p.call = call


def test_a_wait_that_runs_out_is_reported(sv):
    """The tile kernel's waits are bounded: with one arrival withheld its rows report a timeout."""
    import torch
    limit = sv.get_wait_timeout_ns()
    for kind in ("bfloat16", "uint8"):
        p = Problem(sv, 24, 2, 8, 2, 128, 300, [10] * 24, kind, "bfloat16", seed=78)
        out0, lse0 = p.check(rows=[0])
        try:
            sv.set_wait_timeout_ns(2_000_000)
            sv.debug_force_wait_timeout(True)
            out, lse, st = p.call()
            torch.cuda.synchronize()
        finally:
            sv.debug_force_wait_timeout(False)
            sv.set_wait_timeout_ns(limit)
        assert st.tolist() == [6] * 24
        assert float(out.abs().max()) == 0.0 and bool((lse == float("-inf")).all())
        out, lse, st = p.call()
        assert st.tolist() == [0] * 24 and torch.equal(out, out0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("P,D", [(130, 64), (0, 128), (256, 128)])
def test_trees_that_need_no_join(sv, kind, qt, P, D):
    """Enough rows that no part is cut: the kernel writes the answers itself, bad rows, fewer queries
    and values that are not finite among them."""
    import torch
    B, N = 80, 32
    rng = np.random.default_rng(P + D)
    lens = rng.integers(0, 200, B)
    count = rng.integers(0, N + 1, B)
    count[:4] = [N, 0, N, 1]
    p = Problem(sv, B, N, 8, 2, D, P, lens, kind, qt, True, count=count, seed=P)
    out0, lse0 = p.check(rows=[0, 1, 2, 3, 41, 79])
    p.parent[2, 5], p.lens[3] = 5, -3
    bad = int(np.flatnonzero(count[10:] > 8)[0]) + 10
    j = int(count[bad]) - 3
    at = int(p.lens[bad]) + j
    if kind == "uint8":
        p.cache[1, bad, at, 3] = 0x7f                  # a code that stands for NaN: head 0, column 3
    else:
        p.cache[1, bad, at, 0, 3] = float("-inf")
    out, lse, st = p.call()
    want = torch.zeros(B, dtype=torch.int32)
    want[2], want[3] = 4, 8
    assert torch.equal(st.cpu(), want)
    for b in (2, 3):
        assert float(out[b].abs().max()) == 0.0 and bool((lse[b] == float("-inf")).all())
    keep = torch.ones(B, dtype=torch.bool)
    keep[[2, 3, bad]] = False
    assert torch.equal(out[keep], out0[keep]) and torch.equal(lse, lse0.index_put((torch.tensor([2, 3]).cuda(),), torch.tensor(float("-inf")).cuda()))
    sees = torch.from_numpy(seen(N, p.parent[bad])[:, j] & (np.arange(N) < count[bad])).cuda()
    assert torch.equal(out[bad][~sees], out0[bad][~sees])
    hit = out[bad][sees][:, :4, 3]                     # the queries of KV head 0
    assert bool((torch.isnan(hit) if kind == "uint8" else hit == float("-inf")).all())
    rest = out[bad].clone()
    rest[:, :4, 3] = out0[bad][:, :4, 3]
    assert torch.equal(rest, out0[bad])
    limit = sv.get_wait_timeout_ns()
    try:
        sv.set_wait_timeout_ns(2_000_000)
        sv.debug_force_wait_timeout(True)
        out, lse, st = p.call()
        torch.cuda.synchronize()
    finally:
        sv.debug_force_wait_timeout(False)
        sv.set_wait_timeout_ns(limit)
    want[torch.from_numpy(count > 0) & (want == 0)] = 6
    assert torch.equal(st.cpu(), want) and float(out.abs().max()) == 0.0


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("B,N,Hq,H,D,P,top", [(64, 1, 32, 8, 64, 500, 700), (100, 2, 8, 4, 128, 0, 300), (128, 3, 12, 4, 64, 70, 40),
                                             (32, 1, 16, 16, 64, 200, 2000)])
def test_rows_cut_by_a_budget(sv, kind, qt, B, N, Hq, H, D, P, top):
    """Enough rows that they are cut into parts by their lengths: very uneven ones, empty ones, unused ones."""
    rng = np.random.default_rng(B)
    lens = (top * rng.random(B)**3).astype(np.int32)
    lens[3], lens[7], lens[B - 1] = top, 0, 1
    count = rng.integers(0, N + 1, B)
    count[:2], count[3], count[B - 1] = 0, N, N
    p = Problem(sv, B, N, Hq, H, D, P, lens, kind, qt, count=count, seed=B)
    p.check(rows=[0, 2, 3, 7, 8, B // 2, B - 2, B - 1])
    # rows that cannot be used change the cut of the others, so their last bits, and nothing more
    p.lens[5], p.count[6] = -7, N + 1
    bad = [5, 6]
    out, lse = p.check(rows=[2, 3, 7, 8, B - 1], status=[8 if b in bad else 0 for b in range(B)])
    assert bool((lse[bad] == float("-inf")).all())
    assert float(out[bad].abs().max()) == 0.0


@pytest.mark.parametrize("qt", ["bfloat16", "float16"])
@pytest.mark.parametrize("B,N,D,P,top,tree", [
    (1, 50, 64, 200, 20, True),     # prefix and own entries in one item, cut into parts
    (2, 60, 128, 300, 150, True),   # a prefix that is converted once
    (80, 32, 128, 256, 100, True),  # no join
    (40, 6, 64, 500, 60, False),    # the prefix alone
    (16, 2, 128, 700, 40, False),   # the prefix alone, unconverted
])
def test_e4m3_scales_far_apart_in_tiles(sv, qt, B, N, D, P, top, tree):
    """Values and keys 2^40 to 2^100 apart within 128 tokens: a token of the pass that most queries do
    not see, one of the prefix whose weight is nothing, tiny ones and zeros beside them."""
    import torch
    lens = np.random.default_rng(B).integers(0, top, B)
    p = Problem(sv, B, N, 8, 2, D, P, lens, "uint8", qt, tree, seed=D)
    p.q = p.q.abs() + 1
    p.qx = p.q.cpu().double().numpy()
    zeros = torch.zeros(B, dtype=torch.int32, device="cuda")
    total = torch.from_numpy(np.asarray(lens + N, np.int32)).cuda()
    k, v = (torch.from_numpy(x).float().cuda() for x in (p.kx, p.vx))
    for b in range(0, B, 3):
        at = int(lens[b]) + N // 2
        k[b, at] *= 2.0**40
        v[b, at] *= 2.0**40
    sv.spec_kv_append(p.cache, k, v, zeros, count=total)
    kx, vx, _ = sv.spec_kv_read(p.cache, total, p.S, heads=2, head_dim=D, dtype=torch.float32)
    p.kx, p.vx = kx.cpu().double().numpy(), vx.cpu().double().numpy()
    pk, pv = (torch.from_numpy(x).float().cuda()[None] for x in (p.pk, p.pv))
    pk[0, 7], pv[0, 7] = -8.0, pv[0, 7] * 2.0**60      # scores so low that the weight is 0 in 64 bits' reach
    pv[0, 20:30] *= 2.0**-40
    pk[0, 40] *= 2.0**-60
    pk[0, 41], pv[0, 41] = 0.0, 0.0
    sv.spec_kv_append(p.prefix, pk, pv, zeros[:1])
    kx, vx, _ = sv.spec_kv_read(p.prefix, total[:1] * 0 + P, P, heads=2, head_dim=D, dtype=torch.float32)
    p.pk, p.pv = kx[0].cpu().double().numpy(), vx[0].cpu().double().numpy()
    p.check(rows=range(min(B, 4)))


@pytest.mark.parametrize("B,N,D,P,lens", [(1, 4, 64, 0, [100]), (3, 6, 128, 70, [5, 400, 33]), (70, 2, 64, 0, [90] * 70)])
@pytest.mark.parametrize("up", [40, 100])
def test_e4m3_scales_far_apart_in_rows(sv, B, N, D, P, lens, up):
    """Values 2^40 and 2^100 above the rest: the pass's last token, which the queries before it do not
    see, and a token whose weight is nothing; growth after the first blocks, zeros, tiny values."""
    import torch
    p = Problem(sv, B, N, 4, 2, D, P, lens, "uint8", "bfloat16", seed=up + D)
    p.q = p.q.abs() + 1
    p.qx = p.q.cpu().double().numpy()
    total = torch.from_numpy(np.asarray(p.lens + N, np.int32)).cuda()
    k, v = (torch.from_numpy(x).float().cuda() for x in (p.kx, p.vx))
    v[:, :4] = 0.0
    for b in range(0, B, 2):
        at = int(p.lens[b])
        v[b, at + N - 1] *= 2.0**up
        if at > 60:
            k[b, 50], v[b, 50] = -8.0, v[b, 50] * 2.0**up
            v[b, 20:24] *= 2.0**-up
            v[b, 51:55] *= 2.0**30
    zeros = torch.zeros(B, dtype=torch.int32, device="cuda")
    sv.spec_kv_append(p.cache, k, v, zeros, count=total)
    kx, vx, _ = sv.spec_kv_read(p.cache, total, p.S, heads=2, head_dim=D, dtype=torch.float32)
    p.kx, p.vx = kx.cpu().double().numpy(), vx.cpu().double().numpy()
    p.check(rows=range(min(B, 4)))


def test_graphs_have_workspaces_of_their_own(sv):
    """Two graphs captured on one stream and replayed side by side, after eager calls of other sizes."""
    import torch
    from speculative_decoding_verification_32_gb300 import _binding
    ps = [Problem(sv, 4, 6, 8, 2, 128, 600, [30, 900, 5, 77], kind, "bfloat16", seed=40) for kind in ("uint8", "bfloat16")]
    want = [p.check() for p in ps]
    lens = torch.from_numpy(ps[0].lens).cuda()
    before = dict(_binding._ws)
    graphs, got = [], []
    for p in ps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(sv.spec_prefix_attention(p.q, p.cache, lens, prefix=p.prefix, kv_heads=2))
    assert _binding._ws.keys() == before.keys() and all(_binding._ws[x] is before[x] for x in before)
    Problem(sv, 9, 30, 8, 2, 128, 3000, [500] * 9, "uint8", seed=41).call()
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (out, lse), (o, ls, _) in zip(want, got):
        assert torch.equal(out, o) and torch.equal(lse, ls)
