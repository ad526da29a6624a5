"""spec_page_plan and spec_kv_compact_pages against plain restatements (needs a GB300).  Integers
and moved bytes: everything has to be equal."""
import numpy as np
import pytest

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


def live(j, n, c, page, window, sinks):
    """Whether place j holds a token below n + c that a query from position n on can see."""
    tokens = range(j * page, min((j + 1) * page, n + c))
    if not len(tokens):
        return False
    # a page is given back as a whole: all its slots are behind the window and none is a sink
    return not (window > 0 and j * page >= sinks and (j + 1) * page - 1 <= n - window)


def plan(table, free, ring, kv_len, count, N, page, window, sinks):
    """The call, one page at a time: (slots, status); table, free and ring change in place."""
    B, columns = table.shape
    pages = len(free)
    slots, status = np.full((B, N), -1, np.int32), np.zeros(B, np.int32)
    head, have = int(ring[0]), int(ring[1])
    if not (0 <= head < max(1, pages) and 0 <= have <= pages):
        return slots, np.full(B, 8, np.int32)
    wanted, taken, back = 0, 0, []
    for b in range(B):
        n, c = int(kv_len[b]), N if count is None else int(count[b])
        if n < 0 or not 0 <= c <= N or n + c > columns * page or (table[b] >= pages).any():
            status[b] = 8
            continue
        on = [live(j, n, c, page, window, sinks) for j in range(columns)]
        want = [j for j in range(columns) if on[j] and table[b, j] < 0]
        wanted += len(want)
        if want and wanted > have:
            status[b] = 9
        else:
            for j in want:
                page_no = int(free[(head + taken) % pages])
                taken += 1
                if 0 <= page_no < pages:
                    table[b, j] = page_no
                else:
                    status[b] = 8
        for j in range(columns):
            if not on[j] and table[b, j] >= 0:
                back.append((b, int(table[b, j])))
                table[b, j] = -1
        if status[b] != 9:
            for i in range(c):
                e = table[b, (n + i) // page]
                slots[b, i] = e * page + (n + i) % page if e >= 0 else -1
    for k, (b, page_no) in enumerate(back):
        if k < pages - have:
            free[(head + have + k) % pages] = page_no
        else:
            status[b] = 8
    ring[:] = ((head + taken) % max(1, pages), have - taken + min(len(back), pages - have))
    return slots, status


def agree(sv, table, free, ring, kv_len, count, N, page, window=0, sinks=0):
    """One call and the restatement on the same state; returns (slots, status)."""
    t, f, r = i32(table), i32(free), i32(ring)
    slots, status = sv.spec_page_plan(t, f, r, i32(kv_len), N, page, count=None if count is None else i32(count),
                                      window=window, sinks=sinks)
    want_slots, want_status = plan(table, free, ring, kv_len, count, N, page, window, sinks)
    assert np.array_equal(status.cpu().numpy(), want_status)
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(t.cpu().numpy(), table)
    assert np.array_equal(r.cpu().numpy(), ring)
    assert np.array_equal(f.cpu().numpy(), free)
    return want_slots, want_status


@pytest.mark.parametrize("B,N,page,columns,window,sinks", [
    (1, 1, 16, 1, 0, 0), (1, 1, 16, 5, 0, 0), (3, 6, 16, 40, 0, 0), (8, 6, 16, 33, 64, 4), (9, 60, 32, 31, 100, 0),
    (17, 7, 48, 20, 1, 1), (64, 6, 16, 257, 300, 20), (130, 1, 128, 9, 0, 0), (70, 257, 16, 50, 128, 4),
    (2, 1000, 64, 100, 500, 70), (5, 300, 1024, 3, 0, 0), (1100, 2, 16, 12, 50, 3)])
def test_steps(sv, B, N, page, columns, window, sinks):
    """Ten steps from an empty table: rows start, grow, fall back, end and start again."""
    rng = np.random.default_rng(B + N)
    most = columns * page
    table = np.full((B, columns), -1, np.int32)
    pages = B * min(columns, -(-(most // 2) // page) + 2) + 3
    free, ring = rng.permutation(pages).astype(np.int32), np.array([rng.integers(pages), pages], np.int32)
    n = np.zeros(B, np.int64)
    for step in range(10):
        count = rng.integers(0, N + 1, B) if step % 3 else None
        c = np.full(B, N) if count is None else count
        n = np.minimum(n, most - c)
        _, status = agree(sv, table, free, ring, n, count, N, page, window, sinks)
        assert set(status) <= {0, 9}
        # pages are never held twice
        held = table[table >= 0].tolist() + [int(free[(ring[0] + k) % pages]) for k in range(ring[1])]
        assert sorted(held) == list(range(pages))
        kept = np.where(status == 9, 0, rng.integers(0, c + 1))
        n = np.where(rng.random(B) < 0.1, 0, np.minimum(n + kept, most // 2 + rng.integers(0, 50)))
        n = np.where(rng.random(B) < 0.2, n + rng.integers(0, most // 4 + 1, B), n)  # a prompt put in between
        n = np.clip(n, 0, most - N if most >= N else 0)


def test_too_few_pages(sv):
    """Rows are served in order; one that does not get its pages takes none, gives its dead ones back,
    and later rows that want some get none either."""
    table = np.full((6, 8), -1, np.int32)
    table[1, :5] = [3, 1, 7, 9, 11]
    free, ring = np.array([0, 2, 4, 5, 6, 8, 10, -7, -7, -7, -7, -7], np.int32), np.array([0, 7], np.int32)
    kv_len = np.array([40, 20, 60, 0, 16, 1])
    # row 0 wants 3 pages, row 1 none and gives 3 back, row 2 wants 5: too many, row 3 wants none, 4 and 5 some
    _, status = agree(sv, table, free, ring, kv_len, np.array([1, 1, 5, 0, 1, 0]), 6, 16)
    assert status.tolist() == [0, 0, 9, 0, 9, 9]
    assert ring.tolist() == [3, 7]
    # the next step has what came back
    _, status = agree(sv, table, free, ring, kv_len, np.array([1, 1, 5, 0, 1, 0]), 6, 16)
    assert status.tolist() == [0, 0, 0, 0, 0, 9]


@pytest.mark.parametrize("B", [40, 700])
def test_too_few_pages_later(sv, B):
    """The first row that gets nothing may lie in any group of rows."""
    for have in (0, 1, 7, 8, 9, 63, 64, 65, 256, 300, B * 2 - 1):
        table, pages = np.full((B, 3), -1, np.int32), B * 3
        free, ring = np.arange(pages, dtype=np.int32)[::-1].copy(), np.array([pages - 5, have], np.int32)
        agree(sv, table, free, ring, np.full(B, 17), None, 3, 16)


def test_bad_rows(sv):
    """A row that cannot be used is left as it is, and does not disturb the others."""
    table = np.full((8, 4), -1, np.int32)
    table[2] = [50, 0, -1, -1]
    table[5, 0] = 1
    free, ring = np.array([2, 3, 4, 5, 6, 7, 8, 9, -1, -1], np.int32), np.array([0, 8], np.int32)
    kv_len = np.array([-1, 3, 0, 63, 5, 2, 64, 60])
    _, status = agree(sv, table, free, ring, kv_len, np.array([1, 2, 1, 2, -1, 3, 0, 4]), 3, 16)
    assert status.tolist() == [8, 0, 8, 8, 8, 0, 0, 8]


@pytest.mark.parametrize("N", [3, 300])
def test_bad_rows_among_many(sv, N):
    """The same where the rows are too many for one launch, or their slots."""
    B = 300
    table = np.full((B, 20), -1, np.int32)
    table[250] = [2000] + 19 * [-1]
    table[270, 3] = 1
    free, ring = np.roll(np.arange(2, 1202, dtype=np.int32), 7), np.array([7, 1190], np.int32)
    kv_len, count = np.arange(B) % 19, np.arange(B) % (N + 1)
    kv_len[5], count[9], kv_len[10] = -1, N + 1, 20 * 16
    count[10] = 1
    _, status = agree(sv, table, free, ring, kv_len, count, N, 16)
    assert [b for b in range(B) if status[b] == 8] == [5, 9, 10, 250]


@pytest.mark.parametrize("B", [3, 300])
@pytest.mark.parametrize("ring", [(-1, 3), (10, 3), (0, -1), (0, 11)])
def test_bad_ring(sv, ring, B):
    table = np.full((B, 4), -1, np.int32)
    _, status = agree(sv, table, np.arange(10, dtype=np.int32), np.array(ring, np.int32), np.full(B, 5), None, 3, 16)
    assert status.tolist() == [8] * B


def test_broken_ring(sv):
    """Numbers in the ring that are no pages are not put into the table; pages that it has no room for are
    dropped."""
    table = np.full((4, 4), -1, np.int32)
    agree(sv, table, np.array([0, 77, -3, 3, 4, 5, 6, 7], np.int32), np.array([0, 8], np.int32), np.array([20, 0, 15, 20]), None, 2, 16)
    assert table[0].tolist() == [0, -1, -1, -1] and table[1].tolist() == [-1] * 4
    table = np.array([[0, 1, 2, 3], [4, 5, 6, 7]], np.int32)  # and the ring holds five of them as well
    _, status = agree(sv, table, np.arange(8, dtype=np.int32), np.array([3, 5], np.int32), np.array([0, 0]), None, 0, 16)
    assert status.tolist() == [8, 8]


def test_nothing(sv):
    """No rows, no tokens, no pages."""
    import torch
    e = np.zeros((0, 4), np.int32)
    slots, status = sv.spec_page_plan(i32(e), i32(np.arange(4)), i32([0, 4]), i32([]), 3, 16)
    assert slots.shape == (0, 3) and status.shape == (0,)
    agree(sv, np.full((2, 4), -1, np.int32), np.zeros(0, np.int32), np.array([0, 0], np.int32), np.array([0, 20]), None, 0, 16)
    agree(sv, np.full((2, 4), -1, np.int32), np.zeros(0, np.int32), np.array([0, 0], np.int32), np.array([0, 20]), None, 2, 16)
    torch.cuda.synchronize()


def test_slots_feed_append(sv):
    """Tokens written by spec_kv_append through the slot map are where the table says."""
    import torch
    B, N, page, columns, H, D = 5, 7, 16, 6, 2, 64
    rng = np.random.default_rng(1)
    table, pages = np.full((B, columns), -1, np.int32), 40
    t, f, r = i32(table), i32(rng.permutation(pages)), i32([11, pages])
    kv_len, count = i32([0, 30, 15, 63, 80]), i32([7, 7, 0, 3, 6])
    slots, status = sv.spec_page_plan(t, f, r, kv_len, N, page, count=count)
    assert status.tolist() == [0] * B
    pool = torch.full((2, pages, page, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = torch.randn(2, B, N, H, D, device="cuda").bfloat16()
    flat = pool.view(2, 1, pages * page, H, D).expand(2, B * N, pages * page, H, D)
    st = sv.spec_kv_append(flat, k.reshape(B * N, 1, H, D), v.reshape(B * N, 1, H, D), slots.flatten())
    want = torch.full_like(pool, 7.0)
    for b in range(B):
        for i in range(N):
            here = i < int(count[b])
            assert int(st[b * N + i]) == (0 if here else 8)
            if here:
                p = int(kv_len[b]) + i
                want[0, t[b, p // page], p % page] = k[b, i]
                want[1, t[b, p // page], p % page] = v[b, i]
    assert torch.equal(pool, want)


def test_captured(sv):
    """A captured step, replayed on lengths that change in place, beside eager steps of other sizes."""
    import torch
    B, N, page, columns, pages = 6, 4, 16, 10, 80
    table, free, ring = np.full((B, columns), -1, np.int32), np.arange(pages, dtype=np.int32), np.array([0, pages], np.int32)
    t, f, r, n = i32(table), i32(free), i32(ring), i32(np.zeros(B))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sv.spec_page_plan(t, f, r, n, N, page)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            slots, status = sv.spec_page_plan(t, f, r, n, N, page, window=40, sinks=2)
    torch.cuda.current_stream().wait_stream(s)
    plan(table, free, ring, np.zeros(B), None, N, page, 0, 0)
    for step in range(5):
        lens = np.arange(B) * 7 + step * 21
        n.copy_(i32(lens))
        g.replay()
        big = np.full((200, 30), -1, np.int32)
        agree(sv, big, np.arange(7000, dtype=np.int32), np.array([3, 7000], np.int32), np.full(200, 300), None, 20, 16)
        want, st = plan(table, free, ring, lens, None, N, page, 40, 2)
        assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(status.cpu().numpy(), st)
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), ring)


# ------------------------------------------------------------- compaction
def compact(kv, table, kv_len, accepted, path):
    """The moves one at a time: status; kv changes in place."""
    pages, page = kv.shape[1:3]
    status = np.zeros(len(kv_len), np.int32)
    for b in range(len(kv_len)):
        a, n, N = int(accepted[b]), int(kv_len[b]), path.shape[1]
        if a <= 0:
            continue
        p = path[b, :a].astype(np.int64) if a <= N - 1 else None
        if p is None or p[0] < 1 or p[-1] >= N or (np.diff(p) <= 0).any():
            status[b] = 4
            continue
        spots = np.concatenate((n + p, n + 1 + np.arange(a)))
        if n < 0 or spots.max() >= table.shape[1] * page or (table[b, spots // page] < 0).any() or (table[b, spots // page] >= pages).any():
            status[b] = 8
            continue
        for k in range(a):
            f, t = n + int(p[k]), n + 1 + k
            kv[:, table[b, t // page], t % page] = kv[:, table[b, f // page], f % page]
    return status


@pytest.mark.parametrize("B,N,planes,page,entry,depth", [
    (1, 2, 1, 16, 16, 1), (3, 9, 2, 16, 48, 4), (32, 60, 8, 16, 1040, 6), (5, 40, 3, 64, 4112, 39), (2, 200, 2, 32, 64, 150),
    (7, 12, 2, 1024, 2048, 5)])
def test_compact(sv, B, N, planes, page, entry, depth):
    import torch
    rng = np.random.default_rng(N)
    columns = -(-(100 + N) // page)
    pages = B * columns + 3
    table = rng.permutation(pages)[: B * columns].reshape(B, columns).astype(np.int32)
    kv_len = rng.integers(0, 100, B)
    accepted = rng.integers(0, depth + 1, B)
    accepted[0] = depth
    path = np.full((B, N), -1, np.int32)
    for b in range(B):
        path[b, : accepted[b]] = np.sort(rng.choice(np.arange(1, N), accepted[b], replace=False))
    for b in range(B):  # pages that the row does not need
        used = set(((kv_len[b] + 1 + np.arange(N)) // page).tolist())
        for j in range(columns):
            if j not in used:
                table[b, j] = -1 if j % 2 else pages + 5
    kv = rng.integers(0, 256, (planes, pages, page, entry), dtype=np.uint8)
    d = torch.from_numpy(kv.copy()).cuda()
    st = sv.spec_kv_compact_pages(d, i32(table), i32(kv_len), i32(accepted), i32(path))
    want = compact(kv, table, kv_len, accepted, path)
    assert np.array_equal(st.cpu().numpy(), want) and not want.any()
    assert np.array_equal(d.cpu().numpy(), kv)


def test_compact_refuses_rows(sv):
    """Bad paths, lengths and pages: the row is flagged and stays as it is."""
    import torch
    rng = np.random.default_rng(3)
    B, N, page, columns, pages = 10, 8, 16, 3, 20
    table = np.arange(B * columns).reshape(B, columns).astype(np.int32) % pages
    table[:, 2] = -1
    path = np.tile(np.array([2, 3, 5, -1, -1, -1, -1, -1], np.int32), (B, 1))
    path[1, 1] = 2
    path[2, 0] = 0
    path[3, 2] = 8
    kv_len = np.array([3, 3, 3, 3, -1, 27, 45, 26, 3, 3])
    accepted = np.array([3, 3, 3, 3, 3, 3, 3, 3, 8, -1])
    table[9, 0] = 99
    kv = rng.integers(0, 256, (2, pages, page, 32), dtype=np.uint8)
    d = torch.from_numpy(kv.copy()).cuda()
    st = sv.spec_kv_compact_pages(d, i32(table), i32(kv_len), i32(accepted), i32(path))
    want = compact(kv, table, kv_len, accepted, path)
    assert want.tolist() == [0, 4, 4, 4, 8, 8, 8, 0, 4, 0]
    assert st.tolist() == want.tolist()
    assert np.array_equal(d.cpu().numpy(), kv)
