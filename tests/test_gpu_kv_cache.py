"""spec_kv_append and spec_kv_read against a plain 64-bit restatement (needs a GB300).

Stored numbers are exact: a 16-bit cache holds one rounding to nearest even,
an e4m3 cache holds code * 2^(c - 127) with one rounding of x / 2^(c - 127), so
every comparison is for equality."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def e4m3_values(x):
    """What the e4m3 cache stands for, of head vectors x [..., D] (float64), and the scale bytes."""
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(amax)
    f, e = np.frexp(np.where(bad, 1.0, amax) / 448.0)
    e = np.where(f == 0.5, e - 1, e)  # the smallest e with amax <= 448 * 2^e
    c = np.clip(np.where(amax == 0, 1, e + 127), 1, None)
    s = np.ldexp(1.0, c - 127)[..., None]
    y = np.where(bad[..., None], 0.0, x) / s
    _, ye = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(ye - 4, -9))
    y = np.round(y / step) * step * s
    return np.where(bad[..., None], np.nan, y), np.where(bad, 255, c).astype(np.uint8)


def source(torch, B, N, H, D, dtype, seed):
    """Random head vectors of very different sizes, with the borders of the format among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, H, D, generator=g) * torch.exp2(torch.randint(-6, 7, (B, N, H, 1), generator=g).float())
    flat = x.view(-1, D)
    special = [torch.zeros(D), torch.full((D,), 448.0), torch.full((D,), 448.0 * 4), torch.full((D,), -0.0)]
    edge = torch.randn(D, generator=g)
    edge[3] = 449.0
    tiny = torch.randn(D, generator=g) * 1e-40
    inf, nan = torch.randn(D, generator=g), torch.randn(D, generator=g)
    inf[D - 1], nan[0] = float("-inf"), float("nan")
    big = torch.randn(D, generator=g) * (1e38 if dtype != torch.float16 else 1e4)
    halves = torch.arange(D).float() + 17 / 32  # ties of the rounding
    for i, v in enumerate(special + [edge, tiny, inf, nan, big, halves]):
        if i < flat.shape[0]:
            flat[(i * 7) % flat.shape[0]] = v
    return x.to(dtype)


CASES = [  # B, N, heads, D, slots, count, layout
    (1, 1, 8, 128, 1, None, "dense"), (3, 5, 2, 64, 40, [0, 5, 3], "dense"), (2, 7, 3, 80, 19, None, "packed"),
    (4, 3, 1, 16, 9, [3, 1, 0, 2], "dense"), (2, 33, 17, 96, 70, None, "odd"), (1, 200, 5, 112, 333, None, "packed"),
    (65, 2, 4, 48, 6, None, "odd")]


@pytest.mark.parametrize("src", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("cache", ["uint8", "bfloat16", "float16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append_then_read(sv, src, cache, case):
    import torch
    B, N, H, D, S, count, layout = CASES[case]
    dt, ct = getattr(torch, src), getattr(torch, cache)
    k, v = source(torch, B, N, H, D, dt, case), source(torch, B, N, H, D, dt, case + 100)
    if layout == "packed":  # side by side, as one projection leaves them
        both = torch.stack((k, v), 2).cuda()
        kg, vg = both[:, :, 0], both[:, :, 1]
    elif layout == "odd":  # rows that no 16-byte load can take
        both = torch.zeros(2, B, N, H, D + 1, dtype=dt)
        both[0, ..., 1:], both[1, ..., 1:] = k, v
        both = both.cuda()
        kg, vg = both[0, ..., 1:], both[1, ..., 1:]
    else:
        kg, vg = k.cuda(), v.cuda()
    rng = np.random.default_rng(case)
    start = rng.integers(0, S - N + 1, B).astype(np.int32)
    n = np.array(count if count is not None else [N] * B)
    if cache == "uint8":
        buf = torch.full((2, B, S, sv.spec_kv_entry_bytes(H, D)), 0xA5, dtype=torch.uint8, device="cuda")
    else:
        buf = torch.full((2, B, S, H, D), 7.5, dtype=ct, device="cuda")
    before = buf.clone()
    st = sv.spec_kv_append(buf, kg, vg, torch.from_numpy(start).cuda(),
                           count=None if count is None else torch.tensor(count, dtype=torch.int32, device="cuda"))
    assert st.tolist() == [0] * B
    # untouched slots keep their bytes, written ones are whole
    keep = np.ones((B, S), bool)
    for b in range(B):
        keep[b, start[b]:start[b] + n[b]] = False
    kt = torch.from_numpy(keep).cuda()
    assert torch.equal(buf[:, kt], before[:, kt])
    k2, v2, st = sv.spec_kv_read(buf, torch.from_numpy(n.astype(np.int32)).cuda(), N, heads=H, head_dim=D,
                                 start=torch.from_numpy(start).cuda(), dtype=torch.float32)
    assert st.tolist() == [0] * B
    for got, x, plane in ((k2, k, 0), (v2, v, 1)):
        if cache == "uint8":
            want, byte = e4m3_values(x.double().numpy())
        else:
            want = x.to(ct).double().numpy()
        for b in range(B):
            np.testing.assert_array_equal(got[b, :n[b]].cpu().double().numpy(), want[b, :n[b]])
            assert torch.all(got[b, n[b]:] == 0)
            if cache == "uint8" and n[b]:
                raw = buf[plane, b, start[b]:start[b] + n[b]].cpu().numpy()
                np.testing.assert_array_equal(raw[:, H * D:H * D + H], byte[b, :n[b]])
                assert np.all(raw[:, H * D + H:] == 0)
    # a second rounding on the way out, to each output type
    for ot in (torch.bfloat16, torch.float16):
        k3, v3, _ = sv.spec_kv_read(buf, torch.from_numpy(n.astype(np.int32)).cuda(), N, heads=H, head_dim=D,
                                    start=torch.from_numpy(start).cuda(), dtype=ot)
        assert torch.equal(torch.nan_to_num(k3.float(), 9.0), torch.nan_to_num(k2.to(ot).float(), 9.0))
        assert torch.equal(torch.nan_to_num(v3.float(), 9.0), torch.nan_to_num(v2.to(ot).float(), 9.0))


@pytest.mark.parametrize("cache", ["uint8", "bfloat16"])
def test_bad_slots_leave_the_row_alone(sv, cache):
    import torch
    B, N, H, D, S = 6, 4, 2, 64, 10
    k = torch.randn(B, N, H, D, device="cuda", dtype=torch.bfloat16)
    shape = (2, B, S, sv.spec_kv_entry_bytes(H, D)) if cache == "uint8" else (2, B, S, H, D)
    buf = torch.zeros(shape, dtype=getattr(torch, cache), device="cuda")
    start = torch.tensor([-1, 7, 6, 2147483647, 0, 0], dtype=torch.int32, device="cuda")
    count = torch.tensor([1, 4, 4, 1, -1, 5], dtype=torch.int32, device="cuda")
    st = sv.spec_kv_append(buf, k, k, start, count=count)
    assert st.tolist() == [8, 8, 0, 8, 8, 8]
    touched = (buf.view(2, B, -1) != 0).any(-1).any(0)
    assert touched.tolist() == [False, False, True, False, False, False]
    k2, _, st = sv.spec_kv_read(buf, count, N, heads=H, head_dim=D, start=start)
    assert st.tolist() == [8, 8, 0, 8, 8, 8]
    assert torch.equal((k2.view(B, -1) != 0).any(-1).cpu(), touched.cpu())


def test_empty_calls(sv):
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    assert sv.spec_kv_append(z(2, 0, 4, 2, 64), z(0, 3, 2, 64), z(0, 3, 2, 64), i(0)).shape == (0,)
    assert sv.spec_kv_append(z(2, 3, 4, 2, 64), z(3, 0, 2, 64), z(3, 0, 2, 64), i(3)).tolist() == [0, 0, 0]
    k, v, st = sv.spec_kv_read(z(2, 3, 0, 2, 64), i(3), 2)
    assert k.shape == (3, 2, 2, 64) and torch.all(k == 0) and st.tolist() == [0, 0, 0]


def test_append_past_32_bit_offsets(sv):
    """Entries more than 2^31 (and 2^32) bytes from the cache's start."""
    import torch
    H, D = 8, 128
    E = sv.spec_kv_entry_bytes(H, D)
    S = (1 << 32) // E + 100
    buf = torch.zeros(2, 1, S, E, dtype=torch.uint8, device="cuda")
    k = torch.randn(1, 5, H, D, device="cuda", dtype=torch.bfloat16)
    for at in ((1 << 31) // E - 2, S - 5):
        start = torch.tensor([at], dtype=torch.int32, device="cuda")
        assert sv.spec_kv_append(buf, k, -k, start).tolist() == [0]
        k2, v2, _ = sv.spec_kv_read(buf, torch.tensor([5], dtype=torch.int32, device="cuda"), 5, heads=H, head_dim=D,
                                    start=start, dtype=torch.float32)
        want, _ = e4m3_values(k.cpu().double().numpy())
        np.testing.assert_array_equal(k2.cpu().double().numpy(), want)
        np.testing.assert_array_equal(v2.cpu().double().numpy(), -want)
    assert int((buf[0, 0, :100] != 0).sum()) == 0


def test_compaction_moves_quantised_entries_whole(sv):
    """A tree's accepted path, compacted by spec_kv_compact_tree, reads back as the path's own entries."""
    import torch
    B, N, H, D, S = 3, 6, 4, 64, 20
    E = sv.spec_kv_entry_bytes(H, D)
    buf = torch.zeros(2, B, S, E, dtype=torch.uint8, device="cuda")
    k = torch.randn(B, N, H, D, device="cuda") * torch.arange(1, N + 1, device="cuda")[None, :, None, None]
    start = torch.tensor([0, 5, 14], dtype=torch.int32, device="cuda")
    sv.spec_kv_append(buf, k, 2 * k, start)
    path = torch.tensor([[2, 4, -1, -1, -1, -1], [1, 2, 3, -1, -1, -1], [5, -1, -1, -1, -1, -1]], dtype=torch.int32, device="cuda")
    acc = torch.tensor([2, 3, 1], dtype=torch.int32, device="cuda")
    assert sv.spec_kv_compact_tree(buf, start, acc, path).tolist() == [0, 0, 0]
    k2, v2, _ = sv.spec_kv_read(buf, acc + 1, N, heads=H, head_dim=D, start=start, dtype=torch.float32)
    want, _ = e4m3_values(k.cpu().double().numpy())
    for b, nodes in enumerate(([0, 2, 4], [0, 1, 2, 3], [0, 5])):
        np.testing.assert_array_equal(k2[b, :len(nodes)].cpu().double().numpy(), want[b, nodes])
        np.testing.assert_array_equal(v2[b, :len(nodes)].cpu().double().numpy(), 2 * want[b, nodes])


def test_on_another_stream_and_in_a_graph(sv):
    import torch
    B, N, H, D, S = 4, 3, 8, 128, 50
    buf = torch.zeros(2, B, S, sv.spec_kv_entry_bytes(H, D), dtype=torch.uint8, device="cuda")
    k = torch.randn(B, N, H, D, device="cuda", dtype=torch.float16)
    start = torch.tensor([0, 9, 20, 47], dtype=torch.int32, device="cuda")
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    want, _ = e4m3_values(k.cpu().double().numpy())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.spec_kv_append(buf, k, k, start, stream=s)
    k2, _, _ = sv.spec_kv_read(buf, n, N, heads=H, head_dim=D, start=start, dtype=torch.float32, stream=s)
    s.synchronize()
    np.testing.assert_array_equal(k2.cpu().double().numpy(), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_kv_append(buf, k, k, start)
        k3, _, _ = sv.spec_kv_read(buf, n, N, heads=H, head_dim=D, start=start, dtype=torch.float32)
    k.mul_(-0.5)
    graph.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(k3.cpu().double().numpy(), -0.5 * want)
