"""Guard-region checks of the cache, attention and log-probability entry points (needs a GB300).

Every buffer a call receives lies inside a larger allocation with sentinel bytes around
it; after the call the sentinels and the inputs are as they were.  Odd shapes: head
sizes that fill no tile, one token, ragged ends, parts and blocks that end inside a tile."""
import ctypes

import numpy as np
import pytest

from tests.test_gpu_canary import Arena

pytestmark = pytest.mark.gpu
F32, BF16, F16, E4M3 = range(4)


@pytest.fixture(scope="module")
def lib():
    import torch
    assert torch.cuda.is_available()
    from speculative_decoding_verification_32_gb300 import _binding
    return _binding.lib()


def bf16(rng, *shape):
    x = rng.standard_normal(shape).astype(np.float32)
    return (x.view(np.uint32) >> 16).astype(np.uint16)


def stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def cache_of(A, name, rows, heads, D, dtype, slots, rng, writable, k_only=False):
    from speculative_decoding_verification_32_gb300 import _binding as b
    entry = b.lib().spec_kv_entry_bytes(heads, D, dtype)
    pitch = entry + 16  # a gap between entries that must stay as it is
    bufs = []
    for plane in "kv":
        raw = rng.integers(0, 127 if dtype == E4M3 else 256, (rows, slots, pitch), dtype=np.uint8)
        if dtype == E4M3:
            raw[:, :, heads * D:heads * D + heads] = rng.integers(110, 125, (rows, slots, heads))
        else:
            raw[:, :, :entry] = bf16(rng, rows, slots, heads * D).view(np.uint8)
        bufs.append((A.put(name + plane, raw.shape, np.uint8, raw, writable=writable), raw))
    c = b.SpecKvCache(rows, heads, D, dtype, slots, slots * pitch, pitch, A.ptr(bufs[0][0]), A.ptr(bufs[1][0]))
    return c, bufs, entry, pitch


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,N,heads,D,slots", [(1, 1, 1, 16, 1), (3, 5, 3, 80, 11), (2, 70, 8, 128, 75), (5, 3, 17, 48, 6)])
def test_append_and_read(lib, dtype, B, N, heads, D, slots):
    from speculative_decoding_verification_32_gb300 import _binding as b
    rng = np.random.default_rng(B * D)
    A = Arena()
    c, bufs, entry, pitch = cache_of(A, "cache", B, heads, D, dtype, slots, rng, True)
    k, v = (A.put(n, (B, N, heads, D), np.uint16, bf16(rng, B, N, heads, D)) for n in "kv")
    start = rng.integers(0, slots - N + 1, B).astype(np.int32)
    count = rng.integers(0, N + 1, B).astype(np.int32)
    s, n = A.put("start", (B,), np.int32, start), A.put("count", (B,), np.int32, count)
    st = A.put("status", (B,), np.int32)
    i3 = ctypes.c_int64 * 3
    strides = i3(N * heads * D, heads * D, D)
    a = b.SpecKvAppendArgs(c, N, BF16, A.ptr(k), A.ptr(v), strides, strides, A.ptr(s), A.ptr(n))
    assert lib.spec_kv_append(ctypes.byref(a), A.ptr(st), stream()) == 0
    A.check()
    for view, raw in bufs:
        got = A.host(view, np.uint8, raw.shape)
        for r in range(B):
            mine = np.zeros(slots, bool)
            mine[start[r]:start[r] + count[r]] = True
            assert np.array_equal(got[r][~mine], raw[r][~mine])
            assert np.array_equal(got[r][:, entry:], raw[r][:, entry:])  # the gaps
    out = [A.put(f"out{i}", (B, N, heads, D), np.float32) for i in range(2)]
    a = b.SpecKvReadArgs(c, N, F32, A.ptr(out[0]), A.ptr(out[1]), A.ptr(s), A.ptr(n))
    assert lib.spec_kv_read(ctypes.byref(a), A.ptr(st), stream()) == 0
    A.check()
    assert np.all(A.host(st, np.int32, (B,)) == 0)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("B,N,G,heads,D,P,top,tree", [
    (1, 1, 1, 1, 16, 0, 3, False), (2, 3, 4, 2, 80, 77, 40, False), (40, 2, 4, 2, 128, 300, 200, False),
    (3, 33, 4, 2, 64, 130, 70, True), (90, 1, 2, 4, 128, 129, 300, False), (70, 32, 4, 2, 64, 140, 60, True)])
def test_attention(lib, dtype, B, N, G, heads, D, P, top, tree):
    from speculative_decoding_verification_32_gb300 import _binding as b
    rng = np.random.default_rng(B + N)
    A = Arena()
    lens = rng.integers(0, top + 1, B).astype(np.int32)
    lens[0] = top
    slots = top + N
    c, _, _, _ = cache_of(A, "cache", B, heads, D, dtype, slots, rng, False)
    pc = cache_of(A, "prefix", 1, heads, D, dtype, P, rng, False)[0] if P else b.SpecKvCache()
    H = heads * G
    q = A.put("q", (B, N, H, D), np.uint16, bf16(rng, B, N, H, D))
    ln = A.put("len", (B,), np.int32, lens)
    par = None
    if tree:
        p = np.full((B, N), -1, np.int32)
        for i in range(1, N):
            p[:, i] = rng.integers(max(0, i - 5), i, B)
        par = A.put("parent", (B, N), np.int32, p)
    a = b.SpecAttentionArgs(c, pc, P, N, H, BF16, 0.1, A.ptr(q), (ctypes.c_int64 * 3)(N * H * D, H * D, D), A.ptr(ln),
                            None, A.ptr(par))
    need = lib.spec_prefix_attention_workspace_size(ctypes.byref(a))
    ws = A.put("ws", (need,), np.uint8)
    out, lse, st = A.put("out", (B, N, H, D), np.uint16), A.put("lse", (B, N, H), np.float32), A.put("status", (B,), np.int32)
    assert lib.spec_prefix_attention(ctypes.byref(a), A.ptr(out), A.ptr(lse), A.ptr(st), A.ptr(ws), need, stream()) == 0
    A.check()
    assert np.all(A.host(st, np.int32, (B,)) == 0) and np.all(np.isfinite(A.host(lse, np.float32, (B, N, H))))


@pytest.mark.parametrize("B,npos,V,m,dtype", [(1, 1, 1, 1, BF16), (3, 2, 37, 20, F32), (2, 5, 8193, 64, BF16), (300, 1, 4096, 3, F32),
                                              (1, 1, 128256, 50, BF16)])
def test_logprobs(lib, B, npos, V, m, dtype):
    from speculative_decoding_verification_32_gb300 import _binding as b
    rng = np.random.default_rng(V)
    A = Arena()
    x = rng.standard_normal((B, npos, V)).astype(np.float32)
    lg = A.put("logits", x.shape, np.float32, x) if dtype == F32 else A.put("logits", x.shape, np.uint16, bf16(rng, B, npos, V))
    tok = A.put("tokens", (B, npos), np.int32, rng.integers(-1, V, (B, npos)).astype(np.int32))
    o = [A.put(f"o{i}", (B, npos), np.float32) for i in range(2)]
    ids, tops, st = A.put("ids", (B, npos, m), np.int32), A.put("tops", (B, npos, m), np.float32), A.put("st", (B, npos), np.int32)
    a = b.SpecLogprobsArgs(B, npos, V, dtype, m, 0, V, A.ptr(lg), A.ptr(tok), None)
    out = b.SpecLogprobsOut(A.ptr(o[0]), A.ptr(o[1]), A.ptr(ids), A.ptr(tops), A.ptr(st))
    assert lib.spec_token_logprobs(ctypes.byref(a), ctypes.byref(out), stream()) == 0
    A.check()
    assert np.all(A.host(st, np.int32, (B, npos)) == 0)
