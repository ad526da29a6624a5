"""Refusals of the cache and log-probability entry points: every bad argument is
turned down on the host, before anything is launched (runs without a GPU)."""
import ctypes

import pytest

OK, NULL, SHAPE, DTYPE, ALIGN, ARG, CUDA, WORKSPACE = range(8)
F32, BF16, F16, E4M3 = range(4)
P = 0x10000000


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verification_32_gb300 import _binding
    from speculative_decoding_verification_32_gb300 import build as lib_build
    lib_build.build()
    return _binding.lib()


def ptr(a):
    return ctypes.c_void_p(a) if a else None


def cache(rows=2, heads=8, head_dim=128, dtype=E4M3, slots=64, row=64 * 1040, tok=1040, k=P, v=P << 1):
    from speculative_decoding_verification_32_gb300._binding import SpecKvCache
    return SpecKvCache(rows, heads, head_dim, dtype, slots, row, tok, ptr(k), ptr(v))


def test_entry_bytes(L):
    assert L.spec_kv_entry_bytes(8, 128, E4M3) == 1024 + 16
    assert L.spec_kv_entry_bytes(1, 16, E4M3) == 32
    assert L.spec_kv_entry_bytes(17, 64, E4M3) == 17 * 64 + 32
    assert L.spec_kv_entry_bytes(8, 128, BF16) == L.spec_kv_entry_bytes(8, 128, F16) == 2048
    for bad in ((0, 64, BF16), (8, 8, BF16), (8, 72, BF16), (8, 144, BF16), (1025, 64, BF16), (8, 64, F32)):
        assert L.spec_kv_entry_bytes(*bad) == 0, bad


def append(L, c=None, N=3, src=BF16, k=P, v=P, ks=(4096, 1024, 128), kv_len=P, count=None, status=P):
    from speculative_decoding_verification_32_gb300._binding import SpecKvAppendArgs
    i3 = ctypes.c_int64 * 3
    a = SpecKvAppendArgs(c or cache(), N, src, ptr(k), ptr(v), i3(*ks), i3(*ks), ptr(kv_len), ptr(count))
    return L.spec_kv_append(ctypes.byref(a), ptr(status), None)


@pytest.mark.parametrize("kw,want", [
    (dict(src=E4M3), DTYPE), (dict(src=9), DTYPE), (dict(c=dict(dtype=F32)), DTYPE),
    (dict(c=dict(rows=-1)), SHAPE), (dict(c=dict(rows=65536)), SHAPE), (dict(c=dict(head_dim=100)), SHAPE),
    (dict(c=dict(heads=0)), SHAPE), (dict(c=dict(slots=-1)), SHAPE), (dict(c=dict(tok=1024)), SHAPE),
    (dict(N=-1), SHAPE), (dict(N=1 << 30), SHAPE), (dict(ks=(-1, 0, 0)), SHAPE),
    (dict(c=dict(k=P + 8)), ALIGN), (dict(c=dict(row=100)), ALIGN), (dict(c=dict(tok=1048)), ALIGN),
    (dict(k=P + 1), ALIGN), (dict(kv_len=P + 2), ALIGN), (dict(status=P + 2), ALIGN),
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(kv_len=0), NULL), (dict(c=dict(k=0)), NULL),
    (dict(c=dict(rows=0)), OK), (dict(N=0), OK)])
def test_append_refusals(L, kw, want):
    kw = dict(kw)
    if "c" in kw:
        kw["c"] = cache(**kw["c"])
    assert append(L, **kw) == want


def read(L, c=None, T=3, out=BF16, k=P, v=P, start=None, length=P, status=P):
    from speculative_decoding_verification_32_gb300._binding import SpecKvReadArgs
    a = SpecKvReadArgs(c or cache(), T, out, ptr(k), ptr(v), ptr(start), ptr(length))
    return L.spec_kv_read(ctypes.byref(a), ptr(status), None)


@pytest.mark.parametrize("kw,want", [
    (dict(out=E4M3), DTYPE), (dict(c=dict(dtype=7)), DTYPE), (dict(T=-1), SHAPE), (dict(T=1 << 30), SHAPE),
    (dict(c=dict(slots=1 << 31)), SHAPE), (dict(k=P + 8), ALIGN), (dict(length=P + 1), ALIGN),
    (dict(start=P + 1), ALIGN), (dict(k=0), NULL), (dict(length=0), NULL), (dict(c=dict(v=0)), NULL),
    (dict(T=0), OK), (dict(c=dict(rows=0)), OK)])
def test_read_refusals(L, kw, want):
    kw = dict(kw)
    if "c" in kw:
        kw["c"] = cache(**kw["c"])
    assert read(L, **kw) == want


def logprobs(L, B=2, npos=3, V=1000, dtype=BF16, m=5, pitch=None, logits=P, tokens=P, temperature=None,
             logprob=P, entropy=P, ids=P, tops=P, status=P):
    from speculative_decoding_verification_32_gb300._binding import SpecLogprobsArgs, SpecLogprobsOut
    a = SpecLogprobsArgs(B, npos, V, dtype, m, 0, V if pitch is None else pitch, ptr(logits), ptr(tokens),
                         ptr(temperature))
    o = SpecLogprobsOut(ptr(logprob), ptr(entropy), ptr(ids), ptr(tops), ptr(status))
    return L.spec_token_logprobs(ctypes.byref(a), ctypes.byref(o), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(npos=0), SHAPE), (dict(V=0), SHAPE), (dict(V=262145), SHAPE),
    (dict(B=1 << 20, npos=1 << 10), SHAPE), (dict(dtype=F16), DTYPE), (dict(m=-1), ARG), (dict(m=65), ARG),
    (dict(V=4), ARG), (dict(pitch=999), ARG), (dict(logits=0), NULL), (dict(entropy=0), NULL),
    (dict(status=0), NULL), (dict(logprob=0), NULL), (dict(ids=0), NULL), (dict(tops=0), NULL),
    (dict(logits=P + 1), ALIGN), (dict(tokens=P + 2), ALIGN), (dict(temperature=P + 1), ALIGN),
    (dict(tops=P + 1), ALIGN), (dict(B=0), OK)])
def test_logprobs_refusals(L, kw, want):
    assert logprobs(L, **kw) == want


def test_binding_refusals(L):
    """The Python checks that come before any pointer is taken."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    k = torch.zeros(2, 3, 8, 64)
    with pytest.raises(ValueError):
        sv.spec_kv_append(torch.zeros(2, 2, 9, 8, 64), k[0], k, None)
    with pytest.raises(TypeError):  # an fp32 cache
        sv.spec_kv_append(torch.zeros(2, 2, 9, 8, 64), k, k, torch.zeros(2, dtype=torch.int32))
    c = torch.zeros(2, 2, 9, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # another head size
        sv.spec_kv_append(c[..., :48], k, k, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):  # 64-bit lengths
        sv.spec_kv_append(c, k, k, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError):  # one length too few
        sv.spec_kv_append(c, k, k, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        sv.spec_kv_append(c, k, k.double(), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):  # heads unknown
        sv.spec_kv_read(torch.zeros(2, 2, 9, 528, dtype=torch.uint8), None, 3)
    with pytest.raises(ValueError):  # entries of another size
        sv.spec_kv_read(torch.zeros(2, 2, 9, 512, dtype=torch.uint8), None, 3, heads=8, head_dim=64)
    with pytest.raises(ValueError):
        sv.spec_token_logprobs(torch.zeros(3, 5))
    with pytest.raises(TypeError):
        sv.spec_token_logprobs(torch.zeros(3, 5, 7, dtype=torch.float16))
    with pytest.raises(ValueError):
        sv.spec_token_logprobs(torch.zeros(3, 5, 7), torch.zeros(3, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        sv.spec_kv_entry_bytes(8, 100)


def attention(L, c=None, pc=None, P_len=64, N=3, q_heads=16, q_dtype=BF16, scale=0.1, q=P, qs=(6000, 2000, 128),
              kv_len=P, count=None, parent=None, out=P, lse=P, status=P, ws=P, ws_bytes=1 << 40):
    from speculative_decoding_verification_32_gb300._binding import SpecAttentionArgs
    a = SpecAttentionArgs(cache(**(c or {})), cache(**dict(dict(rows=1), **(pc or {}))), P_len, N, q_heads, q_dtype,
                          scale, ptr(q), (ctypes.c_int64 * 3)(*qs), ptr(kv_len), ptr(count), ptr(parent))
    return L.spec_prefix_attention(ctypes.byref(a), ptr(out), ptr(lse), ptr(status), ptr(ws), ws_bytes, None), a


@pytest.mark.parametrize("kw,want", [
    (dict(q_dtype=F32), DTYPE), (dict(q_dtype=E4M3), DTYPE), (dict(c=dict(dtype=F16, tok=2048)), DTYPE),
    (dict(pc=dict(dtype=BF16, tok=2048)), DTYPE), (dict(c=dict(rows=-1)), SHAPE), (dict(pc=dict(rows=0)), SHAPE),
    (dict(P_len=-1), SHAPE), (dict(P_len=65), SHAPE), (dict(pc=dict(heads=4)), SHAPE), (dict(N=-1), SHAPE),
    (dict(N=1025), SHAPE), (dict(q_heads=12), SHAPE), (dict(q_heads=0), SHAPE), (dict(q_heads=8 << 20), SHAPE),
    (dict(c=dict(tok=1 << 27)), SHAPE), (dict(pc=dict(tok=1 << 27)), SHAPE),
    (dict(qs=(0, -1, 0)), SHAPE), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG),
    (dict(c=dict(k=P + 8)), ALIGN), (dict(pc=dict(v=P + 8)), ALIGN), (dict(out=P + 8), ALIGN),
    (dict(q=P + 1), ALIGN), (dict(kv_len=P + 2), ALIGN), (dict(parent=P + 2), ALIGN), (dict(count=P + 1), ALIGN),
    (dict(q=0), NULL), (dict(out=0), NULL), (dict(kv_len=0), NULL), (dict(c=dict(v=0)), NULL),
    (dict(pc=dict(k=0)), NULL), (dict(ws=0), WORKSPACE), (dict(ws=P + 16), WORKSPACE), (dict(ws_bytes=4096), WORKSPACE),
    (dict(c=dict(rows=0)), OK), (dict(N=0), OK)])
def test_attention_refusals(L, kw, want):
    assert attention(L, **kw)[0] == want


def test_attention_workspace_size(L):
    """Sizes only: pointers may be anything; more queries, heads or parts need more."""
    def size(**kw):
        return L.spec_prefix_attention_workspace_size(ctypes.byref(attention(L, **kw)[1]))
    base = size(ws=0)
    assert base >= 2 * 3 * 16 * (128 + 2) * 4 * 2  # two parts at least of 96 output rows
    assert size(ws=0, N=6) > base and size(ws=0, q_heads=32) > base
    assert size(ws=0, q_dtype=F32) == 0 and size(ws=0, N=1025) == 0
    assert L.spec_prefix_attention_workspace_size(None) == 0
