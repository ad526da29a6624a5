"""Refusals of the paged-cache and sampling entry points: every bad argument is turned down on the
host, before anything is launched (runs without a GPU)."""
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


def plan(L, B=3, N=4, columns=10, page=16, pages=50, window=0, sinks=0, table=P, free=P, ring=P, kv_len=P, count=None,
         slots=P, status=P, ws=P, ws_bytes=1 << 30):
    from speculative_decoding_verification_32_gb300._binding import SpecPagePlanArgs
    a = SpecPagePlanArgs(B, N, columns, page, pages, window, sinks, 0, ptr(table), ptr(free), ptr(ring), ptr(kv_len), ptr(count))
    return L.spec_page_plan(ctypes.byref(a), ptr(slots), ptr(status), ptr(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(B=(1 << 20) + 1), SHAPE), (dict(N=-1), SHAPE), (dict(columns=0), SHAPE), (dict(page=8), SHAPE),
    (dict(page=24), SHAPE), (dict(page=2048), SHAPE), (dict(pages=-1), SHAPE), (dict(columns=1 << 27), SHAPE),
    (dict(pages=1 << 27), SHAPE), (dict(B=1 << 16, N=1 << 15), SHAPE), (dict(B=1 << 16, columns=1 << 15), SHAPE),
    (dict(window=-1), ARG), (dict(sinks=-1), ARG), (dict(table=P + 2), ALIGN), (dict(kv_len=P + 1), ALIGN), (dict(count=P + 2), ALIGN),
    (dict(slots=P + 1), ALIGN), (dict(status=P + 3), ALIGN), (dict(ring=P + 2), ALIGN), (dict(free=P + 2), ALIGN),
    (dict(table=0), NULL), (dict(ring=0), NULL), (dict(free=0), NULL), (dict(kv_len=0), NULL), (dict(slots=0), NULL),
    (dict(ws=0), WORKSPACE), (dict(ws=P + 16), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(B=0), OK),
    (dict(B=0, table=0, free=0, ring=0, kv_len=0, slots=0, ws=0), OK)])
def test_plan_refusals(L, kw, want):
    assert plan(L, **kw) == want


def test_plan_workspace_size(L):
    f = L.spec_page_plan_workspace_size
    assert f(-1) == 0 and f((1 << 20) + 1) == 0
    assert f(1) >= 16 and f(1000) >= 8000 and f(1000) % 256 == 0
    assert L.spec_page_plan(None, None, None, None, 0, None) == NULL


def compact(L, B=3, N=4, planes=2, columns=10, page=16, pages=50, E=32, ps=1600, gs=512, ts=32, kv=P, table=P, kv_len=P, acc=P, path=P,
            status=P):
    from speculative_decoding_verification_32_gb300._binding import SpecPageCompactArgs
    a = SpecPageCompactArgs(B, N, planes, columns, page, pages, E, ps, gs, ts, ptr(kv), ptr(table), ptr(kv_len), ptr(acc), ptr(path))
    return L.spec_kv_compact_pages(ctypes.byref(a), ptr(status), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(planes=65536), SHAPE), (dict(planes=-1), SHAPE), (dict(N=0), SHAPE),
    (dict(N=1025), SHAPE), (dict(columns=0), SHAPE), (dict(page=17), SHAPE), (dict(pages=-1), SHAPE), (dict(E=-16), SHAPE),
    (dict(E=1 << 31), SHAPE), (dict(ps=-16), SHAPE), (dict(gs=-16), SHAPE), (dict(ts=-16), SHAPE), (dict(pages=1 << 27), SHAPE),
    (dict(kv=P + 8), ALIGN), (dict(E=24), ALIGN), (dict(ps=8), ALIGN), (dict(gs=8), ALIGN), (dict(ts=8), ALIGN),
    (dict(table=P + 2), ALIGN), (dict(path=P + 1), ALIGN), (dict(status=P + 2), ALIGN),
    (dict(table=0), NULL), (dict(kv_len=0), NULL), (dict(acc=0), NULL), (dict(path=0), NULL), (dict(kv=0), NULL),
    (dict(B=0), OK), (dict(B=0, kv=0, table=0, kv_len=0, acc=0, path=0), OK)])
def test_compact_refusals(L, kw, want):
    assert compact(L, **kw) == want
    assert L.spec_kv_compact_pages(None, None, None) == NULL


def attention(L, B=2, N=3, q_heads=16, heads=8, head_dim=128, q_dtype=BF16, cache_dtype=E4M3, columns=10, page=16, pages=50,
              window=0, sinks=0, scale=0.1, gs=16 * 1040, ts=1040, qs=(6000, 2000, 128), k=P, v=P, q=P, table=P, kv_len=P, count=None,
              parent=None, out=P, lse=P, status=P, ws=P, ws_bytes=1 << 40):
    from speculative_decoding_verification_32_gb300._binding import SpecPagedAttentionArgs
    a = SpecPagedAttentionArgs(B, N, q_heads, heads, head_dim, q_dtype, cache_dtype, columns, page, pages, window, sinks, scale, 0,
                               gs, ts, (ctypes.c_int64 * 3)(*qs), ptr(k), ptr(v), ptr(q), ptr(table), ptr(kv_len), ptr(count),
                               ptr(parent))
    return L.spec_paged_attention(ctypes.byref(a), ptr(out), ptr(lse), ptr(status), ptr(ws), ws_bytes, None), a


@pytest.mark.parametrize("kw,want", [
    (dict(q_dtype=F32), DTYPE), (dict(q_dtype=E4M3), DTYPE), (dict(cache_dtype=F16, ts=2048), DTYPE), (dict(cache_dtype=F32), DTYPE),
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(N=-1), SHAPE), (dict(q_heads=12), SHAPE), (dict(q_heads=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(head_dim=72), SHAPE), (dict(head_dim=144), SHAPE), (dict(columns=0), SHAPE), (dict(page=8), SHAPE),
    (dict(page=40), SHAPE), (dict(pages=-1), SHAPE), (dict(columns=1 << 27), SHAPE), (dict(pages=1 << 27), SHAPE),
    (dict(N=1025, parent=P), SHAPE), (dict(N=1 << 20), SHAPE), (dict(ts=1024), SHAPE), (dict(ts=1 << 27), SHAPE), (dict(gs=-16), SHAPE),
    (dict(qs=(0, -1, 0)), SHAPE), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(window=-1), ARG),
    (dict(sinks=-1), ARG), (dict(k=P + 8), ALIGN), (dict(v=P + 4), ALIGN), (dict(gs=1000), ALIGN), (dict(ts=1048), ALIGN),
    (dict(q=P + 1), ALIGN), (dict(out=P + 8), ALIGN), (dict(lse=P + 4), ALIGN), (dict(table=P + 2), ALIGN), (dict(kv_len=P + 2), ALIGN),
    (dict(parent=P + 2), ALIGN), (dict(count=P + 1), ALIGN), (dict(q=0), NULL), (dict(out=0), NULL), (dict(kv_len=0), NULL),
    (dict(table=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(ws=0), WORKSPACE), (dict(ws=P + 16), WORKSPACE),
    (dict(ws_bytes=256), WORKSPACE), (dict(B=0), OK), (dict(N=0), OK)])
def test_attention_refusals(L, kw, want):
    assert attention(L, **kw)[0] == want


def test_attention_workspace_size(L):
    """Sizes only: pointers may be anything; more queries or heads need more."""
    def size(**kw):
        return L.spec_paged_attention_workspace_size(ctypes.byref(attention(L, ws=0, **kw)[1]))
    assert size() > 0 and size(N=6) > size() and size(q_heads=32) > size()
    assert size(q_dtype=F32) == 0 and size(N=1025, parent=P) == 0 and size(window=-1) == 0
    assert L.spec_paged_attention_workspace_size(None) == 0


def sample(L, B=2, V=1000, dtype=BF16, pitch=None, logits=P, u=P, temperature=None, top_k=None, top_p=None, min_p=None, token=P, prob=P,
           status=P):
    from speculative_decoding_verification_32_gb300._binding import SpecSampleArgs, SpecSampleOut
    a = SpecSampleArgs(B, V, dtype, 0, V if pitch is None else pitch, ptr(logits), ptr(u), ptr(temperature), ptr(top_k), ptr(top_p),
                       ptr(min_p))
    o = SpecSampleOut(ptr(token), ptr(prob), ptr(status))
    return L.spec_sample(ctypes.byref(a), ctypes.byref(o), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(B=1 << 25), SHAPE), (dict(V=0), SHAPE), (dict(V=262145), SHAPE), (dict(dtype=F16), DTYPE),
    (dict(dtype=E4M3), DTYPE), (dict(pitch=999), ARG), (dict(logits=0), NULL), (dict(u=0), NULL), (dict(token=0), NULL),
    (dict(status=0), NULL), (dict(logits=P + 1), ALIGN), (dict(u=P + 2), ALIGN), (dict(temperature=P + 1), ALIGN),
    (dict(top_k=P + 2), ALIGN), (dict(top_p=P + 2), ALIGN), (dict(min_p=P + 2), ALIGN), (dict(prob=P + 1), ALIGN), (dict(B=0), OK)])
def test_sample_refusals(L, kw, want):
    assert sample(L, **kw) == want
    assert L.spec_sample(None, None, None) == NULL


def test_binding_refusals(L):
    """The Python checks that come before any pointer is taken."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        sv.spec_page_plan(z(4), z(9), z(2), z(1), 3, 16)
    with pytest.raises(TypeError):  # 64-bit lengths
        sv.spec_page_plan(z(2, 4), z(9), z(2), z(2).long(), 3, 16)
    with pytest.raises(ValueError):  # one length too few
        sv.spec_page_plan(z(2, 4), z(9), z(2), z(1), 3, 16)
    with pytest.raises(ValueError):  # a ring's state has two numbers
        sv.spec_page_plan(z(2, 4), z(9), z(3), z(2), 3, 16)
    with pytest.raises(ValueError):  # a view of a wider table
        sv.spec_page_plan(z(2, 8)[:, :4], z(9), z(2), z(2), 3, 16)
    kv = torch.zeros(2, 5, 16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        sv.spec_kv_compact_pages(kv[:, :, ::2], z(2, 4), z(2), z(2), z(2, 3))
    with pytest.raises(ValueError):
        sv.spec_kv_compact_pages(kv, z(2, 4), z(2), z(3), z(2, 3))
    q, c = torch.zeros(2, 3, 8, 64).bfloat16(), torch.zeros(2, 9, 16, 4, 64).bfloat16()
    with pytest.raises(TypeError):
        sv.spec_paged_attention(q.float(), c, z(2, 4), z(2))
    with pytest.raises(ValueError):  # another head size
        sv.spec_paged_attention(q, c[..., :48], z(2, 4), z(2))
    with pytest.raises(ValueError):  # heads unknown
        sv.spec_paged_attention(q, torch.zeros(2, 9, 16, 272, dtype=torch.uint8), z(2, 4), z(2))
    with pytest.raises(ValueError):  # rows
        sv.spec_paged_attention(q, c, z(3, 4), z(2))
    with pytest.raises(ValueError):
        sv.spec_paged_attention(q, c, z(2, 4), z(2), parent=z(2, 4))
    with pytest.raises(ValueError):
        sv.spec_sample(torch.zeros(3, 5, 7), torch.zeros(3))
    with pytest.raises(TypeError):
        sv.spec_sample(torch.zeros(3, 5).half(), torch.zeros(3))
    with pytest.raises(TypeError):
        sv.spec_sample(torch.zeros(3, 5), torch.zeros(3).double())
    with pytest.raises(ValueError):
        sv.spec_sample(torch.zeros(3, 5), torch.zeros(3), top_k=z(4))
    with pytest.raises(ValueError):
        sv.spec_sample(torch.zeros(5, 3).T, torch.zeros(3))


@pytest.mark.parametrize("call", [
    lambda sv, t, z: sv.spec_page_plan(z(2, 4), z(9), z(2), z(2), 3, 16),
    lambda sv, t, z: sv.spec_kv_compact_pages(t.zeros(2, 5, 16, 32, dtype=t.uint8), z(2, 4), z(2), z(2), z(2, 3)),
    lambda sv, t, z: sv.spec_paged_attention(t.zeros(2, 3, 8, 64).bfloat16(), t.zeros(2, 9, 16, 4, 64).bfloat16(), z(2, 4), z(2)),
    lambda sv, t, z: sv.spec_sample(t.zeros(3, 5), t.zeros(3))])
def test_host_tensors_are_refused(L, call):
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(sv, torch, lambda *s: torch.zeros(*s, dtype=torch.int32))
