"""What spec_paged_attention asks for: no more than its parts can write (runs without a GPU)."""
import ctypes

import pytest

from tests.test_pages_sample_host import BF16, E4M3, F16, L, attention  # noqa: F401

SMS, WARPS = 152, 16  # parts run side by side: at most 16 of the smallest on an SM


def size(L, **kw):  # noqa: F811
    return L.spec_paged_attention_workspace_size(ctypes.byref(attention(L, ws=0, **kw)[1]))


@pytest.mark.parametrize("B", [1, 2, 17, 64, 128])
@pytest.mark.parametrize("N,q_heads,heads", [(1, 8, 8), (1, 32, 8), (8, 32, 8), (6, 32, 8), (5, 24, 4), (16, 2, 1), (3, 40, 20)])
@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("cache_dtype", [E4M3, BF16])
@pytest.mark.parametrize("window", [0, 2048])
def test_few_rows_of_queries(L, B, N, q_heads, heads, head_dim, cache_dtype, window):  # noqa: F811
    """A few sequences are cut into parts that run side by side, each of a block of query rows of one KV head:
    partial sums in fp32, two numbers a row, a word a part; and at most 32 parts of a sequence."""
    entry = L.spec_kv_entry_bytes(heads, head_dim, cache_dtype)
    got = size(L, B=B, N=N, q_heads=q_heads, heads=heads, head_dim=head_dim, cache_dtype=cache_dtype, columns=4096, page=16, ts=entry,
               gs=16 * entry, window=window)
    rows = -(-N * q_heads // heads // 8) * 8
    assert rows <= 32
    parts = min(SMS * WARPS, B * 32 * heads)
    assert 0 < got <= parts * (rows * (4 * head_dim + 8) + 4) + 8 * B + 8 * 256


@pytest.mark.parametrize("N,parent", [(40, None), (60, 1 << 28)])
def test_many_rows_of_queries(L, N, parent):  # noqa: F811
    """As before for the others: at most 32 parts, each as large as the answers in fp32."""
    got = size(L, B=3, N=N, parent=parent, cache_dtype=F16, q_dtype=F16, ts=2048, gs=16 * 2048, columns=4096)
    assert 0 < got <= 32 * 3 * N * 16 * (4 * 128 + 8) + 3 * N * (4 * 2 + 4) + 32 * 3 * 8 * 4 + 8 * 256 + 3 * 8
