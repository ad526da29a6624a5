"""How few rows are cut into parts by a budget (cut_groups in paged_attention.cu), restated in its own 32-bit
arithmetic: within the lengths for which the call uses it there are never more parts than the budget, nor
more than 32 of a row, and the longer ones go another way (runs without a GPU)."""
import ctypes

import numpy as np
import pytest

from tests.test_pages_sample_host import E4M3, L, attention  # noqa: F401

U = np.uint64(0xffffffff)


def cut(w, budget, splits, rows=128):
    """Parts of each row of w groups, as the kernel's lanes find them (32-bit unsigned, fp32 reciprocals)."""
    w = np.asarray(w, np.uint64)
    B = len(w)
    total, top = w.sum() & U, w.max()
    least = max((int(top) + splits - 1) // splits, 1)
    most = int(total) // (budget - B) + 1
    c = int(total) // budget + 1
    while True:
        c = max(min(c, most), least)
        inv = np.float32(1) / np.float32(c)
        q = (w.astype(np.float32) * inv).astype(np.uint64)
        q = np.where((q * np.uint64(c) & U) >= ((w + np.uint64(c)) & U), q - np.uint64(1), q) & U
        n = np.maximum(1, q + ((q * np.uint64(c) & U) < w))
        if c >= most or n.sum() <= budget:
            return n, c
        c += c // 16 + 1


@pytest.mark.parametrize("top", [40, 3000, 1 << 20, 1 << 24])
@pytest.mark.parametrize("B,budget", [(1, 152), (3, 228), (64, 152), (127, 152), (128, 152), (128, 1824), (100, 2432)])
def test_parts_fit(B, budget, top):
    rng = np.random.default_rng(B + top)
    splits = min(32, budget - B + 1)
    for spread in ("all", "log", "one", "same"):
        for _ in range(3):
            w = {"all": rng.integers(0, top + 1, B), "log": np.exp(rng.uniform(0, np.log(top), B)).astype(np.int64),
                 "one": np.where(np.arange(B) == B // 2, top, 1), "same": np.full(B, top)}[spread]
            n, c = cut(w, budget, splits)
            assert n.sum() <= budget and n.max() <= splits
            assert np.array_equal(n, np.maximum(1, -(-w // c)))


def test_longer_rows_would_not():
    """Beyond it the sum over the rows wraps around, and there are more parts than run."""
    n, _ = cut(np.full(128, 1 << 25), 152, 25)
    assert n.sum() > 152


def test_longer_rows_go_another_way(L):  # noqa: F811
    """Their parts are equal shares of a row: so many as there are to be, times the answers."""
    def size(**kw):
        kw = dict(dict(B=128, N=8, q_heads=32, heads=8, head_dim=128, cache_dtype=E4M3, page=1024, ts=1040, gs=1024 * 1040), **kw)
        return L.spec_paged_attention_workspace_size(ctypes.byref(attention(L, ws=0, **kw)[1]))
    short, long = size(columns=(1 << 18) - 4), size(columns=1 << 18)
    assert short <= 152 * 8 * (32 * (4 * 128 + 8) + 4) + 8 * 128 + 8 * 256
    assert long >= 3 * 128 * 8 * 32 * (4 * 128 + 8)  # 2432 parts of a warp over 128 rows of 8 heads
    # a window that keeps what is seen short
    assert size(columns=1 << 18, window=4096, sinks=4) == size(columns=1 << 12, window=4096, sinks=4)
    assert size(columns=(1 << 21) - 4, window=1 << 29) == size(columns=(1 << 21) - 4)
