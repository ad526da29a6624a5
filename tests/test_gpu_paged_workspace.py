"""spec_paged_attention in a workspace of just the bytes that it asks for, with a mark behind them (needs a
GB300): the parts of rows cut by a budget lie side by side in it."""
import numpy as np
import pytest

from tests.test_gpu_paged_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
@pytest.mark.parametrize("B,N,Hq,H,D,window", [
    (64, 8, 32, 8, 128, 0), (64, 6, 32, 8, 128, 500), (128, 8, 32, 8, 64, 0), (1, 1, 8, 8, 128, 0), (3, 5, 24, 4, 80, 100),
    (100, 1, 40, 20, 64, 0), (127, 3, 10, 2, 48, 200), (150, 2, 8, 2, 64, 0), (2, 130, 8, 2, 64, 0)])
def test_the_bytes_asked_for(kind, B, N, Hq, H, D, window, monkeypatch):
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    from speculative_decoding_verification_32_gb300 import _binding
    rng = np.random.default_rng(B + N)
    lens = rng.integers(0, 900, B)
    lens[B // 2] = 3000  # one long row
    made = []

    def scratch(dev, key, nbytes):
        buf = torch.full((nbytes + 4096,), 0xA5, dtype=torch.uint8, device=dev)
        made.append((buf, nbytes))
        return buf[:nbytes]
    monkeypatch.setattr(_binding, "_scratch", scratch)
    monkeypatch.setattr(_binding, "_ws", {})
    p = Problem(sv, B, N, Hq, H, D, lens, 16, window, 4, kind)
    made.clear()
    p.check(rows=[0, B // 2, B - 1])
    assert len(made) == 1
    buf, nbytes = made[0]
    assert (buf[nbytes:] == 0xA5).all()
