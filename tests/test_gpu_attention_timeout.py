"""Attention whose waits run out in one KV head: a bounded wait that nothing ends, as everywhere in
these tests (needs a GB300)."""
import numpy as np
import pytest

from tests.test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
@pytest.mark.parametrize("B,N,H,D,P,tree,direct", [
    (80, 32, 2, 64, 256, True, True),     # no join: the kernel writes the answers itself
    (100, 16, 2, 64, 0, False, True),     # chains, likewise
    (2, 60, 2, 64, 300, True, False),     # cut into parts
    (24, 2, 2, 128, 300, False, False),   # the prefix alone on the tile kernel
])
def test_one_head_gives_up(kind, B, N, H, D, P, tree, direct):
    """Every row with a query is flagged, whichever CTA of it was done first; the head that gave up
    gets nothing and the other its answers; bad rows stay what they are."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    rng = np.random.default_rng(B)
    count = rng.integers(0, N + 1, B)
    count[:2] = N
    p = Problem(sv, B, N, 8, H, D, P, rng.integers(0, 100, B), kind, "bfloat16", tree, count=count, seed=B)
    p.lens[1] = -1
    out0, lse0, st0 = p.call()
    bad = torch.zeros(B, dtype=torch.int32)
    bad[1] = 8
    assert torch.equal(st0.cpu(), bad)
    limit = sv.get_wait_timeout_ns()
    want = torch.where(torch.from_numpy(count > 0) & (bad == 0), 6, bad)
    try:
        sv.set_wait_timeout_ns(2_000_000)
        for g in range(H):
            sv.debug_force_wait_timeout(2 + g)
            out, lse, st = p.call()
            torch.cuda.synchronize()
            gone = slice(g * 8 // H, (g + 1) * 8 // H)
            assert torch.equal(st.cpu(), want)
            assert float(out[:, :, gone].abs().max()) == 0.0 and bool((lse[:, :, gone] == float("-inf")).all())
            kept = slice(8 // H * (1 - g), 8 // H * (2 - g))
            assert torch.equal(out[:, :, kept], out0[:, :, kept]) and torch.equal(lse[:, :, kept], lse0[:, :, kept])
    finally:
        sv.debug_force_wait_timeout(False)
        sv.set_wait_timeout_ns(limit)
    out, lse, st = p.call()
    assert torch.equal(st.cpu(), bad) and torch.equal(out, out0) and torch.equal(lse, lse0)


def test_statuses_of_chains_without_a_join():
    """The same calls with and without parents of a chain: one status each, no answer apart."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    p = Problem(sv, 100, 16, 8, 2, 64, 0, np.arange(100), "uint8", "bfloat16", count=np.arange(100) % 17, seed=3)
    p.lens[7], p.count[8] = p.S, 17
    out, lse, st = p.call()
    want = torch.zeros(100, dtype=torch.int32)
    want[[7, 8]] = 8
    assert torch.equal(st.cpu(), want)
    p.parent = np.tile(np.arange(-1, 15, dtype=np.int32), (100, 1))
    a, b, c = p.call()
    assert torch.equal(a, out) and torch.equal(b, lse) and torch.equal(c, st)
