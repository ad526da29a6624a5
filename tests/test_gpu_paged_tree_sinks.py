"""spec_paged_attention over trees whose own tokens are sinks (needs a GB300): a node's slot is not its position,
so a sink by its depth may lie in a slot far behind the first ones, before what its descendants' windows
reach."""
import numpy as np
import pytest

from tests.test_gpu_paged_attention import KINDS, Problem, i32, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,qt", KINDS)
@pytest.mark.parametrize("B", [1, 3, 150])
@pytest.mark.parametrize("n,sinks,window,spare", [(0, 4, 1, 2), (0, 4, 1, 400), (2, 6, 3, 2), (1, 20, 2, 30)])
def test_values_of_sinks_among_the_tree(kind, qt, B, n, sinks, window, spare):
    """20 children of the root and a chain of 39 nodes from the last of them: what is no number in a child's
    value reaches the nodes of the chain, in whose windows it is not."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    N, D = 60, 64
    parent = np.array([-1] + [0] * 20 + list(range(20, 59)), np.int32)
    p = Problem(sv, B, N, 4, 2, D, [n] * B, 16, window, sinks, kind, qt, spare=spare)
    p.parent = np.tile(parent, (B, 1))
    p.see = [visible(n, N, window, sinks, parent)] * B
    for b in range(B):  # (the chain that the problem was made for has not needed all pages)
        p.table[b] = np.arange(p.table.shape[1]) + b * p.table.shape[1]
    p.cache.fill_(0)
    g = torch.Generator(device="cuda").manual_seed(1)
    line = torch.zeros(2, B, n + N, *p.cache.shape[3:], dtype=p.cache.dtype, device="cuda")
    k, v = (torch.randn(B, n + N, 2, D, generator=g, device="cuda") for _ in range(2))
    sv.spec_kv_append(line, k, v, i32(np.zeros(B)))
    for b in range(B):
        for t in range(n + N):
            p.cache[:, p.table[b, t // 16], t % 16] = line[:, b, t]
    p.dt = i32(p.table)
    clean = p.run()
    assert not clean[2].any() and torch.isfinite(clean[0]).all()
    b, t = B // 2, n + 20
    sees = p.see[b][:, t]
    assert sees[20:].all() and not sees[:20].any()  # position n + 1 is a sink
    page = p.table[b, t // 16]
    if kind == "uint8":
        p.cache[1, page, t % 16, 2 * D] = 255  # head 0: no scale
        p.cache[1, page, t % 16, D + 5] = 0x7f  # head 1: one code
    else:
        p.cache[1, page, t % 16, 0, 3] = float("nan")
        p.cache[1, page, t % 16, 1, 5] = float("-inf")
    out, lse, status = p.run()
    assert not status.any() and torch.equal(lse, clean[1])
    want = clean[0].clone()
    if kind == "uint8":
        want[b, 20:, :2] = float("nan")
        want[b, 20:, 2:, 5] = float("nan")
    else:
        want[b, 20:, :2, 3] = float("nan")
        want[b, 20:, 2:, 5] = float("-inf")
    assert torch.equal(out.nan_to_num(nan=7e4), want.nan_to_num(nan=7e4))
