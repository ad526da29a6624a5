"""Attention over caches whose entries are extreme: value vectors that are NaN (needs a GB300).  The plain restatement and its
tolerances are those of test_gpu_attention.py."""
import numpy as np
import pytest

from tests.test_gpu_attention import Problem, seen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def lse_bound(p, b, lse):
    """Twice the bound of one lse of row b (two of them are compared): a score is a sum of D products
    in fp32, |q . k| at most |q| |k|; see test_gpu_attention.py."""
    keys = [p.kx[b]] + ([p.pk] if p.P else [])
    size = p.scale * np.linalg.norm(p.qx[b], axis=-1).max() * max(np.nanmax(np.linalg.norm(k, axis=-1)) for k in keys)
    return 2 * (2.0**-23 * (p.D + 8) * size + 2.0**-20 + 2.0**-23 * (p.P + p.S) + 2.0**-20 * lse.abs())


@pytest.mark.parametrize("qt", ["bfloat16", "float16"])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("B,N,G,D,P,tree", [(2, 1, 4, 64, 40, False), (2, 5, 4, 128, 40, False), (1, 6, 2, 80, 0, False),
                                           (40, 2, 4, 64, 300, False), (2, 50, 4, 64, 40, True)])
def test_a_nan_value_vector_is_no_matter_for_lse(sv, qt, zeros, B, N, G, D, P, tree):
    """A value vector whose scale byte stands for NaN makes NaN of what its head's queries get, as far
    as they see it, and nothing else: lse comes from the keys."""
    import torch
    H = 2
    p = Problem(sv, B, N, G * H, H, D, P, [30] * B, "uint8", qt, tree, seed=B + N)
    out0, lse0 = p.check(rows=[0])
    whole = torch.ones(N, dtype=torch.bool)
    own = max(0, N - 2)
    sees = torch.from_numpy(seen(N, None if p.parent is None else p.parent[0])[:, own])
    for where in ("own", "history") + (("prefix",) if P else ()):
        buf, row, slot = (p.prefix, 0, 7) if where == "prefix" else (p.cache, 0, 30 + own if where == "own" else 11)
        keep = buf[1, row, slot].clone()
        buf[1, row, slot, H * D + 1] = 255
        if zeros:  # as the append leaves it; else codes of another writer
            buf[1, row, slot, D:2 * D] = 0
        out, lse, st = p.call()
        buf[1, row, slot].copy_(keep)
        assert st.tolist() == [0] * B
        for b in range(B):
            hit = sees if where == "own" else whole
            if where != "prefix" and b > 0:
                hit = torch.zeros(N, dtype=torch.bool)
            hit = hit.cuda()
            assert torch.equal(out[b, :, :G], out0[b, :, :G]) and torch.equal(lse[b, :, :G], lse0[b, :, :G])
            assert torch.equal(out[b, ~hit, G:], out0[b, ~hit, G:])
            assert bool(torch.isnan(out[b, hit, G:]).all())
            assert bool(((lse[b] - lse0[b]).abs().double() <= lse_bound(p, b, lse0[b].double())).all()), where
