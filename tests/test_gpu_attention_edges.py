"""Attention over caches whose entries are extreme: value vectors that are NaN, scales of
tokens that carry no weight, no slots at all (needs a GB300).  The plain restatement and its tolerances are those of
test_gpu_attention.py."""
import ctypes

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


@pytest.mark.parametrize("qt", ["bfloat16", "float16"])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("up", [3, 5, 9, 12, 15])
@pytest.mark.parametrize("B,N,G,D,P,tree", [
    (16, 2, 4, 128, 5000, False),   # the prefix alone, unconverted
    (40, 3, 4, 64, 5000, False),    # the prefix alone, converted
    (2, 60, 4, 128, 5000, True),    # prefix and own entries in one item
    (1, 50, 4, 64, 0, True),        # own entries
    (1, 5, 4, 64, 3000, False),     # few query rows
])
def test_scales_of_tokens_without_weight(sv, qt, up, sink, B, N, G, D, P, tree):
    """Tokens of no weight whose values lie 2^up above the others' or (sink) a token of zeros that has 2^13.7
    times any other's weight: thousands of tokens 2^-11 below the largest weight behind them count all the same."""
    import torch
    H = 16  # enough that a part is many blocks long
    own = 4000 if P == 0 else 40
    p = Problem(sv, B, N, G * H, H, D, P, [own] * B, "uint8", qt, tree, seed=up)
    p.q = torch.ones_like(p.q)
    p.qx = p.q.cpu().double().numpy()
    rng = np.random.default_rng(up)
    unit = 1.0 / (D * p.scale)

    def keys(shape):
        """[..., H, D] of constant vectors: scores 0, or -4 to -8.5 in nats."""
        s = rng.choice([-4.0, -6.5, -7.75, -8.5], shape)
        s[..., 3::600] = 0.0
        return np.broadcast_to((s * unit)[..., None, None], shape + (H, D)).copy()

    k, v = keys((B, own + N)), np.abs(p.vx[:, :own + N])
    pk, pv = (keys((1, P)), np.abs(p.pv[None])) if P else (None, None)
    for kk, vv in ((pk, pv), (k, v)):
        if kk is None or (kk is k and P):
            continue
        kk[:, 7::600] = -30.0 * unit
        vv[:, 7::600] *= 2.0**up
        if sink:
            kk[:, 9], vv[:, 9] = 9.5 * unit, 0.0
    if tree:  # a token of the pass that few see
        v[:, own + N // 2] *= 2.0**up
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    total = torch.full((B,), own + N, dtype=torch.int32, device="cuda")
    f32 = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    sv.spec_kv_append(p.cache, f32(k), f32(v), zero)
    kx, vx, _ = sv.spec_kv_read(p.cache, total, p.S, heads=H, head_dim=D, dtype=torch.float32)
    p.kx, p.vx = kx.cpu().double().numpy(), vx.cpu().double().numpy()
    if P:
        sv.spec_kv_append(p.prefix, f32(pk), f32(pv), zero[:1])
        kx, vx, _ = sv.spec_kv_read(p.prefix, zero[:1] + P, P, heads=H, head_dim=D, dtype=torch.float32)
        p.pk, p.pv = kx[0].cpu().double().numpy(), vx[0].cpu().double().numpy()
    p.check(rows=[B - 1])


def test_a_cache_without_slots(sv):
    """No slots at all: rows that ask for none are right and empty, others are refused."""
    import torch
    from speculative_decoding_verification_32_gb300 import _binding as b
    L = b.lib()
    for B, H, N in ((64, 8, 1), (64, 8, 20), (3, 2, 2)):
        D, Hq = 64, 2 * H
        q = torch.randn(B, N, Hq, D, device="cuda").bfloat16()
        some = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
        count = torch.arange(B, dtype=torch.int32, device="cuda") % 2
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        c = b.SpecKvCache(B, H, D, b.SPEC_BF16, 0, 0, 0, some.data_ptr(), some.data_ptr())
        a = b.SpecAttentionArgs(c, b.SpecKvCache(), 0, N, Hq, b.SPEC_BF16, 0.1, q.data_ptr(),
                                (ctypes.c_int64 * 3)(N * Hq * D, Hq * D, D), lens.data_ptr(), count.data_ptr(), None)
        need = L.spec_prefix_attention_workspace_size(ctypes.byref(a))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out, lse = torch.full_like(q, 7), torch.full((B, N, Hq), 7.0, device="cuda")
        status = torch.full((B,), 77, dtype=torch.int32, device="cuda")
        assert L.spec_prefix_attention(ctypes.byref(a), out.data_ptr(), lse.data_ptr(), status.data_ptr(), ws.data_ptr(), need,
                                       ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
        assert status.tolist() == [8 * (i % 2) for i in range(B)]
        assert float(out.abs().max()) == 0 and bool((lse == float("-inf")).all())
