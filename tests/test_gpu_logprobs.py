"""spec_token_logprobs against a plain 64-bit restatement (needs a GB300).

Tolerances.  y = (l - M) log2(e) / T carries three fp32 roundings, at most
3 * 2^-24 |y|; ex2 is within 2^-22 relative and a sum of V terms in chunks of
32 and trees adds at most 2^-19, so log2 S is within 2^-18 absolute, and
  |logprob error| <= 2^-18 + 2^-21 |logprob|.
U / S is a mean of -y over p with the same relative errors, so
  |entropy error| <= 2^-17 (1 + entropy).
Ids are exact: order by logit, ties to the lower id."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def plain(x, tokens, temp, m):
    """x [B, n, V] float64."""
    y = x / temp[:, None, None]
    M = y.max(-1, keepdims=True)
    lse = M + np.log(np.exp(y - M).sum(-1, keepdims=True))
    lp = y - lse
    p = np.exp(lp)
    ent = -np.where(p > 0, p * np.where(p > 0, lp, 0), 0).sum(-1)
    V = x.shape[-1]
    ids = np.lexsort((np.broadcast_to(np.arange(V), x.shape), -x), axis=-1)[..., :m]
    tops = np.take_along_axis(lp, ids, -1)
    given = np.take_along_axis(lp, np.clip(tokens, 0, None)[..., None].astype(np.int64), -1)[..., 0]
    return given, ent, ids, tops


def close(got, want, atol, rtol):
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)  # what fp32 can hold: past its range, -inf
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf])
    got, want = got[~inf], want[~inf]
    assert np.all(np.abs(got - want) <= atol + rtol * np.abs(want)), np.max(np.abs(got - want))


def check(sv, x, tokens, temp, m, used=None):
    """x: a CUDA tensor [B, n, V]."""
    import torch
    g = sv.spec_token_logprobs(x, torch.from_numpy(tokens).cuda(),
                               None if temp is None else torch.from_numpy(temp).cuda(), m=m)
    g = {k: v.cpu().numpy() for k, v in g.items()}
    t = np.ones(x.shape[0], np.float32) if temp is None else temp
    given, ent, ids, tops = plain(x.double().cpu().numpy(), tokens, t.astype(np.float64), m)
    on = tokens >= 0
    assert np.all(g["status"] == 0)
    close(g["logprob"][on], given[on], 2.0**-18, 2.0**-21)
    close(g["entropy"][on], ent[on], 2.0**-17, 2.0**-17)
    assert np.array_equal(g["top_ids"][on], ids[on])
    close(g["top_logprobs"][on], tops[on], 2.0**-18, 2.0**-21)
    for k in ("logprob", "entropy", "top_logprobs"):
        assert np.all(np.isnan(g[k][~on]))
    assert np.all(g["top_ids"][~on] == -1)
    return g


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,n,V,m", [(1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 37, 20), (3, 1, 257, 0), (5, 2, 4096, 1),
                                     (2, 2, 8192, 64), (2, 1, 8193, 33), (4, 6, 32000, 20), (1, 2, 128256, 50),
                                     (1, 1, 262144, 64)])
def test_against_plain(sv, dtype, B, n, V, m):
    import torch
    g = torch.Generator().manual_seed(V + m)
    x = (3 * torch.randn(B, n, V, generator=g)).to(getattr(torch, dtype)).cuda()
    rng = np.random.default_rng(V)
    tokens = rng.integers(0, V, (B, n)).astype(np.int32)
    tokens[rng.random((B, n)) < 0.3] = -1
    tokens[0, 0] = V - 1
    check(sv, x, tokens, (0.3 + rng.random(B)).astype(np.float32), m)
    check(sv, x, tokens, None, m)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [50, 5000, 40001])
def test_ties_masks_and_flat_rows(sv, dtype, V):
    """Masses of equal logits (the whole-position search), -inf masks with
    fewer finite logits than alternatives, the type's lowest value, zeros of
    both signs, a one-hot law."""
    import torch
    dt = getattr(torch, dtype)
    m = min(40, V)
    x = torch.randn(8, 1, V, generator=torch.Generator().manual_seed(V))
    x[0] = 1.25                                   # all equal
    x[1] = x[1].clamp_max(0.5)                    # a plateau on top
    x[2] = float("-inf")
    x[2, 0, 3::11] = 0.25                         # masked, ties among the rest
    x[3] = float("-inf")
    x[3, 0, V - 1] = -4.0                         # one finite logit
    x[4] = torch.finfo(dt).min
    x[4, 0, 7] = 1.0                              # masked with the lowest value
    x[5, 0, ::2] = 0.0
    x[5, 0, 1::2] = -0.0                          # signed zeros are equal
    x[6, 0, 11] = 80.0                            # one token has it all
    x[7] = torch.round(x[7] * 4) / 4              # coarse: ties everywhere
    x = x.to(dt).cuda()
    tokens = np.full((8, 1), 0, np.int32)
    tokens[3], tokens[6] = V - 1, 11
    g = check(sv, x, tokens, np.full(8, 0.7, np.float32), m)
    assert g["entropy"][3, 0] == 0.0 and g["logprob"][3, 0] == 0.0
    assert abs(g["entropy"][0, 0] - np.log(V)) < 1e-4


def test_flags(sv):
    """NaN, +inf, no finite logit, a bad token or temperature: the position
    is flagged, the others are not."""
    import torch
    V, m = 9000, 4
    x = torch.randn(5, 3, V, generator=torch.Generator().manual_seed(3))
    x[0, 1, 8999] = float("nan")
    x[1, 2, 0] = float("inf")
    x[2, 0] = float("-inf")
    tokens = torch.zeros(5, 3, dtype=torch.int32)
    tokens[2, 1], tokens[2, 2] = V, -2
    tokens[0, 2] = -1
    temp = torch.tensor([1.0, 2.0, 0.5, 0.0, float("nan")])
    want = [[0, 1, 0], [0, 0, 1], [5, 2, 2], [7] * 3, [7] * 3]
    for dt in (torch.bfloat16, torch.float32):
        g = sv.spec_token_logprobs(x.to(dt).cuda(), tokens.cuda(), temp.cuda(), m=m)
        assert g["status"].tolist() == want
        bad = torch.tensor(want) != 0
        bad[0, 2] = True  # skipped
        for k in ("logprob", "entropy", "top_logprobs"):
            nan = torch.isnan(g[k].cpu())
            assert torch.equal(nan.view(5, 3, -1).any(-1), bad) and torch.equal(nan.view(5, 3, -1).all(-1), bad)
        assert torch.equal((g["top_ids"].cpu() == -1).all(-1), bad)


def test_strided_positions_and_no_tokens(sv):
    import torch
    B, n, V = 3, 4, 1000
    for pad in (8, 3):  # 16-byte rows and odd ones
        wide = torch.randn(B, n, V + pad, generator=torch.Generator().manual_seed(1)).cuda()
        wide[..., V:] = float("nan")
        x = wide[..., :V]
        tokens = np.tile(np.arange(n, dtype=np.int32), (B, 1))
        a = check(sv, x, tokens, None, 7)
        b = sv.spec_token_logprobs(x, m=7)
        assert "logprob" not in b and np.array_equal(b["top_ids"].cpu().numpy(), a["top_ids"])
        assert np.array_equal(b["entropy"].cpu().numpy(), a["entropy"])


def test_verified_tokens_in_a_graph_and_on_a_stream(sv):
    """The emitted tokens of a verify step, as they come (with its -1 filler)."""
    import torch
    from workloads import synthetic as S
    from tests.gpu_util import cuda
    inp = S.make("c2")
    t = [cuda(inp[k]) for k in ("target", "draft", "draft_tokens", "temperature", "u_accept", "u_sample")]
    out = sv.spec_verify_chain(*t)
    tokens = out["out_tokens"].cpu().numpy()
    assert (tokens == -1).any()
    a = check(sv, t[0], tokens, t[3].cpu().numpy(), 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = sv.spec_token_logprobs(t[0], out["out_tokens"], t[3], m=5, stream=s)
    s.synchronize()
    for k in a:
        np.testing.assert_array_equal(a[k], b[k].cpu().numpy())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = sv.spec_token_logprobs(t[0], out["out_tokens"], t[3], m=5)
    out["out_tokens"].clamp_min_(3)
    graph.replay()
    torch.cuda.synchronize()
    on = tokens >= 3
    np.testing.assert_array_equal(c["logprob"].cpu().numpy()[on], a["logprob"][on])
    assert not torch.isnan(c["logprob"]).any()
