"""spec_sample against a plain 64-bit restatement (needs a GB300).

The kernel's weights are 2^-y with y = (M - l) log2(e) / T: three roundings of y (3 y 2^-24, of the
weight 3 y ln 2 2^-24) and a hardware power of two (2^-22 by its specification); its sums are exact but
for rounding each vector's part to 2^-44 and an fp32 sum of up to 8 terms (7 * 2^-24).  Over a law the
mean of y is at most log2 V <= 17.3 here, so a running sum over a sum is within
17.3 * 3 ln 2 2^-24 + 2^-22 + 7 * 2^-24 = 2.8e-6 < 2^-18 of the law's, and a probability, of tokens drawn
at all (y <= 25), within twice that, relative.  So: the token must be the law's at some uniform within
2^-18 of the given one, where a group of equal logits may be in or out of top-p's set if its
mass is within 2^-18 of the border."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
BAND = 2.0**-18


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def laws(l, T, k, p, m):
    """The truncated laws (one, or two where top_p is within BAND of a border) over the vocabulary."""
    V = len(l)
    M = l.max()
    w = np.exp((l - M) / T)
    keep = np.ones(V, bool)
    if k is not None and 1 <= k < V:
        keep = l >= np.sort(l)[::-1][k - 1]
    found = []
    if p is not None and 0 < p < 1:
        values, member = np.unique(l[keep], return_inverse=True)
        group = np.bincount(member, w[keep])
        values, group = values[::-1], group[::-1]
        mass = np.cumsum(group) / group.sum()
        for q in {float(p) - BAND, float(p), float(p) + BAND}:
            last = min(int((mass < q).sum()), len(values) - 1)
            found.append(keep & (l >= values[last]))
    else:
        found.append(keep)
    out = []
    for keep in found:
        if m is not None and 0 < m <= 1:
            keep = keep & (l - M >= T * np.log(np.float64(np.float32(m))))
        q = np.where(keep, w, 0.0)
        out.append(q / q.sum())
    return out


def fits(token, prob, l, u, T, k, p, m):
    """Whether the token is what some law gives at a uniform within BAND of u."""
    for q in laws(l, T, k, p, m):
        if q[token] == 0:
            continue
        upto = np.cumsum(q)
        low = upto[token] - q[token]
        last = token == np.nonzero(q)[0][-1]
        if low - BAND <= u and (last or u < upto[token] + BAND) and abs(prob - q[token]) <= 2 * BAND * q[token]:
            return True
    return False


def run(sv, x, u, T=None, k=None, p=None, m=None):
    import torch
    f = lambda a: None if a is None else torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    r = sv.spec_sample(x, f(u), f(T), top_k=None if k is None else torch.tensor(k, dtype=torch.int32, device="cuda"),
                       top_p=f(p), min_p=f(m))
    return {a: b.cpu().numpy() for a, b in r.items()}


def check(sv, x, u, T=None, k=None, p=None, m=None):
    got = run(sv, x, u, T, k, p, m)
    l = x.double().cpu().numpy()
    B = len(l)
    one = lambda a, b, d: d if a is None else a[b]  # noqa: E731
    for b in range(B):
        assert got["row_status"][b] == 0
        T32 = np.float64(np.float32(one(T, b, 1.0)))
        p32 = None if p is None else np.float64(np.float32(p[b]))
        assert fits(int(got["token"][b]), got["prob"][b], l[b], float(np.float32(u[b])), T32, one(k, b, None), p32, one(m, b, None)), \
            (b, got["token"][b], got["prob"][b])
    return got


def logits(rng, B, V, dtype, spread=3.0, peaks=True):
    import torch
    x = rng.normal(0, spread, (B, V))
    if peaks:
        x[:, rng.integers(0, V, max(1, V // 5000))] += 3 * spread
    return torch.from_numpy(x).to(getattr(torch, dtype)).cuda()


MIXES = {"plain": {}, "k": dict(k=40), "k1": dict(k=1), "p": dict(p=0.9), "p_small": dict(p=0.05), "p_near_1": dict(p=0.9999),
         "m": dict(m=0.05), "m1": dict(m=1.0), "kp": dict(k=50, p=0.8), "kpm": dict(k=60, p=0.95, m=0.02), "pm": dict(p=0.99, m=0.001),
         "k_many": dict(k=900), "k_more": dict(k=5000, p=0.9)}


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4099, 16384, 32000, 65537, 128256])
@pytest.mark.parametrize("mix", MIXES)
def test_law(sv, mix, V, dtype):
    rng = np.random.default_rng(V)
    B = 3
    kw = {a: np.full(B, b) for a, b in MIXES[mix].items()}
    x = logits(rng, B, V, dtype)
    for _ in range(2):
        check(sv, x, rng.random(B), T=0.4 + rng.random(B), **kw)


@pytest.mark.parametrize("spread", [0.0, 0.01, 0.5])
@pytest.mark.parametrize("mix", ["plain", "p", "p_near_1", "k", "k_many", "k_more", "m", "kpm"])
def test_flat(sv, spread, mix):
    """Laws that keep most of the vocabulary, masses of equal logits among them: more than can be listed."""
    rng = np.random.default_rng(5)
    for dtype in ("bfloat16", "float32"):
        x = logits(rng, 2, 50000, dtype, spread, peaks=False)
        check(sv, x, rng.random(2), **{a: np.full(2, b) for a, b in MIXES[mix].items()})


def test_uniforms(sv):
    """The ends of the interval, and the borders of a law of four tokens in between."""
    import torch
    x = torch.log(torch.tensor([0.0, 0.125, 0.0, 0.5, 0.25, 0.125, 0.0], dtype=torch.float64)).float()
    u = [0.0, 0.1, 0.2, 0.3, 0.6, 0.63, 0.8, 0.88, 0.9999, float(np.nextafter(np.float32(1), np.float32(0)))]
    want = [1, 1, 3, 3, 3, 4, 4, 5, 5, 5]
    got = run(sv, x.cuda().expand(len(u), 7).contiguous(), u)
    assert got["token"].tolist() == want
    assert np.allclose(got["prob"], [0.125, 0.125, 0.5, 0.5, 0.5, 0.25, 0.25, 0.125, 0.125, 0.125], rtol=2 * BAND)
    # the same law where the vocabulary runs over all CTAs of a row
    y = torch.full((len(u), 200000), float("-inf"))
    at = [5, 40000, 90000, 199999]
    y[:, at] = x[[1, 3, 4, 5]]
    got = run(sv, y.cuda(), u)
    assert got["token"].tolist() == [dict(zip([1, 3, 4, 5], at))[w] for w in want]


def test_ties(sv):
    """Equal logits stay together at every border."""
    import torch
    x = torch.tensor([[2.0, 1.0, 2.0, 1.0, 0.0, 1.0, -0.0, 0.0]]).cuda()
    for u in np.linspace(0, 0.999, 40):
        assert int(run(sv, x, [u], k=[1])["token"][0]) in (0, 2)
        assert int(run(sv, x, [u], k=[3])["token"][0]) in (0, 1, 2, 3, 5)
        assert int(run(sv, x, [u], p=[0.7])["token"][0]) in (0, 1, 2, 3, 5)
        check(sv, x, [u], k=[6])  # -0 and 0 are one value: all eight stay
    got = [int(run(sv, x, [u], k=[6])["token"][0]) for u in np.linspace(0, 0.9999, 200)]
    assert set(got) == set(range(8))


def test_off_switches(sv):
    """Values that turn a truncation off."""
    rng = np.random.default_rng(2)
    x = logits(rng, 6, 3000, "bfloat16")
    u = rng.random(6)
    base = run(sv, x, u)
    off = run(sv, x, u, k=[0, -3, 3000, 5000, 0, 0], p=[0.0, 1.0, -1.0, 2.0, np.nan, np.inf], m=[0.0, -1.0, 1.5, np.nan, 0.0, np.inf])
    assert np.array_equal(base["token"], off["token"]) and np.array_equal(base["prob"], off["prob"])


def test_statuses(sv):
    """Bad rows are flagged, the others stay right."""
    import torch
    rng = np.random.default_rng(4)
    for V in (100, 128256):
        x = logits(rng, 9, V, "bfloat16")
        x[1, V // 2] = float("nan")
        x[2, V - 1] = float("inf")
        x[3] = float("-inf")
        x[8, : V - 1] = float("-inf")
        u = [0.5, 0.5, 0.5, 0.5, 1.0, -0.1, np.nan, 0.3, 0.7]
        T = [1, 1, 1, 1, 1, 1, 1, 0, 1]
        for kw in ({}, dict(k=np.full(9, 30)), dict(p=np.full(9, 0.9)), dict(m=np.full(9, 0.1))):
            got = run(sv, x, u, T, **kw)
            assert got["row_status"].tolist() == [0, 1, 1, 5, 3, 3, 3, 7, 0]
            assert got["token"][1:8].tolist() == [-1] * 7 and np.isnan(got["prob"][1:8]).all()
            assert got["token"][8] == V - 1 and got["prob"][8] == 1.0
            check(sv, x[:1], u[:1], **{a: b[:1] for a, b in kw.items()})


@pytest.mark.parametrize("T", [1e-30, 2.0**-130, 1e-3, 50.0, 1e30])
def test_temperatures(sv, T):
    import torch
    rng = np.random.default_rng(6)
    x = logits(rng, 2, 5000, "float32")
    x[1, ::3] = float("-inf")
    x[0, 77] = x[0].max()
    for kw in ({}, dict(k=[20, 20]), dict(p=[0.9, 0.9]), dict(m=[0.5, 0.5])):
        check(sv, x, rng.random(2), T=[T, T], **kw)


def test_rows_apart(sv):
    """Strided rows, odd sizes and unaligned bases read the same."""
    import torch
    rng = np.random.default_rng(7)
    for dtype in ("bfloat16", "float32"):
        wide = logits(rng, 4, 4099, dtype)
        view = wide[:, 3:4002]
        u, T = rng.random(4), 0.5 + rng.random(4)
        a, b = run(sv, view, u, T, p=np.full(4, 0.95)), run(sv, view.contiguous(), u, T, p=np.full(4, 0.95))
        assert np.array_equal(a["token"], b["token"])
        check(sv, view, u, T, k=np.full(4, 25))


def test_many_rows_and_repeats(sv):
    """A large batch; the same call twice gives the same bits."""
    rng = np.random.default_rng(8)
    x = logits(rng, 700, 2000, "bfloat16", 1.0)
    u = rng.random(700)
    a = check(sv, x, u, T=np.full(700, 0.8), p=np.full(700, 0.9), m=np.full(700, 0.01))
    b = run(sv, x, u, np.full(700, 0.8), p=np.full(700, 0.9), m=np.full(700, 0.01))
    assert np.array_equal(a["token"], b["token"]) and np.array_equal(a["prob"], b["prob"])


def test_draft_law(sv):
    """Drafts drawn here under top-k and top-p are never outside what spec_verify_chain's truncated law keeps:
    with draft = target, every one of them is accepted."""
    import torch
    rng = np.random.default_rng(9)
    B, K, V = 16, 3, 6000
    t = logits(rng, B * (K + 1), V, "bfloat16").view(B, K + 1, V)
    T = torch.from_numpy((0.5 + rng.random(B)).astype(np.float32)).cuda()
    k, p = torch.full((B,), 30, dtype=torch.int32, device="cuda"), torch.full((B,), 0.8, device="cuda")
    u = lambda *s: torch.from_numpy(rng.random(s).astype(np.float32)).cuda()  # noqa: E731
    drafts = torch.stack([sv.spec_sample(t[:, j].contiguous(), u(B), T, top_k=k, top_p=p)["token"] for j in range(K)], 1)
    out = sv.spec_verify_chain(t, t[:, :K].contiguous(), drafts.contiguous(), T, u(B, K), u(B, K + 1), top_k=k, top_p=p)
    assert out["row_status"].tolist() == [0] * B
    assert out["accepted_len"].tolist() == [K] * B


def test_frequencies(sv):
    """200000 draws recover a small law within four standard deviations."""
    import torch
    rng = np.random.default_rng(10)
    l = np.array([1.0, 0.5, 0.0, -1.0, -2.0, 0.25, 0.75, -0.5])
    n = 200000
    x = torch.from_numpy(l).float().cuda().expand(n, 8).contiguous()
    got = run(sv, x, rng.random(n), np.full(n, 0.9), p=np.full(n, 0.9))
    q = laws(l, np.float64(np.float32(0.9)), None, 0.9, None)[0]
    f = np.bincount(got["token"], minlength=8) / n
    assert np.all(np.abs(f - q) <= 4 * np.sqrt(q * (1 - q) / n) + 1e-12)
