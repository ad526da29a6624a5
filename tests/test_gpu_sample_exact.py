"""spec_sample's token is the 64-bit law's, without a band (needs a GB300).

The kernel decides by weights good to 2^-36 of themselves where fp32 ones leave a decision open.  A running
sum S over the whole Z is then off by at most 2 S/Z (1 - S/Z) 2^-36 <= 2^-37, so the token can differ from the
law's only where u lies that near a border between two tokens, or top_p that near a group's mass: rows
where the restatement here (2^-52 a term) finds one within NEAR are left out, by its own numbers.  A
probability from fp32 weights: the weight 3.25 ln 2 2^-24 y + 2^-22 with y <= 25 for tokens drawn at all, the
whole as much with y <= 18, and its sums 2^-20: below 2^-17 together."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
NEAR = 2.0**-36


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def law(x, u, T, k=0, p=1.0, m=0.0):
    """(token, its probability, whether some decision was nearer than NEAR) per row, in 64 bits."""
    import torch
    x = x.double()
    B, V = x.shape
    T = torch.ones(B, 1, dtype=torch.float64, device=x.device) if T is None else T.double()[:, None]
    top = x.amax(1, keepdim=True)
    floor = torch.full_like(top, float("-inf"))
    near = torch.zeros(B, dtype=torch.bool, device=x.device)
    if k or p < 1:
        xs = torch.sort(x, 1, descending=True).values
        if k and k < V:
            floor = xs[:, k - 1:k]
        if p < 1:
            p = float(np.float32(p))
            mass = torch.cumsum(torch.where(xs >= floor, torch.exp((xs - top) / T), 0.0), 1)
            share = mass / mass[:, -1:]
            # groups of equal logits: a border is where the next logit differs
            end = torch.cat((xs[:, 1:] != xs[:, :-1], torch.ones_like(near)[:, None]), 1)
            near |= (((share - p).abs() < NEAR) & end).any(1)
            floor = torch.maximum(floor, torch.gather(xs, 1, (share < p).sum(1, keepdim=True).clamp_max(V - 1)))
    keep = x >= floor
    if m:
        keep &= x - top >= T * np.log(np.float64(np.float32(m)))
    w = torch.where(keep, torch.exp((x - top) / T), 0.0)
    upto = torch.cumsum(w, 1)
    Z = upto[:, -1:]
    at = (upto <= u.double()[:, None] * Z).sum(1, keepdim=True)
    at = torch.minimum(at, V - 1 - (w > 0).flip(1).int().argmax(1, keepdim=True))
    q = torch.gather(w, 1, at)
    gap = torch.minimum((torch.gather(upto, 1, at) - u.double()[:, None] * Z).abs(), (torch.gather(upto, 1, at) - q - u.double()[:, None] * Z).abs())
    near |= (gap < NEAR * Z)[:, 0]
    return at[:, 0].int(), (q / Z)[:, 0], near


def sample(sv, x, u, T=None, k=0, p=1.0, m=0.0):
    import torch
    B = len(x)
    f = lambda a: torch.full((B,), a, device="cuda")  # noqa: E731
    return sv.spec_sample(x, u, T, top_k=torch.full((B,), k, dtype=torch.int32, device="cuda") if k else None,
                          top_p=f(p) if p < 1 else None, min_p=f(m) if m else None)


def rows(g, B, V, dtype, spread):
    import torch
    x = spread * torch.randn(B, V, generator=g, device="cuda")
    x[:, torch.randint(0, V, (max(1, V // 6000),), generator=g, device="cuda")] += 3 * spread
    return x.to(getattr(torch, dtype)), torch.rand(B, generator=g, device="cuda"), 0.5 + 0.7 * torch.rand(B, generator=g, device="cuda")


MIXES = {"plain": {}, "p": dict(p=0.95), "p_low": dict(p=0.6), "m": dict(m=0.02), "pm": dict(p=0.95, m=0.02), "kp": dict(k=50, p=0.9),
         "k": dict(k=300), "kp_many": dict(k=3000, p=0.9)}


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V,B", [(128256, 256), (32000, 300), (32000, 64), (5000, 700), (4099, 40)])
@pytest.mark.parametrize("spread", [3.0, 1.0, 0.1])
@pytest.mark.parametrize("mix", MIXES)
def test_tokens(sv, mix, spread, V, B, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(V + B)
    for _ in range(2):
        x, u, T = rows(g, B, V, dtype, spread)
        got = sample(sv, x, u, T, **MIXES[mix])
        token, prob, near = law(x, u, T, **MIXES[mix])
        assert not got["row_status"].any() and near.sum() <= 1
        assert torch.equal(got["token"][~near], token[~near])
        assert ((got["prob"].double() - prob).abs() <= 2.0**-17 * prob)[~near].all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [200, 128256])
@pytest.mark.parametrize("mix", ["plain", "p", "m", "kp"])
def test_borders(sv, mix, V, dtype):
    """Uniforms right below and right above a token's borders."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    B = 256
    x, _, T = rows(g, 1, V, dtype, 2.0)
    one = lambda a: law(x, torch.tensor([a], device="cuda"), T, **MIXES[mix])  # noqa: E731
    at, q, _ = one(0.0)
    w = torch.exp((x.double() - x.double().amax()) / T.double())[0]
    # a law's borders from its members: those that some uniform draws
    kept = set(one(float(a))[0].item() for a in np.linspace(0, 1, 60)[:-1])
    lows = []
    for t in sorted(kept):
        lo, hi = 0.0, 1.0
        for _ in range(60):  # the border in front of the token, by halving
            mid = (lo + hi) / 2
            tok = law(x, torch.tensor([mid], dtype=torch.float64, device="cuda"), T, **MIXES[mix])[0].item()
            lo, hi = (lo, mid) if tok >= t else (mid, hi)
        lows.append(hi)
    u = []
    for a in lows:
        f = np.float32(a)
        u += [np.nextafter(f, np.float32(0)), f, np.nextafter(f, np.float32(1))]
    u = torch.tensor(np.clip(np.array(u, np.float32), 0, np.nextafter(np.float32(1), np.float32(0)))[:B], device="cuda")
    n = len(u)
    x, T = x.expand(n, V).contiguous(), T.expand(n).contiguous()
    got = sample(sv, x, u, T, **MIXES[mix])
    token, _, near = law(x, u, T, **MIXES[mix])
    assert near.sum() <= n // 8
    assert torch.equal(got["token"][~near], token[~near])
    assert w.numel() == V and q.item() > 0 and at.item() >= 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("mix", ["plain", "p", "pm", "k"])
@pytest.mark.parametrize("V", [32000, 128256, 100001])
def test_alone_and_in_batches(sv, V, mix, dtype):
    """A row draws the same token whatever batch it is in."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    x, u, T = rows(g, 700, V, dtype, 1.0)
    whole = sample(sv, x, u, T, **MIXES[mix])["token"]
    for B in (1, 64, 300):
        for b in (0, 64, 300):
            part = sample(sv, x[b:b + B], u[b:b + B], T[b:b + B], **MIXES[mix])["token"]
            assert torch.equal(part, whole[b:b + B])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [4, 1024, 16384, 131072])
@pytest.mark.parametrize("B", [2, 300])
def test_ties_of_a_flat_law(sv, V, dtype, B):
    """V = 2^n equal logits: u V is exact, so the token is its integer part, on the borders too."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.full((B, V), 1.375, dtype=getattr(torch, dtype), device="cuda")
    n = torch.randint(0, V, (B,), generator=g, device="cuda")
    for off in (0.0, -1.0, 1.0):
        u = (n.double() / V).float()
        if off:
            u = torch.nextafter(u, torch.full_like(u, off)).clamp(0, 1 - 2.0**-24)
        want = (u.double() * V).floor().int()
        for kw in ({}, dict(m=0.5), dict(p=0.9), dict(k=min(7, V - 1))):
            got = sample(sv, x, u, None, **kw)
            assert torch.equal(got["token"], want), (off, kw)
            assert (got["prob"] * V - 1).abs().max() <= 2.0**-17


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kw", [{}, dict(k=30), dict(m=1e-30), dict(k=2000), dict(p=0.9999999)])
def test_next_to_zero(sv, kw, dtype):
    """The first tokens of the law weigh next to nothing; u = 0 draws the very first, and small uniforms those that
    their running sums say."""
    import torch
    V, B = 40000, 12
    l = torch.zeros(V, dtype=torch.float64)
    l[:] = -60.0
    l[5:25] = torch.linspace(-52, -34, 20).double()
    l[V - 3] = 0.0
    l[:3] = float("-inf")
    x = l.to(getattr(torch, dtype)).cuda().expand(B, V).contiguous()
    u = torch.tensor([0.0, 1e-40, 1e-30, 1e-25, 1e-23, 1e-22, 1e-20, 1e-18, 1e-16, 1e-15, 2.0**-30, 2.0**-24], device="cuda")
    got = sample(sv, x, u, None, **kw)
    token, prob, _ = law(x, u, None, **kw)
    assert not got["row_status"].any()
    assert torch.equal(got["token"], token), (got["token"].tolist(), token.tolist())
    assert ((got["prob"].double() - prob).abs() <= 2.0**-17 * prob).all()


@pytest.mark.parametrize("T", [1e-44, 2.0**-140, 2.0**-66, 2.0**-63, 2.0**63, 2.0**66, 1e30, 3e38])
@pytest.mark.parametrize("mix", ["plain", "p", "m", "kp", "k"])
@pytest.mark.parametrize("V", [300, 20000])
def test_temperatures_out_of_range(sv, T, mix, V):
    """Logits of the temperature's size, where fp32's reciprocals and differences end."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    B = 20
    T32 = float(np.float32(T))
    x = (torch.randn(B, V, generator=g, device="cuda").double().clamp(-3, 3) * (T32 if T < 1e38 else 1e38)).float()
    u = torch.rand(B, generator=g, device="cuda")
    t = torch.full((B,), T32, device="cuda")
    got = sample(sv, x, u, t, **MIXES[mix])
    token, prob, near = law(x, u, t, **MIXES[mix])
    assert not got["row_status"].any() and near.sum() <= 1
    assert torch.equal(got["token"][~near], token[~near])
    assert ((got["prob"].double() - prob).abs() <= 2.0**-17 * prob)[~near].all()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [5, 300, 60000])
@pytest.mark.parametrize("p", [1e-5, 1e-7, 1e-12, 1e-16, 1e-30, 1e-45])
def test_top_p_next_to_zero(sv, p, V, dtype):
    """The largest logits alone are kept, however small top_p is."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(6)
    B = 6
    for spread in (0.1, 2.0):
        x = (spread * torch.randn(B, V, generator=g, device="cuda")).to(getattr(torch, dtype))
        top = x.amax(1, keepdim=True)
        at = torch.randint(0, V, (B, 3), generator=g, device="cuda")
        x.scatter_(1, at, top.expand(B, 3) + (2 if dtype == "bfloat16" else 2.0**-10))
        u = torch.rand(B, generator=g, device="cuda")
        for kw in (dict(p=p), dict(p=p, m=0.9), dict(p=p, k=min(4, V - 1))):
            got = sample(sv, x, u, None, **kw)
            assert not got["row_status"].any()
            best = x == x.amax(1, keepdim=True)
            n = best.sum(1)
            want = torch.stack([best[b].nonzero()[min(int(float(u[b]) * int(n[b])), int(n[b]) - 1), 0] for b in range(B)])
            if p < 1e-6 or V < 1000:  # (a larger share of a flat law is more than these)
                assert torch.equal(got["token"].long(), want)
                assert (got["prob"] * n - 1).abs().max() <= 2.0**-17
