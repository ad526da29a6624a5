"""spec_token_logprobs at the ends of the temperature's range (needs a GB300)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [300, 50000])
@pytest.mark.parametrize("T", [1e-45, 1e-40, 4e-39, 1e-38, 1e-30, 1e30, 3e38])
def test_temperatures_of_any_size(dtype, V, T):
    """Any finite temperature above zero is a law: towards zero all of it on the largest logit (here by
    itself, or shared by three), towards the largest numbers the uniform one."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    x = torch.randn(3, 2, V, generator=torch.Generator().manual_seed(V)).clamp_max(3.0)
    x[:, 0, 5] = 4.0
    x[:, 1, [7, 100, V - 1]] = 4.0
    x = x.to(getattr(torch, dtype)).cuda()
    T = torch.tensor(T, dtype=torch.float32)
    tokens = torch.tensor([[5, 7], [6, 100], [5, 6]], dtype=torch.int32, device="cuda")
    g = {k: v.cpu().numpy() for k, v in sv.spec_token_logprobs(x, tokens, T.repeat(3).cuda(), m=4).items()}
    assert not g["status"].any()
    # the tolerances of test_gpu_logprobs.py: y = (l - M) / T carries three fp32 roundings at most
    xd = x.double().cpu().numpy()
    y = (xd - xd.max(-1, keepdims=True)) / float(T)
    lse = np.log(np.exp(y).sum(-1, keepdims=True))
    lp = y - lse
    p = np.exp(lp)
    entropy = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(-1)
    given = np.take_along_axis(lp, tokens.cpu().numpy()[..., None].astype(np.int64), -1)[..., 0]
    tops = np.take_along_axis(lp, g["top_ids"].astype(np.int64), -1)
    for got, want, rtol, atol in ((g["logprob"], given, 2.0**-21, 2.0**-18), (g["top_logprobs"], tops, 2.0**-21, 2.0**-18),
                                  (g["entropy"], entropy, 2.0**-17, 2.0**-17)):
        with np.errstate(over="ignore"):
            far = np.isinf(want.astype(np.float32))
        assert not np.isnan(got).any()
        assert np.array_equal(got[far], np.full(far.sum(), -np.inf))
        assert np.all(np.abs(got[~far] - want[~far]) <= atol + rtol * np.abs(want[~far]))
