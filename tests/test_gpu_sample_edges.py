"""spec_sample where hardly any weight lies before the token drawn (needs a GB300)."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import torch
    import speculative_decoding_verification_32_gb300 as m
    assert torch.cuda.is_available()
    return m


def into(sv, x, u):
    """The call into outputs that hold something else: (token, prob, row_status)."""
    import torch
    from speculative_decoding_verification_32_gb300 import _binding as b
    B, V = x.shape
    u = torch.tensor(u, dtype=torch.float32, device="cuda")
    token, status = (torch.full((B,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    prob = torch.full((B,), -77.0, device="cuda")
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    a = b.SpecSampleArgs(B, V, b._dtype_code(x), 0, V, P(x), P(u), None, None, None, None)
    o = b.SpecSampleOut(P(token), P(prob), P(status))
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert b.lib().spec_sample(ctypes.byref(a), ctypes.byref(o), stream) == 0
    return token.cpu().numpy(), prob.cpu().numpy(), status.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("B,V", [(1, 128256), (1, 200000), (300, 128256), (700, 32000), (2, 4099)])
@pytest.mark.parametrize("above", [31, 32, 33, 34, 35, 36, 60])
def test_little_weight_at_the_start(sv, B, V, dtype, above):
    """One late logit holds all but a 2^-44th of the law, the rest is spread over so many tokens that a vector's
    share of it is next to nothing: every row is answered, at the start of the interval as well."""
    import torch
    x = torch.zeros(B, V, dtype=getattr(torch, dtype), device="cuda")
    x[:, V - 1] = above
    u = [[0.0, 1e-30, 2.0**-44, 2.0**-24, 0.5][b % 5] for b in range(B)]
    token, prob, status = into(sv, x, u)
    assert not status.any()
    q = np.exp(-float(above))
    Z = 1.0 + (V - 1) * q
    for b in range(B):
        assert 0 <= token[b] < V
        want = (1.0 if token[b] == V - 1 else q) / Z
        assert abs(prob[b] - want) <= 2.0**-17 * want
        if token[b] == V - 1:
            assert u[b] >= (V - 1) * q / Z - 2.0**-18
        else:
            assert token[b] * q / Z <= u[b] + 2.0**-18
