"""spec_paged_attention over rows of more than 2^28 tokens, whose table names a few pages again and again (needs
a GB300)."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [(1 << 28) - 5000, (1 << 28) + 77, (1 << 30) + 5])
def test_the_last_token_counts(tokens):
    """The last token of a row weighs 2^8 times all the others: an answer that leaves a part of the row out is far
    off.  What remains is the fp32 sum of up to 2^20 equal terms in a thread, 2^-5 of the others' share."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    B, H, D, page = 2, 1, 16, 1024
    pages = 6
    cache = torch.zeros(2, pages, page, sv.spec_kv_entry_bytes(H, D), dtype=torch.uint8, device="cuda")
    # keys are zero but one number of the last page's tokens; values: 1 and 2 in the last page's
    n = tokens - 1
    columns = -(-tokens // page) + 1
    table = torch.zeros(B, columns, dtype=torch.int32, device="cuda")
    k, v = torch.zeros(1, pages * page, H, D, device="cuda"), torch.ones(1, pages * page, H, D, device="cuda")
    last = n // page
    for b in range(B):
        table[b, last] = 2 + b
        at = (2 + b) * page + n % page
        k[0, at, 0, 0] = 1.0
        v[0, at, 0] = 3.0 + b
    sv.spec_kv_append(cache.view(2, 1, pages * page, -1), k, v, torch.zeros(1, dtype=torch.int32, device="cuda"))
    x = np.log(256.0 * n)  # its score; the others' is 0
    q = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 32.0
    kv_len = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out, lse, status = sv.spec_paged_attention(q, cache, table, kv_len, scale=float(x / 32), kv_heads=H)
    assert not status.any()
    want_lse = np.log(257.0 * n)
    assert (lse.cpu().double() - want_lse).abs().max() <= 2.0**-5 / 256 + 2.0**-18 * x + 2.0**-20
    for b in range(B):
        want = (256 * (3.0 + b) + 1) / 257
        assert (out[b].cpu().double() - want).abs().max() <= 2.0**-8 * want + 2.0**-5 / 256 * want + 2.0**-10 * want
