"""spec_paged_attention with scales at the small end of fp32 and numbers that make up for it (needs a GB300)."""
import numpy as np
import pytest

from tests.test_gpu_attention import check_row
from tests.test_gpu_paged_attention import i32, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
@pytest.mark.parametrize("N", [1, 8, 40, 200])
@pytest.mark.parametrize("scale", [2.0**-124, -2.0**-124, 2.0**-126, 2.0**-118])
def test_small_scales(kind, N, scale):
    """q.k of 2^120 and more: scores of a few units, by the rows kernel and by the tile kernel."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    B, Hq, H, D, page, n = 2, 4, 2, 64, 16, 90
    g = torch.Generator().manual_seed(N)
    up = round(-np.log2(abs(scale)) / 2)
    q = torch.zeros(B, N, Hq, D)
    k = torch.zeros(B, n + N, H, D)
    q[..., 0] = 2.0**up
    k[..., 0] = 2.0**up * torch.randint(-16, 17, k.shape[:3], generator=g) / 8
    v = torch.randn(B, n + N, H, D, generator=g)
    q = q.bfloat16()
    pages = -(-(n + N) // page)
    line = torch.zeros((2, B, pages * page) + ((sv.spec_kv_entry_bytes(H, D),) if kind == "uint8" else (H, D)),
                       dtype=getattr(torch, kind), device="cuda")
    total = i32([n + N] * B)
    sv.spec_kv_append(line, k.cuda(), v.cuda(), i32([0] * B), count=total)
    kx, vx, _ = sv.spec_kv_read(line, total, n + N, heads=H, head_dim=D, dtype=torch.float32)
    pool = line.view(2, B * pages, page, *line.shape[3:])
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    out, lse, status = sv.spec_paged_attention(q.cuda(), pool, table, i32([n] * B), scale=scale, kv_heads=H)
    assert not status.any()
    rounded = "bfloat16" if kind == "uint8" and N * Hq // H > 32 else kind
    for b in range(B):
        check_row(out[b].cpu().double().numpy(), lse[b].cpu().double().numpy(), q[b].double().numpy(), kx[b].cpu().double().numpy(),
                  vx[b].cpu().double().numpy(), visible(n, N, 0, 0, None), scale, rounded, 2.0**-8)
