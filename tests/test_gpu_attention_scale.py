"""spec_prefix_attention with scales at the small end of fp32 and numbers that make up for it (needs a GB300)."""
import numpy as np
import pytest

from tests.test_gpu_attention import check_row
from tests.test_gpu_paged_attention import i32, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bfloat16", "uint8"])
@pytest.mark.parametrize("P", [0, 200])
@pytest.mark.parametrize("N", [1, 8, 40, 200])
@pytest.mark.parametrize("scale", [2.0**-124, -2.0**-124, 2.0**-126, 2.0**-118])
def test_small_scales(kind, P, N, scale):
    """q.k of 2^120 and more: scores of a few units, by the rows kernel and by the tile kernel."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    B, Hq, H, D, n = 2, 4, 2, 64, 90
    g = torch.Generator().manual_seed(N)
    up = round(-np.log2(abs(scale)) / 2)
    q = torch.zeros(B, N, Hq, D)
    q[..., 0] = 2.0**up
    q = q.bfloat16()

    def cache(rows, T):
        k = torch.zeros(rows, T, H, D)
        k[..., 0] = 2.0**up * torch.randint(-16, 17, k.shape[:3], generator=g) / 8
        v = torch.randn(rows, T, H, D, generator=g)
        c = torch.zeros((2, rows, T) + ((sv.spec_kv_entry_bytes(H, D),) if kind == "uint8" else (H, D)),
                        dtype=getattr(torch, kind), device="cuda")
        sv.spec_kv_append(c, k.cuda(), v.cuda(), i32([0] * rows))
        kx, vx, _ = sv.spec_kv_read(c, i32([T] * rows), T, heads=H, head_dim=D, dtype=torch.float32)
        return c, kx.cpu().double().numpy(), vx.cpu().double().numpy()
    own, kx, vx = cache(B, n + N)
    kw = {}
    if P:
        pre, kp, vp = cache(1, P)
        kw = dict(prefix=pre)
        kx, vx = (np.concatenate((np.repeat(a, B, 0), b), 1) for a, b in ((kp, kx), (vp, vx)))
    out, lse, status = sv.spec_prefix_attention(q.cuda(), own, i32([n] * B), scale=scale, kv_heads=H, **kw)
    assert not status.any()
    for b in range(B):
        # (the rounding of fp16 where the kernels go by codes, else of bf16: what is coarser)
        check_row(out[b].cpu().double().numpy(), lse[b].cpu().double().numpy(), q[b].double().numpy(), kx[b], vx[b],
                  visible(P + n, N, 0, 0, None), scale, kind, 2.0**-8)
