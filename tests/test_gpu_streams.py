"""Calls on a stream that is not the current one: nothing of theirs waits in the current one's queue
(needs a GB300)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [("c2",), ("c1", "c2")])
def test_a_new_workspace_is_the_streams_own(sizes):
    """A verify call on a named stream makes (or replaces) that stream's workspace: what the call has
    left in it stays, whatever the current stream was still busy with."""
    import torch
    import speculative_decoding_verification_32_gb300 as sv
    from speculative_decoding_verification_32_gb300 import _binding
    from tests.gpu_util import cuda
    from workloads import synthetic as S
    s = torch.cuda.Stream()
    for size in sizes:
        inp = S.make(size)
        t = [cuda(inp[k]) for k in ("target", "draft", "draft_tokens", "temperature", "u_accept", "u_sample")]
        want = sv.spec_verify_chain(*t)
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)  # about 0.1 s of the current stream
        with torch.cuda.stream(s):
            out = {k: torch.empty_like(v) for k, v in want.items()}
        got = sv.spec_verify_chain(*t, out=out, stream=s)
        s.synchronize()
        ws = _binding._ws[(t[0].device, s.cuda_stream)]
        with torch.cuda.stream(s):
            after = ws.cpu()
        torch.cuda.synchronize()
        assert bool(after.any()) and torch.equal(after, ws.cpu())
        for k in want:
            assert torch.equal(got[k], want[k])
