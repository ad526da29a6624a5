"""Where the binding's calls launch: on their tensors' device, and on no other (runs without a GPU)."""
from types import SimpleNamespace

import pytest
import torch

import speculative_decoding_verification_32_gb300 as sv
from speculative_decoding_verification_32_gb300 import _binding


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    """A library that must not be called."""
    from speculative_decoding_verification_32_gb300 import build as lib_build
    lib_build.build()

    def refuse(name, nargs):
        raise AssertionError(f"{name} was about to be launched")
    monkeypatch.setattr(_binding, "_fn", refuse)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


STREAM = SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 0))


@pytest.mark.parametrize("stream", [None, STREAM])
@pytest.mark.parametrize("call", [
    lambda **kw: sv.spec_kv_append(torch.zeros(2, 2, 9, 8, 64).bfloat16(), torch.zeros(2, 3, 8, 64), torch.zeros(2, 3, 8, 64), i32(2), **kw),
    lambda **kw: sv.spec_kv_read(torch.zeros(2, 2, 9, 8, 64).bfloat16(), i32(2), 4, **kw),
    lambda **kw: sv.spec_prefix_attention(torch.zeros(2, 3, 8, 64).bfloat16(), torch.zeros(2, 2, 9, 8, 64).bfloat16(), i32(2), **kw),
    lambda **kw: sv.spec_token_logprobs(torch.zeros(2, 3, 50), i32(2, 3), **kw),
    lambda **kw: sv.spec_verify_tree(torch.zeros(2, 3, 50), i32(2, 3), i32(2, 3), **kw),
    lambda **kw: sv.spec_rollback_lengths(i32(2), i32(2), i32(2), i32(2, 3), **kw),
    lambda **kw: sv.spec_kv_compact_tree(torch.zeros(2, 2, 9, 8), i32(2), i32(2), i32(2, 3), **kw),
])
def test_host_tensors_are_refused(call, stream):
    with pytest.raises(ValueError, match="CUDA tensors"):
        call(stream=stream)


def test_the_tensors_device_becomes_the_current_one(monkeypatch):
    monkeypatch.setattr(_binding, "_current_device", lambda: 0)
    assert _binding._on(torch.device("cuda", 0), None) is _binding._here
    other = _binding._on(torch.device("cuda", 1), None)
    assert isinstance(other, torch.cuda.device) and other.idx == 1
    with pytest.raises(ValueError, match="stream"):
        _binding._on(torch.device("cuda", 1), STREAM)
