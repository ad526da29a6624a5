"""Scales that spec_paged_attention cannot hold in base 2 are turned down (runs without a GPU)."""
import ctypes

import pytest

from tests.test_pages_sample_host import ARG, OK, L, attention  # noqa: F401


@pytest.mark.parametrize("scale,want", [(3.0e38, ARG), (-3.0e38, ARG), (2.4e38, ARG), (2.3e38, OK), (-2.3e38, OK), (1e-45, OK), (0.0, OK)])
def test_scales(L, scale, want):  # noqa: F811
    """(B = 0: what is left once the arguments are accepted)"""
    code, a = attention(L, scale=scale, B=0)
    assert code == want
    assert (L.spec_paged_attention_workspace_size(ctypes.byref(a)) > 0) == (want == OK)
