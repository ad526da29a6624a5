"""The example that runs append, attention, tree verification, log probabilities, compaction and
rollback together, checking each step against the cache as it reads back (needs a GB300)."""
import importlib.util
import os

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,prompt", [(1, 33), (8, 700), (40, 1000)])
def test_decode_steps(batch, prompt):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    lines = []
    emitted = m.main(steps=4, batch=batch, prompt=prompt, check=True, out=lines.append)
    assert len(lines) == 4
    assert emitted > 4 * batch  # some drafts were kept: the mask's branches and the compaction were at work
