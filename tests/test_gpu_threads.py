"""Two host threads on one stream: each call's results are those of the same call made alone
(needs a GB300)."""
import threading

import pytest

from tests.test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


def test_attention_from_two_threads():
    """Different prefixes, trees, lengths and kernels through one workspace."""
    import numpy as np
    import torch
    import speculative_decoding_verification_32_gb300 as sv

    def i32(a):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    problems = [[Problem(sv, 6, 40, 8, 2, 64, 700, [9, 30, 0, 64, 12, 50], "uint8", "bfloat16", True, seed=1),
                 Problem(sv, 3, 4, 8, 2, 128, 500, [20, 0, 77], "bfloat16", "bfloat16", seed=2)],
                [Problem(sv, 5, 50, 8, 2, 64, 300, [100, 3, 0, 7, 55], "uint8", "bfloat16", True, seed=3),
                 Problem(sv, 64, 1, 16, 8, 64, 100, list(range(0, 320, 5)), "uint8", "bfloat16", seed=4)]]
    calls = []
    for ps in problems:
        mine = []
        for p in ps:
            lens, parent = i32(p.lens), i32(p.parent)
            mine.append(lambda p=p, lens=lens, parent=parent: sv.spec_prefix_attention(
                p.q, p.cache, lens, prefix=p.prefix, parent=parent, kv_heads=p.H))
        calls.append(mine)
    want = [[c() for c in mine] for mine in calls]
    torch.cuda.synchronize()
    wrong = [None, None]

    def work(t):
        bad = torch.zeros((), dtype=torch.int64, device="cuda")
        for i in range(1500):
            out, lse, status = calls[t][i % 2]()
            o, ls, st = want[t][i % 2]
            bad += (out != o).sum() + (lse != ls).sum() + (status != st).sum()
        wrong[t] = bad

    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert [int(x) for x in wrong] == [0, 0]
