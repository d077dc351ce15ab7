"""Calls from several threads at once, each with its own sizes, buffers and stream."""
import threading

import numpy as np
import pytest
import torch

from bit_mixed_precision_channel_b200 import binding as kb

from _spec import Cache
from test_gpu_select import run_select
from test_gpu_tree import call, check, make

pytestmark = pytest.mark.gpu


def test_threads_with_different_sizes_of_one_kernel():
    """Page sizes and table lengths ask for different shared memory of the same kernels."""
    trees = [make(kb.Config(num_q_heads=4, num_kv_heads=1, page_tokens=P, num_boost=64), [5], [9], 7, [7], seed=P) for P in (32, 64, 128)]
    chosen = []
    for n in (40, 300, 9000):
        c = Cache(kb.Config(num_q_heads=2, num_kv_heads=1, page_tokens=64, num_boost=64), [n], [0], seed=n, distinct=8)
        c.d["page_table"] = c.ints(np.pad(c.table, ((0, 0), (0, n % 7))))
        chosen.append((c, c.queries(1)))
    torch.cuda.synchronize()
    gate, bad, sels = threading.Barrier(6), [], {}

    def run(i):
        try:
            gate.wait()
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    if i < 3:
                        call(trees[i])
                    else:
                        sels[i] = run_select(*chosen[i - 3], 6, 1, 1)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    for c in trees:
        assert c.err.item() == 0
        check(c)
    for i, (c, q) in enumerate(chosen):
        sel, n_sel = run_select(c, q, 6, 1, 1)
        assert c.err.item() == 0 and torch.equal(sel, sels[3 + i][0]) and torch.equal(n_sel, sels[3 + i][1])
