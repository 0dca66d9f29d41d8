"""Calls from several host threads at once."""
import sys
import threading

import pytest
import torch

from gated_delta_rule_57_gb300 import kda

pytestmark = pytest.mark.gpu


def test_plans_of_different_sizes_from_several_threads():
    """Their kernels need different amounts of shared memory; one thread's call must not
    take from the other's."""
    L, results = kda.lib(), []

    def ints(n, value=0):
        return torch.full((n,), value, dtype=torch.int32, device="cuda")

    def work(n):
        stream = torch.cuda.Stream()
        old, new, table, ring, at = ints(n), ints(n), ints(n, -1), ints(n), ints(2)
        ring_out, kv, cu, slot = ints(2, 7), ints(n, 7), ints(n + 1, 7), ints(8, 7)
        torch.cuda.synchronize()
        args = [x.data_ptr() for x in (old, new, table, ring, at, ring_out, kv, cu, slot)]
        codes = {L.kda_kv_plan(*args, n, 1, n, 16, 8, None, stream.cuda_stream) for _ in range(5000)}
        stream.synchronize()
        results.append((codes, int(kv.abs().sum()), int(cu.abs().sum()), slot.tolist()))

    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        threads = [threading.Thread(target=work, args=(n,)) for n in (16000, 5000, 16384, 4200)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert results == [({kda.KDA_OK}, 0, 0, [-1] * 8)] * 4
