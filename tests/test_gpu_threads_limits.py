"""Host threads that call the same kernels at once with different amounts of dynamic shared memory: the limit that a
launch may use belongs to the function, so no call may lower it below another's.  Each thread has its own stream and
its own batch, and repeats its call, whose outputs do not depend on how often it ran."""
import threading

import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from test_gpu_blocks import Problem, lengths

pytestmark = pytest.mark.gpu


def at_once(*calls, times=400):
    """Each call(stream) `times` times in a thread of its own, all threads at once."""
    errors, start = [], threading.Barrier(len(calls))

    def run(call):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            start.wait()
            for _ in range(times):
                call(stream)
            stream.synchronize()
        except Exception as e:  # reported on the main thread
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("new", [60, 3])  # with a launch of the slots' own (more than 131072), and without
def test_block_assignment(new):
    kv.load()
    rng = np.random.default_rng(31)
    problems = [Problem(*lengths(rng, B, 300, new, 0.3), 16, seed=5) for B in (3000, 8192)]
    for p in problems:
        p.place()
    at_once(*[p.call for p in problems])
    for p in problems:
        p.check()
