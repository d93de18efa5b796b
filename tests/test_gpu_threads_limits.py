"""Host threads that call the same kernels at once with different amounts of dynamic shared memory: the limit that a
launch may use belongs to the function, so no call may lower it below another's.  Each thread has its own stream and
its own batch, and repeats its call, whose outputs do not depend on how often it ran."""
import threading

import numpy as np
import pytest
import torch

import oracle
import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import workloads as W
from dequant_kvc8_store_gb300.device import DecodeAttention, DeviceBatch
from test_gpu_blocks import Problem, lengths
from test_gpu_parity import _assert_bits_equal, _oracle_store

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


@pytest.mark.parametrize("new", [60, 3])  # with a launch of the slots' own, and without
def test_block_assignment(new):
    kv.load()
    rng = np.random.default_rng(31)
    problems = [Problem(*lengths(rng, B, 300, new, 0.3), 16, seed=5) for B in (3000, 8192)]
    for p in problems:
        p.place()
    at_once(*[p.call for p in problems])
    for p in problems:
        p.check()


def wide(heads, seed):
    """A batch whose static scales, kept in shared memory by the gather and the attention, take more than 48 KB."""
    return W.make_workload(f"limits{heads}", q_lens=[5, 1, 30], ctx_before=[9, 40, 0], kv_heads=heads, head_dim=128,
                           block_size=16, num_blocks=16, quant_mode=1, seed=seed)


def test_gather():
    batches = [DeviceBatch(wide(heads, heads)) for heads in (48, 64)]
    for d in batches:
        d.store()
    at_once(*[d.gather for d in batches])
    for d in batches:
        assert d.error_code() == 0
        ko, vo = oracle.dequant_gather(1, *_oracle_store(d.w), d.w.block_table, d.w.context_lengths)
        gk, gv = d.host_outputs()
        _assert_bits_equal(gk, ko, "k_out")
        _assert_bits_equal(gv, vo, "v_out")


def test_decode_attention():
    calls = []
    for heads in (48, 64):
        d = DeviceBatch(wide(heads, heads))
        d.store()
        calls.append(DecodeAttention(d, 2, seed=heads))
        calls[-1]()
    alone = [a.out.clone() for a in calls]
    at_once(*calls)
    for a, want in zip(calls, alone):
        assert a.d.error_code() == 0 and torch.equal(a.out, want)
