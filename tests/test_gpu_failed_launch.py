"""A launch that the device refuses is reported by the call that made it, and by no later one."""
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import workloads as W
from dequant_kvc8_store_gb300.device import DeviceBatch

pytestmark = pytest.mark.gpu


def batch(heads):
    return DeviceBatch(W.make_workload(f"heads{heads}", q_lens=[3], ctx_before=[9], kv_heads=heads, head_dim=128,
                                       block_size=16, num_blocks=2, quant_mode=1, seed=heads))


def test_scales_beyond_shared_memory():
    kv.load()
    few, many = batch(8), batch(256)  # of 256 heads the channels' scales take more than an SM's shared memory
    few.store()
    few.gather()
    want = few.k_out.clone()
    for _ in range(2):
        with pytest.raises(kv.Kvc8Error) as e:
            many.gather()
        assert e.value.status == kv.ERR_CUDA
        few.k_out.zero_()
        few.gather()
        torch.cuda.synchronize()
        assert few.error_code() == 0 and torch.equal(few.k_out, want)
