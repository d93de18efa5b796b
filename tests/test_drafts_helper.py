"""The drafts' helper refuses host arrays that do not fit its batch, before anything reaches the GPU."""
import numpy as np
import pytest

from dequant_kvc8_store_gb300 import workloads as W
from dequant_kvc8_store_gb300.device import DeviceBatch, TreeAttention


@pytest.fixture(scope="module")
def batch():
    return DeviceBatch(W.make_workload("refused", q_lens=[3, 2], ctx_before=[5, 0], kv_heads=2, head_dim=64, block_size=16,
                                       num_blocks=4, quant_mode=0, seed=1), device="cpu")


@pytest.mark.parametrize("shape", [(4, 1), (6, 1), (5,), (5, 1, 1)])
def test_masks_of_another_number_of_drafts(batch, shape):
    TreeAttention(batch, 2, masks=np.ones((5, 1), np.uint64))
    with pytest.raises(ValueError):
        TreeAttention(batch, 2, masks=np.ones(shape, np.uint64))


@pytest.mark.parametrize("accepted,num", [((1, 3), (2,)), ((2, 3), (1,)), ((3, 3), (3,)), ((6,), (2,)), ((2, 3), (2, 1))])
def test_kept_drafts_of_another_number_of_sequences(batch, accepted, num):
    with pytest.raises(ValueError):
        TreeAttention(batch, 2).keep(np.zeros(accepted, np.int32), np.zeros(num, np.int32))
