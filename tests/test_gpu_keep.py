"""TreeAttention.keep on a stream that is not torch's current one."""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import workloads as W
from dequant_kvc8_store_gb300.device import DeviceBatch, TreeAttention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["current", "stream", "address", "default"])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_keep_on_a_stream_that_is_behind(mode, form):
    """The stream is held back while torch's current one takes and overwrites whatever memory is free."""
    kv.load()
    w = W.make_workload("keep", q_lens=[9, 4, 30], ctx_before=[40, 0, 77], kv_heads=2, head_dim=64, block_size=16,
                        num_blocks=32, quant_mode=mode, seed=mode)
    accepted = np.zeros((3, 12), np.int32)
    num = [5, 0, 12]
    for b, path in enumerate(([1, 2, 5, 6, 8], [], [0, 2, 3, 7, 9, 11, 14, 15, 20, 22, 28, 29])):
        accepted[b, :len(path)] = path
    want = DeviceBatch(w)
    want.store()
    lens = TreeAttention(want, 2).keep(accepted, num)
    assert lens.tolist() == [45, 0, 89]
    d = DeviceBatch(w)
    d.store()
    tree, behind = TreeAttention(d, 2), torch.cuda.Stream()
    torch.cuda.synchronize()
    on = {"current": torch.cuda.current_stream(), "default": torch.cuda.default_stream()}.get(form, behind)
    with torch.cuda.stream(on):
        torch.cuda._sleep(200_000_000)
    got = tree.keep(accepted, num, {"current": None, "stream": behind, "address": behind.cuda_stream, "default": 0}[form])
    junk = [torch.full((n,), 1 << 20, dtype=torch.int32, device="cuda") for n in (3, 36) for _ in range(64)]
    torch.cuda.synchronize()
    assert d.error_code() == 0 and torch.equal(got, lens) and len(junk) == 128
    for x, y in zip(d.host_caches(), want.host_caches()):
        assert np.array_equal(x, y)
