"""The tree attention's outputs are the same bits whenever and beside whatever it runs: no sum's order depends on time."""
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from _drafts_ref import TreeProblem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("ctx,new", [([3000, 40, 700, 0], [20, 64, 1, 9]), ([20000, 20001], [64, 64]), ([900] * 40, [4] * 40)])
def test_the_same_bits_every_time(ctx, new, mode):
    kv.load()
    x = TreeProblem(ctx, new, H=4, G=4, D=128, mode=mode, sharp=False, seed=18)
    first = x.run().clone()
    other, side = torch.ones(1 << 22, device="cuda"), torch.cuda.Stream()
    for i in range(30):
        x.out.fill_(float("nan"))
        if i % 2:
            x.d["ws"].fill_(i)
        if i % 3 == 0:  # beside work of another stream
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(20):
                    other.mul_(1.0)
        assert torch.equal(first, x.run()), i
    torch.cuda.synchronize()
    assert x.error() == 0
