"""The inputs, bounds and loops of the drafted tokens' GPU tests, on the CPU."""
import numpy as np
import pytest
import torch

import _drafts_ref as R

CASES = [([37], [4]), ([0, 5, 300], [1, 7, 33]), ([100, 0, 64, 1], [2, 1, 65, 16])]


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
def test_bound_holds_for_the_kernels_roundings(kind, mode, sharp):
    for ctx, new in CASES:
        for D, G, H in ((64, 4, 2), (128, 7, 3)):
            x = R.TreeProblem(ctx, new, H=H, G=G, D=D, mode=mode, kind=kind, sharp=sharp, seed=1, device="cpu")
            x.check(x.rounded())


def test_a_wrong_answer_does_not_pass():
    x = R.TreeProblem([100, 0, 64], [20, 3, 33], D=128, bs=32, sharp=False, device="cpu")
    good = x.rounded()
    x.check(good)
    for name, (out, _) in x.answers()[2].items():
        with pytest.raises(AssertionError):
            x.check(out.to(torch.bfloat16))
    one = good.clone()
    one[5, 3, 77] = float("nan")
    with pytest.raises(AssertionError):
        x.check(one)


def test_assignment_by_hand():
    # blocks of 4; row 0 gives its second and third block, row 1 needs two, row 2 stays
    table = [[7, 8, 9], [1, -1, -1], [2, 3, -1]]
    free, count, table, lens, slots, errors = R.assign([9, 3, 5], [2, 9, 7], [5, 6] + [0] * 8, 2, table, 4, 10)
    assert free[:4] == [5, 6, 8, 9] and count == 2 and table[1] == [1, 9, 8] and not errors
    assert lens == [2, 9, 7] and slots == [1 * 4 + 3, 36, 37, 38, 39, 32, 13, 14]
    # one block is too few: sequence 0 gets it, 1 does not, 2 needs none, 3 would fit but comes later
    out = R.assign([0, 4, 5, 0], [3, 12, 6, 2], [0], 1, [[-1, -1, -1], [1, -1, -1], [2, 3, -1], [-1, -1, -1]], 4, 10)
    assert out[1] == 0 and out[3] == [3, 4, 6, 0] and out[4] == [0, 1, 2] + [-1] * 8 + [13] + [-1] * 2
    assert out[5] == {6}


def test_compaction_by_hand():
    k = np.arange(2 * 1 * 4 * 16, dtype=np.int64).reshape(2, 1, 4, 16) % 101 - 50
    k = k.astype(np.int8)
    v, want = k[::-1].copy(), k.copy()
    s = np.array([[0.5], [0.25]], np.float32)
    # positions 0..3 in block 1, 4..7 in block 0; context 3, drafts 0, 2, 3 kept: position 3 stays, 5 -> 4, 6 -> 5
    want[0, 0, 0], want[0, 0, 1] = k[0, 0, 1], k[0, 0, 2]
    assert R.compact(2, k, v, s, s.copy(), [[1, 0]], [3], [[0, 2, 3]], [3], 4) == [6]
    assert np.array_equal(k, want)
    # from block 0 (scale 1/2) to block 1 (1/4): codes double, clamped
    x = k[0, 0, 1].copy()
    R.compact(2, k, v, s, s.copy(), [[1, 0]], [3], [[2]], [1], 4)
    assert np.array_equal(k[1, 0, 3], np.clip(2 * x.astype(int), -127, 127))
