"""Decode attention behind a shared prefix on inputs whose answers differ between heads,
sequences, and prefix and own positions, within a bound of about 1 % of an output (5 % where
single positions decide): _prefix_ref.py makes the inputs and derives the bound, and each check
also asserts that the answers of some mistakes would not pass it."""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from _prefix_ref import Problem

pytestmark = pytest.mark.gpu

LENGTHS = [(p, lens, D) for D in (64, 128) for p, lens in (
    (0, [0, 1, 5, 16, 17, 33]), (1, [0, 1, 5, 16, 17, 33]), (15, [3, 0, 64]), (16, [65, 2]), (17, [1, 1]),
    (127, [0, 31, 7]), (128, [0, 0, 48]), (129, [50]), (255, [12, 0]), (256, [9, 100]), (257, [0, 20]),
    (384, [40, 1, 5]), (1000, [70, 5, 16, 17, 33]))]
HEADS = [(1, 1, 128, 16), (2, 8, 128, 128), (3, 7, 64, 48), (8, 3, 128, 32), (5, 5, 64, 80), (1, 8, 64, 112),
         (4, 2, 128, 64)]
ROWS = [(B, G, D) for D in (64, 128) for B, G in ((1, 1), (1, 8), (15, 8), (16, 8), (17, 8), (31, 8), (32, 8),
                                                  (33, 8), (65, 4), (131, 3), (300, 1))]


def row_lens(B):
    return np.random.default_rng(B).integers(0, 50, B).tolist()


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


def _run(x):
    x.run()
    assert x.error() == 0
    x.check(x.out)


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("prefix,lens,D", LENGTHS)
def test_lengths(prefix, lens, D, mode, sharp):
    _run(Problem(prefix, lens, D=D, mode=mode, sharp=sharp, seed=1))


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("H,G,D,bs", HEADS)
def test_heads_and_blocks(H, G, D, bs, mode, sharp):
    _run(Problem(777, [40, 0, 130, 1, 64, 99, 3], H=H, G=G, D=D, bs=bs, mode=mode, sharp=sharp, seed=2))


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("B,G,D", ROWS)
def test_query_rows(B, G, D, mode, sharp):
    """Rows of a kv head around every multiple of a tile."""
    _run(Problem(400, row_lens(B), H=2, G=G, D=D, mode=mode, sharp=sharp, seed=3))


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_many_parts_and_own_splits(mode, sharp):
    _run(Problem(9001, [200, 0, 2049, 4100, 6200], H=2, G=3, D=128, bs=64, mode=mode, sharp=sharp, seed=4))


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("G", [3, 8])
def test_tables_with_room(G, mode, sharp):
    """Own positions and the prefix end far before their tables do."""
    lens = [500, 0, 7, 64] * 10
    _run(Problem(3000, lens, H=2, G=G, D=64, bs=32, mode=mode, sharp=sharp, seed=5, spare_prefix=400, spare_own=60))


@pytest.mark.parametrize("mode,H,G,D,lens_most", [(0, 8, 4, 128, 1024), (1, 8, 4, 128, 1024), (2, 8, 4, 128, 1024),
                                                  (0, 8, 8, 64, 300), (2, 3, 5, 128, 600)])
def test_a_large_batch_behind_a_long_prefix(mode, H, G, D, lens_most):
    """Several tiles of rows, hundreds of steps, every SM."""
    lens = np.random.default_rng(7).integers(0, lens_most, 256).tolist()
    _run(Problem(32768 - 7 * mode, lens, H=H, G=G, D=D, bs=128, mode=mode, sharp=mode != 1, seed=6))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_a_single_sequence_behind_the_longest_prefix(mode):
    _run(Problem(100003, [77], H=8, G=8, D=128, bs=64, mode=mode, sharp=False, seed=7))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_a_replayed_graph_follows_its_lengths(mode):
    x = Problem(2000, [100, 64, 31, 700], H=2, G=8, D=128, bs=32, mode=mode, sharp=False, seed=8)
    x.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.run()
    for prefix, lens in ((1999, [0, 5, 31, 64]), (0, [1, 1, 0, 700]), (17, [0, 0, 0, 0]), (2000, [100, 64, 31, 700])):
        x.prefix, x.lens = prefix, lens
        x.d["plen"].fill_(prefix)
        x.d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        x.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert x.error() == 0
        want, tol, wrong = x.answers()
        assert bool(((x.out.double() - want).abs() <= tol).all()), prefix
        # (the weights were balanced for the first lengths: not every mistake shows at the others)
        x.tells(want, tol, {k: wrong[k] for k in ("zeros", "the next head's")})


LIMITS = [  # modes, and powers of two on value scales, key scales and queries
    ((0, 2), -66, 0, 0), ((0, 2), 65, 0, 0), ((0, 2), 0, -106, 0), ((0, 2), 0, 105, 0), ((0, 1, 2), 0, 0, -103),
    ((0, 1, 2), 0, 0, 96), ((0, 2), -66, -50, -53), ((1,), -66, -90, 0), ((1,), 65, 90, 0)]


@pytest.mark.parametrize("mode,values,keys,query",
                         [(m, v, k, q) for modes, v, k, q in LIMITS for m in modes])
def test_scales_and_queries_at_the_ends_of_their_range(mode, values, keys, query):
    """Value scales from 2^-74 to 2^60, key scales from 2^-114 to 2^100, queries from 2^-100 to
    2^100 (the softmax's scale takes the powers of the last two back)."""
    x = Problem(300, [40, 0, 130], H=2, G=4, D=128, bs=32, mode=mode, seed=9)
    x.vs *= 2.0 ** values
    x.ks *= 2.0 ** keys
    x.q = (x.q.float() * 2.0 ** query).to(torch.bfloat16)
    x.scale *= 2.0 ** -(keys + query)
    _run(x)


@pytest.mark.parametrize("mode", [0, 2])
@pytest.mark.parametrize("values", [-70, -76, -84, -100])
def test_value_scales_below_their_range(mode, values):
    """A prefix's value is then off by 2^-78 at most, its own positions' as above."""
    x = Problem(300, [40, 0, 130], H=2, G=4, D=128, bs=32, mode=mode, seed=10)
    x.vs *= 2.0 ** values
    x.run()
    assert x.error() == 0
    want, tol, _ = x.answers(least=2.0 ** -78)
    assert bool(((x.out.double() - want).abs() <= tol).all())
    x.prefix, x.out = 0, torch.full_like(x.out, float("nan"))
    x.d["plen"].fill_(0)
    _run(x)
