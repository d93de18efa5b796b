"""kvc8_assign_blocks against a loop over its definition: tables, stack, slots and reports, bit for bit."""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from _drafts_ref import assign

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


def up(a, b):
    return -(-a // b)


class Problem:
    def __init__(self, held, want, bs, MB=None, free=None, spare=5, seed=0, slot_rows=None, NB=None):
        rng = np.random.default_rng([seed, len(held), bs])
        self.held, self.want, self.bs, self.slot_rows = list(held), list(want), bs, slot_rows
        self.MB = MB if MB is not None else max([1] + [up(max(h, w), bs) + 1 for h, w in zip(held, want)])
        cap = self.MB * bs
        have = [up(min(max(h, 0), cap), bs) for h in held]
        need = sum(max(0, up(w, bs) - up(h, bs)) for h, w in zip(held, want) if 0 <= h <= cap and 0 <= w <= cap)
        free = need + spare if free is None else free
        self.NB = NB if NB is not None else max(1, sum(have) + max(free, 0) + 3)
        ids = rng.permutation(max(self.NB, sum(have) + max(free, 0))).astype(np.int32)
        self.table = np.full((len(held), self.MB), -1, np.int32)
        at = 0
        for b, n in enumerate(have):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.free = np.full(self.NB, -7, np.int32)
        n = min(max(free, 0), self.NB)
        self.free[:n] = ids[at:at + n]
        self.count = free

    def place(self):
        i32 = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
        rows = sum(max(0, w - max(h, 0)) for h, w in zip(self.held, self.want)) if self.slot_rows is None else self.slot_rows
        self.d = dict(held=i32(self.held), want=i32(self.want), free=i32(self.free), count=i32([self.count]),
                      out=i32([-9]), table=i32(self.table), lens=i32([-9] * len(self.held)), err=i32([0]),
                      slots=torch.full((rows + 8,), -99, dtype=torch.int64, device="cuda"), rows=rows)
        self.g = kv.Geom(len(self.held), 2, 64, self.bs, self.NB, self.MB, 0)

    def call(self, stream=None, **other):
        d = {**self.d, **other}
        kv.kvc8_assign_blocks(self.g, d["held"], d["want"], d["free"], d["count"], d["out"], d["table"], d["lens"],
                              d["slots"], d["rows"], d["err"], stream)

    def want_all(self):
        return assign(self.held, self.want, self.free, self.count, self.table, self.bs, self.NB, self.d["rows"])

    def check(self, want=None, errors=None):
        free, count, table, lens, slots, codes = self.want_all() if want is None else want
        d, got = self.d, {}
        code = kv.kvc8_get_error(d["err"])
        assert code in codes if codes else code == 0, (code, codes)
        assert d["table"].cpu().numpy().tolist() == [list(map(int, r)) for r in table]
        assert d["free"].cpu().tolist() == list(map(int, free))
        assert d["lens"].cpu().tolist() == lens
        assert int(d["out"]) == count
        assert d["slots"].cpu().tolist() == list(map(int, slots)) + [-99] * (d["slots"].numel() - len(slots))

    def run(self):
        self.place()
        self.call()
        self.check()


def lengths(rng, B, most, new, gone):
    held = rng.integers(0, most + 1, B).tolist()
    want = [int(rng.choice([0, h // 2, max(0, h - 1)])) if rng.random() < gone else h + int(rng.integers(0, new + 1)) for h in held]
    return held, want


@pytest.mark.parametrize("bs", [1, 3, 16, 128])
@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 257])
def test_growth_and_release(B, bs):
    rng = np.random.default_rng([B, bs])
    for gone in (0.0, 0.4, 1.0):
        for most, new in ((0, 1), (5, 3), (200, 90)):
            Problem(*lengths(rng, B, most, new, gone), bs, seed=B).run()


@pytest.mark.parametrize("B", [0, 1])
def test_nothing_to_do(B):
    x = Problem([17] * B, [17] * B, 16, free=4)
    x.run()
    assert int(x.d["out"]) == 4


@pytest.mark.parametrize("B", [1023, 1024, 1025, 4096, 8192])
def test_many_sequences(B):
    rng = np.random.default_rng(B)
    Problem(*lengths(rng, B, 300, 60, 0.3), 32, seed=1).run()
    x = Problem(*lengths(rng, B, 300, 60, 0.1), 16, seed=2)
    x = Problem(x.held, x.want, 16, free=x.count // 3, seed=3)  # the stack runs short
    x.run()
    assert kv.kvc8_get_error(x.d["err"]) == kv.DEV_NO_FREE_BLOCK


def test_long_prompts():
    Problem([0, 5, 0, 70000], [131072, 9, 40000, 131000], 16, seed=4).run()
    Problem([0], [30011], 1, seed=5).run()


@pytest.mark.parametrize("free", [0, 1, 2, 3, 7, 8])
def test_a_stack_that_runs_short_serves_whole_sequences_in_order(free):
    # needs 1, 3, 0, 2, 1 blocks; one is given back by the last
    Problem([0, 4, 9, 8, 3, 12], [4, 14, 11, 13, 8, 8], 4, free=free).run()


def test_popped_blocks_are_the_ones_just_pushed():
    x = Problem([64, 0, 48], [0, 40, 16], 16, free=0, spare=0)
    x.run()
    assert int(x.d["out"]) == 3 and set(x.d["table"][1, :3].tolist()) <= set(x.table[0, :4].tolist() + x.table[2, :3].tolist())


@pytest.mark.parametrize("held,want,code", [
    ([5, -1, 5], [9, 4, 30], kv.DEV_BAD_LENGTH), ([5, 7, 5], [9, -4, 30], kv.DEV_BAD_LENGTH),
    ([5, 7, 5], [9, 65, 30], kv.DEV_POS_BEYOND_TABLE), ([5, 65, 5], [9, 3, 30], kv.DEV_POS_BEYOND_TABLE),
    ([64, 0, 0], [0, 64, 64], 0)])
def test_lengths_out_of_range(held, want, code):
    x = Problem(held, want, 8, MB=8)
    x.run()
    assert kv.kvc8_get_error(x.d["err"]) == code


@pytest.mark.parametrize("count,NB", [(-3, 40), (41, 40), (39, 40), (40, 40)])
def test_counts_out_of_range_and_a_full_stack(count, NB):
    """Pushes beyond the pool's size are dropped."""
    Problem([33, 20, 0], [1, 0, 9], 4, free=count, NB=NB).run()


def test_slots_beyond_their_room_are_not_written():
    x = Problem([3, 0, 9], [30, 11, 12], 4, slot_rows=20)
    x.run()
    assert kv.kvc8_get_error(x.d["err"]) == kv.DEV_OUT_ROW_RANGE
    x = Problem([3, 0, 9], [30, 11, 12], 4)  # without a slot map
    x.place()
    x.call(slots=None, rows=0)
    x.check(want=x.want_all()[:4] + ([], set()))


def test_ids_outside_the_pool_are_reported_and_moved():
    x = Problem([9, 0], [0, 9], 4, free=2)
    x.table[0, 1] = 10 ** 6
    x.run()
    assert kv.kvc8_get_error(x.d["err"]) == kv.DEV_BAD_BLOCK_ID


@pytest.mark.parametrize("alias", ["held", "want"])
def test_outputs_in_place_of_inputs(alias):
    rng = np.random.default_rng(5)
    for B in (3, 700, 5000):
        x = Problem(*lengths(rng, B, 90, 70, 0.4), 16, seed=6)
        x.place()
        want = x.want_all()
        x.d["lens"], x.d["out"] = x.d[alias], x.d["count"]
        x.call()
        x.check(want)


def test_a_replayed_graph_follows_its_lengths_on_another_stream():
    rng = np.random.default_rng(6)
    x = Problem(*lengths(rng, 300, 200, 100, 0.3), 16, seed=7, MB=40, slot_rows=40000)
    x.place()
    x.call()
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        x.call()
    for seed in (8, 9):
        y = Problem(*lengths(rng, 300, 200, 100, 0.5), 16, seed=seed, MB=40, slot_rows=40000, NB=x.NB)
        y.place()
        for k in ("held", "want", "free", "count", "table"):
            x.d[k].copy_(y.d[k])
        x.d["slots"].fill_(-99)
        x.d["err"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        y.d, y.g = x.d, x.g
        y.check()


@pytest.mark.parametrize("alias", ["held", "want", None])
def test_slots_of_a_launch_of_their_own_with_outputs_in_place_and_replayed(alias):
    rng = np.random.default_rng(11)
    x = Problem(*lengths(rng, 4096, 90, 150, 0.2), 16, seed=12)
    x.place()
    want = x.want_all()
    assert x.d["slots"].numel() > 1 << 17
    if alias is not None:
        x.d["lens"], x.d["out"] = x.d[alias], x.d["count"]
    first = {k: x.d[k].clone() for k in ("held", "want", "free", "count", "table")}
    x.call()
    x.check(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # the inputs again, the call, twice
        for _ in range(2):
            for k, v in first.items():
                x.d[k].copy_(v)
            x.call()
    x.d["slots"].fill_(-99)
    graph.replay()
    torch.cuda.synchronize()
    x.check(want)
