"""kvc8_compact_drafts and its bf16 form against a loop over the definition: whole pools, bit for bit."""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from _drafts_ref import compact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


class Problem:
    """mode None: bf16 pages."""

    def __init__(self, ctx, new, num, H=2, D=64, bs=16, mode=0, seed=0, most=None):
        rng = np.random.default_rng([seed, D, bs, H])
        B = len(ctx)
        self.mode, self.bs, self.ctx, self.num = mode, bs, np.array(ctx, np.int32), np.array(num, np.int32)
        self.MB = max(1, max([-(-(c + q) // bs) for c, q in zip(ctx, new)], default=1))
        NB = B * self.MB + 2
        self.table = rng.permutation(NB)[:B * self.MB].reshape(B, self.MB).astype(np.int32)
        self.most = most if most is not None else max([1] + list(num))
        self.acc = np.full((B, self.most), -5, np.int32)
        for b, (q, n) in enumerate(zip(new, num)):
            self.acc[b, :n] = np.sort(rng.permutation(q)[:n])
        shape = (NB, H, bs, D)
        if mode is None:
            self.k, self.v = (rng.integers(0, 65536, shape).astype(np.uint16).view(np.int16) for _ in range(2))
            self.ks = self.vs = None
        else:
            self.k, self.v = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
            s = [(NB, H, bs), (H, D), (NB, H)][mode]
            self.ks, self.vs = (np.exp2(rng.uniform(-9, -5, s)).astype(np.float32) for _ in range(2))
            if mode == 2:
                self.ks[::3] = self.ks[0]  # equal scales: rows move as they are
                self.vs[1::4] = 0.0
        self.g = kv.Geom(B, H, D, bs, NB, self.MB, 0 if mode is None else mode)

    def place(self):
        to = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.d = dict(k=to(self.k), v=to(self.v), table=to(self.table), ctx=to(self.ctx), acc=to(self.acc),
                      num=to(self.num), lens=torch.full((len(self.ctx),), -9, dtype=torch.int32, device="cuda"),
                      err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        if self.mode is not None:
            self.d.update(ks=to(self.ks), vs=to(self.vs))

    def call(self):
        d = self.d
        if self.mode is None:
            kv.kvc8_compact_drafts_bf16(self.g, d["k"], d["v"], d["table"], d["ctx"], d["acc"], self.most, d["num"],
                                        d["lens"], d["err"])
        else:
            kv.kvc8_compact_drafts(self.g, d["k"], d["v"], d["ks"], d["vs"], d["table"], d["ctx"], d["acc"], self.most,
                                   d["num"], d["lens"], d["err"])

    def check(self, num=None, lens=None, code=0):
        """num: the moves that are made (0 where a sequence is left as it is)."""
        k, v = self.k.copy(), self.v.copy()
        ks, vs = (None, None) if self.ks is None else (self.ks.copy(), self.vs.copy())
        made = self.num if num is None else num
        out = compact(self.mode, k, v, ks, vs, self.table, np.maximum(self.ctx, 0), self.acc, made, self.bs)
        assert kv.kvc8_get_error(self.d["err"], reset=True) == code
        for name, want in (("k", k), ("v", v), ("ks", ks), ("vs", vs)):
            if want is not None:
                assert np.array_equal(self.d[name].cpu().numpy().view(np.uint8), want.view(np.uint8)), name
        if self.d["lens"] is not None:
            assert self.d["lens"].cpu().tolist() == (out if lens is None else lens)

    def run(self):
        self.place()
        self.call()
        self.check()


MODES = [0, 1, 2, None]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("H,D,bs", [(1, 16, 1), (2, 64, 16), (5, 80, 24), (8, 128, 128), (3, 192, 77), (2, 256, 32),
                                    (40, 128, 16)])
def test_heads_and_blocks(H, D, bs, mode):
    Problem([37, 0, 15, 16, 100], [12, 1, 40, 9, 64], [5, 1, 17, 0, 8], H=H, D=D, bs=bs, mode=mode).run()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("num", [0, 1, 2, 7, 8, 9, 15, 16, 17, 64, 255, 256])
def test_counts(num, mode):
    """Moves around every multiple of what is in flight, dense paths among them: a row's place is another's source."""
    for extra in (0, 1, 3, 100):
        Problem([5, 30], [num + extra, num + 2 * extra], [num, num], mode=mode, seed=num + extra, most=256).run()


@pytest.mark.parametrize("mode", MODES)
def test_a_large_batch(mode):
    rng = np.random.default_rng(3)
    ctx = rng.integers(0, 200, 300).tolist()
    new = rng.integers(16, 65, 300).tolist()
    Problem(ctx, new, rng.integers(0, 17, 300).tolist(), H=3, D=128, bs=32, mode=mode).run()


@pytest.mark.parametrize("mode", MODES)
def test_bad_sequences_are_left_and_the_others_done(mode):
    def bad(change, sequence, code, lens):
        x = Problem([20, 21, 22], [16, 16, 16], [4, 4, 4], mode=mode, bs=16)
        change(x)
        x.place()
        x.call()
        made = [4, 4, 4]
        made[sequence] = 0
        x.check(made, lens, code)
    def set_acc(b, row):
        return lambda x: x.acc.__setitem__(b, row)
    bad(set_acc(1, [0, 3, 3, 5]), 1, kv.DEV_BAD_INDEX, [24, 21, 26])
    bad(set_acc(1, [2, 1, 4, 5]), 1, kv.DEV_BAD_INDEX, [24, 21, 26])
    bad(set_acc(2, [-1, 1, 4, 5]), 2, kv.DEV_BAD_INDEX, [24, 25, 22])
    bad(set_acc(0, [1, 4, 5, 1000]), 0, kv.DEV_POS_BEYOND_TABLE, [20, 25, 26])
    bad(lambda x: x.num.__setitem__(1, 5), 1, kv.DEV_BAD_LENGTH, [24, 21, 26])
    bad(lambda x: x.num.__setitem__(1, -1), 1, kv.DEV_BAD_LENGTH, [24, 21, 26])
    bad(lambda x: x.ctx.__setitem__(1, -1), 1, kv.DEV_BAD_LENGTH, [24, -1, 26])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_rows_of_blocks_outside_the_pool_do_not_move(bad, mode):
    x = Problem([16, 15], [30, 30], [3, 3], mode=mode, bs=16)
    x.acc[0], x.acc[1] = [1, 14, 18], [0, 1, 4]  # the third of sequence 0 lies in its third block
    kept = x.table.copy()
    x.table[0, 2] = bad
    x.place()
    x.call()
    x.table = kept
    x.check([2, 3], [19, 18], kv.DEV_BAD_BLOCK_ID)


@pytest.mark.parametrize("lens", ["context", None])
def test_lengths_in_place_or_not_wanted(lens):
    x = Problem([37, 0, 15], [12, 1, 40], [5, 1, 17], mode=1)
    x.place()
    x.d["lens"] = x.d["ctx"] if lens == "context" else None
    x.call()
    x.check()


def test_requantised_rows_near_ties_and_at_the_ends():
    """Ratios of powers of two and halves: every code's product is exact, ties go to even."""
    x = Problem([15], [40], [10], H=4, D=128, bs=16, mode=2, most=10)
    for s in (x.ks, x.vs):
        s[:] = np.array([1.0, 2.0, 0.5, 0.375], np.float32)[np.arange(s.shape[0]) % 4][:, None]
    for c in (x.k, x.v):
        c[:] = (np.arange(c.size) % 255 - 127).astype(np.int8).reshape(c.shape)
    x.run()


def test_a_replayed_graph_follows_its_lists():
    x = Problem([37, 0, 15], [12, 8, 40], [5, 3, 17], mode=0)
    x.place()
    x.call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.call()
    y = Problem([30, 9, 11], [19, 8, 33], [4, 0, 12], mode=0, seed=4, most=x.most)
    y.MB = x.MB
    for n in ("k", "v", "ks", "vs", "table"):
        setattr(y, n, getattr(x, n))
    for n in ("k", "v", "ks", "vs", "ctx", "acc", "num"):
        x.d[n].copy_(torch.from_numpy(getattr(y, n)))
    graph.replay()
    torch.cuda.synchronize()
    y.d = x.d
    y.check()
