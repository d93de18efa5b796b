"""Decode attention behind a shared prefix (kvc8_shared_prefix_attention) against
an fp64 evaluation over fp32(code) * scale.

The operands of the products are allowed the rounding of bf16 (the kernel rounds most
of them to fp16, eight times finer): each weight (times a row's or block's value
scale) moves by a relative 2^-8 at most, the query (times the key scale) and the
keys move a score by 2^-8 * scale * sum_d |q_d k_d| each, each value moves by 2^-8.  The
fp32 accumulation of D products moves a score by D * 2^-24 of the same sum.  So with
    delta = scale * max_p sum_d |q_d k_pd| * (2 * 2^-8 + D * 2^-24)
a weight is off by a relative eps = 2^-8 + expm1(delta), the normalised average of
values by 2 eps max|V| + 2^-8 max|V|, and the output's rounding adds 2^-8 |out|.
"""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300.device import bf16_bits
from _rope_ref import (BF16, U, attend, bf16_f64, bf16_tensor, fixed_point, inv_freq, norm_rotate,
                       to_bf16_bits)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


class Batch:
    """A pool, a prefix, own pages and queries."""

    def __init__(self, prefix, lens, H=2, G=4, D=64, bs=16, mode=0, seed=0, spare_prefix=1,
                 spare_own=1):
        rng = np.random.default_rng([seed, prefix, len(lens), D])
        self.prefix, self.lens, self.H, self.G, self.D, self.bs, self.mode = prefix, list(lens), H, G, D, bs, mode
        B = len(self.lens)
        self.PB = max(1, -(-prefix // bs) + spare_prefix)
        self.MB = max(1, -(-max(self.lens, default=0) // bs) + spare_own)
        NB = self.PB + B * self.MB + 2
        ids = rng.permutation(NB).astype(np.int32)
        self.ptab, self.tab = ids[:self.PB].copy(), ids[self.PB:self.PB + B * self.MB].reshape(B, self.MB).copy()
        shape = (NB, H, bs, D)
        self.kc, self.vc = (rng.integers(-127, 128, shape).astype(np.int8) for _ in range(2))
        sshape = [(NB, H, bs), (H, D), (NB, H)][mode]
        self.ks, self.vs = (rng.uniform(0.004, 0.02, sshape).astype(np.float32) for _ in range(2))
        self.qb = to_bf16_bits(rng.standard_normal((B, H * G, D)))
        self.scale = D ** -0.5
        self.g = kv.Geom(B, H, D, bs, NB, self.MB, mode)
        self.dev()

    def dev(self):
        c = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.d = dict(kc=c(self.kc), vc=c(self.vc), ks=c(self.ks), vs=c(self.vs), ptab=c(self.ptab),
                      tab=c(self.tab), q=bf16_tensor(self.qb).cuda(),
                      plen=torch.tensor([self.prefix], dtype=torch.int32).cuda(),
                      lens=torch.tensor(self.lens, dtype=torch.int32).cuda(),
                      err=torch.zeros(1, dtype=torch.int32).cuda())
        need = kv.kvc8_shared_prefix_workspace_bytes(self.g, self.H * self.G, self.PB)
        self.d["ws"] = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        self.out = torch.full_like(self.d["q"], float("nan"))

    def run(self, out=None, q=None, stream=None, scale=None):
        d, o = self.d, self.out if out is None else out
        q = d["q"] if q is None else q
        kv.kvc8_shared_prefix_attention(self.g, self.H * self.G, q, q.stride(0), q.stride(1), d["kc"],
                                        d["vc"], d["ks"], d["vs"], d["ptab"], self.PB, d["plen"],
                                        d["tab"], d["lens"], self.scale if scale is None else scale, o,
                                        o.stride(0), o.stride(1), d["ws"], d["ws"].numel(), d["err"],
                                        stream)
        return o

    def error(self):
        return kv.kvc8_get_error(self.d["err"], reset=True)

    def rows(self, cache, scale, table, count, h):
        p = np.array([i for i in range(count) if 0 <= table[i // self.bs] < self.g.num_blocks], np.int64)
        ids, at = table[p // self.bs], p % self.bs
        x = cache[ids, h, at].astype(np.float64)
        s = scale.astype(np.float64)
        return x * (s[ids, h, at][:, None] if self.mode == 0 else s[h][None] if self.mode == 1 else s[ids, h][:, None])

    def check(self, out=None, scale=None):
        scale = self.scale if scale is None else scale
        got = bf16_f64(bf16_bits(self.out if out is None else out))
        for h in range(self.H):
            pk, pv = (self.rows(c, s, self.ptab, min(self.prefix, self.PB * self.bs), h)
                      for c, s in ((self.kc, self.ks), (self.vc, self.vs)))
            for b in range(len(self.lens)):
                n = min(self.lens[b], self.MB * self.bs)
                k = np.concatenate([pk, self.rows(self.kc, self.ks, self.tab[b], n, h)])
                v = np.concatenate([pv, self.rows(self.vc, self.vs, self.tab[b], n, h)])
                j = slice(h * self.G, (h + 1) * self.G)
                want = attend(self.qb[b, j], k, v, scale)
                if not len(k):
                    assert not got[b, j].any()
                    continue
                size = np.abs(bf16_f64(self.qb[b, j])) @ np.abs(k).T
                delta = abs(scale) * size.max(-1, keepdims=True) * (2 * BF16 + self.D * U)
                top = np.abs(v).max(0)[None]
                tol = (2 * (BF16 + np.expm1(delta)) + BF16) * top + BF16 * np.abs(want)
                bad = ~(np.abs(got[b, j] - want) <= tol)
                fine = not bad.any()
                assert fine, (b, h, np.argwhere(bad)[:4], got[b, j][bad][:4], want[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 384, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_prefix_lengths(prefix, D):
    x = Batch(prefix, [0, 1, 5, 16, 17, 33], D=D, seed=1)
    x.run()
    assert x.error() == 0
    x.check()


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("H,G,D,bs", [(1, 1, 128, 16), (2, 8, 128, 128), (3, 7, 64, 48), (8, 3, 128, 32),
                                      (5, 5, 64, 80), (1, 8, 64, 112), (4, 2, 128, 64)])
def test_heads_blocks_and_modes(H, G, D, bs, mode):
    x = Batch(777, [40, 0, 130, 1, 64, 99, 3], H=H, G=G, D=D, bs=bs, mode=mode, seed=2)
    x.run()
    assert x.error() == 0
    x.check()


@pytest.mark.parametrize("B,G", [(1, 1), (1, 8), (15, 8), (16, 8), (17, 8), (31, 8), (32, 8), (33, 8),
                                 (65, 4), (131, 3), (300, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_query_row_counts(B, G, D):
    """Rows of a kv head around every multiple of a tile."""
    rng = np.random.default_rng(B)
    x = Batch(400, rng.integers(0, 50, B).tolist(), H=2, G=G, D=D, seed=3)
    x.run()
    assert x.error() == 0
    x.check()


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_long_prefix_many_parts(mode):
    x = Batch(9001, [200, 0, 2049, 4100], H=2, G=3, D=128, bs=64, mode=mode, seed=4)
    x.run()
    assert x.error() == 0
    x.check()


@pytest.mark.parametrize("lens", [[0] * 40, [0] * 39 + [2500], [2500, 0, 7, 64] * 10, [2500] * 40])
@pytest.mark.parametrize("G", [3, 8])
def test_tables_with_room_for_more(lens, G):
    """The same tables more or less full: the work is cut by what is in them."""
    x = Batch(5000, lens, H=2, G=G, D=64, bs=32, mode=1, seed=30, spare_own=80 - max(lens) // 32)
    x.run()
    assert x.error() == 0
    x.check()


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_many_calls_of_many_sequences(mode):
    """Enough work items for every SM to take several, twice, with other data in between
    (nothing left over from an earlier item or call is read)."""
    rng = np.random.default_rng(40)
    lens = rng.integers(0, 40, 200).tolist()
    x = Batch(300, lens, H=4, G=8, D=128, bs=32, mode=mode, seed=21)
    y = Batch(150, lens, H=4, G=8, D=64, bs=16, mode=mode, seed=22)
    y.qb[:] = to_bf16_bits(30 * rng.standard_normal(y.qb.shape))
    y.dev()
    y.run(scale=0.01)
    x.run()
    first = x.out.clone()
    y.run(scale=0.01)
    x.run()
    assert torch.equal(first, x.out)
    assert x.error() == 0 and y.error() == 0
    x.check()
    y.check(scale=0.01)


def test_equal_values_come_back():
    """Weights that sum to one: a constant V gives that constant, whatever the split of the
    positions."""
    for mode in (0, 1, 2):
        x = Batch(1234, [0, 7, 300], H=2, G=8, D=128, bs=32, mode=mode, seed=5)
        x.vc[:] = 100
        x.vs[:] = 0.5  # a power of two: the product with a weight is exact
        x.dev()
        x.run()
        assert x.error() == 0
        got = bf16_f64(bf16_bits(x.out))
        # numerator and denominator see weights rounded differently: 2^-8, and the output's 2^-8
        fine = bool((np.abs(got - 50.0) <= 50.0 * (2 * BF16 + 2.0 ** -12)).all())
        assert fine


@pytest.mark.parametrize("D,mode", [(64, 0), (128, 0), (128, 1), (64, 2)])
def test_each_position_reaches_its_own_value(D, mode):
    """One position holds the only key along the query, far above the rest: the output is its
    value.  Walks over tile, page and part borders, in the prefix and behind it."""
    prefix, own = 530, 70
    x = Batch(prefix, [own] * 3, H=1, G=2, D=D, bs=16, mode=mode, seed=6)
    x.ks[:], x.vs[:] = 0.01, 0.01
    x.qb[:] = to_bf16_bits(np.ones(D))
    x.dev()
    spots = [0, 1, 15, 16, 63, 64, 127, 128, 129, 255, 256, 383, 384, 511, 512, prefix - 1]
    for where, p in [("pre", s) for s in spots] + [("own", s) for s in (0, 15, 16, 17, 63, 64, own - 1)]:
        x.kc[:] = 0
        if where == "pre":
            x.kc[x.ptab[p // 16], :, p % 16] = 127
            want = np.stack([x.vc[x.ptab[p // 16], 0, p % 16]] * 3)
        else:
            for b in range(3):
                x.kc[x.tab[b, p // 16], :, p % 16] = 127
            want = x.vc[x.tab[:, p // 16], 0, p % 16]
        x.d["kc"].copy_(torch.from_numpy(x.kc))
        x.run(scale=4.0)  # e^-(4 * 1.27 * 64) is nothing beside 1
        got = bf16_f64(bf16_bits(x.out))
        want = want.astype(np.float64)[:, None] * np.float64(np.float32(0.01))
        # weight 1 times the scale in bf16, and the output in bf16
        fine = bool((np.abs(got - want) <= (2 * BF16 + 2.0 ** -15) * np.abs(want) + 1e-30).all())
        assert fine, (where, p)
    assert x.error() == 0


def test_growing_scores_rescale_the_sums():
    """Keys that get longer along the prefix: the running maximum keeps moving."""
    for D in (64, 128):
        x = Batch(1500, [100, 0, 31], H=2, G=4, D=D, bs=32, mode=0, seed=7)
        grow = np.linspace(0.0001, 0.05, x.PB * 32).astype(np.float32)
        for i in range(x.PB * 32):
            x.ks[x.ptab[i // 32], :, i % 32] = grow[i]
        x.dev()
        x.run(scale=1.0)
        assert x.error() == 0
        x.check(scale=1.0)


def test_scores_far_below_and_above_zero():
    """Scores in the thousands, positive and negative, and a scale of zero."""
    x = Batch(300, [20, 0], H=1, G=8, D=128, bs=16, mode=2, seed=8)
    x.kc[:] = np.abs(x.kc)
    x.qb[:, :4] = to_bf16_bits(np.full((2, 4, 128), 3.0))
    x.qb[:, 4:] = to_bf16_bits(np.full((2, 4, 128), -3.0))
    x.dev()
    for scale in (0.0, 1e-3):
        x.run(scale=scale)
        assert x.error() == 0
        x.check(scale=scale)
    x.run(scale=2.0)  # a single weight is left: finite and inside the values' range
    got = bf16_f64(bf16_bits(x.out))
    assert np.isfinite(got).all() and (np.abs(got) <= 127 * 0.02 * 1.01).all()


def test_values_of_very_different_scales():
    """A position with most of the weight and a tiny value scale beside large ones."""
    x = Batch(260, [9], H=1, G=2, D=64, bs=16, mode=0, seed=9)
    x.vs[:] = 1e4
    x.vs[x.ptab[0], :, 0] = 1e-6
    x.ks[x.ptab[0], :, 0] = 0.2
    x.dev()
    x.run()
    assert x.error() == 0
    x.check()


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_many_faint_positions_behind_one_strong(mode, where):
    """The strong position's value is zero, so that the output is the sum of weights 2^-20.4 of
    its own: each is still held to bf16's precision."""
    x = Batch(*((600, [0, 0]) if where == "prefix" else (0, [600, 600])), H=1, G=2, D=64, mode=mode, seed=23)
    x.ks[:], x.vs[:] = 2.0 ** -7, 2.0 ** -7
    x.qb[:] = to_bf16_bits(np.ones(64))
    x.kc[:] = 0
    x.vc[:] = np.maximum(np.abs(x.vc), 1)
    first = [x.ptab[0]] if where == "prefix" else list(x.tab[:, 0])
    x.kc[first, :, 0], x.vc[first, :, 0] = 127, 0
    x.dev()
    scale = 20.4 * np.log(2.0) / (64 * 127 * 2.0 ** -7)
    x.run(scale=scale)
    assert x.error() == 0
    got = bf16_f64(bf16_bits(x.out))
    for b in range(2):
        table, n = (x.ptab, 600) if where == "prefix" else (x.tab[b], 600)
        k, v = x.rows(x.kc, x.ks, table, n, 0), x.rows(x.vc, x.vs, table, n, 0)
        want = attend(x.qb[b], k, v, scale)
        # all terms are positive: the weights' and the output's 2^-8, the scale's 2^-11 or less,
        # and 2^-11 for fp32 sums and the strong score (24 bits of 14)
        assert (np.abs(got[b] - want) <= (2 * BF16 + 2.0 ** -10) * want).all()


def test_zero_rows_beside_others():
    """Rows of zeros are kept with scale 0: alone in their sixteen, among others, everywhere."""
    x = Batch(500, [40, 0], H=2, G=4, D=128, mode=0, seed=24)
    for i in [*range(32, 48), 50, 51, 200]:
        b, at = x.ptab[i // 16], i % 16
        for cache, s in ((x.kc, x.ks), (x.vc, x.vs)):
            cache[b, :, at], s[b, :, at] = 0, 0.0
    x.dev()
    x.run()
    assert x.error() == 0
    x.check()
    x.vc[:], x.vs[:] = 0, 0.0
    x.dev()
    x.run(scale=40.0)  # scores that keep moving the maximum
    assert x.error() == 0
    assert not (bf16_bits(x.out) & 0x7FFF).any()


def test_more_splits_than_the_grid_takes_at_once():
    """Thousands of sequences with room for long contexts: a block walks several splits."""
    rng = np.random.default_rng(25)
    B, H = 2100, 2
    x = Batch(40, [1] * B, H=H, G=1, D=64, mode=0, seed=26)
    x.MB = 400
    x.tab = rng.integers(0, x.g.num_blocks, (B, x.MB)).astype(np.int32)
    x.lens = rng.integers(0, 20, B).tolist()
    x.lens[0], x.lens[1234], x.lens[B - 1] = 6400, 4097, 2049
    x.g = kv.Geom(B, H, 64, 16, x.g.num_blocks, x.MB, 0)
    x.dev()
    x.run()
    assert x.error() == 0
    x.check()


def test_output_on_any_element():
    x = Batch(300, [40, 0, 3], H=2, G=4, D=128, seed=27)
    first = x.run().clone()
    base = torch.full((x.out.numel() + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    for at in (1, 3, 8):
        base.fill_(7.0)
        out = base[at:at + x.out.numel()].view(x.out.shape)
        x.run(out=out)
        assert torch.equal(out, first)
        assert (base[:at] == 7).all() and (base[at + x.out.numel():] == 7).all()
    assert x.error() == 0


def test_two_graphs_share_a_workspace():
    """Replayed in turn on one stream: a call leaves nothing in the workspace that a later one
    reads."""
    xs = [Batch(900, [70, 0, 9], H=2, G=8, D=128, bs=32, mode=0, seed=28),
          Batch(2500, [5, 2100], H=4, G=3, D=64, bs=16, mode=1, seed=29)]
    ws = torch.full((max(x.d["ws"].numel() for x in xs),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for x in xs:
        x.d["ws"] = ws
        x.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            x.run()
    for _ in range(3):
        for x, graph in zip(xs, graphs):
            x.out.fill_(float("nan"))
            graph.replay()
    torch.cuda.synchronize()
    for x in xs:
        assert x.error() == 0
        x.check()


def test_strided_query_and_output_rows_beyond_untouched():
    x = Batch(333, [10, 0, 44], H=2, G=4, D=128, bs=16, seed=10)
    hm = x.d["q"].transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.full((5, 11, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    o = wide[1:4, 2:10]
    x.run(out=o, q=hm)
    assert x.error() == 0
    x.check(out=o)
    assert (wide[0] == 7).all() and (wide[4] == 7).all() and (wide[:, :2] == 7).all() and (wide[:, 10:] == 7).all()


@pytest.mark.parametrize("mode", [0, 2])
def test_bad_pages_are_left_out_and_reported(mode):
    x = Batch(700, [40, 64, 3], H=2, G=4, D=128, bs=16, mode=mode, seed=11)
    x.ptab[3], x.ptab[20], x.ptab[43] = -1, x.g.num_blocks, 2 ** 31 - 1
    x.tab[1, 2] = -5
    x.dev()
    x.run()
    assert x.error() == kv.DEV_BAD_BLOCK_ID
    x.check()
    # nothing left at all: zeros
    y = Batch(50, [20, 0], H=1, G=2, D=64, bs=16, mode=mode, seed=12)
    y.ptab[:] = -1
    y.tab[:] = -1
    y.dev()
    y.run()
    assert y.error() == kv.DEV_BAD_BLOCK_ID
    assert not bf16_bits(y.out).any()


def test_bad_lengths_are_clamped_and_reported():
    x = Batch(64, [16, 8], H=1, G=2, D=64, bs=16, seed=13, spare_prefix=0, spare_own=0)
    x.prefix = 10 ** 6
    x.dev()
    x.run()
    assert x.error() == kv.DEV_POS_BEYOND_TABLE
    x.check()
    x.prefix, x.lens = 30, [-3, 500]
    x.dev()
    x.run()
    assert x.error() in (kv.DEV_BAD_LENGTH, kv.DEV_POS_BEYOND_TABLE)
    x.lens[0] = 0
    x.check()
    x.prefix, x.lens = -7, [16, 8]
    x.dev()
    x.run()
    assert x.error() == kv.DEV_BAD_LENGTH
    x.prefix = 0
    x.check()


def test_same_call_twice_is_bit_identical_and_graph_replays_follow():
    x = Batch(2000, [100, 0, 31, 700], H=2, G=8, D=128, bs=32, seed=14)
    first = x.run().clone()
    again = x.run(out=torch.zeros_like(x.out))
    torch.cuda.synchronize()
    assert torch.equal(first, again)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x.run(stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.run()
    for prefix, lens in ((1999, [0, 5, 31, 64]), (0, [1, 1, 0, 700]), (17, [0, 0, 0, 0]), (2000, [100, 0, 31, 700])):
        x.prefix, x.lens = prefix, lens
        x.d["plen"].fill_(prefix)
        x.d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert x.error() == 0
        x.check()
    assert torch.equal(first, x.out)


def test_two_streams_with_their_own_workspaces():
    xs = [Batch(1500 + 100 * i, [50, 9, 0], H=2, G=4, D=128, bs=16, mode=i, seed=15 + i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for x, s in zip(xs, streams):
            x.run(stream=s)
    torch.cuda.synchronize()
    for x in xs:
        assert x.error() == 0
        x.check()


def test_offsets_past_32_bits():
    """Pages whose byte offset in the pool passes 2^32."""
    H, D, bs, G = 2, 128, 128, 2
    NB = (1 << 32) // (H * bs * D) + 40
    x = Batch(300, [130, 4], H=H, G=G, D=D, bs=bs, mode=0, seed=18)
    small = x.g
    far = [NB - 1 - i for i in range(x.g.num_blocks)]
    at = torch.tensor(far).cuda()
    for n, a, t in (("kc", x.kc, torch.int8), ("vc", x.vc, torch.int8), ("ks", x.ks, torch.float32),
                    ("vs", x.vs, torch.float32)):
        big = torch.zeros((NB,) + a.shape[1:], dtype=t, device="cuda")
        big[at] = torch.from_numpy(a).cuda()
        x.d[n] = big
    x.d["ptab"] = torch.tensor([far[i] for i in x.ptab], dtype=torch.int32).cuda()
    x.d["tab"] = torch.tensor([[far[i] for i in r] for r in x.tab], dtype=torch.int32).cuda()
    x.g = kv.Geom(2, H, D, bs, NB, x.MB, 0)
    need = kv.kvc8_shared_prefix_workspace_bytes(x.g, H * G, x.PB)
    x.d["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    x.run()
    assert x.error() == 0
    x.g = small
    x.check()


def test_agrees_with_decode_attention_over_copied_prefixes():
    """Prefix pages named in every sequence's own table give the same attention through
    kvc8_paged_decode_attention (each within its tolerance of the exact one)."""
    x = Batch(512, [32, 64, 1], H=2, G=4, D=128, bs=32, mode=0, seed=19, spare_prefix=0)
    x.run()
    x.check()
    tab = torch.from_numpy(np.concatenate([np.stack([x.ptab] * 3), x.tab], 1)).cuda()
    g = kv.Geom(3, 2, 128, 32, x.g.num_blocks, tab.shape[1], 0)
    need = kv.kvc8_attention_workspace_bytes(g, 8)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(x.out)
    d = x.d
    kv.kvc8_paged_decode_attention(g, 8, d["q"], d["q"].stride(0), d["q"].stride(1), d["kc"], d["vc"],
                                   d["ks"], d["vs"], tab, d["lens"] + 512, x.scale, out, out.stride(0),
                                   out.stride(1), ws, need, d["err"])
    assert x.error() == 0
    x.check(out=out)


def test_a_decode_step_behind_a_prefix():
    """The operators as they are used together: the prefix is appended once, each sequence's new
    token is appended behind it with its own position, and its rotated query attends over both."""
    rng = np.random.default_rng(20)
    B, H, G, D, bs, P = 5, 2, 4, 128, 16, 75
    NB, MB, PB = 40, 4, 5
    kc, vc = (torch.zeros(NB, H, bs, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(NB, H, bs, device="cuda") for _ in range(2))
    ids = rng.permutation(NB).astype(np.int32)
    ptab = torch.from_numpy(ids[:PB].copy()).cuda()
    tab = torch.from_numpy(ids[PB:PB + B * MB].reshape(B, MB).copy()).cuda()
    freqs = fixed_point(inv_freq(D))
    fd = torch.from_numpy(freqs.view(np.int64)).cuda()
    wk = to_bf16_bits(1 + 0.1 * rng.standard_normal(D))
    wkd = bf16_tensor(wk).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    pk, pv = (to_bf16_bits(rng.standard_normal((P, H, D))) for _ in range(2))
    pkd, pvd = bf16_tensor(pk).cuda(), bf16_tensor(pv).cuda()
    rope = kv.Rope(D, fd, k_norm_weight=wkd, q_norm_weight=wkd)
    kv.kvc8_rope_store(kv.Geom(1, H, D, bs, NB, PB, 0), rope, P, 0, None, 0, 0, None, 0, 0, pkd, pvd,
                       H * D, D, kc, vc, ks, vs, ptab, i32([0, P]), i32([0]), err)
    steps, keys, vals = 3, [[] for _ in range(B)], [[] for _ in range(B)]
    g = kv.Geom(B, H, D, bs, NB, MB, 0)
    need = kv.kvc8_shared_prefix_workspace_bytes(g, H * G, PB)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    pky, _ = norm_rotate(pk, wk, 1e-6, np.arange(P), freqs, D, False, 1.0)
    for step in range(steps):
        nk, nv = (to_bf16_bits(rng.standard_normal((B, H, D))) for _ in range(2))
        qb = to_bf16_bits(rng.standard_normal((B, H * G, D)))
        nkd, nvd, q = bf16_tensor(nk).cuda(), bf16_tensor(nv).cuda(), bf16_tensor(qb).cuda()
        rope = kv.Rope(D, fd, k_norm_weight=wkd, q_norm_weight=wkd, positions=i32([P + step] * B))
        kv.kvc8_rope_store(g, rope, B, H * G, q, q.stride(0), q.stride(1), q, q.stride(0), q.stride(1),
                           nkd, nvd, H * D, D, kc, vc, ks, vs, tab, None, i32([step] * B), err)
        out = torch.empty_like(q)
        kv.kvc8_shared_prefix_attention(g, H * G, q, q.stride(0), q.stride(1), kc, vc, ks, vs, ptab, PB,
                                        i32([P]), tab, i32([step + 1] * B), D ** -0.5, out, out.stride(0),
                                        out.stride(1), ws, need, err)
        torch.cuda.synchronize()
        qy, _ = norm_rotate(qb, wk, 1e-6, [P + step] * B, freqs, D, False, 1.0)
        got = bf16_f64(bf16_bits(out))
        for b in range(B):
            keys[b].append(nk[b])
            vals[b].append(nv[b])
            ky, _ = norm_rotate(np.stack(keys[b]), wk, 1e-6, P + np.arange(step + 1), freqs, D, False, 1.0)
            for h in range(H):
                k = np.concatenate([pky[:, h], ky[:, h]])
                v = np.concatenate([bf16_f64(pv)[:, h], bf16_f64(np.stack(vals[b]))[:, h]])
                for j in range(G):
                    y = qy[b, h * G + j]
                    z = k @ y * D ** -0.5
                    w = np.exp(z - z.max())
                    want = (w / w.sum()) @ v
                    # codes: half a step of max|row| / 127 on every key and value;
                    # bf16: the query, the weights, the own rows
                    kerr = np.abs(k).max(-1) / 254 * np.abs(y).sum() * D ** -0.5
                    qerr = 2 * BF16 * (np.abs(k) @ np.abs(y)) * D ** -0.5
                    eps = BF16 + np.expm1((kerr + qerr).max())
                    top = np.abs(v).max()
                    fine = bool((np.abs(got[b, h * G + j] - want) <= 2 * eps * top + top / 254 + 2 * BF16 * top).all())
                    assert fine, (step, b, h, j)
    assert kv.kvc8_get_error(err) == 0
