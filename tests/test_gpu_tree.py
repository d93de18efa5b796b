"""Attention of drafted tokens, within the bound of _drafts_ref.py, whose checks also assert that the
answers of some mistakes would not pass it."""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from _drafts_ref import F32, U16, UB, TreeProblem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


def run(x):
    x.run()
    assert x.error() == 0
    x.check(x.out)


LENGTHS = [([0], [1]), ([1], [1]), ([0, 5, 16, 17], [1, 2, 3, 4]), ([127, 128, 129, 126], [1, 1, 1, 2]),
           ([0, 100, 128], [128, 28, 129]), ([250, 255, 256, 257], [7, 1, 16, 33]), ([1000, 0, 3], [64, 65, 1]),
           ([40, 700], [256, 255])]


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new", LENGTHS)
def test_lengths(ctx, new, D, mode, sharp):
    run(TreeProblem(ctx, new, D=D, mode=mode, sharp=sharp, seed=1))


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("kind", ["chain", "any", "none"])
@pytest.mark.parametrize("ctx,new", LENGTHS)
def test_masks(ctx, new, kind, mode):
    """Chains; any bits, rows without one among them; no bit at all (the context alone, or nothing)."""
    run(TreeProblem(ctx, new, D=128, mode=mode, kind=kind, sharp=False, seed=2))


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("H,G,D,bs", [(1, 1, 128, 16), (2, 8, 128, 128), (3, 7, 64, 48), (8, 3, 128, 32), (5, 5, 64, 80),
                                      (1, 8, 64, 112), (4, 2, 128, 64)])
def test_heads_and_blocks(H, G, D, bs, mode, sharp):
    run(TreeProblem([300, 0, 77, 1], [9, 31, 1, 40], H=H, G=G, D=D, bs=bs, mode=mode, sharp=sharp, seed=3))


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("T,G", [(1, 1), (4, 4), (16, 1), (8, 4), (33, 1), (16, 8), (17, 8), (32, 8), (33, 8), (128, 1),
                                 (64, 7), (256, 8)])
def test_query_rows(T, G, mode):
    """Rows of a kv head around every multiple of a tile."""
    run(TreeProblem([260, 31], [T, max(1, T - 1)], H=2, G=G, D=128, mode=mode, sharp=False, seed=4))


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 128])
def test_a_batch_of_ragged_trees(D, mode):
    rng = np.random.default_rng(D + mode)
    ctx, new = rng.integers(0, 700, 70).tolist(), rng.integers(0, 30, 70).tolist()
    run(TreeProblem(ctx, new, H=3, G=5, D=D, bs=32, mode=mode, sharp=mode != 1, seed=5))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_many_sequences(mode):
    rng = np.random.default_rng(7 + mode)
    ctx, new = rng.integers(0, 40, 1500).tolist(), rng.integers(0, 4, 1500).tolist()
    run(TreeProblem(ctx, new, H=1, G=2, D=64, bs=16, mode=mode, sharp=False, seed=6))


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("ctx,new,G", [([40003], [64], 4), ([20000, 3, 9001], [5, 100, 1], 8), ([70001], [1], 1)])
def test_long_contexts(ctx, new, G, mode):
    run(TreeProblem(ctx, new, H=2, G=G, D=128, bs=64, mode=mode, sharp=False, seed=7))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_tables_with_room_and_wide_masks(mode):
    run(TreeProblem([500, 0, 7], [3, 9, 1], H=2, G=8, D=64, bs=32, mode=mode, seed=8, spare=300, words=7, most=256))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_one_draft_each_without_prefix_sums(mode):
    x = TreeProblem([40, 0, 129, 300], [1, 1, 1, 1], H=2, G=4, D=128, mode=mode, kind="chain", seed=9)
    x.place()
    x.d["cu"] = None
    run(x)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_rows_behind_the_last_sequence_and_strides(mode):
    x = TreeProblem([40, 130], [5, 17], H=2, G=4, D=64, mode=mode, seed=10)
    x.place(rows=x.N + 7)
    wide = torch.full((x.N + 7, 8, 3 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:x.N, :, 64:128] = x.q
    out = torch.full((8, x.N + 7, 64 + 1), 3.0, dtype=torch.bfloat16, device="cuda")
    q, o = wide[:, :, 64:128], out.transpose(0, 1)[:, :, 1:]  # rows that start on odd elements
    d = x.d
    kv.kvc8_tree_attention(x.g, 8, x.N + 7, x.most, q, q.stride(0), q.stride(1), x.kc, x.vc, x.ks, x.vs, x.tab, d["cu"],
                           d["ctx"], d["mask"], x.words, x.scale, o, o.stride(0), o.stride(1), d["ws"], d["ws"].numel(),
                           d["err"])
    assert x.error() == 0
    x.check(o)
    assert bool((o[x.N:] == 3.0).all()) and bool((out[:, :, 0] == 3.0).all())


@pytest.mark.parametrize("scale", [-1.0, 0.0, 1e-30])
def test_softmax_scales(scale):
    x = TreeProblem([40, 130], [5, 17], H=2, G=4, D=64, seed=11)
    x.scale *= scale
    want, tol, _ = x.answers()
    x.run()
    assert x.error() == 0 and bool(((x.out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("mode", [0, 2])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_scales_that_are_no_numbers_where_nothing_looks(bad, mode):
    """Rows behind the end, and drafts that nobody sees (padding that was never stored): of these the row's scales
    (mode 0) or the block's (mode 2) may be anything."""
    x = TreeProblem([40, 0, 128, 33], [5, 17, 64, 3], H=2, G=4, D=64, mode=mode, kind="any", sharp=False, seed=12, spare=3)
    x.mask[:, 0] &= np.uint64(0x00FFFF0F0FF00003)
    for b in range(x.B):
        c, q = x.ctx[b], x.new[b]
        seen = x.sees(b)[:, c:].any(0).tolist()
        for p in range(x.MB * x.bs):
            dead = p >= c + q or (p >= c and not seen[p - c])
            blk, at = int(x.tab[b, p // x.bs]), p % x.bs
            if mode == 0 and dead:
                x.ks[blk, :, at] = x.vs[blk, :, at] = bad
            elif mode == 2 and at == 0:
                lo, hi = p, min(p + x.bs, c + q)
                if all(i >= c and not seen[i - c] for i in range(lo, hi)):
                    x.ks[blk] = x.vs[blk] = bad
    clean = TreeProblem([40, 0, 128, 33], [5, 17, 64, 3], H=2, G=4, D=64, mode=mode, kind="any", sharp=False, seed=12, spare=3)
    clean.mask = x.mask
    x.run()
    assert x.error() == 0
    want, tol, _ = clean.answers()
    assert bool(((x.out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("which", ["ks", "vs"])
def test_a_scale_that_is_no_number_reaches_those_who_see_it(which):
    x = TreeProblem([40], [6], H=2, G=4, D=64, mode=0, kind="chain", sharp=False, seed=13)
    p = 43
    getattr(x, which)[int(x.tab[0, p // x.bs]), 1, p % x.bs] = float("nan")
    x.run()
    bad = torch.isnan(x.out).flatten(2).any(2)
    assert bool(bad[3:, 4:].all()) and not bool(bad[:3].any()) and not bool(bad[:, :4].any())


def test_reports():
    def go(change, code, bad=(), lens=None):
        x = TreeProblem([40, 60, 33], [5, 7, 3], H=2, G=4, D=64, sharp=False, seed=14, spare=0)
        x.place()
        want, tol, _ = x.answers()
        change(x)
        x.run()
        assert x.error() == code
        n0 = 0
        for b, q in enumerate(x.new):
            ok = ((x.out[n0:n0 + q].double() - want[n0:n0 + q]).abs() <= tol[n0:n0 + q])
            if b not in bad:
                assert bool(ok.all()), b
            elif lens == "unwritten":
                assert bool(torch.isnan(x.out[n0:n0 + q]).all())
            n0 += q
    cu = lambda *v: lambda x: x.d["cu"].copy_(torch.tensor(v, dtype=torch.int32))  # noqa: E731
    go(lambda x: None, 0)
    go(cu(0, 5, 4, 15), kv.DEV_BAD_LENGTH, (1, 2), None)  # decreasing, and one that then has too many
    go(cu(0, 5, 12, 16), kv.DEV_BAD_LENGTH, (2,), "unwritten")  # beyond num_tokens
    go(cu(-1, 5, 12, 15), kv.DEV_BAD_LENGTH, (0,), "unwritten")
    go(lambda x: setattr(x, "most", 6), kv.DEV_BAD_LENGTH, (1,), "unwritten")
    go(lambda x: x.d["ctx"].__setitem__(1, -1), kv.DEV_BAD_LENGTH, (1,), None)
    go(lambda x: x.d["ctx"].__setitem__(1, 1000), kv.DEV_POS_BEYOND_TABLE, (1,), None)
    go(lambda x: x.tab.__setitem__((1, 1), -1), kv.DEV_BAD_BLOCK_ID, (1,), None)
    go(lambda x: x.tab.__setitem__((1, 1), 10 ** 6), kv.DEV_BAD_BLOCK_ID, (1,), None)


def test_positions_of_bad_blocks_and_beyond_the_table_are_left_out():
    x = TreeProblem([40, 64], [8, 8], H=1, G=2, D=64, bs=16, kind="none", sharp=False, seed=15, spare=0)
    y = TreeProblem([40, 64], [8, 8], H=1, G=2, D=64, bs=16, kind="none", sharp=False, seed=15, spare=0)
    x.place()
    x.tab[0, 1] = -1
    x.d["ctx"][1] = 2 ** 31 - 1  # all five blocks of the table, which are the 64 positions and eight more
    x.run()
    assert x.error() != 0
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[16:32] = False
    for b, rows in ((0, keep), (1, torch.ones(80, dtype=torch.bool, device="cuda"))):
        y.lens[b] = rows.numel()
        k, v = y.rows(y.kc, y.ks, b, 0)[rows], y.rows(y.vc, y.vs, b, 0)[rows]
        w = torch.softmax(torch.matmul(y.q[8 * b:8 * b + 8].double(), k.T) * y.scale, -1)
        assert torch.allclose(x.out[8 * b:8 * b + 8].double(), torch.matmul(w, v), rtol=0.02, atol=0.02 * float(v.abs().max()))


def test_a_negative_context_counts_as_none():
    x = TreeProblem([0, 50], [9, 4], H=2, G=4, D=64, seed=16)
    x.place()
    x.d["ctx"][0] = -7
    x.run()
    assert x.error() == kv.DEV_BAD_LENGTH
    x.check(x.out)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_a_replayed_graph_follows_its_lengths_and_masks(mode):
    x = TreeProblem([2000, 100, 31, 700], [9, 16, 1, 30], H=2, G=8, D=128, bs=32, mode=mode, sharp=False, seed=17)
    x.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.run()
    for seed, ctx, new in ((1, [1999, 0, 5, 64], [10, 15, 3, 28]), (2, [0, 0, 0, 0], [1, 30, 24, 1]),
                           (3, [2000, 100, 31, 700], [9, 16, 1, 30])):
        y = TreeProblem(ctx, new, H=2, G=8, D=128, bs=32, mode=mode, kind="any", sharp=False, seed=17, most=30)
        x.ctx, x.new, x.mask, x.lens = ctx, new, y.mask, y.lens
        x.d["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        x.d["cu"].copy_(torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32))
        x.d["mask"].copy_(torch.from_numpy(y.mask.view(np.int64)))
        x.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert x.error() == 0
        want, tol, _ = x.answers()
        assert bool(((x.out.double() - want).abs() <= tol).all()), seed


def test_two_streams_with_their_own_workspaces():
    xs = [TreeProblem([3000, 40], [20, 64], H=4, G=4, D=128, bs=32, mode=m, sharp=False, seed=18) for m in (0, 1)]
    streams = [torch.cuda.Stream() for _ in xs]
    for x in xs:
        x.place()
    torch.cuda.synchronize()
    for _ in range(20):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                x.run()
    torch.cuda.synchronize()
    for x in xs:
        assert x.error() == 0
        x.check(x.out)


LIMITS = [((0, 2), -66, 0, 0), ((0, 2), 65, 0, 0), ((0, 2), 0, -106, 0), ((0, 2), 0, 105, 0), ((0, 1, 2), 0, 0, -103),
          ((0, 1, 2), 0, 0, 96), ((0, 2), -66, -50, -53), ((1,), -66, -90, 0), ((1,), 65, 90, 0)]


@pytest.mark.parametrize("mode,values,keys,query", [(m, v, k, q) for modes, v, k, q in LIMITS for m in modes])
def test_scales_and_queries_at_the_ends_of_their_range(mode, values, keys, query):
    x = TreeProblem([300, 0, 40], [9, 40, 3], H=2, G=4, D=128, bs=32, mode=mode, seed=19)
    x.vs *= 2.0 ** values
    x.ks *= 2.0 ** keys
    x.q = (x.q.float() * 2.0 ** query).to(torch.bfloat16)
    x.scale *= 2.0 ** -(keys + query)
    run(x)


def test_a_step_of_drafts_from_pages_to_pages():
    """Blocks assigned, drafts rotated and stored, looked at, some kept, the rest given back; three times, against a
    plain model of the conversation."""
    B, H, G, D, bs, NB, MB = 5, 2, 4, 64, 16, 64, 12
    rng = np.random.default_rng(20)
    g = kv.Geom(B, H, D, bs, NB, MB, 0)
    i32 = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    err, lens, count = i32([0]), i32([0] * B), i32([NB])
    free = i32(rng.permutation(NB))
    table = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros(NB, H, bs, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((NB, H, bs), float("nan"), device="cuda") for _ in range(2))
    freqs, _ = kv.kvc8_rope_frequencies(kv.RopeScaling(kv.ROPE_PLAIN, 1e4), D)
    freqs = torch.from_numpy(freqs.view(np.int64)).cuda()
    inv = torch.from_numpy(1e4 ** (-2.0 * np.arange(D // 2) / D)).cuda()
    kept = [[] for _ in range(B)]  # (key, value) rows in fp64 of each sequence, as the cache should hold them

    def turned(x, pos):
        a, b = x[..., :D // 2].double(), x[..., D // 2:].double()
        t = pos.double()[:, None, None] * inv
        return torch.cat([a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()], -1)

    def quantised(x):
        s = x.abs().amax(-1, keepdim=True) / 127.0
        return torch.round(x / s) * s

    for step in range(3):
        T = [int(t) for t in rng.integers(1, 14, B)] if step else [30, 1, 17, 16, 45]
        cu = np.concatenate([[0], np.cumsum(T)])
        parent = [[int(rng.integers(-1, i)) if step else i - 1 for i in range(q)] for q in T]
        depth, anc = [], []
        for q, par in zip(T, parent):
            d, a = [], []
            for i, p in enumerate(par):
                d.append(0 if p < 0 else d[p] + 1)
                a.append((a[p] if p >= 0 else 0) | 1 << i)
            depth.append(d)
            anc.append(a)
        N = int(cu[-1])
        base = [len(x) for x in kept]
        pos = i32([base[b] + d for b in range(B) for d in depth[b]])
        new = torch.randn(N, H * (G + 2), D, device="cuda").to(torch.bfloat16)
        q, k, v = new[:, :H * G], new[:, H * G:H * G + H], new[:, H * G + H:]
        grown, served = i32([a + b for a, b in zip(base, T)]), i32([0] * B)
        slots = torch.zeros(N, dtype=torch.int64, device="cuda")
        kv.kvc8_assign_blocks(g, lens, grown, free, count, count, table, served, slots, N, err)
        assert torch.equal(served, grown) and int(slots.min()) >= 0 and slots.unique().numel() == N
        rope, qo = kv.Rope(D, freqs, positions=pos), torch.empty_like(q)
        kv.kvc8_rope_store(g, rope, N, H * G, q, q.stride(0), q.stride(1), qo, qo.stride(0), qo.stride(1), k, v,
                           k.stride(0), k.stride(1), kc, vc, ks, vs, table, i32(cu), lens, err)
        # the slots say where the store put each row
        at = ks.transpose(1, 2).reshape(NB * bs, H)[slots]
        assert torch.allclose(at.double(), turned(k, pos).abs().amax(-1) / 127.0, rtol=1e-5)
        words = torch.tensor([a for row in anc for a in row], dtype=torch.int64, device="cuda")[:, None].contiguous()
        out = torch.empty(N, H * G, D, dtype=torch.bfloat16, device="cuda")
        most = max(T)
        ws = torch.empty(kv.kvc8_tree_attention_workspace_bytes(g, H * G, N, most), dtype=torch.uint8, device="cuda")
        kv.kvc8_tree_attention(g, H * G, N, most, qo, qo.stride(0), qo.stride(1), kc, vc, ks, vs, table, i32(cu), lens, words,
                               1, D ** -0.5, out, out.stride(0), out.stride(1), ws, ws.numel(), err)
        kr, vr = quantised(turned(k, pos)), quantised(v.double())
        # as stored: codes and scales at the slots
        stored = [(c.transpose(1, 2).reshape(NB * bs, H, D)[slots].double() * s.transpose(1, 2).reshape(NB * bs, H)[slots].double()[..., None])
                  for c, s in ((kc, ks), (vc, vs))]
        for got, want in zip(stored, (kr, vr)):  # a code's step at most: fp32 rotations move a tie
            assert bool(((got - want).abs() <= want.abs().amax(-1, keepdim=True) / 127 * 1.01).all())
        kr, vr = stored
        path = []
        for b in range(B):
            for i in range(T[b]):
                n = int(cu[b]) + i
                rows = kept[b] + [(kr[cu[b] + j], vr[cu[b] + j]) for j in range(T[b]) if anc[b][i] >> j & 1]
                kk, vv = (torch.stack([r[x] for r in rows]) for x in (0, 1))
                for h in range(H):
                    qh = qo[n, h * G:(h + 1) * G].double()
                    z = torch.matmul(qh, kk[:, h].T) * D ** -0.5
                    w = torch.softmax(z, -1)
                    want = torch.matmul(w, vv[:, h])
                    # the bound of _drafts_ref, with the largest delta of a row for all its positions
                    delta = torch.matmul(qh.abs(), kk[:, h].abs().T) * D ** -0.5 * (2 * U16 + D * F32)
                    delta = delta + qh.abs().amax(-1, keepdim=True) * kk[:, h].abs().sum(-1) * D ** -0.5 * 2.0 ** -25
                    off = torch.expm1(delta.amax(-1, keepdim=True) + 2.0 ** -20 * (1 + z.abs().amax(-1, keepdim=True)))
                    sums = (len(rows) + 64) / 8 * F32
                    num = torch.matmul(w, vv[:, h].abs()) * ((1 + off) * (1 + 5.01 * U16) - 1 + sums)
                    num = num + len(rows) * 2.0 ** -31 * vv[:, h].abs().max()
                    tol = (num + want.abs() * (off + sums)) / (1 - off - sums)
                    tol = tol + UB * (want.abs() + tol)
                    assert bool(((out[n, h * G:(h + 1) * G].double() - want).abs() <= tol).all()), (step, b, i, h)
            leaf = int(rng.integers(0, T[b]))
            path.append([j for j in range(T[b]) if anc[b][leaf] >> j & 1])
        depth_most = max(len(p) for p in path)
        acc = i32([p + [-1] * (depth_most - len(p)) for p in path])
        held = grown.clone()
        kv.kvc8_compact_drafts(g, kc, vc, ks, vs, table, lens, acc, depth_most, i32([len(p) for p in path]), lens, err)
        for b in range(B):
            kept[b] += [(kr[cu[b] + j], vr[cu[b] + j]) for j in path[b]]
        assert lens.tolist() == [len(x) for x in kept]
        kv.kvc8_assign_blocks(g, held, lens, free, count, count, table, served, None, 0, err)
        used = sum(-(-len(x) // bs) for x in kept)
        assert int(count) == NB - used
        ids = [int(table[b, j]) for b in range(B) for j in range(-(-len(kept[b]) // bs))]
        assert sorted(ids + free[:int(count)].tolist()) == list(range(NB))
        total = sum(len(x) for x in kept)
        rows = torch.empty(total, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(total, H, D, dtype=torch.bfloat16, device="cuda")
        n = kv.kvc8_gather_workspace_bytes(g)
        gws = torch.empty(n, dtype=torch.uint8, device="cuda")
        kv.kvc8_dequant_gather(g, kc, vc, ks, vs, table, lens, None, rows[0], rows[1], total, H * D, D, gws, n, err)
        assert kv.kvc8_get_error(err) == 0
        for got, x in zip(rows, (0, 1)):
            want = torch.stack([r[x] for seq in kept for r in seq])
            assert bool(((got.double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -22)).all())


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(31, 1), (32, 1), (33, 1), (4, 8), (11, 3), (63, 1), (64, 1), (65, 1), (8, 8), (13, 5), (128, 1), (129, 1)])
def test_rows_at_the_edges_of_a_tile_s_quarters(T, G, D, mode):
    # full and shorter trees, contexts of none, of less and of more than a step, and long enough for several CTAs
    run(TreeProblem([0, 1000, 77, 301, 5000], [T, T, 1, max(1, T // 2), T], G=G, D=D, mode=mode, seed=T))


@pytest.mark.parametrize("T,G", [(4, 8), (16, 4)])
def test_many_short_tiles_of_few_rows(T, G):
    rng = np.random.default_rng(3)
    run(TreeProblem(rng.integers(0, 40, 150).tolist(), rng.integers(0, T + 1, 149).tolist() + [T], G=G, D=128, seed=4))
