"""What is measured of the block assignment, the tree attention and the compaction of
drafted tokens: cases, inputs, the calls, and their plain forms.

Operators (``op`` of a case):

* ``assign``        kvc8_assign_blocks: block tables and slots of sequences that grow
                    and shrink, from their lengths and a stack of free blocks.
* ``tree``          kvc8_tree_attention: the drafted tokens of each sequence over its
                    cached positions and, by a mask, over each other, in the int8 pages.
* ``compact``       kvc8_compact_drafts: the accepted drafts' rows moved behind the
                    context; the pages are read back as the values they stand for with
                    kvc8_dequant_gather.
* ``compact_bf16``  kvc8_compact_drafts_bf16: the same in bf16 pages.
"""
import math
import random

import torch

own = False


# ---- cases ------------------------------------------------------------------

def listed():
    tree = dict(op="tree")
    grow = dict(op="assign", short=False)
    keep = dict(op="compact")
    return [
        # one conversation with a short chain of drafts: the smallest call, where latency counts
        dict(tree, name="tree 4 of 1 x 500", seqs=1, ctx_lo=500, ctx_hi=500, new_lo=4, new_hi=4, kv_heads=2, group=4,
             dim=64, block=16, mode=0, chain=True, lens=1),
        # a serving batch, a tree of 8 drafts each
        dict(tree, name="tree 8 of 16 x 8192", seqs=16, ctx_lo=1, ctx_hi=8192, new_lo=8, new_hi=8, kv_heads=8, group=4,
             dim=128, block=128, mode=0, chain=False, lens=2),
        # odd sizes: ragged trees, 7 queries to a head, per-block scales, empty contexts, a draft that sees nothing
        dict(tree, name="tree 1-37 of 23 x 1000", seqs=23, ctx_lo=0, ctx_hi=1000, new_lo=1, new_hi=37, kv_heads=4,
             group=7, dim=128, block=48, mode=2, chain=False, lens=3),
        # two long documents with a wide tree
        dict(tree, name="tree 64 of 2 x 131072", seqs=2, ctx_lo=130000, ctx_hi=131008, new_lo=64, new_hi=64, kv_heads=8,
             group=4, dim=128, block=128, mode=0, chain=False, lens=4),
        # the benchmark's decode batch with a chain of 4 drafts, per-channel scales
        dict(tree, name="tree 4 of 256 x 8192", seqs=256, ctx_lo=1, ctx_hi=8192, new_lo=4, new_hi=4, kv_heads=8,
             group=4, dim=128, block=128, mode=1, chain=True, lens=5),
        # a decode step's growth, a few tokens each: most sequences keep their last block
        dict(grow, name="assign decode 256", seqs=256, held_lo=1, held_hi=8192, new_lo=1, new_hi=8, finished=0.0,
             block=128, lens=6),
        # prompts admitted into small blocks
        dict(grow, name="assign prompts 16", seqs=16, held_lo=0, held_hi=0, new_lo=512, new_hi=4096, finished=0.0,
             block=16, lens=7),
        # a large batch between two steps: a quarter has finished, the others grow; the pool runs short
        dict(grow, name="assign mixed 4096", seqs=4096, held_lo=0, held_hi=4000, new_lo=0, new_hi=500, finished=0.25,
             block=32, short=True, lens=8),
        # one accepted draft or two of a short tree, dynamic scales
        dict(keep, name="keep of 1 x 12", seqs=1, ctx_lo=37, ctx_hi=37, new_lo=12, new_hi=12, most=4, kv_heads=2,
             dim=64, block=16, mode=0, lens=9),
        # a batch of trees, short contexts (which are read back), dynamic scales
        dict(keep, name="keep of 64 x 24", seqs=64, ctx_lo=0, ctx_hi=64, new_lo=24, new_hi=24, most=8, kv_heads=8,
             dim=128, block=128, mode=0, lens=10),
        # per-block scales: rows that change blocks are requantised; odd sizes
        dict(keep, name="keep of 33 x 9-61", seqs=33, ctx_lo=0, ctx_hi=130, new_lo=9, new_hi=61, most=9, kv_heads=5,
             dim=80, block=24, mode=2, lens=11),
        # the benchmark's decode batch with wide trees, bf16 pages
        dict(keep, op="compact_bf16", name="keep bf16 of 256 x 64", seqs=256, ctx_lo=1, ctx_hi=700, new_lo=64,
             new_hi=64, most=16, kv_heads=8, dim=128, block=64, mode=0, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: lengths over their logarithm, odd sizes, every mode and layout."""
    op = rng.choice(["tree", "tree", "tree", "assign", "assign", "compact", "compact_bf16"])
    lens = rng.randrange(1 << 30)
    if op == "assign":
        seqs = _log_int(rng, 1, 4096)
        new = _log_int(rng, 1, max(1, min(4096, 1 << 20) // seqs + 1))
        held = rng.choice([0, _log_int(rng, 1, max(2, min(8192, (1 << 23) // seqs)))])
        return dict(op=op, seqs=seqs, held_lo=0, held_hi=held, new_lo=0, new_hi=new,
                    finished=rng.choice([0.0, 0.25, 0.5]) if held else 0.0,
                    block=rng.choice([1, 16, 24, 32, 64, 77, 128]) if held < 1000 else rng.choice([16, 32, 64, 77, 128]),
                    short=rng.random() < 0.3, lens=lens)
    if op == "tree":
        kv, group, dim = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 8), rng.choice([64, 128])
        seqs, new = _log_int(rng, 1, 256), _log_int(rng, 1, 128)
        new = min(new, max(1, 8192 // seqs))
        most = min(131008, 8 * 256 * 4096 // (seqs * kv), 8 * 4 * 64 * 262144 // (seqs * kv * group * new))
        return dict(op=op, seqs=seqs, ctx_lo=0, ctx_hi=_log_int(rng, 1, max(2, most)),
                    new_lo=rng.choice([1, new]), new_hi=new, kv_heads=kv, group=group, dim=dim,
                    block=16 * rng.randint(1, 8), mode=rng.randrange(3), chain=rng.random() < 0.3, lens=lens)
    kv, dim = rng.choice([1, 2, 3, 5, 8]), rng.choice([16, 64, 80, 128, 128, 192, 256])
    seqs, most = _log_int(rng, 1, 256), rng.randint(1, 16)
    new = most + _log_int(rng, 1, 48)
    # (read back, a position of an int8 page costs six bytes a channel)
    room = 700 if op == "compact_bf16" else max(1, min(700, 16_000_000 // (6 * seqs * kv * dim) - most))
    ctx = _log_int(rng, 1, room)
    return dict(op=op, seqs=seqs, ctx_lo=0, ctx_hi=ctx, new_lo=most + 1, new_hi=new, most=most, kv_heads=kv, dim=dim,
                block=rng.choice([1, 16, 24, 32, 64, 77, 128]), mode=rng.randrange(3) if op == "compact" else 0, lens=lens)


def _lens(case):
    """Lengths of a case's sequences (they belong to the case, not to the seed)."""
    c, rng = case, random.Random(case["lens"])
    n = c["seqs"]
    if c["op"] == "assign":
        held = [rng.randint(c["held_lo"], c["held_hi"]) for _ in range(n)]
        gone = [rng.random() < c["finished"] for _ in range(n)]
        # finished sequences give all back, or, as after rejected drafts, some
        want = [rng.choice([0, h // 2]) if g else h + rng.randint(c["new_lo"], c["new_hi"]) for h, g in zip(held, gone)]
        return held, want
    ctx = [c["ctx_lo"]] + [rng.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(n - 1)]
    new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(n)]
    if c["op"] == "tree":
        return ctx, new
    return ctx, new, [rng.randint(0, min(c["most"], q)) for q in new]


def _up(a, b):
    return -(-a // b)


def _counts(case):
    """(blocks needed, given up, new positions) of an assignment, and the free blocks before it."""
    held, want = _lens(case)
    bs = case["block"]
    need = sum(max(0, _up(w, bs) - _up(h, bs)) for h, w in zip(held, want))
    give = sum(max(0, _up(h, bs) - _up(w, bs)) for h, w in zip(held, want))
    new = sum(max(0, w - h) for h, w in zip(held, want))
    return need, give, new, max(0, need * 3 // 4 - give) if case["short"] else need + 37


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(g, need, per_seq, spare):
    """Rows of distinct blocks in random order, as many as each sequence needs, -1 behind them; the pool's size, and the rest."""
    total = sum(need)
    ids = torch.randperm(total + spare, device="cuda", generator=g).to(torch.int32)
    n = torch.tensor(need, device="cuda")
    j = torch.arange(per_seq, device="cuda")
    at = (n.cumsum(0) - n)[:, None] + j
    table = torch.where(j < n[:, None], ids[at.clamp(max=max(0, total + spare - 1))], torch.full_like(ids[:1], -1))
    return table.contiguous(), total + spare, ids[total:]


def _pool(g, s, blocks, heads, block, dim, mode):
    """Pages as a store leaves them: N(0, 1) rows, four channels of each key head ten times as large, values around a
    mean of their head, quantised by row, channel or block."""
    for n in ("k", "v"):
        big = torch.where(torch.rand(heads, dim, device="cuda", generator=g).argsort(1) < 4, 10.0, 1.0)[:, None]
        mean = 0.7 * torch.randn(heads, 1, dim, device="cuda", generator=g)
        s[n + "_cache"] = torch.empty(blocks, heads, block, dim, dtype=torch.int8, device="cuda")
        shape = [(blocks, heads, block), (heads, dim), (blocks, heads)][mode]
        s[n + "_scale"] = torch.empty(shape, device="cuda")
        if mode == 1:
            s[n + "_scale"][:] = ((big * torch.ones_like(mean) if n == "k" else 1.0 + mean.abs()) * (4.0 / 127.0))[:, 0]
        part = max(1, (1 << 26) // (heads * block * dim))
        for i in range(0, blocks, part):
            m = min(part, blocks - i)
            x = torch.randn(m, heads, block, dim, device="cuda", generator=g)
            x = x * big if n == "k" else x + mean
            if mode == 0:
                by = x.abs().amax(-1) / 127.0
                s[n + "_scale"][i : i + m] = by
                by = by[..., None]
            elif mode == 1:
                by = s[n + "_scale"][:, None]
            else:
                by = x.abs().amax((-1, -2)) / 127.0
                s[n + "_scale"][i : i + m] = by
                by = by[..., None, None]
            s[n + "_cache"][i : i + m] = torch.round(x / by).clamp(-127, 127).to(torch.int8)


def _masks(rng, new, words):
    """Ancestors of every draft in random trees, as bits; the last draft of the first sequence, and of one in five, is
    padding that sees no draft."""
    rows = []
    for b, q in enumerate(new):
        seen = []
        for i in range(q):
            parent = rng.randint(-1, i - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << i))
        if q > 1 and (b == 0 or rng.random() < 0.2):
            seen[-1] = 0
        rows += [[(x >> (64 * w)) & (2 ** 64 - 1) for w in range(words)] for x in seen]
    return torch.tensor([[w - 2 ** 64 if w >= 2 ** 63 else w for w in r] for r in rows], dtype=torch.int64, device="cuda")


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": case}
    n, block = c["seqs"], c["block"]
    if c["op"] == "assign":
        held, want = _lens(c)
        need, give, new, free = s["counts"] = _counts(c)
        per_seq = max(1, max(_up(max(h, w), block) for h, w in zip(held, want)))
        s["table"], s["blocks"], rest = _table(g, [_up(h, block) for h in held], per_seq, max(1, free))
        s["free"] = torch.full((s["blocks"],), -1, dtype=torch.int32, device="cuda")
        s["free"][:free] = rest[:free]
        s["count"], s["count_out"] = _i32([free]), _i32([0])
        s["held"], s["want"] = _i32(held), _i32(want)
        s["lens_out"] = torch.empty_like(s["held"])
        s["slots"] = torch.empty(new, dtype=torch.int64, device="cuda")
        return s
    heads, dim = c["kv_heads"], c["dim"]
    ctx, new = s["lens"] = _lens(c)[:2]
    need = [_up(a + b, block) for a, b in zip(ctx, new)]
    s["table"], blocks, _ = _table(g, need, max(1, max(need)), 3)
    s["ctx"] = _i32(ctx)
    if c["op"] == "tree":
        _pool(g, s, blocks, heads, block, dim, c["mode"])
        cu = [0]
        for q in new:
            cu.append(cu[-1] + q)
        s["cu"], s["rows"], s["most"] = _i32(cu), cu[-1], max(new)
        s["words"] = _up(s["most"], 64)
        s["mask"] = None if c["chain"] else _masks(random.Random(seed), new, s["words"])
        s["query"] = torch.randn(cu[-1], heads * c["group"], dim, device="cuda", generator=g).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["query"])
        s["scale"] = dim ** -0.5
        return s
    take = _lens(c)[2]
    rng = random.Random(seed)
    # a path through a tree whose first level is as wide as the longest path: the first draft or one behind the path
    most = max(1, c["most"])
    idx = []
    for q, a in zip(new, take):
        keep = rng.randint(0, min(a, 2))
        rest = sorted(rng.sample(range(a, q), min(a - keep, q - a)))
        row = list(range(a - len(rest))) + rest
        idx.append(row + [-1] * (most - a))
    s["accepted"], s["num"] = _i32(idx), _i32(take)
    s["lens_out"] = torch.empty_like(s["ctx"])
    s["rows"] = sum(ctx) + sum(take)
    if c["op"] == "compact_bf16":
        for k in ("k_cache", "v_cache"):
            s[k] = torch.randn(blocks, heads, block, dim, device="cuda", generator=g).to(torch.bfloat16)
    else:
        _pool(g, s, blocks, heads, block, dim, c["mode"])
        for k in ("k_rows", "v_rows"):
            s[k] = torch.empty(s["rows"], heads, dim, dtype=torch.bfloat16, device="cuda")
    return s


# ---- the framework's calls --------------------------------------------------

def _space(s, size):
    """A workspace that the program keeps."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    import dequant_kvc8_store_gb300 as kv
    c, t = s["case"], s["table"]
    if "geom" not in s:
        blocks = s["blocks"] if c["op"] == "assign" else s["k_cache"].shape[0]
        s["geom"] = kv.Geom(c["seqs"], c.get("kv_heads", 1), c.get("dim", 128), c["block"], blocks, t.shape[1],
                            c.get("mode", 0))
    g = s["geom"]
    if c["op"] == "assign":
        kv.kvc8_assign_blocks(g, s["held"], s["want"], s["free"], s["count"], s["count_out"], t, s["lens_out"],
                              s["slots"], s["slots"].shape[0])
        return _assigned(s)
    if c["op"] == "tree":
        q, o, heads = s["query"], s["out"], c["kv_heads"] * c["group"]
        if "ws_bytes" not in s:
            s["ws_bytes"] = kv.kvc8_tree_attention_workspace_bytes(g, heads, s["rows"], s["most"])
        kv.kvc8_tree_attention(g, heads, s["rows"], s["most"], q, q.stride(0), q.stride(1), s["k_cache"], s["v_cache"],
                               s["k_scale"], s["v_scale"], t, s["cu"], s["ctx"], s["mask"], s["words"], s["scale"], o,
                               o.stride(0), o.stride(1), _space(s, s["ws_bytes"]), s["ws_bytes"])
        return o
    if c["op"] == "compact_bf16":
        kv.kvc8_compact_drafts_bf16(g, s["k_cache"], s["v_cache"], t, s["ctx"], s["accepted"], s["accepted"].shape[1],
                                    s["num"], s["lens_out"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens_out"]}
    kv.kvc8_compact_drafts(g, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], t, s["ctx"], s["accepted"],
                           s["accepted"].shape[1], s["num"], s["lens_out"])
    if "ws_bytes" not in s:
        s["ws_bytes"] = kv.kvc8_gather_workspace_bytes(g)
    kr, vr = s["k_rows"], s["v_rows"]
    kv.kvc8_dequant_gather(g, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], t, s["lens_out"], None, kr, vr,
                           s["rows"], kr.stride(0), kr.stride(1), _space(s, s["ws_bytes"]), s["ws_bytes"])
    return {"k_rows": kr, "v_rows": vr, "lens": s["lens_out"]}


def _assigned(s):
    return {"table": s["table"], "free": s["free"], "count": s["count_out"], "lens": s["lens_out"], "slots": s["slots"]}


# ---- the plain forms --------------------------------------------------------

def _plain_assign(s):
    bs, table, free = s["case"]["block"], s["table"], s["free"]
    need_all, give_all, new_all, _ = s["counts"]
    held, want = s["held"].long(), s["want"].long()
    hb, wb = (held + bs - 1) // bs, (want + bs - 1) // bs
    need, give, count = (wb - hb).clamp(min=0), (hb - wb).clamp(min=0), s["count"].long()

    def spread(n, total):
        """Sequence and index of each of the `total` items that the sequences have n of."""
        b = torch.repeat_interleave(n, output_size=total)
        return b, torch.arange(total, device="cuda") - (n.cumsum(0) - n)[b]

    b, j = spread(give, give_all)
    free[count + torch.arange(give_all, device="cuda")] = table[b, wb[b] + j]
    have = count + give_all
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= have)
    b, j = spread(need, need_all)
    k = torch.arange(need_all, device="cuda")
    ids = free[(have - 1 - k).clamp(min=0)]
    table[b, hb[b] + j] = torch.where(served[b], ids, table[b, hb[b] + j])
    s["count_out"].copy_((have - torch.where(served, need, torch.zeros_like(need)).sum()).int())
    s["lens_out"].copy_(torch.where(served, want, held).int())
    b, j = spread((want - held).clamp(min=0), new_all)
    p = held[b] + j
    s["slots"].copy_(torch.where(served[b], table[b, p // bs].long() * bs + p % bs, torch.full_like(p, -1)))
    return _assigned(s)


def _rows(s, n, b, count, h=slice(None)):
    """[count][heads][dim] fp32 values of the first positions of sequence b."""
    c = s["case"]
    bs = c["block"]
    ids = s["table"][b, : _up(count, bs)].long()
    x = s[n + "_cache"][ids].float()
    scale = s[n + "_scale"]
    x = x * (scale[ids][..., None] if c["mode"] == 0 else scale[:, None] if c["mode"] == 1 else scale[ids][..., None, None])
    return x.transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])[:count]


def _plain_tree(s):
    c, out = s["case"], s["out"]
    h, g, d = c["kv_heads"], c["group"], c["dim"]
    ctx, new = s["lens"]
    bit = torch.arange(64 * s["words"], device="cuda")
    first = 0
    for b, (x, q) in enumerate(zip(ctx, new)):
        k, v = _rows(s, "k", b, x + q), _rows(s, "v", b, x + q)
        qs = s["query"][first : first + q].float().view(q, h, g, d).permute(1, 0, 2, 3).reshape(h, q * g, d)
        z = (torch.matmul(qs, k.permute(1, 2, 0)) * s["scale"]).view(h, q, g, x + q)
        if s["mask"] is None:
            seen = bit[:q] <= bit[:q, None]
        else:
            m = s["mask"][first : first + q]
            seen = ((m[:, bit // 64] >> (bit % 64)) & 1).bool()[:, :q]
        z[..., x:].masked_fill_(~seen[None, :, None], -math.inf)
        top = z.amax(-1, keepdim=True)
        w = torch.exp(z - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        total = w.sum(-1, keepdim=True)
        o = torch.matmul(w.view(h, q * g, -1), v.transpose(0, 1)).view(h, q, g, d)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out[first : first + q] = o.permute(1, 0, 2, 3).reshape(q, h * g, d).to(torch.bfloat16)
        first += q
    return out


def _plain_compact(s):
    c, bs = s["case"], s["case"]["block"]
    k = torch.arange(s["accepted"].shape[1], device="cuda")
    live = k < s["num"][:, None]
    b = torch.arange(c["seqs"], device="cuda")[:, None].expand_as(live)
    src, dst = s["ctx"][:, None] + s["accepted"], s["ctx"][:, None] + k
    src = torch.where(live, src, 0 * src).long()
    dst = torch.where(live, dst, 0 * dst).long()  # (a sequence's first position stands in for what is not moved)
    si, sa, di, da = s["table"][b, src // bs].long(), src % bs, s["table"][b, dst // bs].long(), dst % bs
    si, sa, di, da = (x[live] for x in (si, sa, di, da))
    s["lens_out"].copy_(s["ctx"] + s["num"])
    rows = {}
    for n in ("k", "v"):
        cache = s[n + "_cache"]
        x = cache[si, :, sa]
        if c["op"] == "compact" and c["mode"] == 2:
            scale = s[n + "_scale"]
            y = torch.round(x.float() * scale[si][..., None] / scale[di][..., None]).clamp(-127, 127)
            x = torch.where((scale[di] == 0)[..., None], torch.zeros_like(y), y).to(torch.int8)
        cache[di, :, da] = x
        if c["op"] == "compact" and c["mode"] == 0:
            s[n + "_scale"][di, :, da] = s[n + "_scale"][si, :, sa]
        if c["op"] == "compact":  # the values that the pages stand for, sequence by sequence
            end = s["lens_out"].long().cumsum(0)
            r = torch.arange(s["rows"], device="cuda")
            rb = torch.bucketize(r, end, right=True)
            p = r - end[rb] + s["lens_out"][rb]
            ri, ra = s["table"][rb, p // bs].long(), p % bs
            scale = s[n + "_scale"]
            by = scale[ri, :, ra][..., None] if c["mode"] == 0 else scale if c["mode"] == 1 else scale[ri][..., None]
            rows[n + "_rows"] = (cache[ri, :, ra].float() * by).to(torch.bfloat16)
    if c["op"] == "compact_bf16":
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "lens": s["lens_out"]}
    return {"k_rows": rows["k_rows"], "v_rows": rows["v_rows"], "lens": s["lens_out"]}


def run(state):
    if own:
        return _own(state)
    return {"assign": _plain_assign, "tree": _plain_tree}.get(state["case"]["op"], _plain_compact)(state)


# ---- what a pass cannot do without --------------------------------------------

def work(case):
    c = case
    if c["op"] == "assign":
        need, give, new, _ = _counts(c)
        # lengths in and out, ids read and written, slots
        return {"bytes": 12 * c["seqs"] + 8 * (need + give) + 8 * new, "flops": 0}
    h, d = c["kv_heads"], c["dim"]
    if c["op"] == "tree":
        ctx, new = _lens(c)
        held, hq = sum(ctx) + sum(new), h * c["group"]
        scales = {0: 8 * h * held, 1: 8 * h * d, 2: 8 * h * (held / c["block"])}[c["mode"]]
        return {"bytes": 2 * h * held * d + scales + 4 * sum(new) * hq * d,
                "flops": 4 * hq * d * sum(q * (x + q) for x, q in zip(ctx, new))}
    ctx, _, take = _lens(c)
    if c["op"] == "compact_bf16":
        return {"bytes": 8 * h * d * sum(take) + 12 * c["seqs"], "flops": 0}
    row = d + (4 if c["mode"] == 0 else 0)
    held = sum(ctx) + sum(take)
    return {"bytes": 4 * h * row * sum(take) + 2 * h * (row + 2 * d) * held + 12 * c["seqs"], "flops": 2 * h * d * held}


# ---- the definition in 64 bits -------------------------------------------------

def _exact_assign(c, s):
    held, want = _lens(c)
    bs = c["block"]
    table, free = s["table"].tolist(), s["free"].tolist()
    count, lens, slots = int(s["count"]), [], []
    for b, (h, w) in enumerate(zip(held, want)):
        for j in range(_up(w, bs), _up(h, bs)):
            free[count] = table[b][j]
            count += 1
    asked = 0
    have = count
    for b, (h, w) in enumerate(zip(held, want)):
        need = range(_up(h, bs), _up(w, bs))
        asked += len(need)
        good = len(need) == 0 or asked <= have
        if good:
            for j in need:
                count -= 1
                table[b][j] = free[count]
        lens.append(w if good else h)
        slots += [table[b][p // bs] * bs + p % bs if good else -1 for p in range(h, w)]
    return {"table": _i32(table), "free": _i32(free), "count": _i32([count]), "lens": _i32(lens),
            "slots": torch.tensor(slots, dtype=torch.int64, device="cuda")}


def _exact_values(c, s, n):
    """The pages as fp64 values."""
    x, scale = s[n + "_cache"], s[n + "_scale"].double()
    return x, scale[..., None] if c["mode"] == 0 else scale[None, :, None, :] if c["mode"] == 1 else scale[..., None, None]


def _exact_tree(c, s):
    ctx, new = _lens(c)
    h, g, d = c["kv_heads"], c["group"], c["dim"]
    pages = {n: _exact_values(c, s, n) for n in ("k", "v")}
    out, at = torch.zeros(sum(new), h * g, d, dtype=torch.float64, device="cuda"), 0
    masks = None if s["mask"] is None else [[w % 2 ** 64 for w in r] for r in s["mask"].tolist()]
    for b, (x, q) in enumerate(zip(ctx, new)):
        ids = s["table"][b].long()
        ids = ids[: _up(x + q, c["block"])]
        seen = torch.ones(q, x + q, dtype=torch.bool)
        for t in range(q):
            for i in range(q):
                seen[t, x + i] = i <= t if masks is None else bool(masks[at + t][i // 64] >> (i % 64) & 1)
        seen = seen.cuda()
        for j in range(h):
            k, v = ((p[ids, j].double() * (sc[0, j] if c["mode"] == 1 else sc[ids, j])).reshape(-1, d)[: x + q]
                    for p, sc in (pages["k"], pages["v"]))
            z = torch.einsum("tgd,pd->gtp", s["query"][at : at + q, j * g : (j + 1) * g].double(), k) * s["scale"]
            w = torch.softmax(z.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)
            out[at : at + q, j * g : (j + 1) * g] = torch.einsum("gtp,pd->tgd", w, v)
        at += q
    return out


def _exact_compact(c, s):
    ctx, _, take = _lens(c)
    bs = c["block"]
    idx, table = s["accepted"].tolist(), s["table"].tolist()
    moves = [(table[b][(x + i) // bs], (x + i) % bs, table[b][(x + k) // bs], (x + k) % bs)
             for b, (x, a) in enumerate(zip(ctx, take)) for k, i in enumerate(idx[b][:a])]
    si, sa, di, da = (torch.tensor([m[i] for m in moves], dtype=torch.long, device="cuda") for i in range(4))
    lens = [x + a for x, a in zip(ctx, take)]
    out = {"lens": _i32(lens)}
    places = [(table[b][p // bs], p % bs) for b, n in enumerate(lens) for p in range(n)]
    ri, ra = (torch.tensor([p[i] for p in places], dtype=torch.long, device="cuda") for i in range(2))
    for n in ("k", "v"):
        if c["op"] == "compact_bf16":
            cache = s[n + "_cache"].double()
            cache[di, :, da] = cache[si, :, sa]
            out[n + "_cache"] = cache
            continue
        cache, scale = _exact_values(c, s, n)
        cache, scale = cache.double(), scale.expand(cache.shape[0], -1, bs, -1).clone()
        if c["mode"] == 2:
            code = (cache[si, :, sa] * scale[si, :, sa] / scale[di, :, da]).round().clamp(-127, 127)
            cache[di, :, da] = code
        else:
            cache[di, :, da] = cache[si, :, sa]
            scale[di, :, da] = scale[si, :, sa]
        out[n + "_rows"] = cache[ri, :, ra] * scale[ri, :, ra]
    return out


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "tree":
        return _exact_tree(c, s)
    return _exact_assign(c, s) if c["op"] == "assign" else _exact_compact(c, s)
