"""What is measured of the rotary append, the norm-and-rotate pass and the
shared-prefix attention: cases, inputs, the calls, and their plain forms.

Operators (``op`` of a case):

* ``rope_store``       kvc8_rope_store: per-head RMS norm and rotary rotation
                       of the new queries and keys, keys and values quantised
                       into the int8 pages; the pages are read back as the
                       values they stand for with kvc8_dequant_gather.
* ``rope_store_bf16``  kvc8_rope_store_bf16: the same into bf16 pages.
* ``qk_norm_rope``     kvc8_qk_norm_rope: the same norm and rotation of query
                       and key rows, without a cache.
* ``shared_prefix``    kvc8_shared_prefix_attention: one decode query per
                       sequence over a prefix that all sequences share and
                       each sequence's own pages.
"""
import math
import random

import torch

own = False

_EPS = 1e-6
_TURN = 2.0 * math.pi


# ---- cases ------------------------------------------------------------------

def listed():
    rope = dict(op="rope_store", rot=128, interleaved=False, norm=True, base=1e6, scaling="none", factor=1.0, offset=0)
    pre = dict(op="shared_prefix")
    return [
        # one new token of one conversation: the smallest call, where latency counts
        dict(rope, name="append 1 token", seqs=1, new_lo=1, new_hi=1, ctx_lo=37, ctx_hi=37, q_heads=8, kv_heads=2,
             dim=64, block=16, mode=0, rot=64, lens=1),
        # a decode step of the benchmark's batch of 256, short contexts, behind a prefix of 4000
        dict(rope, name="append decode 256", seqs=256, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=255, q_heads=64,
             kv_heads=8, dim=128, block=128, mode=0, offset=4000, lens=2),
        # the benchmark's prompts (16 of 512 to 4096 tokens), dynamic scales, positions scaled by parts
        dict(rope, name="append prompts", seqs=16, new_lo=512, new_hi=4096, ctx_lo=0, ctx_hi=0, q_heads=32,
             kv_heads=8, dim=128, block=128, mode=0, scaling="by_parts", factor=8.0, lens=3),
        # chunks and single tokens mixed, per-channel scales, part of the head rotated, interleaved pairs
        dict(rope, name="append mixed static", seqs=33, new_lo=1, new_hi=611, ctx_lo=0, ctx_hi=1201, q_heads=24,
             kv_heads=8, dim=128, block=64, mode=1, rot=64, interleaved=True, norm=False, base=1e4, lens=4),
        # a decode step into bf16 pages
        dict(rope, op="rope_store_bf16", name="append bf16 decode", seqs=61, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=500,
             q_heads=32, kv_heads=4, dim=128, block=32, mode=0, norm=False, lens=5),
        # prompts into bf16 pages, with the norms
        dict(rope, op="rope_store_bf16", name="append bf16 prompts", seqs=16, new_lo=256, new_hi=2048, ctx_lo=0,
             ctx_hi=0, q_heads=32, kv_heads=8, dim=128, block=128, mode=0, scaling="linear", factor=4.0, lens=6),
        # the queries and keys of a single token, in place of two small passes
        dict(op="qk_norm_rope", name="rotate 1 token", tokens=1, q_heads=32, kv_heads=8, dim=128, rot=128,
             interleaved=False, norm=True, base=1e6, scaling="none", factor=1.0, first=131071),
        # a long prompt's queries and keys, odd count, interleaved, a quarter of the head left alone
        dict(op="qk_norm_rope", name="rotate prompt 20011", tokens=20011, q_heads=32, kv_heads=8, dim=128, rot=96,
             interleaved=True, norm=True, base=1e4, scaling="none", factor=1.0, first=3),
        # a handful of short conversations behind a short prefix
        dict(pre, name="prefix 1000 x 4", seqs=4, prefix=1000, own_lo=0, own_hi=64, kv_heads=2, group=4, dim=64,
             block=16, mode=0, lens=7),
        # an ordinary serving batch behind a prompt of 8192, dynamic scales
        dict(pre, name="prefix 8192 x 64", seqs=64, prefix=8192, own_lo=0, own_hi=512, kv_heads=8, group=8, dim=128,
             block=128, mode=0, lens=8),
        # odd sizes: per-block scales, 7 queries to a head, ragged prefix
        dict(pre, name="prefix 10007 x 23", seqs=23, prefix=10007, own_lo=1, own_hi=300, kv_heads=4, group=7, dim=128,
             block=48, mode=2, lens=9),
        # the benchmark's batch of 256 behind a long shared document, per-channel scales
        dict(pre, name="prefix 32768 x 256", seqs=256, prefix=32768, own_lo=1, own_hi=1024, kv_heads=8, group=4,
             dim=128, block=128, mode=1, lens=10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ranges: lengths over their logarithm, odd sizes, every mode and layout."""
    op = rng.choice(["rope_store", "rope_store", "rope_store_bf16", "qk_norm_rope", "shared_prefix", "shared_prefix"])
    lens = rng.randrange(1 << 30)
    if op == "shared_prefix":
        kv, group, dim = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 8), rng.choice([64, 128])
        seqs = _log_int(rng, 1, 256)
        most = 256 * 32 * 32768 // (seqs * kv * group)  # no more products than the largest listed case
        return dict(op=op, seqs=seqs, prefix=_log_int(rng, 1, max(1, min(32768, most))), own_lo=0,
                    own_hi=_log_int(rng, 1, 1024), kv_heads=kv, group=group, dim=dim,
                    block=16 * rng.randint(1, 8), mode=rng.randrange(3), lens=lens)
    dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
    kv, group = rng.choice([1, 2, 4, 5, 8]), rng.randint(1, 8)
    q_heads = kv * group
    rot = rng.choice([dim, dim, dim // 2 // 16 * 16, 16 * rng.randint(1, dim // 16)])
    more = dict(op=op, q_heads=q_heads, kv_heads=kv, dim=dim, rot=rot, interleaved=rng.random() < 0.5,
                norm=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]))
    scaling = rng.choice(["none", "linear", "by_parts"])
    more.update(scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]))
    rows = min(40000, 33883 * 48 * 128 // ((q_heads + 2 * kv) * dim))  # tokens of the largest listed case's work
    if op == "qk_norm_rope":
        return dict(more, tokens=_log_int(rng, 1, min(20011, rows)), first=rng.randrange(1 << 17))
    seqs = _log_int(rng, 1, 256)
    new = _log_int(rng, 1, max(1, min(4096, rows // seqs)))
    return dict(more, seqs=seqs, new_lo=1 if rng.random() < 0.5 else (new + 1) // 2, new_hi=new, ctx_lo=0,
                ctx_hi=_log_int(rng, 1, max(1, min(1201, 2 * rows // seqs))), block=rng.choice([1, 16, 24, 32, 64, 77, 128]),
                mode=rng.randrange(3) if op == "rope_store" else 0, offset=rng.choice([0, 0, rng.randrange(1 << 17)]),
                lens=lens)


def _lens(case):
    """Per-sequence lengths of a case (they belong to the case, not to the seed)."""
    rng = random.Random(case["lens"])
    n = case["seqs"]
    if case["op"] == "shared_prefix":
        return [rng.randint(case["own_lo"], case["own_hi"]) for _ in range(n)]
    return ([rng.randint(case["new_lo"], case["new_hi"]) for _ in range(n)],
            [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)])


def _inv_freq(case):
    """Radians per position of each rotated pair (64 bits), and the factor of cos and sin."""
    rot = case["rot"]
    inv = [case["base"] ** (-2.0 * i / rot) for i in range(rot // 2)]
    f = case["factor"]
    if case["scaling"] == "linear":
        return [v / f for v in inv], 1.0
    if case["scaling"] == "by_parts":  # pairs that turn often over the original length keep their speed
        out = []
        for v in inv:
            keep = min(1.0, max(0.0, (4096.0 * v / _TURN - 1.0) / (32.0 - 1.0)))
            out.append(v / f * (1.0 - keep) + v * keep)
        return out, 0.1 * math.log(f) + 1.0
    return inv, 1.0


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _heads(g, tokens, heads, dim):
    """bf16 N(0, 1) rows, four channels of each head far larger, as trained keys have them."""
    x = _normal(g, tokens, heads, dim)
    big = torch.rand(heads, dim, device="cuda", generator=g).argsort(1) < 4
    return torch.where(big, x * 20.0, x).to(torch.bfloat16)


def _table(g, seqs, per_seq, blocks):
    return torch.randperm(blocks, device="cuda", generator=g)[: seqs * per_seq].to(torch.int32).view(seqs, per_seq)


def _pool(g, s, blocks, heads, block, dim, mode, lo, hi):
    """Seeded codes on [-127, 127] in every page, and the scales of the mode."""
    for n in ("k", "v"):
        s[n + "_cache"] = torch.randint(-127, 128, (blocks, heads, block, dim), dtype=torch.int8, device="cuda", generator=g)
        shape = [(blocks, heads, block), (heads, dim), (blocks, heads)][mode]
        s[n + "_scale"] = torch.rand(shape, device="cuda", generator=g) * (hi - lo) + lo


def _rope_inputs(case, g, s):
    inv, s["mult"] = _inv_freq(case)
    s["inv"] = torch.tensor(inv, dtype=torch.float64, device="cuda")
    # turns per position as fractions of 2^64, what a program keeps beside its weights
    turns = [round(v / _TURN * 2.0 ** 64) & (2 ** 64 - 1) for v in inv]
    s["freqs"] = torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device="cuda")
    s["wq"] = s["wk"] = None
    if case["norm"]:
        s["wq"], s["wk"] = ((1.0 + 0.2 * _normal(g, case["dim"])).to(torch.bfloat16) for _ in range(2))


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "shared_prefix":
        heads, dim, block, n = case["kv_heads"], case["dim"], case["block"], case["seqs"]
        lens = _lens(case)
        own_blocks = max(1, -(-max(lens) // block))
        pre_blocks = max(1, -(-case["prefix"] // block))
        blocks = n * own_blocks + pre_blocks + 3
        _pool(g, s, blocks, heads, block, dim, case["mode"], 0.005, 0.03)
        ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
        s["prefix_table"] = ids[:pre_blocks].contiguous()
        s["table"] = ids[pre_blocks : pre_blocks + n * own_blocks].contiguous().view(n, own_blocks)
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["query"] = _normal(g, n, heads * case["group"], dim).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["query"])
        s["scale"] = dim ** -0.5
        return s
    _rope_inputs(case, g, s)
    if case["op"] == "qk_norm_rope":
        n = case["tokens"]
        s["query"], s["key"] = _heads(g, n, case["q_heads"], case["dim"]), _heads(g, n, case["kv_heads"], case["dim"])
        s["q_out"], s["k_out"] = torch.empty_like(s["query"]), torch.empty_like(s["key"])
        s["positions"] = torch.arange(case["first"], case["first"] + n, dtype=torch.int32, device="cuda")
        return s
    new, ctx = _lens(case)
    n, total, heads, dim, block = case["seqs"], sum(new), case["kv_heads"], case["dim"], case["block"]
    per_seq = max(-(-(a + b) // block) for a, b in zip(new, ctx))
    blocks = n * per_seq + 2
    cu = [0]
    for q in new:
        cu.append(cu[-1] + q)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["after"] = torch.tensor([a + b for a, b in zip(new, ctx)], dtype=torch.int32, device="cuda")
    s["rows"] = sum(new) + sum(ctx)
    s["query"], s["key"], s["value"] = (_heads(g, total, h, dim) for h in (case["q_heads"], heads, heads))
    s["q_out"] = torch.empty_like(s["query"])
    s["table"] = _table(g, n, per_seq, blocks)
    s["positions"] = None
    if case["offset"]:  # the pages hold what follows a shared prefix: positions go on behind it
        seq = torch.bucketize(torch.arange(total, device="cuda"), s["cu"][1:].long(), right=True)
        s["positions"] = (case["offset"] + s["ctx"][seq] + torch.arange(total, device="cuda") - s["cu"][seq]).to(torch.int32)
    if case["op"] == "rope_store_bf16":
        for k in ("k_cache", "v_cache"):
            s[k] = _normal(g, blocks, heads, block, dim).to(torch.bfloat16)
    else:
        _pool(g, s, blocks, heads, block, dim, case["mode"], 0.02, 0.05)
        for k in ("k_rows", "v_rows"):
            s[k] = torch.empty(s["rows"], heads, dim, dtype=torch.bfloat16, device="cuda")
    return s


# ---- the framework's calls --------------------------------------------------

def _space(s, key, size):
    """A workspace that the program keeps."""
    if key not in s:
        s[key] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")
    return s[key]


def _rope(kv, s):
    if "rope" not in s:
        c = s["case"]
        s["rope"] = kv.Rope(rotary_dim=c["rot"], interleaved=int(c["interleaved"]), attention_factor=s["mult"],
                            norm_eps=_EPS, freqs=s["freqs"], q_norm_weight=s["wq"], k_norm_weight=s["wk"],
                            positions=s["positions"])
    return s["rope"]


def _own(s):
    import dequant_kvc8_store_gb300 as kv
    c = s["case"]
    q = s["query"]
    if c["op"] == "qk_norm_rope":
        k, qo, ko = s["key"], s["q_out"], s["k_out"]
        kv.kvc8_qk_norm_rope(_rope(kv, s), c["tokens"], c["dim"], c["q_heads"], q, q.stride(0), q.stride(1), qo,
                             qo.stride(0), qo.stride(1), c["kv_heads"], k, k.stride(0), k.stride(1), ko,
                             ko.stride(0), ko.stride(1))
        return {"q": qo, "k": ko}
    if "geom" not in s:
        t = s["table"]
        s["geom"] = kv.Geom(c["seqs"], c["kv_heads"], c["dim"], c["block"], s["k_cache"].shape[0], t.shape[1], c["mode"])
    g = s["geom"]
    if c["op"] == "shared_prefix":
        o, heads = s["out"], c["kv_heads"] * c["group"]
        if "ws_bytes" not in s:
            s["ws_bytes"] = kv.kvc8_shared_prefix_workspace_bytes(g, heads, s["prefix_table"].shape[0])
        kv.kvc8_shared_prefix_attention(g, heads, q, q.stride(0), q.stride(1), s["k_cache"], s["v_cache"],
                                        s["k_scale"], s["v_scale"], s["prefix_table"], s["prefix_table"].shape[0],
                                        s["prefix_len"], s["table"], s["lens"], s["scale"], o, o.stride(0),
                                        o.stride(1), _space(s, "ws", s["ws_bytes"]), s["ws_bytes"])
        return o
    k, v, qo = s["key"], s["value"], s["q_out"]
    n = k.shape[0]
    if c["op"] == "rope_store_bf16":
        kv.kvc8_rope_store_bf16(g, _rope(kv, s), n, c["q_heads"], q, q.stride(0), q.stride(1), qo, qo.stride(0),
                                qo.stride(1), k, v, k.stride(0), k.stride(1), s["k_cache"], s["v_cache"],
                                s["table"], s["cu"], s["ctx"])
        return {"q": qo, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    kv.kvc8_rope_store(g, _rope(kv, s), n, c["q_heads"], q, q.stride(0), q.stride(1), qo, qo.stride(0), qo.stride(1),
                       k, v, k.stride(0), k.stride(1), s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                       s["table"], s["cu"], s["ctx"])
    if "ws_bytes" not in s:
        s["ws_bytes"] = kv.kvc8_gather_workspace_bytes(g)
    kr, vr = s["k_rows"], s["v_rows"]
    kv.kvc8_dequant_gather(g, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["after"], None,
                           kr, vr, s["rows"], kr.stride(0), kr.stride(1), _space(s, "ws", s["ws_bytes"]), s["ws_bytes"])
    return _int8_outputs(s, qo, kr, vr)


def _int8_outputs(s, q, k_rows, v_rows):
    out = {"q": q, "k_rows": k_rows, "v_rows": v_rows}
    if s["case"]["mode"] == 0:  # the scale of each row is written beside its codes
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


# ---- the plain forms --------------------------------------------------------

def _norm_rotate(x, w, pos, s):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()
    rot = c["rot"]
    angle = pos.double()[:, None] * s["inv"]  # 64 bits: far positions turn many times
    cos, sin = (torch.cos(angle) * s["mult"]).float()[:, None], (torch.sin(angle) * s["mult"]).float()[:, None]
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
        y[..., : rot // 2], y[..., rot // 2 : rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _quantise(x, scale):
    """Codes of fp32 rows for a scale that broadcasts over them."""
    q = torch.round(x / scale).clamp(-127, 127)
    return torch.where(scale == 0, torch.zeros_like(q), q).to(torch.int8)


def _plain_attention(s):
    c = s["case"]
    n, h, g, d, bs = c["seqs"], c["kv_heads"], c["group"], c["dim"], c["block"]

    def rows(cache, scale, ids, slot):
        """[...][h][d] fp32 values of positions (ids, slot)."""
        x = cache[ids, :, slot].float()
        if c["mode"] == 0:
            return x * scale[ids, :, slot][..., None]
        return x * (scale if c["mode"] == 1 else scale[ids][..., None])

    q = s["query"].float().view(n, h, g, d)
    p = torch.arange(c["prefix"], device="cuda")
    pid, pslot = s["prefix_table"].long()[p // bs], p % bs
    own = torch.arange(s["table"].shape[1] * bs, device="cuda")[: max(1, c["own_hi"])]
    oid, oslot = s["table"].long()[:, own // bs], (own % bs).expand(n, -1)
    qp = q.permute(1, 0, 2, 3).reshape(h, n * g, d)  # every query row of a kv head against the one prefix
    sp = torch.matmul(qp, rows(s["k_cache"], s["k_scale"], pid, pslot).permute(1, 2, 0)) * s["scale"]
    ko = rows(s["k_cache"], s["k_scale"], oid, oslot).permute(0, 2, 3, 1)  # [n][h][d][own]
    so = torch.matmul(q, ko) * s["scale"]
    live = (own < s["lens"][:, None])[:, None, None]
    so = so.masked_fill(~live, -math.inf).permute(1, 0, 2, 3).reshape(h, n * g, -1)
    top = so.amax(-1, keepdim=True)
    if c["prefix"]:
        top = torch.maximum(top, sp.amax(-1, keepdim=True))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    wp, wo = torch.exp(sp - top), torch.exp(so - top)
    total = wp.sum(-1, keepdim=True) + wo.sum(-1, keepdim=True)
    acc = torch.matmul(wp, rows(s["v_cache"], s["v_scale"], pid, pslot).transpose(0, 1))
    vo = rows(s["v_cache"], s["v_scale"], oid, oslot).transpose(1, 2)  # [n][h][own][d]
    acc = acc + torch.matmul(wo.view(h, n, g, -1).transpose(0, 1), vo).transpose(0, 1).reshape(h, n * g, d)
    out = torch.where(total > 0, acc / total, torch.zeros_like(acc))
    return out.view(h, n, g, d).transpose(0, 1).reshape(n, h * g, d).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        return _own(s)
    c = s["case"]
    if c["op"] == "shared_prefix":
        return _plain_attention(s)
    if c["op"] == "qk_norm_rope":
        return {"q": _norm_rotate(s["query"], s["wq"], s["positions"], s).to(torch.bfloat16),
                "k": _norm_rotate(s["key"], s["wk"], s["positions"], s).to(torch.bfloat16)}
    total, bs = s["key"].shape[0], c["block"]
    t = torch.arange(total, device="cuda")
    seq = torch.bucketize(t, s["cu"][1:].long(), right=True)
    slot = s["ctx"][seq].long() + t - s["cu"][seq]
    pos = slot if s["positions"] is None else s["positions"]
    q = _norm_rotate(s["query"], s["wq"], pos, s).to(torch.bfloat16)
    k, v = _norm_rotate(s["key"], s["wk"], pos, s), s["value"].float()
    ids, at = s["table"][seq, slot // bs].long(), slot % bs
    if c["op"] == "rope_store_bf16":
        s["k_cache"][ids, :, at], s["v_cache"][ids, :, at] = k.to(torch.bfloat16), v.to(torch.bfloat16)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    rows = []
    for x, n in ((k, "k"), (v, "v")):
        cache, scale = s[n + "_cache"], s[n + "_scale"]
        if c["mode"] == 0:
            by = x.abs().amax(-1) / 127.0
            scale[ids, :, at] = by
            by = by[..., None]
        else:
            by = scale if c["mode"] == 1 else scale[ids][..., None]
        cache[ids, :, at] = _quantise(x, by.expand_as(x))
        # the values that the pages stand for, sequence by sequence
        end = s["after"].long().cumsum(0)
        r = torch.arange(s["rows"], device="cuda")
        b = torch.bucketize(r, end, right=True)
        p = r - end[b] + s["after"][b]
        rid, rat = s["table"][b, p // bs].long(), p % bs
        y = cache[rid, :, rat].float()
        y = y * (scale[rid, :, rat][..., None] if c["mode"] == 0 else scale if c["mode"] == 1 else scale[rid][..., None])
        rows.append(y.to(torch.bfloat16))
    return _int8_outputs(s, q, rows[0], rows[1])


# ---- what a pass cannot do without --------------------------------------------

def work(case):
    c = case
    d = c["dim"]
    if c["op"] == "shared_prefix":
        h, hq, held = c["kv_heads"], c["kv_heads"] * c["group"], c["prefix"] + sum(_lens(c))
        # each cached position once, its scales, the queries and the outputs
        scales = {0: 8 * h * held, 1: 8 * h * d, 2: 8 * h * (held / c["block"])}[c["mode"]]
        return {"bytes": 2 * h * held * d + scales + 4 * c["seqs"] * hq * d,
                "flops": 4 * hq * d * (c["seqs"] * c["prefix"] + sum(_lens(c)))}
    hq, h = c["q_heads"], c["kv_heads"]
    if c["op"] == "qk_norm_rope":
        return {"bytes": 4 * d * c["tokens"] * (hq + h), "flops": 8 * d * c["tokens"] * (hq + h)}
    new, ctx = (sum(x) for x in _lens(c))
    if c["op"] == "rope_store_bf16":
        return {"bytes": 4 * d * new * (hq + 2 * h), "flops": 8 * d * new * (hq + h)}
    row = d + (4 if c["mode"] == 0 else 0)
    store = new * (4 * d * hq + 2 * h * (2 * d + row))
    read = (new + ctx) * 2 * h * (row + 2 * d)
    return {"bytes": store + read, "flops": new * 8 * d * (hq + 2 * h) + 2 * d * h * (new + ctx)}


# ---- the definition in 64 bits -------------------------------------------------

def _exact_turned(x, w, pos, inv, mult, c):
    """Norm, then each pair as a complex number times mult * e^(i pos inv)."""
    z = x.double()
    if w is not None:
        z = z / (z.pow(2).sum(-1, keepdim=True) / c["dim"] + _EPS).sqrt() * w.double()
    rot = c["rot"]
    shape = z.shape[:-1]
    pairs = z[..., :rot].reshape(*shape, rot // 2, 2) if c["interleaved"] else z[..., :rot].reshape(*shape, 2, rot // 2).transpose(-1, -2)
    turn = torch.polar(torch.full_like(inv, mult).expand(pos.numel(), -1).contiguous(), torch.outer(pos.double(), inv))
    r = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn[:, None])
    r = r.reshape(*shape, rot) if c["interleaved"] else r.transpose(-1, -2).reshape(*shape, rot)
    return torch.cat([r, z[..., rot:]], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d, bs = c["dim"], c["block"] if "block" in c else 1
    if c["op"] == "qk_norm_rope":
        return {n[0]: _exact_turned(s[n], s["w" + n[0]], s["positions"], s["inv"], s["mult"], c) for n in ("query", "key")}
    if c["op"] == "shared_prefix":
        h, g, n = c["kv_heads"], c["group"], c["seqs"]
        full = {}
        for k in ("k", "v"):
            sc = s[k + "_scale"].double()
            sc = sc[..., None] if c["mode"] == 0 else sc[None, :, None, :] if c["mode"] == 1 else sc[..., None, None]
            full[k] = (s[k + "_cache"], sc)

        def span(k, ids, count):
            """[h][count][d]: the first count positions of these blocks."""
            cache, sc = full[k]
            sc = sc.expand(1, h, 1, d) if c["mode"] == 1 else sc[ids]
            return (cache[ids].double() * sc).transpose(0, 1).reshape(h, -1, d)[:, :count]

        shared = {k: span(k, s["prefix_table"].long(), c["prefix"]) for k in ("k", "v")}
        q = s["query"].double().view(n, h, g, d) * s["scale"]
        first = torch.einsum("nhgd,hpd->nhgp", q, shared["k"])
        out = torch.zeros(n, h, g, d, dtype=torch.float64, device="cuda")
        for b, count in enumerate(_lens(c)):
            k, v = (span(x, s["table"][b].long(), count) for x in ("k", "v"))
            z = torch.cat([first[b], torch.matmul(q[b], k.transpose(1, 2))], -1)
            if z.shape[-1]:
                w = torch.softmax(z, -1)
                out[b] = torch.matmul(w[..., : c["prefix"]], shared["v"]) + torch.matmul(w[..., c["prefix"] :], v)
        return out.view(n, h * g, d)
    new, ctx = _lens(c)
    seq = torch.tensor([b for b, q in enumerate(new) for _ in range(q)], device="cuda")
    slot = torch.tensor([x + i for q, x in zip(new, ctx) for i in range(q)], device="cuda")
    pos = slot + c["offset"]
    q = _exact_turned(s["query"], s["wq"], pos, s["inv"], s["mult"], c)
    rows = {"k": _exact_turned(s["key"], s["wk"], pos, s["inv"], s["mult"], c), "v": s["value"].double()}
    ids, at = s["table"].long()[seq, slot.div(bs, rounding_mode="floor")], slot.remainder(bs)
    if c["op"] == "rope_store_bf16":
        out = {"q": q}
        for k in ("k", "v"):
            p = s[k + "_cache"].double()
            p[ids, :, at] = rows[k]
            out[k + "_cache"] = p
        return out
    out = {"q": q}
    places = [(b, p) for b, (x, y) in enumerate(zip(new, ctx)) for p in range(x + y)]
    places = torch.tensor(places, device="cuda")
    rid, rat = s["table"].long()[places[:, 0], places[:, 1].div(bs, rounding_mode="floor")], places[:, 1].remainder(bs)
    for k in ("k", "v"):
        sc = s[k + "_scale"].double()
        if c["mode"] == 0:
            per = rows[k].abs().max(-1).values / 127.0
            sc[ids, :, at] = per
            out[k + "_scale"] = sc
            per, every = per[..., None], sc[rid, :, rat][..., None]
        else:
            per, every = (sc, sc) if c["mode"] == 1 else (sc[ids][..., None], sc[rid][..., None])
        cache = s[k + "_cache"].double()
        code = torch.nan_to_num(rows[k] / per).round().clamp(-127, 127)
        cache[ids, :, at] = code
        out[k + "_rows"] = cache[rid, :, rat] * every
    return out
