"""Block assignment and compaction as loops over the definition, and tree-attention problems
with their 64-bit answers and how far a call may be off.

Tree attention, data: as in _prefix_ref (a value's code is a mean of its sequence and head, one
of its page and noise), and four channels of queries and draft keys that give the drafts about
as much weight as the context, so that a wrong mask shows.

Bound, with u = 2^-11 (fp16), b = 2^-8 (bf16) and f = 2^-23 (an fp32 step that may truncate), as
derived in _prefix_ref for a prefix's rows, which all positions are here:
* score: delta_p = A_p (r + D f) + |scale| 2^-25 max|q| sum_d |k_pd| + 2^-20 (1 + max|z|), A_p =
  |scale| sum_d |q_d k_pd|, r = 2 u with a row's or block's scale (fp16(code * fp16(scale))), u with
  the channels' (fp16(q s));
* weight u, value 2 u with a row's or block's scale; below 2^-21 of the largest, weights are off by
  2^-31 of it;
* sums of n: (n + 64) / 8 f of their size;
* numerator N = sum w |V| (e^delta ... - 1), denominator E, output (N + |out| E) / (1 - E), rounded: b.
"""
import numpy as np
import torch

import dequant_kvc8_store_gb300 as kv

U16, UB, F32 = 2.0 ** -11, 2.0 ** -8, 2.0 ** -23
BIAS = 4


def assign(held, want, free, count, table, bs, num_blocks, slot_rows=None):
    """(free, count, table, lens, slots, error codes) of kvc8_assign_blocks."""
    free, table, errors = list(free), [list(r) for r in table], set()
    cap = len(table[0]) * bs if len(table) else 0
    if not 0 <= count <= num_blocks:
        errors.add(kv.DEV_BAD_LENGTH)
        count = min(max(count, 0), num_blocks)
    good = []
    for h, w in zip(held, want):
        good.append(0 <= h <= cap and 0 <= w <= cap)
        if not good[-1]:
            errors.add(kv.DEV_BAD_LENGTH if h < 0 or w < 0 else kv.DEV_POS_BEYOND_TABLE)
    up = lambda x: -(-x // bs)  # noqa: E731
    for b, (h, w) in enumerate(zip(held, want)):
        for j in range(up(w), up(h)) if good[b] else ():
            if not 0 <= table[b][j] < num_blocks:
                errors.add(kv.DEV_BAD_BLOCK_ID)
            if count < num_blocks:
                free[count] = table[b][j]
                count += 1
            else:
                errors.add(kv.DEV_BAD_LENGTH)
    have, asked, lens, slots = count, 0, [], []
    for b, (h, w) in enumerate(zip(held, want)):
        need = range(up(h), up(w)) if good[b] else range(0)
        asked += len(need)
        served = good[b] and (len(need) == 0 or asked <= have)
        if good[b] and not served:
            errors.add(kv.DEV_NO_FREE_BLOCK)
        for j in need if served else ():
            count -= 1
            table[b][j] = free[count]
            if not 0 <= free[count] < num_blocks:
                errors.add(kv.DEV_BAD_BLOCK_ID)
        lens.append(w if served else h)
        for p in range(max(h, 0), w) if h >= 0 else ():
            if slot_rows is None or len(slots) <= slot_rows:
                slots.append(table[b][p // bs] * bs + p % bs if served else -1)
    if slot_rows is not None and len(slots) > slot_rows:
        errors.add(kv.DEV_OUT_ROW_RANGE)
        slots = slots[:slot_rows]
    return free, count, table, lens, slots, errors


def compact(mode, k_cache, v_cache, k_scale, v_scale, table, ctx, accepted, num, bs):
    """kvc8_compact_drafts in place on numpy arrays (mode None: bf16 bits); returns the lengths."""
    lens = []
    for b, n in enumerate(num):
        for k in range(n):
            f, t = int(ctx[b]) + int(accepted[b][k]), int(ctx[b]) + k
            fb, tb = table[b][f // bs], table[b][t // bs]
            if f == t:
                continue
            for cache, scale in ((k_cache, k_scale), (v_cache, v_scale)):
                x = cache[fb, :, f % bs].copy()
                if mode == 2:
                    s, d = scale[fb].astype(np.float32), scale[tb].astype(np.float32)
                    with np.errstate(divide="ignore", invalid="ignore"):
                        y = np.clip(np.rint((x.astype(np.float32) * s[:, None]) / d[:, None]), -127, 127)
                    y[d == 0] = 0
                    x = np.where((s == d)[:, None], x, y.astype(np.int8))
                cache[tb, :, t % bs] = x
                if mode == 0:
                    scale[tb, :, t % bs] = scale[fb, :, f % bs]
        lens.append(int(ctx[b]) + n)
    return lens


def random_masks(rng, news, words, kind):
    """uint64 [N][words]: ancestors in random trees ('tree'), any bits ('any'), or none ('none')."""
    out = np.zeros((max(1, sum(news)), words), np.uint64)
    n = 0
    for q in news:
        seen = []
        for i in range(q):
            if kind == "tree":
                p = int(rng.integers(-1, i)) if i else -1
                seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            elif kind == "any":
                seen.append(int.from_bytes(rng.bytes(8 * words), "little") if rng.random() > 0.15 else 0)
            else:
                seen.append(0)
            for w in range(words):
                out[n, w] = np.uint64(seen[-1] >> (64 * w) & (2 ** 64 - 1))
            n += 1
    return out


class TreeProblem:
    """A pool, tables, drafts and queries on `device`."""

    def __init__(self, ctx, new, H=2, G=4, D=64, bs=16, mode=0, kind="tree", sharp=True, seed=0, spare=1,
                 words=None, most=None, device="cuda"):
        self.ctx, self.new, self.H, self.G, self.D, self.bs, self.mode = list(ctx), list(new), H, G, D, bs, mode
        self.kind, self.sharp, self.device = kind, sharp, device
        B, N = len(self.ctx), sum(new)
        self.B, self.N = B, N
        gen = torch.Generator()
        gen.manual_seed(seed * 1000003 + 101 * sum(ctx) + 7 * N + D + 2 * H + mode + sharp)
        rng = np.random.default_rng([seed, N, sum(ctx)])
        uni = lambda lo, hi, *s: torch.rand(*s, generator=gen).to(device) * (hi - lo) + lo  # noqa: E731
        normal = lambda *s: torch.randn(*s, generator=gen).to(device)  # noqa: E731
        self.lens = [c + q for c, q in zip(ctx, new)]
        self.MB = max(1, -(-max(self.lens) // bs) + spare)
        NB = B * self.MB + 2
        ids = torch.randperm(NB, generator=gen).to(device)
        self.tab = ids[:B * self.MB].view(B, self.MB).to(torch.int32).contiguous()
        owner = torch.full((NB,), B, dtype=torch.long, device=device)
        owner[self.tab.long()] = torch.arange(B, device=device)[:, None]
        sign = (torch.rand(B + 1, H, D, generator=gen) < 0.5).to(device).float() * 2 - 1
        mean = uni(30, 60, B + 1, H, D) * sign
        self.vc = torch.empty(NB, H, bs, D, dtype=torch.int8, device=device)
        self.kc = torch.empty_like(self.vc)
        for i in range(0, NB, 256):
            n = min(256, NB - i)
            page = mean[owner[i:i + n]][:, :, None] + uni(-35, 35, n, H, 1, D) + 25 * normal(n, H, bs, D)
            self.vc[i:i + n] = page.round().clamp(-127, 127).to(torch.int8)
            self.kc[i:i + n] = torch.randint(-127, 128, (n, H, bs, D), generator=gen, dtype=torch.int8).to(device)
        shape = [(NB, H, bs), (H, D), (NB, H)][mode]
        self.ks, self.vs = (2.0 ** uni(-8, -5, *shape) for _ in range(2))
        q = normal(max(N, 1), H * G, D)
        q[..., :BIAS] = 8.0 if sharp else 40.0
        self.q = q.to(torch.bfloat16)
        s2 = float(self.ks.double().pow(2).mean()) ** 0.5
        self.scale = (3.0 if sharp else 0.25) / (73.3 * s2 * (D - BIAS) ** 0.5)
        self.kc[:, :, :, :BIAS] = 0
        for b in range(B):  # the drafts' keys: a few of them have about the context's weight
            gain = float(np.log(max(1.0, self.ctx[b] / 2))) + (2.0 if sharp and self.ctx[b] else 0.0)
            gain /= float(self.q[0, 0, 0]) * BIAS * self.scale
            for p in range(self.ctx[b], self.lens[b]):
                blk, at = int(self.tab[b, p // bs]), p % bs
                s = self.ks[blk, :, at] if mode == 0 else self.ks[:, :BIAS].mean(-1) if mode == 1 else self.ks[blk]
                self.kc[blk, :, at, :BIAS] = (gain / s).round().clamp(-127, 127).to(torch.int8)[:, None]
        self.most = most if most is not None else max(1, max(new, default=1))
        self.words = words if words is not None else -(-self.most // 64)
        self.mask = None if kind == "chain" else random_masks(rng, self.new, self.words, kind)
        self.g = kv.Geom(B, H, D, bs, NB, self.MB, mode)
        self.d = None

    def sees(self, b, shift=0):
        """bool [T][ctx + T] of sequence b (shift: of that many drafts on, for a wrong answer)."""
        c, q = self.ctx[b], self.new[b]
        out = torch.ones(q, c + q, dtype=torch.bool)
        n = sum(self.new[:b])
        for t in range(q):
            for i in range(q):
                out[t, c + i] = i <= t if self.mask is None else bool(int(self.mask[n + t][i // 64]) >> (i % 64) & 1)
        if shift:
            out = torch.cat([out[:, :c], out[:, c:].roll(-shift, 0)], 1)
        return out.to(self.device)

    def rows(self, cache, scale, b, h):
        ids = self.tab[b, :-(-self.lens[b] // self.bs)].long()
        x, s = cache[ids, h].double(), scale.double()
        if self.mode == 0:
            x = x * s[ids, h][..., None]
        elif self.mode == 1:
            x = x * s[h]
        else:
            x = x * s[ids, h][:, None, None]
        return x.reshape(-1, self.D)[:self.lens[b]]

    def answers(self, heads=None):
        """want, tol [N][Hq][D], and wrong answers {name: (out, applies [N])}."""
        B, H, G, D = self.B, self.H, self.G, self.D
        want = torch.zeros(self.N, H * G, D, dtype=torch.float64, device=self.device)
        tol = torch.zeros_like(want)
        wrong = {k: torch.zeros_like(want) for k in ("context left out", "drafts left out", "every draft seen",
                                                     "the next draft's mask")}
        applies = {k: torch.zeros(self.N, dtype=torch.bool, device=self.device) for k in wrong}
        scaled = self.mode != 1
        r, wr = (2 * U16, 3 * U16 + 2 * U16 ** 2) if scaled else (U16, U16)
        n0 = 0
        for b in range(B):
            c, q = self.ctx[b], self.new[b]
            if q == 0:
                continue
            row = slice(n0, n0 + q)
            seen = self.sees(b)[:, None]
            is_draft = torch.arange(c + q, device=self.device) >= c
            masks = {"context left out": seen & is_draft, "drafts left out": seen & ~is_draft,
                     "every draft seen": torch.ones_like(seen), "the next draft's mask": self.sees(b, 1)[:, None]}
            n_seen, n_draft = seen.sum((1, 2)), (seen & is_draft).sum((1, 2))
            most = {k: (masks[k] ^ seen).sum((1, 2)) >= 1 + n_draft // 2 for k in masks if "left out" not in k}
            for h in range(H):
                j = slice(h * G, (h + 1) * G)
                qs = self.q[row, j].double()
                k, v = self.rows(self.kc, self.ks, b, h), self.rows(self.vc, self.vs, b, h)
                z = torch.matmul(qs, k.T) * self.scale
                size = torch.matmul(qs.abs(), k.abs().T) * abs(self.scale)
                low = qs.abs().amax(-1, keepdim=True) * k.abs().sum(-1) * abs(self.scale)

                def mean(m):
                    top = z.masked_fill(~m, -np.inf).amax(-1, keepdim=True)
                    e = torch.exp(z - torch.where(torch.isfinite(top), top, 0.0)) * m
                    w = torch.where(m, e, 0.0) / e.sum(-1, keepdim=True).clamp(min=1e-300)
                    return w, torch.matmul(w, v)

                w, o = mean(seen)
                want[row, j] = o
                # (a side that weighs less than a twentieth in every head may be missed)
                share = (w * is_draft).sum(-1).amax(-1)
                applies["drafts left out"][row] |= (share > 0.05) & (c > 0)
                applies["context left out"][row] |= ((w * ~is_draft).sum(-1).amax(-1) > 0.05) & (n_draft > 0)
                for name, m in masks.items():
                    u, wrong[name][row, j] = mean(m)
                    if name in most:  # what sees too much, or too little, weighs something
                        gap = torch.maximum((u * ~seen).sum(-1), (w * ~m).sum(-1)).amax(-1)
                        applies[name][row] |= most[name] & (gap > 0.05)
                # (only positions that a row sees matter to it)
                big = (z.abs() * seen).amax(-1, keepdim=True)
                delta = size * (r + D * F32) + low * 2.0 ** -25 + 2.0 ** -20 * (1 + big)
                off = torch.expm1(delta) * seen
                sums = (c + q + 64) / 8 * F32
                N = torch.matmul(w * ((1 + off) * (1 + wr) - 1 + sums), v.abs())
                N = N + (c + q) * 2.0 ** -31 * v.abs().max()
                E = (w * (off + sums)).sum(-1, keepdim=True)
                assert float(E.max()) < 0.2
                err = (N + o.abs() * E) / (1 - E)
                tol[row, j] = torch.where(n_seen[:, None, None] > 0, err + UB * (o.abs() + err), 0.0)
            n0 += q
        out = {k: (wrong[k], applies[k]) for k in wrong}
        some = torch.zeros(self.N, dtype=torch.bool, device=self.device)
        n0 = 0
        for b in range(B):
            some[n0:n0 + self.new[b]] = (self.sees(b).sum(1) > 0)
            n0 += self.new[b]
        out["zeros"] = (torch.zeros_like(want), some)
        if H > 1:
            out["the next head's"] = (want.roll(-G, 1), some)
        if G > 1 and self.sharp:
            turned = want.view(-1, H, G, D).roll(-1, 2).reshape(-1, H * G, D)
            enough = torch.cat([(self.sees(b).sum(1) > 16) for b in range(B)]) if self.N else some
            out["the next query's"] = (turned, enough)
        return want, tol, out

    def check(self, got):
        want, tol, wrong = self.answers()
        got = got[:self.N].double().to(want.device)
        bad = ~((got - want).abs() <= tol)
        assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                                     tol[bad][:4].tolist(), int(bad.sum()))
        for name, (out, applies) in wrong.items():
            seen = ((out - want).abs() > 2 * tol).flatten(1).any(1)
            # (with sharp scores a single position may weigh nearly all, or one of few next to nothing)
            part = (0.5 if self.sharp else 0.75) if "draft" in name or "left out" in name else 0.9 if "query" in name else 1.0
            assert int((applies & seen).sum()) >= part * int(applies.sum()), (name, (applies & ~seen).nonzero()[:8].tolist())

    def place(self, rows=None):
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=self.device)  # noqa: E731
        rows = self.N if rows is None else rows
        cu = np.concatenate([[0], np.cumsum(self.new)])
        need = kv.kvc8_tree_attention_workspace_bytes(self.g, self.H * self.G, rows, self.most)
        mask = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).to(self.device)
        self.d = dict(cu=i32(cu), ctx=i32(self.ctx), mask=mask, err=i32([0]), rows=rows,
                      ws=torch.full((need,), 0xFF, dtype=torch.uint8, device=self.device))
        self.out = torch.full((rows, *self.q.shape[1:]), float("nan"), dtype=torch.bfloat16, device=self.device)

    def run(self):
        if self.d is None:
            self.place()
        d, q, o = self.d, self.q, self.out
        kv.kvc8_tree_attention(self.g, self.H * self.G, d["rows"], self.most, q, q.stride(0), q.stride(1), self.kc,
                               self.vc, self.ks, self.vs, self.tab, d["cu"], d["ctx"], d["mask"], self.words,
                               self.scale, o, o.stride(0), o.stride(1), d["ws"], d["ws"].numel(), d["err"])
        return o

    def error(self):
        return kv.kvc8_get_error(self.d["err"], reset=True)

    def rounded(self):
        """The attention with each operand rounded as the kernel rounds it (on the CPU, against the bound)."""
        out = torch.zeros(self.N, self.H * self.G, self.D, dtype=torch.float64)
        half = lambda x, p: (x * 2.0 ** p).to(torch.float16).double() * 2.0 ** -p  # noqa: E731
        n0 = 0
        for b in range(self.B):
            c, q = self.ctx[b], self.new[b]
            seen = self.sees(b)[:, None]
            for h in range(self.H):
                j = slice(h * self.G, (h + 1) * self.G)
                ids = self.tab[b, :-(-(c + q) // self.bs)].long()
                code = [x[ids, h].double().reshape(-1, self.D)[:c + q] for x in (self.kc, self.vc)]
                qs = self.q[n0:n0 + q, j].double()
                if self.mode == 1:
                    qs = qs * self.ks[h].double()
                    k, v = code
                else:
                    def by(s):
                        s = s[ids, h].double()
                        return (s if self.mode == 0 else s[:, None].expand(-1, self.bs)).reshape(-1, 1)[:c + q]
                    k, v = (half(x * half(by(s), 6), 6) for x, s in zip(code, (self.ks, self.vs)))
                top = 2.0 ** torch.floor(torch.log2(qs.abs().amax(-1, keepdim=True)))
                qs = (qs / top).to(torch.float16).double() * top
                z = (torch.matmul(qs, k.T) * self.scale).float().masked_fill(~seen, -np.inf)
                m = z.amax(-1, keepdim=True)
                w = torch.exp(z - torch.where(torch.isfinite(m), m, 0.0)).double()
                o = torch.matmul(half(w, 7), v) / w.sum(-1, keepdim=True).clamp(min=1e-300)
                out[n0:n0 + q, j] = o * self.vs[h].double() if self.mode == 1 else o
            n0 += q
        return out.to(torch.bfloat16)
