"""Shared-prefix attention problems whose answers tell one mistake from another, their 64-bit
answers, and how far a call may be off.

Data.  A value's code is a mean of its owner (the prefix, or the sequence) and head, a mean of
its page and noise, so that an output is a good part of the largest value and differs between
heads, sequences, and prefix and own positions.  Four channels of the queries hold a constant, and
of a sequence's own keys a code that gives prefix and own positions about equal weight.
`sharp` scores have a standard deviation of 3 (a few positions decide, so every key counts),
the others of 1/4 (all positions count).

Bound.  With half a step u = 2^-11 of fp16, b = 2^-8 of bf16, and f = 2^-23 for an fp32
accumulation that may truncate:
* score of position p: A_p = |scale| sum_d |q_d k_pd|.  Queries enter as fp16 (a bf16 value is
  exact, below 2^-14 of the row's largest it is off by 2^-25 of that); prefix rows with a row's or a
  block's scale as fp16(code * fp16(scale)), so 2 u; with channel scales the products q_d s_d
  as fp16, u, on either side; own rows otherwise exact.  D fp32 products, and the factors, the
  subtraction of the maximum and the exponential on top:
    delta_p = A_p (r_p + D f) + |scale| 2^-25 max|q| sum_d |k_pd| + 2^-20 (1 + max|z|)
* weight in the numerator: fp16, u; own positions of modes 0 and 2, times the scale, bf16, b.
  Below 2^-21 of the largest, fp16 weights are off by 2^-32 of that (2^-31 with the values' power).
* value: prefix rows in modes 0 and 2, 2 u.
* sums over n positions: (n + 64) / 8 f of the sum of sizes (the products add 16 at a time).
So numerator and denominator are off by N = sum_p w_p |V_p| (e^delta_p - 1 + ...) and
E = sum_p w_p (e^delta_p - 1 + ...), the output by (N + |out| E) / (1 - E), and by its rounding, b.
"""
import numpy as np
import torch

import dequant_kvc8_store_gb300 as kv

U16 = 2.0 ** -11
UB = 2.0 ** -8
F32 = 2.0 ** -23
BIAS = 4  # channels that weigh own against prefix positions


class Problem:
    """A pool, a prefix, own pages and queries on `device`."""

    def __init__(self, prefix, lens, H=2, G=4, D=64, bs=16, mode=0, sharp=True, seed=0, spare_prefix=1,
                 spare_own=1, device="cuda"):
        self.prefix, self.lens, self.H, self.G, self.D, self.bs, self.mode = prefix, list(lens), H, G, D, bs, mode
        self.sharp, self.device = sharp, device
        B = len(self.lens)
        gen = torch.Generator()
        gen.manual_seed(seed * 1000003 + prefix * 101 + B * 7 + D + 2 * H + mode + sharp)
        uni = lambda lo, hi, *s: torch.rand(*s, generator=gen).to(device) * (hi - lo) + lo  # noqa: E731
        normal = lambda *s: torch.randn(*s, generator=gen).to(device)  # noqa: E731
        self.PB = max(1, -(-prefix // bs) + spare_prefix)
        self.MB = max(1, -(-max(self.lens, default=0) // bs) + spare_own)
        NB = self.PB + B * self.MB + 2
        ids = torch.randperm(NB, generator=gen).to(device)
        self.ptab = ids[:self.PB].to(torch.int32)
        self.tab = ids[self.PB:self.PB + B * self.MB].view(B, self.MB).to(torch.int32).contiguous()
        owner = torch.full((NB,), B + 1, dtype=torch.long, device=device)
        owner[self.ptab.long()] = 0
        owner[self.tab.long()] = torch.arange(1, B + 1, device=device)[:, None]
        sign = lambda *s: (torch.rand(*s, generator=gen) < 0.5).to(device).float() * 2 - 1  # noqa: E731
        mean = uni(30, 60, B + 2, H, D) * sign(B + 2, H, D)
        self.vc = torch.empty(NB, H, bs, D, dtype=torch.int8, device=device)
        self.kc = torch.empty_like(self.vc)
        for i in range(0, NB, 256):  # (in parts: the fp32 forms are large)
            n = min(256, NB - i)
            page = mean[owner[i:i + n]][:, :, None] + uni(-35, 35, n, H, 1, D) + 12 * normal(n, H, bs, D)
            self.vc[i:i + n] = page.round().clamp(-127, 127).to(torch.int8)
            self.kc[i:i + n] = torch.randint(-127, 128, (n, H, bs, D), generator=gen, dtype=torch.int8).to(device)
        self.kc[:, :, :, :BIAS] = 0
        shape = [(NB, H, bs), (H, D), (NB, H)][mode]
        self.ks, self.vs = (2.0 ** uni(-8, -5, *shape) for _ in range(2))
        q = normal(B, H * G, D)
        q[..., :BIAS] = 8.0 if sharp else 40.0
        self.q = q.to(torch.bfloat16)
        # the standard deviation of <q, k> over all but the four channels
        k2 = (73.3 * float(self.ks.double().pow(2).mean()) ** 0.5) ** 2 * (D - BIAS)
        self.scale = (3.0 if sharp else 0.25) / k2 ** 0.5
        self._weigh(owner)
        self.g = kv.Geom(B, H, D, bs, NB, self.MB, mode)
        self.d = None

    def _weigh(self, owner):
        """Own keys' codes in the four channels, for about equal weights of both sides."""
        P, most = self.prefix, max(self.lens, default=0)
        if P == 0 or most == 0:
            return
        lens = torch.tensor(self.lens, device=self.device)
        live = (torch.arange(most, device=self.device) < lens[:, None])[..., None]
        code = torch.zeros(len(self.lens) + 2, self.H, dtype=torch.int8, device=self.device)
        for h in range(self.H):
            z = self.scores(h)[0]
            gap = (torch.logsumexp(z[..., :P], -1) - torch.logsumexp(z[..., P:], -1)).mean(-1)
            s = self.row_scales(self.ks, self.tab.long(), h)[:, :most]
            s = (s[..., :BIAS] * live).sum((1, 2)) / (live.sum((1, 2)) * min(s.shape[-1], BIAS)).clamp(min=1)
            t = gap / (float(self.q[0, 0, 0]) * BIAS * self.scale * s).clamp(min=1e-30)
            code[1:-1, h] = torch.where(lens > 0, t, torch.zeros_like(t)).round().clamp(-127, 127).to(torch.int8)
        self.kc[:, :, :, :BIAS] = code[owner][:, :, None, None]

    # ---- rows ------------------------------------------------------------------
    def row_scales(self, scale, ids, h):
        """[...][positions][D or 1] of the pages `ids` [...][pages]."""
        s = scale.double()
        n = (*ids.shape[:-1], ids.shape[-1] * self.bs)
        if self.mode == 0:
            return s[ids, h].reshape(*n, 1)
        if self.mode == 1:
            return s[h].expand(*n, self.D)
        return s[ids, h][..., None].expand(*ids.shape, self.bs).reshape(*n, 1)

    def rows(self, cache, scale, ids, h):
        x = cache[ids, h].double()
        return x.reshape(*ids.shape[:-1], ids.shape[-1] * self.bs, self.D) * self.row_scales(scale, ids, h)

    def _sides(self, cache, scale, h):
        most = max(self.lens, default=0)
        pages = lambda t, n: t[..., :-(-n // self.bs)].long()  # noqa: E731
        return (self.rows(cache, scale, pages(self.ptab, self.prefix), h)[:self.prefix],
                self.rows(cache, scale, pages(self.tab, most), h)[:, :most])

    def scores(self, h):
        """(z [B][G][P + most], live [B][1][P + most], |scale| sum |q k|, |scale| max|q| sum |k|)."""
        B, P, most = len(self.lens), self.prefix, max(self.lens, default=0)
        q = self.q.double()[:, h * self.G:(h + 1) * self.G]
        kp, ko = self._sides(self.kc, self.ks, h)
        own = torch.arange(most, device=self.device) < torch.tensor(self.lens, device=self.device)[:, None]
        live = torch.cat([torch.ones(B, P, dtype=torch.bool, device=self.device), own], 1)[:, None]
        dots = lambda q, kp, ko: torch.cat([torch.matmul(q, kp.T), torch.matmul(q, ko.transpose(1, 2))], -1)  # noqa: E731
        z = (dots(q, kp, ko) * self.scale).masked_fill(~live, -np.inf)
        size = dots(q.abs(), kp.abs(), ko.abs()) * abs(self.scale)
        ones = q.abs().amax(-1, keepdim=True).expand_as(q)
        return z, live, size, dots(ones, kp.abs(), ko.abs()) * abs(self.scale)

    def answers(self, least=0.0):
        """want, tol [B][Hq][D], and the wrong answers {name: (out, applies [B][H])}.  least: an
        absolute error of each value."""
        B, H, G, D, P = len(self.lens), self.H, self.G, self.D, self.prefix
        want, tol, pre, own = (torch.zeros(B, H * G, D, dtype=torch.float64, device=self.device) for _ in range(4))
        most = max(self.lens, default=0)
        is_pre = torch.arange(P + most, device=self.device) < P
        scaled = self.mode != 1
        r = torch.where(is_pre, 2 * U16 if scaled else U16, 0.0 if scaled else U16).double()
        wr = torch.where(is_pre, U16, UB if scaled else U16).double() + torch.where(is_pre, 2 * U16 if scaled else 0.0, 0.0)
        n = torch.tensor(self.lens, device=self.device).double()[:, None, None] + P
        for h in range(H):
            j = slice(h * G, (h + 1) * G)
            z, live, size, low = self.scores(h)
            vp, vo = self._sides(self.vc, self.vs, h)
            mix = lambda w, a, b: torch.matmul(w[..., :P], a) + torch.matmul(w[..., P:], b)  # noqa: E731
            top = z.amax(-1, keepdim=True) if z.shape[-1] else z.new_full((B, G, 1), -np.inf)
            top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
            e = torch.exp(z - top)

            def mean(keep):
                w = e * keep
                return mix(w / w.sum(-1, keepdim=True).clamp(min=1e-300), vp, vo)

            want[:, j], pre[:, j], own[:, j] = mean(1.0), mean(is_pre.double()), mean((~is_pre).double())
            w = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
            largest = z.masked_fill(~live, 0.0).abs().amax(-1, keepdim=True) if z.shape[-1] else 0.0
            delta = size * (r + D * F32) + low * 2.0 ** -25 + 2.0 ** -20 * (1 + largest)
            off = torch.expm1(delta)
            sums = (n + 64) / 8 * F32
            N = mix(w * ((1 + off) * (1 + wr) - 1 + sums), vp.abs(), vo.abs())
            N = N + n * 2.0 ** -31 * max([float(v.abs().max()) for v in (vp, vo) if v.numel()], default=0.0) + least
            E = (w * (off + sums)).sum(-1, keepdim=True)
            assert E.numel() == 0 or float(E.max()) < 0.2
            err = (N + want[:, j].abs() * E) / (1 - E)
            tol[:, j] = err + UB * (want[:, j].abs() + err)
        lens = torch.tensor(self.lens, device=self.device)
        some = ((lens + P) > 0)[:, None].expand(B, H)
        both = ((lens > 0) & (P > 0))[:, None].expand(B, H)
        wrong = {"zeros": (torch.zeros_like(want), some), "own positions left out": (pre, both),
                 "prefix left out": (own, both)}
        if H > 1:
            wrong["the next head's"] = (want.roll(-G, 1), some)
        if B > 1:
            owns = ((lens > 0) & (lens.roll(-1) > 0))[:, None].expand(B, H)
            wrong["the next sequence's"] = (want.roll(-1, 0), some if self.sharp and P > 1 else owns)
        if G > 1 and self.sharp:
            turned = want.view(B, H, G, D).roll(-1, 2).reshape(B, H * G, D)
            wrong["the next query's"] = (turned, ((lens + P) > 16)[:, None].expand(B, H))
        return want, tol, wrong

    def check(self, got):
        """`got` is within the bound, and none of the wrong answers would be."""
        want, tol, wrong = self.answers()
        got = got.double().to(want.device)
        bad = ~((got - want).abs() <= tol)
        assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                                     tol[bad][:4].tolist())
        self.tells(want, tol, wrong)

    def tells(self, want, tol, wrong):
        """None of the wrong answers would pass: not for any head of any sequence, but that nine in
        ten are enough where one position may weigh next to nothing (one own key left out of a
        thousand) or nearly all (two queries that meet the same key), and half where, with sharp
        scores, a side is left out."""
        B, H, G, D = len(self.lens), self.H, self.G, self.D
        for name, (out, applies) in wrong.items():
            seen = ((out - want).abs() > 2 * tol).view(B, H, G * D).any(-1)
            part = (0.5 if self.sharp else 0.9) if "left out" in name else 0.9 if "query" in name else 1.0
            enough = int((applies & seen).sum()) >= part * int(applies.sum())
            assert enough, (name, (applies & ~seen).nonzero()[:8].tolist())

    # ---- the call -----------------------------------------------------------------
    def place(self):
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=self.device)  # noqa: E731
        need = kv.kvc8_shared_prefix_workspace_bytes(self.g, self.H * self.G, self.PB)
        self.d = dict(plen=i32([self.prefix]), lens=i32(self.lens), err=i32([0]),
                      ws=torch.full((need,), 0xFF, dtype=torch.uint8, device=self.device))
        self.out = torch.full_like(self.q, float("nan"))

    def run(self):
        if self.d is None:
            self.place()
        d, q, o = self.d, self.q, self.out
        kv.kvc8_shared_prefix_attention(self.g, self.H * self.G, q, q.stride(0), q.stride(1), self.kc, self.vc,
                                        self.ks, self.vs, self.ptab, self.PB, d["plen"], self.tab, d["lens"],
                                        self.scale, o, o.stride(0), o.stride(1), d["ws"], d["ws"].numel(), d["err"])
        return o

    def error(self):
        return kv.kvc8_get_error(self.d["err"], reset=True)
