"""The inputs and the bound of the shared-prefix attention's GPU tests, on the CPU: the bound holds
for a restatement of the kernels' roundings, and lets none of the wrong answers pass."""
import numpy as np
import pytest
import torch

from _prefix_ref import Problem
from test_gpu_prefix_values import HEADS, LENGTHS, ROWS, row_lens


def _half(x, power=0):
    """fp16 after a power of two."""
    return (x * 2.0 ** power).to(torch.float16).double() * 2.0 ** -power


def _normal(x):
    """fp16 after the power of two that brings a row's largest to [1, 2)."""
    top = 2.0 ** torch.floor(torch.log2(x.abs().amax(-1, keepdim=True)))
    return (x / top).to(torch.float16).double() * top


def _rounded(x):
    """The attention with each operand rounded as the kernels round it."""
    B, G, P, most, mode = len(x.lens), x.G, x.prefix, max(x.lens, default=0), x.mode
    out = torch.zeros(x.q.shape, dtype=torch.float64)
    pages = [t[..., :-(-n // x.bs)].long() for t, n in ((x.ptab, P), (x.tab, most))]
    live = torch.arange(most) < torch.tensor(x.lens)[:, None]
    if P + most == 0:
        return out
    for h in range(x.H):
        j = slice(h * G, (h + 1) * G)
        code = lambda c, i, n: c[pages[i], h].double().reshape(*pages[i].shape[:-1], -1, x.D)[..., :n, :]  # noqa: E731
        by = lambda s, i, n: x.row_scales(s, pages[i], h)[..., :n, :]  # noqa: E731
        kp, vp, ko, vo = code(x.kc, 0, P), code(x.vc, 0, P), code(x.kc, 1, most), code(x.vc, 1, most)
        q, so = x.q.double()[:, j], torch.ones(B, 1, most, dtype=torch.float64)
        if mode == 1:
            q = _normal(q * x.ks[h].double())
            zo = torch.matmul(q, ko.transpose(1, 2))
        else:
            q = _normal(q)
            kp, vp = (_half(c * _half(by(s, 0, P), 6), 6) for c, s in ((kp, x.ks), (vp, x.vs)))
            zo = torch.matmul(q, ko.transpose(1, 2)) * by(x.ks, 1, most)[..., 0][:, None]
            so = by(x.vs, 1, most)[..., 0][:, None]
        z = torch.cat([torch.matmul(q, kp.T), zo.masked_fill(~live[:, None], -np.inf)], -1)
        z = (z * x.scale).float()
        top = z.amax(-1, keepdim=True)
        w = torch.exp(z - torch.where(torch.isfinite(top), top, torch.zeros_like(top))).double()
        own = _half(w[..., P:], 7) if mode == 1 else (w[..., P:] * so).to(torch.bfloat16).double()
        o = torch.matmul(_half(w[..., :P], 7), vp) + torch.matmul(own.masked_fill(~live[:, None], 0.0), vo)
        if mode == 1:
            o = o * x.vs[h].double()
        out[:, j] = o / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return out.to(torch.bfloat16)


@pytest.mark.parametrize("sharp", [False, True])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_bound_holds_and_tells_mistakes_apart(mode, sharp):
    for x in [Problem(p, lens, D=D, mode=mode, sharp=sharp, seed=1, device="cpu") for p, lens, D in LENGTHS] + \
             [Problem(777, [40, 0, 130, 1, 64, 99, 3], H=H, G=G, D=D, bs=bs, mode=mode, sharp=sharp, seed=2,
                      device="cpu") for H, G, D, bs in HEADS] + \
             [Problem(400, row_lens(B), H=2, G=G, D=D, mode=mode, sharp=sharp, seed=3, device="cpu")
              for B, G, D in ROWS]:
        x.check(_rounded(x))


def test_a_wrong_answer_does_not_pass():
    x = Problem(777, [40, 0, 130], D=128, bs=32, sharp=False, device="cpu")
    good = _rounded(x)
    x.check(good)
    for name, (out, _) in x.answers()[2].items():
        with pytest.raises(AssertionError):
            x.check(out.to(torch.bfloat16))
    one = good.clone()
    one[1, 3, 77] += 0.05 * one.abs().max()
    with pytest.raises(AssertionError):
        x.check(one)
    one[1, 3, 77] = float("nan")
    with pytest.raises(AssertionError):
        x.check(one)
