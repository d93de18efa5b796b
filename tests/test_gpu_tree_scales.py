"""Tree attention where a scale is no number: rows that do not see its position keep their values."""
import numpy as np
import pytest
import torch

import dequant_kvc8_store_gb300 as kv
from _drafts_ref import TreeProblem

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


def at(x, b, p):
    """Places of position p of sequence b in the caches' scales of mode 0."""
    return int(x.tab[b, p // x.bs]), slice(None), p % x.bs


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,draft", [([40, 9], [6, 3], 3), ([130, 0], [64, 40], 33), ([0, 300], [17, 9], 0)])
def test_one_bad_scale_beside_a_large_one(ctx, new, draft, D, which, bad):
    """The key's scale alone, and the value's alone, of a draft whose other scale is 16 times the others': a chain, of
    which the earlier drafts do not see it."""
    make = lambda: TreeProblem(ctx, new, H=2, G=4, D=D, mode=0, kind="chain", sharp=False, seed=21)  # noqa: E731
    x, clean = make(), make()
    place, other = at(x, 0, ctx[0] + draft), {"ks": "vs", "vs": "ks"}[which]
    for y in (x, clean):
        getattr(y, other)[place] *= 16.0
    getattr(x, which)[place] = bad
    x.run()
    assert x.error() == 0
    want, tol, _ = clean.answers()
    sees = torch.zeros(x.N, dtype=torch.bool, device="cuda")
    sees[draft:new[0]] = True
    good = ((x.out.double() - want).abs() <= tol).flatten(1).all(1)
    assert bool((good | sees).all()), (~good & ~sees).nonzero().flatten().tolist()
    assert bool(torch.isnan(x.out[sees]).all())


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_one_bad_scale_of_a_draft_that_nobody_sees(which, bad):
    make = lambda: TreeProblem([40, 0, 250], [5, 17, 70], H=2, G=4, D=64, mode=0, kind="any", sharp=False, seed=22)  # noqa: E731
    x, clean = make(), make()
    clean.mask[:, 0] &= ~np.uint64(1 << 2)
    x.mask = clean.mask
    for b in range(3):
        place = at(x, b, x.ctx[b] + 2)
        for y in (x, clean):
            y.ks[place] *= 16.0
            y.vs[place] *= 16.0
        getattr(x, which)[place] = bad
    x.run()
    assert x.error() == 0
    want, tol, _ = clean.answers()
    assert bool(((x.out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ctx,new,H", [([0], [5], 2), ([0], [256], 1), ([40, 0, 0], [3, 30, 200], 2)])
def test_rows_without_a_position_are_zero_whatever_the_channels_scales(ctx, new, H, D, bad, which):
    """Tiles that one CTA has whole, and tiles that are joined from several."""
    x = TreeProblem(ctx, new, H=H, G=4, D=D, mode=1, kind="none", sharp=False, seed=23)
    getattr(x, which)[:, 7] = bad
    x.run()
    n = new[0] if ctx[0] else 0
    assert x.error() == 0 and bool((x.out[n:] == 0).all())
    if n and np.isnan(bad):  # the others are what such scales make of them
        assert bool(torch.isnan(x.out[:n, :, 7]).all())


@pytest.mark.parametrize("size", [2.0 ** 16, 2.0 ** 40, 1e38])
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("ctx,new,G,D", [([40, 0, 250], [5, 17, 70], 4, 64), ([40, 0, 250], [5, 17, 70], 4, 128),
                                         ([1000, 3], [256, 130], 8, 64), ([77, 128], [200, 4], 1, 128)])
def test_large_scales_of_drafts_that_nobody_sees(ctx, new, G, D, which, size):
    """Padding that was never stored: its scales are whatever the page held."""
    make = lambda: TreeProblem(ctx, new, H=2, G=G, D=D, mode=0, kind="any", sharp=False, seed=24)  # noqa: E731
    x, clean = make(), make()
    hidden = [2, 3, 64, 66, 127, 128, 199]
    for i in hidden:
        if i < 64 * clean.words:
            clean.mask[:, i // 64] &= ~np.uint64(1 << (i % 64))
    x.mask = clean.mask
    for b in range(len(ctx)):
        for i in hidden:
            if i < new[b]:
                getattr(x, which)[at(x, b, ctx[b] + i)] = size
    x.run()
    assert x.error() == 0
    want, tol, _ = clean.answers()
    assert bool(((x.out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("D", [64, 128])
def test_a_bad_scale_of_a_block_that_the_earlier_drafts_do_not_see(D, bad, which):
    make = lambda: TreeProblem([32, 5], [40, 3], H=2, G=4, D=D, bs=16, mode=2, kind="chain", sharp=False, seed=25)  # noqa: E731
    x, clean = make(), make()
    getattr(x, which)[int(x.tab[0, 3])] = bad  # positions 48 to 63: drafts 16 to 31
    x.run()
    assert x.error() == 0
    want, tol, _ = clean.answers()
    sees = torch.zeros(x.N, dtype=torch.bool, device="cuda")
    sees[16:40] = True
    good = ((x.out.double() - want).abs() <= tol).flatten(1).all(1)
    assert bool((good | sees).all()), (~good & ~sees).nonzero().flatten().tolist()
    assert bool(torch.isnan(x.out[sees]).all())
