"""The rotating append where a warp works through several tokens, some of them skipped, and through
more than the 32 whose slots it looks up at once.  A launch has at most 20 warps per SM (five
blocks of four), so that many tokens are one each.  Bounds as in test_gpu_rope.py."""
import numpy as np
import pytest
import torch

import oracle
import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import workloads as W
from dequant_kvc8_store_gb300.device import Bf16Batch, DeviceBatch, bf16_bits
from _rope_ref import BF16, U, bf16_f64, bf16_tensor, norm_rotate, to_bf16_bits
from test_gpu_rope import Turn, _append, _check_rows, _rows, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


def _warps():
    return 20 * torch.cuda.get_device_properties(0).multi_processor_count


def _spoil(d, w, rng, share):
    """Bad pages, and sequences of negative length, in the device's copies: which tokens stay, and
    the codes that may be reported."""
    table, ctx = w.block_table.copy(), w.context_kv_lens.copy()
    hit = rng.random(table.shape) < share
    table[hit] = rng.choice([-1, w.num_blocks, 2 ** 31 - 1, -2 ** 31], hit.sum())
    ctx[rng.random(len(ctx)) < share / 4] = -1
    d.block_table.copy_(torch.from_numpy(table))
    d.context_kv_lens.copy_(torch.from_numpy(ctx))
    seq, pos = _tokens(w)
    return ~hit[seq, pos // w.block_size] & (ctx[seq] >= 0)


def _int8_pool(w, d, turn, keep):
    """Values and every slot that is not a kept token's bit for bit, rotated keys within the bound."""
    seq, pos = _tokens(w)
    ids, at = w.block_table[seq, pos // w.block_size], pos % w.block_size
    was = (w.k_cache, w.v_cache, w.k_scale, w.v_scale)
    want = [x.copy() for x in was]
    oracle.store(w.quant_mode, w.k_states, w.v_states, *want, w.block_table, w.cu_q_lens, w.context_kv_lens)
    off = ids[~keep], slice(None), at[~keep]
    for x, y in zip(want[:2] + (want[2:] if w.quant_mode == 0 else []), was):
        x[off] = y[off]
    kc, vc, ks, vs = d.host_caches()
    np.testing.assert_array_equal(vc, want[1])
    np.testing.assert_array_equal(vs, want[3])
    same = np.ones((w.num_blocks, w.block_size), bool)
    same[ids[keep], at[keep]] = False
    np.testing.assert_array_equal(kc.transpose(0, 2, 1, 3)[same], w.k_cache.transpose(0, 2, 1, 3)[same])
    if w.quant_mode == 0:
        np.testing.assert_array_equal(ks.transpose(0, 2, 1)[same], w.k_scale.transpose(0, 2, 1)[same])
    else:
        np.testing.assert_array_equal(ks, w.k_scale)
    ids, at = ids[keep], at[keep]
    y, e = turn.exact(w.k_states[keep], "k", pos[keep])
    code = kc[ids, :, at].astype(np.float64)
    if w.quant_mode == 0:
        s = ks[ids, :, at].astype(np.float64)[..., None]
        top = np.abs(y).max(-1, keepdims=True)
        assert (np.abs(s - top / 127) <= e.max(-1, keepdims=True) / 127 + U * top / 127 + 2.0 ** -149).all()
    elif w.quant_mode == 1:
        s = np.broadcast_to(ks.astype(np.float64)[None], y.shape)
    else:
        s = ks[ids].astype(np.float64)[..., None]
    assert np.abs(code).max(initial=0) <= 127
    bad = np.abs(code * s - np.clip(y, -127 * s, 127 * s)) > s * (0.5 + 127 * U) + e
    assert not bad.any(), np.argwhere(bad)[:5]


def _bf16_pool(w, d, before, turn, keep):
    seq, pos = _tokens(w)
    ids, at = w.block_table[seq, pos // w.block_size][keep], (pos % w.block_size)[keep]
    vw = before[1].copy()
    vw[ids, :, at] = w.v_states[keep]
    np.testing.assert_array_equal(bf16_bits(d.v_cache), vw)
    got = bf16_bits(d.k_cache)
    _check_rows(got[ids, :, at], turn, "k", w.k_states[keep], pos[keep])
    same = np.ones((w.num_blocks, w.block_size), bool)
    same[ids, at] = False
    np.testing.assert_array_equal(got.transpose(0, 2, 1, 3)[same], before[0].transpose(0, 2, 1, 3)[same])


def _append_and_check(w, turn, rng, heads, bf16, share):
    d = Bf16Batch(w, seed=3) if bf16 else DeviceBatch(w)
    before = (bf16_bits(d.k_cache), bf16_bits(d.v_cache)) if bf16 else None
    keep = _spoil(d, w, rng, share)
    qb = _rows(rng, w.num_tokens, heads, w.head_dim)
    q = bf16_tensor(qb).cuda()
    out = torch.full_like(q, 7.0)
    _append(d, w, turn, q, out, bf16=bf16)
    assert d.error_code(reset=True) in ((kv.DEV_BAD_BLOCK_ID, kv.DEV_BAD_LENGTH) if share else (0,))
    pos = _tokens(w)[1]
    _check_rows(bf16_bits(out), turn, "q", qb, pos, keep)
    assert (out[torch.from_numpy(~keep).cuda()] == 7).all()
    if bf16:
        _bf16_pool(w, d, before, turn, keep)
    else:
        _int8_pool(w, d, turn, keep)
    return keep


@pytest.mark.parametrize("share", [0.0, 0.3])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sink", [0, 1, 2, "bf16"])
def test_several_tokens_to_a_warp(sink, inter, share):
    """About four tokens to a warp, kept and skipped ones in turn."""
    rng = np.random.default_rng([100, inter, int(10 * share)])
    q_lens = rng.integers(0, 60, 4 * _warps() // 30)
    H, D, bs = (2, 128, 16) if inter else (3, 80, 24)
    ctx = rng.integers(0, 70, len(q_lens))
    mb = int((-(-(ctx + q_lens) // bs)).max())
    w = W.make_workload("ropeunits", q_lens=q_lens, ctx_before=ctx, kv_heads=H, head_dim=D, block_size=bs,
                        num_blocks=len(ctx) * mb + 5, quant_mode=0 if sink == "bf16" else sink, seed=101,
                        outlier_channels=2)
    keep = _append_and_check(w, Turn(rng, D, 64, inter, positions=None), rng, 8, sink == "bf16", share)
    n, step = len(keep), _warps()
    assert n > 3 * step
    if share:  # skipped then kept, kept then skipped, both twice over, in many warps
        a, b, c = keep[:n - 2 * step], keep[step:n - step], keep[2 * step:]
        assert (a & ~b & c).sum() > 50 and (~a & b & ~c).sum() > 50


@pytest.mark.parametrize("sink", [0, 2, "bf16"])
@pytest.mark.parametrize("share", [0.0, 0.3])
def test_more_tokens_to_a_warp_than_it_looks_up_at_once(sink, share):
    rng = np.random.default_rng([110, int(10 * share)])
    n = -(-35 * _warps() // 400)
    q_lens, ctx = rng.integers(300, 560, n), rng.integers(0, 30, n)
    w = W.make_workload("ropelookups", q_lens=q_lens, ctx_before=ctx, kv_heads=1, head_dim=16, block_size=37,
                        num_blocks=n * 16 + 3, quant_mode=0 if sink == "bf16" else sink, seed=111)
    keep = _append_and_check(w, Turn(rng, 16, 16, positions=None), rng, 1, sink == "bf16", share)
    assert len(keep) > 33 * _warps()


def test_rows_of_more_tokens_than_a_warp_looks_up_at_once():
    """The same without pages: positions of a lane above 0, and of later looks."""
    rng = np.random.default_rng(120)
    n = 35 * _warps() + 11
    pos = rng.integers(-2 ** 31, 2 ** 31, n)
    turn = Turn(rng, 32, 32, positions=pos)
    qb, kb = _rows(rng, n, 1, 32), _rows(rng, n, 1, 32)
    q, k = bf16_tensor(qb).cuda(), bf16_tensor(kb).cuda()
    kv.kvc8_qk_norm_rope(turn.rope, n, 32, 1, q, 32, 32, q, 32, 32, 1, k, 32, 32, k, 32, 32)
    _check_rows(bf16_bits(q), turn, "q", qb, pos)
    _check_rows(bf16_bits(k), turn, "k", kb, pos)


@pytest.mark.parametrize("power,eps", [(56, 1e-6), (56, 0.0), (-51, 0.0), (-20, 1e-6), (-100, 2.0 ** -110)])
@pytest.mark.parametrize("D", [16, 128, 256])
def test_norm_at_the_ends_of_its_range(D, power, eps):
    """Rows of values up to 2^58, and down to a mean of squares plus eps of 2^-110."""
    rng = np.random.default_rng([130, D])
    x = np.clip(rng.standard_normal((40, 3, D)), -4.0, 4.0)
    x[:, :, 0] = 1.5  # a mean of squares of no less than 2.25 / D
    bits = to_bf16_bits(x * 2.0 ** power)
    turn = Turn(rng, D, 16, positions=np.arange(40))
    turn.rope.struct.norm_eps = eps
    q = bf16_tensor(bits).cuda()
    out = torch.full_like(q, float("nan"))
    kv.kvc8_qk_norm_rope(turn.rope, 40, D, 3, q, 3 * D, D, out, 3 * D, D, 0, None, 0, 0, None, 0, 0)
    y, e = norm_rotate(bits, turn.wq, float(np.float32(eps)), np.arange(40), turn.freqs, 16, False, 1.0)
    got = bf16_f64(bf16_bits(out))
    # (squares below fp32's normal numbers: 2^-149 each of a mean of 2^-110, far below U)
    bad = ~(np.abs(got - y) <= e + BF16 * (np.abs(y) + e) + 2.0 ** -133)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], y[bad][:4])
