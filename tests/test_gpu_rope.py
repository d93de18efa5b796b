"""The rotating append (kvc8_rope_store, kvc8_rope_store_bf16) and the
norm-and-rotate pass (kvc8_qk_norm_rope) against an fp64 evaluation.

A rotated value is off by the bound that tests/_rope_ref.py derives for fp32,
e.  Then
* a bf16 output is off by e plus half a step of what is rounded:
  e + 2^-8 (|y| + e);
* a dynamic scale max|y| / 127 is off by e / 127 (the largest e of the row) and one
  rounding of 2^-24;
* the value that a code stands for, code * s with the stored scale s, is off by
  half a step s / 2, by e, and by the quotient's rounding, which moves the
  border between two codes by 127 * 2^-24 s at most.
Values take kvc8_store's arithmetic: their codes and scales are equal to the
oracle's bit for bit, and so is every slot that the call does not write.
"""
import numpy as np
import pytest
import torch

import oracle
import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import workloads as W
from dequant_kvc8_store_gb300.device import Bf16Batch, DeviceBatch, bf16_bits
from _rope_ref import BF16, U, bf16_f64, bf16_tensor, fixed_point, inv_freq, norm_rotate, to_bf16_bits

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    kv.load()
    yield
    torch.cuda.synchronize()


def _rows(rng, n, h, d):
    x = rng.standard_normal((n, h, d)).astype(np.float32)
    x[:, :, rng.integers(0, d, 2)] *= 20.0
    return to_bf16_bits(x)


class Turn:
    """A rotation on the device and its host form."""

    def __init__(self, rng, dim, rot, interleaved=False, norm=True, factor=1.0, positions=None,
                 base=1e4):
        self.rot, self.interleaved, self.factor = rot, interleaved, factor
        self.freqs = fixed_point(inv_freq(rot, base))
        self.wq = self.wk = None
        if norm:
            self.wq, self.wk = (to_bf16_bits(1 + 0.3 * rng.standard_normal(dim)) for _ in range(2))
        self.positions = positions
        dev = lambda b: None if b is None else bf16_tensor(b).cuda()  # noqa: E731
        self.rope = kv.Rope(rotary_dim=rot, interleaved=int(interleaved), attention_factor=factor,
                            norm_eps=EPS, freqs=torch.from_numpy(self.freqs.view(np.int64)).cuda(),
                            q_norm_weight=dev(self.wq), k_norm_weight=dev(self.wk),
                            positions=None if positions is None else
                            torch.from_numpy(np.asarray(positions, np.int32)).cuda())

    def exact(self, bits, side, pos):
        return norm_rotate(bits, self.wq if side == "q" else self.wk, EPS, pos, self.freqs,
                           self.rot, self.interleaved, np.float64(np.float32(self.factor)))


def _check_rows(bits, turn, side, src, pos, keep=None):
    y, e = turn.exact(src, side, pos)
    got = bf16_f64(bits)
    if keep is not None:
        y, e, got = y[keep], e[keep], got[keep]
    tol = e + BF16 * (np.abs(y) + e) + 2.0 ** -133
    bad = np.abs(got - y) > tol
    fine = not bad.any()
    assert fine, (side, np.argwhere(bad)[:5], np.abs(got - y)[bad][:5], tol[bad][:5])


def _tokens(w):
    """(sequence, slot position) of each new token."""
    q = w.q_lens()
    seq = np.repeat(np.arange(w.num_seqs), q)
    first = np.concatenate([[0], np.cumsum(q)])[:-1]
    return seq, w.context_kv_lens[seq].astype(np.int64) + np.arange(len(seq)) - first[seq]


def _slots(w):
    seq, pos = _tokens(w)
    return w.block_table[seq, pos // w.block_size], pos % w.block_size, pos


def _append(d, w, turn, q, q_out, bf16=False, k=None, v=None, stream=None):
    ks, vs = (d.k_states, d.v_states) if k is None else (k, v)
    n = w.num_tokens
    hq = 0 if q is None else q.shape[1]
    st = lambda t, i: 0 if t is None else t.stride(i)  # noqa: E731
    head = (d.g, turn.rope, n, hq, q, st(q, 0), st(q, 1), q_out, st(q_out, 0), st(q_out, 1), ks, vs,
            ks.stride(0), ks.stride(1), d.k_cache, d.v_cache)
    tail = (d.block_table, d.cu_q_lens, d.context_kv_lens, d.dev_error, stream)
    if bf16:
        kv.kvc8_rope_store_bf16(*head, *tail)
    else:
        kv.kvc8_rope_store(*head, d.k_scale, d.v_scale, *tail)


def _check_pool(w, d, turn, rot_pos):
    """The int8 pages after an append: values and untouched slots bit for bit,
    rotated keys within the bound."""
    ids, at, pos = _slots(w)
    kc, vc, ks, vs = d.host_caches()
    want = [x.copy() for x in (w.k_cache, w.v_cache, w.k_scale, w.v_scale)]
    # values: the oracle's store; keys: what was there, but for the slots written
    oracle.store(w.quant_mode, w.k_states, w.v_states, *want, w.block_table, w.cu_q_lens,
                 w.context_kv_lens)
    np.testing.assert_array_equal(vc, want[1])
    np.testing.assert_array_equal(vs, want[3])
    same = np.ones((w.num_blocks, w.block_size), bool)
    same[ids, at] = False
    np.testing.assert_array_equal(kc.transpose(0, 2, 1, 3)[same], w.k_cache.transpose(0, 2, 1, 3)[same])
    if w.quant_mode == 0:
        np.testing.assert_array_equal(ks.transpose(0, 2, 1)[same], w.k_scale.transpose(0, 2, 1)[same])
    else:
        np.testing.assert_array_equal(ks, w.k_scale)
    y, e = turn.exact(w.k_states, "k", rot_pos)
    code = kc[ids, :, at].astype(np.float64)
    if w.quant_mode == 0:
        s = ks[ids, :, at].astype(np.float64)[..., None]
        top = np.abs(y).max(-1, keepdims=True)
        fine = bool((np.abs(s - top / 127) <= e.max(-1, keepdims=True) / 127 + U * top / 127 + 2.0 ** -149).all())
        assert fine
    elif w.quant_mode == 1:
        s = np.broadcast_to(ks.astype(np.float64)[None], y.shape)
    else:
        s = ks[ids].astype(np.float64)[..., None]
    assert np.abs(code).max(initial=0) <= 127
    clamped = np.clip(y, -127 * s, 127 * s)
    tol = s * (0.5 + 127 * U) + e
    bad = np.abs(code * s - clamped) > tol
    fine = not bad.any()
    assert fine, (np.argwhere(bad)[:5], (np.abs(code * s - clamped) / s)[bad][:5])


GRID = [
    # heads, dim, block, rot, interleaved, norm, group, mode
    (2, 64, 16, 64, False, True, 4, 0),
    (8, 128, 128, 128, False, True, 4, 0),
    (1, 128, 64, 64, True, False, 7, 0),
    (8, 128, 64, 128, True, True, 1, 1),
    (3, 80, 24, 32, False, True, 5, 1),
    (4, 96, 7, 96, True, True, 2, 2),
    (5, 256, 32, 192, False, False, 3, 2),
    (2, 16, 1, 16, False, True, 8, 0),
    (6, 48, 33, 0, False, True, 1, 0),
    (16, 240, 20, 240, True, True, 1, 1),
    (1, 32, 16, 16, False, False, 33, 2),
    (4, 192, 128, 64, False, True, 2, 0),
]


@pytest.mark.parametrize("H,D,bs,rot,inter,norm,group,mode", GRID)
def test_append_int8(H, D, bs, rot, inter, norm, group, mode):
    rng = np.random.default_rng([H, D, bs, rot])
    w = W.make_workload("rope", q_lens=[5, 0, 41, 1, 64], ctx_before=[0, 9, 30, 63, 1], kv_heads=H,
                        head_dim=D, block_size=bs, num_blocks=5 * (-(-71 // bs)) + 3, quant_mode=mode,
                        seed=40 + H, outlier_channels=2)
    d = DeviceBatch(w)
    turn = Turn(rng, D, rot, inter, norm, factor=1.25 if rot == D else 1.0)
    qb = _rows(rng, w.num_tokens, H * group, D)
    q = bf16_tensor(qb).cuda()
    out = torch.full_like(q, float("nan"))
    _append(d, w, turn, q, out)
    assert d.error_code() == 0
    pos = _slots(w)[2]
    _check_rows(bf16_bits(out), turn, "q", qb, pos)
    _check_pool(w, d, turn, pos)


@pytest.mark.parametrize("H,D,bs,rot,inter,norm,group,mode", GRID)
def test_append_bf16_pages_and_rows_agree(H, D, bs, rot, inter, norm, group, mode):
    """The bf16 pages hold kvc8_qk_norm_rope's key rows and the values, bit for bit."""
    rng = np.random.default_rng([H, D, bs, rot, 1])
    w = W.make_workload("rope16", q_lens=[5, 0, 41, 1, 64], ctx_before=[0, 9, 30, 63, 1], kv_heads=H,
                        head_dim=D, block_size=bs, num_blocks=5 * (-(-71 // bs)) + 3, quant_mode=0,
                        seed=50 + H)
    d = Bf16Batch(w, seed=3)
    before = bf16_bits(d.k_cache), bf16_bits(d.v_cache)
    ids, at, pos = _slots(w)
    turn = Turn(rng, D, rot, inter, norm, positions=pos + 777)
    qb = _rows(rng, w.num_tokens, H * group, D)
    q = bf16_tensor(qb).cuda()
    out, rows_q, rows_k = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(d.k_states)
    _append(d, w, turn, q, out, bf16=True)
    assert d.error_code() == 0
    k = d.k_states
    kv.kvc8_qk_norm_rope(turn.rope, w.num_tokens, D, H * group, q, q.stride(0), q.stride(1), rows_q,
                         q.stride(0), q.stride(1), H, k, k.stride(0), k.stride(1), rows_k,
                         k.stride(0), k.stride(1))
    _check_rows(bf16_bits(rows_q), turn, "q", qb, pos + 777)
    _check_rows(bf16_bits(rows_k), turn, "k", w.k_states, pos + 777)
    np.testing.assert_array_equal(bf16_bits(out), bf16_bits(rows_q))
    kw, vw = before[0].copy(), before[1].copy()
    kw[ids, :, at] = bf16_bits(rows_k)
    vw[ids, :, at] = w.v_states
    np.testing.assert_array_equal(bf16_bits(d.k_cache), kw)
    np.testing.assert_array_equal(bf16_bits(d.v_cache), vw)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_no_rotation_and_no_norm_is_the_store(mode):
    """rotary_dim 0 and no weights: the same pages as kvc8_store, bit for bit, and the queries
    unchanged."""
    rng = np.random.default_rng(90 + mode)
    w = W.make_workload("rope0", q_lens=[130, 0, 7], ctx_before=[5, 3, 60], kv_heads=3, head_dim=96,
                        block_size=24, num_blocks=30, quant_mode=mode, seed=91, outlier_channels=3)
    d = DeviceBatch(w)
    turn = Turn(rng, 96, 0, norm=False)
    q = bf16_tensor(_rows(rng, w.num_tokens, 5, 96)).cuda()
    out = torch.zeros_like(q)
    _append(d, w, turn, q, out)
    assert d.error_code() == 0
    want = [x.copy() for x in (w.k_cache, w.v_cache, w.k_scale, w.v_scale)]
    oracle.store(mode, w.k_states, w.v_states, *want, w.block_table, w.cu_q_lens, w.context_kv_lens)
    for got, x in zip(d.host_caches(), want):
        np.testing.assert_array_equal(got, x)
    assert torch.equal(out, q)


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_decode_form_in_place_and_strided(mode):
    """cu_q_lens NULL, query rotated in place in a wider tensor, keys and values
    views of one packed projection."""
    rng = np.random.default_rng(60 + mode)
    B, H, D, HQ = 37, 4, 128, 12
    w = W.make_workload("ropedec", q_lens=np.ones(B, int), ctx_before=rng.integers(0, 90, B),
                        kv_heads=H, head_dim=D, block_size=32, num_blocks=3 * B + 5, quant_mode=mode,
                        seed=61, decode_null_cu=True)
    d = DeviceBatch(w)
    turn = Turn(rng, D, 64, norm=True)
    qb = _rows(rng, B, HQ, D)
    packed = torch.zeros(B, HQ + 2 * H + 1, D, dtype=torch.bfloat16, device="cuda")
    packed[:, :HQ] = bf16_tensor(qb).cuda()
    packed[:, HQ:HQ + H], packed[:, HQ + H:HQ + 2 * H] = d.k_states, d.v_states
    q, k, v = packed[:, :HQ], packed[:, HQ:HQ + H], packed[:, HQ + H:HQ + 2 * H]
    _append(d, w, turn, q, q, k=k, v=v)
    assert d.error_code() == 0
    pos = _slots(w)[2]
    _check_rows(bf16_bits(q), turn, "q", qb, pos)
    _check_pool(w, d, turn, pos)
    assert torch.equal(packed[:, HQ:HQ + H], d.k_states) and not packed[:, -1].any()


def test_head_major_rows_and_no_queries():
    rng = np.random.default_rng(70)
    H, D = 3, 64
    w = W.make_workload("ropehm", q_lens=[33, 2], ctx_before=[4, 0], kv_heads=H, head_dim=D,
                        block_size=16, num_blocks=9, quant_mode=0, seed=71)
    d = DeviceBatch(w)
    turn = Turn(rng, D, 64, True, norm=False)
    hm = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    _append(d, w, turn, None, None, k=hm(d.k_states), v=hm(d.v_states))
    assert d.error_code() == 0
    _check_pool(w, d, turn, _slots(w)[2])


@pytest.mark.parametrize("inter", [False, True])
def test_far_and_negative_positions(inter):
    rng = np.random.default_rng(72)
    pos = np.array([0, 1, -1, 131071, 131072, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], np.int64)
    turn = Turn(rng, 128, 128, inter, positions=pos, base=1e6)
    n = len(pos)
    qb, kb = _rows(rng, n, 5, 128), _rows(rng, n, 2, 128)
    q, k = bf16_tensor(qb).cuda(), bf16_tensor(kb).cuda()
    kv.kvc8_qk_norm_rope(turn.rope, n, 128, 5, q, 640, 128, q, 640, 128, 2, k, 256, 128, k, 256, 128)
    _check_rows(bf16_bits(q), turn, "q", qb, pos)
    _check_rows(bf16_bits(k), turn, "k", kb, pos)


@pytest.mark.parametrize("n", [1, 2, 31, 1000, 5003])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (256, 256)])
def test_rows_of_every_count(n, D, rot):
    rng = np.random.default_rng(n + D)
    pos = rng.integers(0, 1 << 17, n)
    turn = Turn(rng, D, rot, positions=pos)
    hq, hk = (3, 1) if n > 1000 else (9, 4)
    qb, kb = _rows(rng, n, hq, D), _rows(rng, n, hk, D)
    q, k = bf16_tensor(qb).cuda(), bf16_tensor(kb).cuda()
    qo = torch.full((n + 2, hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko = torch.full((n + 2, hk, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kv.kvc8_qk_norm_rope(turn.rope, n, D, hq, q, hq * D, D, qo, hq * D, D, hk, k, hk * D, D, ko,
                         hk * D, D)
    _check_rows(bf16_bits(qo[:n]), turn, "q", qb, pos)
    _check_rows(bf16_bits(ko[:n]), turn, "k", kb, pos)
    assert (qo[n:] == 7).all() and (ko[n:] == 7).all()


def test_one_side_only():
    rng = np.random.default_rng(73)
    turn = Turn(rng, 64, 64, positions=np.arange(9))
    kb = _rows(rng, 9, 2, 64)
    k = bf16_tensor(kb).cuda()
    out = torch.zeros_like(k)
    kv.kvc8_qk_norm_rope(turn.rope, 9, 64, 0, None, 0, 0, None, 0, 0, 2, k, 128, 64, out, 128, 64)
    _check_rows(bf16_bits(out), turn, "k", kb, np.arange(9))
    kv.kvc8_qk_norm_rope(turn.rope, 9, 64, 2, k, 128, 64, out, 128, 64, 0, None, 0, 0, None, 0, 0)
    _check_rows(bf16_bits(out), turn, "q", kb, np.arange(9))


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_zero_rows_tiny_rows_and_zero_scales(mode):
    """Rows of zeros get scale 0 and code 0; rows near the bottom of bf16 and
    scales of 0 are handled."""
    rng = np.random.default_rng(74)
    w = W.make_workload("ropezero", q_lens=[6], ctx_before=[0], kv_heads=2, head_dim=64,
                        block_size=16, num_blocks=3, quant_mode=mode, seed=75)
    w.k_states[1] = 0
    w.v_states[2] = 0
    w.k_states[3] = to_bf16_bits(rng.standard_normal((2, 64)) * 2.0 ** -125)
    w.k_states[4] = to_bf16_bits(rng.standard_normal((2, 64)) * 2.0 ** 100)
    if mode == 1:
        w.k_scale[:, 5] = 0.0
    if mode == 2:
        w.k_scale[:, 1] = 0.0
    d = DeviceBatch(w)
    turn = Turn(rng, 64, 64, norm=False)
    _append(d, w, turn, None, None)
    assert d.error_code() == 0
    kc, _, ks, _ = d.host_caches()
    ids, at, pos = _slots(w)
    assert not kc[ids[1], :, at[1]].any()
    if mode == 1:
        assert not kc[ids[0], :, at[0]][:, 5].any()
    elif mode == 2:
        assert not kc[ids[0], 1, at[0]].any()
    else:
        assert not ks[ids[1], :, at[1]].any()
        _check_pool(w, d, turn, pos)


def test_a_rotation_past_the_fp32_range():
    """Finite rows whose rotated values pass the fp32 range: scale infinity and codes 0 by the
    definition (finite / inf = 0, inf / inf is no number: 0)."""
    rng = np.random.default_rng(92)
    w = W.make_workload("ropebig", q_lens=[3], ctx_before=[0], kv_heads=2, head_dim=64,
                        block_size=16, num_blocks=2, quant_mode=0, seed=93)
    w.k_states[1] = to_bf16_bits(np.full((2, 64), 2.0 ** 127))
    d = DeviceBatch(w)
    _append(d, w, Turn(rng, 64, 64, norm=False, factor=4.0), None, None)
    assert d.error_code() == 0
    kc, _, ks, _ = d.host_caches()
    ids, at, _ = _slots(w)
    assert np.isinf(ks[ids[1], :, at[1]]).all() and not kc[ids[1], :, at[1]].any()
    assert np.isfinite(ks[ids[2], :, at[2]]).all() and kc[ids[2], :, at[2]].any()


def test_bad_pages_and_lengths_are_skipped_and_reported():
    rng = np.random.default_rng(76)
    H, D = 2, 128
    for what, code in (("id", kv.DEV_BAD_BLOCK_ID), ("negative id", kv.DEV_BAD_BLOCK_ID),
                       ("beyond", kv.DEV_POS_BEYOND_TABLE), ("length", kv.DEV_BAD_LENGTH),
                       ("padding", kv.DEV_BAD_LENGTH)):
        w = W.make_workload("ropebad", q_lens=[3, 4, 2], ctx_before=[0, 14, 5], kv_heads=H,
                            head_dim=D, block_size=16, num_blocks=9, max_blocks_per_seq=2,
                            quant_mode=0, seed=77)
        d = DeviceBatch(w)
        if what == "id":
            d.block_table[1, 1] = w.num_blocks
            skip = {5, 6}
        elif what == "negative id":
            d.block_table[1, 1] = -1
            skip = {5, 6}
        elif what == "beyond":
            d.context_kv_lens[1] = 30
            skip = {5, 6}
        elif what == "length":
            d.context_kv_lens[1] = -1
            skip = {3, 4, 5, 6}
        else:  # tokens behind the last sequence: a padded batch
            d.cu_q_lens[3] = 7
            skip = {7, 8}
        turn = Turn(rng, D, 128)
        qb = _rows(rng, 9, 4, D)
        q = bf16_tensor(qb).cuda()
        out = torch.full_like(q, 7.0)
        _append(d, w, turn, q, out)
        assert d.error_code(reset=True) == code, what
        kc, vc, _, _ = d.host_caches()
        ids, at, pos = _slots(w)
        if what == "beyond":
            pos = pos.copy()
            pos[3:7] = [30, 31, 32, 33]
            ids, at = ids.copy(), at.copy()
            ids[3:5], at[3:5] = w.block_table[1, 1], [14, 15]
        keep = np.array([t not in skip for t in range(9)])
        _check_rows(bf16_bits(out), turn, "q", qb, pos, keep)
        assert (out[torch.from_numpy(~keep).cuda()] == 7).all(), what
        same = np.ones((w.num_blocks, 16), bool)
        same[ids[keep], at[keep]] = False
        for c, before in ((kc, w.k_cache), (vc, w.v_cache)):
            np.testing.assert_array_equal(c.transpose(0, 2, 1, 3)[same],
                                          before.transpose(0, 2, 1, 3)[same])
            # what is kept was written (the random codes do not all stay)
            assert (c[ids[keep], :, at[keep]] != before[ids[keep], :, at[keep]]).any((1, 2)).all()


def test_graph_replay_follows_its_inputs():
    """A captured append replayed with other tokens, lengths and positions."""
    rng = np.random.default_rng(78)
    mk = lambda seed, ctx: W.make_workload(  # noqa: E731
        "ropegraph", q_lens=np.ones(5, int), ctx_before=ctx, kv_heads=2, head_dim=64, block_size=16,
        num_blocks=17, max_blocks_per_seq=3, quant_mode=0, seed=seed, decode_null_cu=True)
    w = mk(79, [0, 3, 15, 16, 40])
    d = DeviceBatch(w)
    turn = Turn(rng, 64, 64)
    qb = _rows(rng, 5, 4, 64)
    q = bf16_tensor(qb).cuda()
    out = torch.zeros_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _append(d, w, turn, q, out, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _append(d, w, turn, q, out)
    w2 = mk(80, [1, 4, 16, 17, 41])
    qb2 = _rows(rng, 5, 4, 64)
    fresh = DeviceBatch(w2)
    for name in ("k_states", "v_states", "k_cache", "v_cache", "k_scale", "v_scale", "block_table",
                 "context_kv_lens"):
        getattr(d, name).copy_(getattr(fresh, name))
    q.copy_(bf16_tensor(qb2))
    graph.replay()
    torch.cuda.synchronize()
    assert d.error_code() == 0
    _check_rows(bf16_bits(out), turn, "q", qb2, _slots(w2)[2])
    _check_pool(w2, d, turn, _slots(w2)[2])


def test_append_then_gather_and_attention_use_the_rotated_keys():
    """The calls as a decode step makes them: append, then the gather's rows and
    the decode attention see the rotated key."""
    rng = np.random.default_rng(81)
    B, H, D, G = 6, 2, 128, 4
    w = W.make_workload("ropestep", q_lens=np.ones(B, int), ctx_before=[0, 1, 15, 16, 40, 63],
                        kv_heads=H, head_dim=D, block_size=16, num_blocks=B * 4 + 1, quant_mode=0,
                        seed=82, decode_null_cu=True)
    d = DeviceBatch(w)
    turn = Turn(rng, D, 128)
    qb = _rows(rng, B, H * G, D)
    q = bf16_tensor(qb).cuda()
    qo = torch.zeros_like(q)
    _append(d, w, turn, q, qo)
    d.gather()
    out = torch.zeros_like(q)
    need = kv.kvc8_attention_workspace_bytes(d.g, H * G)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    scale = D ** -0.5
    kv.kvc8_paged_decode_attention(d.g, H * G, qo, qo.stride(0), qo.stride(1), d.k_cache, d.v_cache,
                                   d.k_scale, d.v_scale, d.block_table, d.context_lengths, scale,
                                   out, out.stride(0), out.stride(1), ws, need, d.dev_error)
    assert d.error_code() == 0
    pos = _slots(w)[2]
    y, e = turn.exact(w.k_states, "k", pos)
    rows, _ = d.host_outputs()
    last = np.cumsum(w.context_lengths.astype(np.int64)) - 1
    got = bf16_f64(rows[last])
    step = np.abs(y).max(-1, keepdims=True) / 127
    # half a step of the code, the fp32 bounds, and bf16 of the gather
    fine = bool((np.abs(got - y) <= 0.51 * step + 3 * e + BF16 * (np.abs(y) + step)).all())
    assert fine
    caches = d.host_caches()
    want = oracle.paged_decode_attention(0, bf16_bits(qo), *caches, w.block_table,
                                         w.context_lengths, scale)
    _, vr = oracle.dequant_gather(0, *caches, w.block_table, w.context_lengths)
    top = np.abs(bf16_f64(vr)).max()
    # the decode attention's own tolerance (weights in bf16), see test_gpu_attention.py
    fine = bool((np.abs(bf16_f64(bf16_bits(out)) - want) <= 2.0 ** -7 * top + BF16 * np.abs(want)).all())
    assert fine
