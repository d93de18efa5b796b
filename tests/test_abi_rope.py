"""Host side of the rotating append, the norm-and-rotate pass and the shared-prefix
attention on the CPU: frequencies, and arguments refused before anything is
enqueued."""
import ctypes
import math

import numpy as np
import pytest

import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import binding as B

FAKE = 1 << 20  # an aligned, never-dereferenced address: checks fail before any launch


def _rope(**kw):
    a = dict(rotary_dim=128, freqs=FAKE, interleaved=0, attention_factor=1.0, norm_eps=1e-6,
             q_norm_weight=FAKE, k_norm_weight=FAKE, positions=FAKE)
    a.update(kw)
    return kv.Rope(**a)


GEOM = dict(num_seqs=2, kv_heads=8, head_dim=128, block_size=16, num_blocks=64,
            max_blocks_per_seq=8, quant_mode=0)


def _store(bf16=False, n=4, geom=None, rope=None, **kw):
    g = kv.Geom(**{**GEOM, **(geom or {})})
    a = dict(hq=16, q=FAKE, qt=16 * 128, qh=128, qo=FAKE, qot=16 * 128, qoh=128, k=FAKE, v=FAKE,
             xt=8 * 128, xh=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, cu=FAKE, ctx=FAKE)
    a.update(kw)
    r = rope if rope is not None else _rope()
    head = [ctypes.byref(g), ctypes.byref(r.struct), n, a["hq"], a["q"], a["qt"], a["qh"], a["qo"],
            a["qot"], a["qoh"], a["k"], a["v"], a["xt"], a["xh"], a["kc"], a["vc"]]
    tail = [a["bt"], a["cu"], a["ctx"], None, None]
    if bf16:
        return kv.load().kvc8_rope_store_bf16(*head, *tail)
    return kv.load().kvc8_rope_store(*head, a["ks"], a["vs"], *tail)


@pytest.mark.parametrize("bf16", [False, True])
def test_rope_store_refusals(bf16):
    bad, uns = kv.ERR_INVALID_ARG, kv.ERR_UNSUPPORTED
    names = ["q", "qo", "k", "v", "kc", "vc", "bt", "ctx"] + ([] if bf16 else ["ks", "vs"])
    for name in names:
        assert _store(bf16, **{name: None}) == bad, name
    for name in ("q", "qo", "k", "v", "kc", "vc"):
        assert _store(bf16, **{name: FAKE + 2}) == bad, name
    for name in ("qt", "qh", "qot", "qoh", "xt", "xh"):
        assert _store(bf16, **{name: 1028}) == bad, name
        assert _store(bf16, **{name: -128}) == bad, name
    assert _store(bf16, n=-1) == bad and _store(bf16, hq=-1) == bad
    assert _store(bf16, n=1 << 31) == uns and _store(bf16, hq=1 << 20) == uns
    assert _store(bf16, n=3, cu=None) == bad  # decode form: one token per sequence
    assert _store(bf16, n=1, geom=dict(num_seqs=0)) == bad
    assert _store(bf16, geom=dict(head_dim=24)) == bad
    assert _store(bf16, geom=dict(head_dim=512)) == uns
    if not bf16:
        assert _store(geom=dict(quant_mode=3)) == bad
        assert _store(ks=FAKE + 4) == bad
    # nothing to do is a no-op, whatever the pointers
    assert _store(bf16, n=0, k=None, q=None) == kv.OK
    assert _store(bf16, n=0, geom=dict(num_seqs=0)) == kv.OK


def test_rope_refusals():
    bad, uns = kv.ERR_INVALID_ARG, kv.ERR_UNSUPPORTED
    for want, kw in [(bad, dict(rotary_dim=-2)), (bad, dict(rotary_dim=130)),
                     (bad, dict(rotary_dim=144)), (bad, dict(rotary_dim=33)),
                     (uns, dict(rotary_dim=8)), (uns, dict(rotary_dim=120)),
                     (bad, dict(interleaved=2)), (bad, dict(freqs=None)),
                     (bad, dict(freqs=FAKE + 4)), (bad, dict(attention_factor=math.inf)),
                     (bad, dict(attention_factor=math.nan)), (bad, dict(norm_eps=-1e-6)),
                     (bad, dict(norm_eps=math.nan)), (bad, dict(q_norm_weight=FAKE + 2)),
                     (bad, dict(k_norm_weight=FAKE + 8)), (bad, dict(positions=FAKE + 2))]:
        assert _store(rope=_rope(**kw)) == want, kw
        assert _rows(rope=_rope(**kw)) == want, kw
    g = kv.Geom(**GEOM)
    for geom, rope in ((ctypes.byref(g), None), (None, ctypes.byref(_rope().struct))):
        assert kv.load().kvc8_rope_store(geom, rope, 1, 0, None, 0, 0, None, 0, 0, FAKE, FAKE, 8,
                                         8, *([FAKE] * 7), None, None) == bad


def _rows(n=4, rope=None, **kw):
    a = dict(d=128, hq=16, q=FAKE, qt=2048, qh=128, qo=FAKE, qot=2048, qoh=128, hk=8, k=FAKE,
             kt=1024, kh=128, ko=FAKE, kot=1024, koh=128)
    a.update(kw)
    r = rope if rope is not None else _rope()
    return kv.load().kvc8_qk_norm_rope(ctypes.byref(r.struct), n, a["d"], a["hq"], a["q"], a["qt"],
                                       a["qh"], a["qo"], a["qot"], a["qoh"], a["hk"], a["k"],
                                       a["kt"], a["kh"], a["ko"], a["kot"], a["koh"], None)


def test_qk_norm_rope_refusals():
    bad, uns = kv.ERR_INVALID_ARG, kv.ERR_UNSUPPORTED
    for name in ("q", "qo", "k", "ko"):
        assert _rows(**{name: None}) == bad, name
        assert _rows(**{name: FAKE + 8}) == bad, name
    for name in ("qt", "qh", "qot", "qoh", "kt", "kh", "kot", "koh"):
        assert _rows(**{name: 4}) == bad, name
        assert _rows(**{name: -8}) == bad, name
    assert _rows(d=8) == bad and _rows(d=100) == bad and _rows(d=272) == uns
    assert _rows(n=-1) == bad and _rows(n=1 << 31) == uns
    assert _rows(hq=-1) == bad and _rows(hk=-1) == bad and _rows(hk=1 << 17) == uns
    assert _rows(rope=_rope(positions=None)) == bad
    assert _rows(n=0, q=None) == kv.OK and _rows(hq=0, hk=0, k=None, q=None) == kv.OK
    assert kv.load().kvc8_qk_norm_rope(None, 1, 128, 0, None, 0, 0, None, 0, 0, 0, None, 0, 0,
                                       None, 0, 0, None) == bad


def _prefix(geom=None, hq=32, mpb=8, wsb=1 << 40, scale=0.088, **kw):
    g = kv.Geom(**{**GEOM, **(geom or {})})
    a = dict(q=FAKE, qs=32 * 128, qh=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, pl=FAKE,
             bt=FAKE, lens=FAKE, out=FAKE, os=32 * 128, oh=128, ws=FAKE)
    a.update(kw)
    return kv.load().kvc8_shared_prefix_attention(
        ctypes.byref(g), hq, a["q"], a["qs"], a["qh"], a["kc"], a["vc"], a["ks"], a["vs"], a["pt"],
        mpb, a["pl"], a["bt"], a["lens"], scale, a["out"], a["os"], a["oh"], a["ws"], wsb, None,
        None)


def test_shared_prefix_refusals():
    bad, uns = kv.ERR_INVALID_ARG, kv.ERR_UNSUPPORTED
    for name in ("q", "kc", "vc", "ks", "vs", "pt", "pl", "bt", "lens", "out"):
        assert _prefix(**{name: None}) == bad, name
    assert _prefix(hq=30) == bad and _prefix(hq=0) == bad and _prefix(hq=72) == uns
    assert _prefix(mpb=0) == bad and _prefix(mpb=1 << 28) == uns
    assert _prefix(qs=100) == bad and _prefix(qh=-128) == bad and _prefix(os=-8) == bad
    assert _prefix(q=FAKE + 8) == bad and _prefix(out=FAKE + 1) == bad
    assert _prefix(scale=math.inf) == bad and _prefix(scale=math.nan) == bad
    assert _prefix(geom=dict(head_dim=96)) == uns and _prefix(geom=dict(block_size=24)) == uns
    assert _prefix(geom=dict(quant_mode=3)) == bad
    g = kv.Geom(**GEOM)
    need = kv.kvc8_shared_prefix_workspace_bytes(g, 32, 8)
    assert need >= 256 and need % 256 == 0
    assert _prefix(wsb=need - 1) == kv.ERR_WORKSPACE
    assert _prefix(ws=None) == kv.ERR_WORKSPACE and _prefix(ws=FAKE + 16) == kv.ERR_WORKSPACE
    assert _prefix(geom=dict(num_seqs=0), q=None) == kv.OK
    # 2^21 tiles of rows or more by 1024 steps of positions: not in 32 bits
    many = dict(num_seqs=1 << 24, max_blocks_per_seq=1)
    steps = dict(block_size=128, kv_heads=8)
    assert _prefix(geom=dict(many, **steps), mpb=1 << 10) == uns
    assert kv.kvc8_shared_prefix_workspace_bytes(kv.Geom(**{**GEOM, **many, **steps}), 32, 1 << 8) > 0
    for hq, mpb in ((30, 8), (32, 0)):
        assert kv.kvc8_shared_prefix_workspace_bytes(g, hq, mpb) == 0


def _scaling(kind, base=1e4, factor=4.0, original=4096.0, low=1.0, high=32.0):
    return kv.RopeScaling(kind, base, factor, original, low, high)


@pytest.mark.parametrize("rot", [16, 64, 128, 256])
@pytest.mark.parametrize("kind", [kv.ROPE_PLAIN, kv.ROPE_LINEAR, kv.ROPE_BASE, kv.ROPE_BY_PARTS])
def test_frequencies(rot, kind):
    s = _scaling(kind)
    freqs, factor = kv.kvc8_rope_frequencies(s, rot)
    assert freqs.dtype == np.uint64 and freqs.shape == (rot // 2,)
    i = np.arange(rot // 2)
    base = s.base * (s.factor ** (rot / (rot - 2)) if kind == kv.ROPE_BASE else 1.0)
    f = base ** (-2.0 * i / rot)
    if kind == kv.ROPE_LINEAR:
        f = f / 4.0
    if kind == kv.ROPE_BY_PARTS:
        turns = 4096.0 * f / (2 * np.pi)
        g = (turns - 1.0) / 31.0
        mid = (turns > 1.0) & (turns < 32.0)
        f = np.where(mid, f / 4.0 * (1 - g) + f * g, np.where(turns <= 1.0, f / 4.0, f))
        assert mid.any() or rot == 16
        assert factor == pytest.approx(0.1 * math.log(4.0) + 1.0, rel=2.0 ** -23)
    else:
        assert factor == 1.0
    # a handful of fp64 roundings, and pow's last bits
    np.testing.assert_allclose(freqs.astype(np.float64) / 2.0 ** 64, f / (2 * np.pi), rtol=2.0 ** -46)
    if kind == kv.ROPE_BASE:  # the slowest pair is slowed by the factor, the fastest is kept
        plain, _ = kv.kvc8_rope_frequencies(_scaling(kv.ROPE_PLAIN), rot)
        assert float(plain[-1]) / float(freqs[-1]) == pytest.approx(4.0, rel=1e-9)
        assert freqs[0] == plain[0]


def test_frequencies_are_fractions_of_a_turn():
    # more than a turn per position: only the fraction counts
    freqs, _ = kv.kvc8_rope_frequencies(_scaling(kv.ROPE_LINEAR, factor=0.01), 16)
    want = (100.0 / (2 * np.pi)) % 1.0
    assert float(freqs[0]) / 2.0 ** 64 == pytest.approx(want, rel=1e-12)
    assert kv.kvc8_rope_frequencies(_scaling(kv.ROPE_PLAIN), 0)[0].size == 0


def test_frequencies_refusals():
    lib = kv.load()
    buf = (ctypes.c_uint64 * 64)()
    f = ctypes.c_float()

    def call(s, rot=128, out=buf):
        return lib.kvc8_rope_frequencies(None if s is None else ctypes.byref(s), rot, out,
                                         ctypes.byref(f))
    bad = kv.ERR_INVALID_ARG
    assert call(None) == bad and call(_scaling(0), out=None) == bad
    assert call(_scaling(0), rot=-2) == bad and call(_scaling(0), rot=7) == bad
    assert call(_scaling(4)) == bad and call(_scaling(-1)) == bad
    assert call(_scaling(0, base=0.0)) == bad and call(_scaling(0, base=math.nan)) == bad
    assert call(_scaling(1, factor=0.0)) == bad and call(_scaling(1, factor=math.inf)) == bad
    assert call(_scaling(2), rot=2) == bad
    assert call(_scaling(3, original=0.0)) == bad and call(_scaling(3, low=32.0)) == bad
    assert call(_scaling(0, factor=math.nan)) == kv.OK  # not used there
    assert lib.kvc8_rope_frequencies(ctypes.byref(_scaling(0)), 128, buf, None) == kv.OK
    assert B.DEV_TIMEOUT == 5 and kv.kvc8_version() >= 10100
