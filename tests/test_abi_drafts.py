"""Refusals of the drafted tokens' entry points, on the host, before anything is enqueued."""
import ctypes

import pytest

import dequant_kvc8_store_gb300 as kv
from dequant_kvc8_store_gb300 import binding as B

FAKE = 1 << 20  # an aligned, never-dereferenced address: checks fail before any launch


def geom(**kw):
    return kv.Geom(**{**dict(num_seqs=2, kv_heads=8, head_dim=128, block_size=16, num_blocks=64,
                             max_blocks_per_seq=8, quant_mode=0), **kw})


def assign(g, **kw):
    a = dict(held=FAKE, want=FAKE, free=FAKE, count=FAKE, out=FAKE, bt=FAKE, lens=FAKE, slots=FAKE, rows=4)
    a.update(kw)
    return kv.load().kvc8_assign_blocks(ctypes.byref(g), a["held"], a["want"], a["free"], a["count"], a["out"], a["bt"],
                                        a["lens"], a["slots"], a["rows"], None, None)


def tree(g, heads=32, n=5, most=4, **kw):
    a = dict(q=FAKE, qts=32 * 128, qhs=128, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, cu=FAKE, ctx=FAKE, mask=FAKE,
             words=1, scale=0.1, out=FAKE + 4096, ots=32 * 128, ohs=128, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return kv.load().kvc8_tree_attention(ctypes.byref(g), heads, n, most, a["q"], a["qts"], a["qhs"], a["kc"], a["vc"],
                                         a["ks"], a["vs"], a["bt"], a["cu"], a["ctx"], a["mask"], a["words"], a["scale"],
                                         a["out"], a["ots"], a["ohs"], a["ws"], a["wsb"], None, None)


def compact(g, bf16=False, **kw):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, ctx=FAKE, acc=FAKE, most=4, num=FAKE, lens=FAKE)
    a.update(kw)
    lib = kv.load()
    if bf16:
        return lib.kvc8_compact_drafts_bf16(ctypes.byref(g), a["kc"], a["vc"], a["bt"], a["ctx"], a["acc"], a["most"],
                                            a["num"], a["lens"], None, None)
    return lib.kvc8_compact_drafts(ctypes.byref(g), a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["ctx"], a["acc"],
                                   a["most"], a["num"], a["lens"], None, None)


BAD_GEOMS = [("head_dim", 24), ("head_dim", 8), ("quant_mode", 3), ("kv_heads", 0), ("block_size", 0), ("num_blocks", 0),
             ("max_blocks_per_seq", 0), ("num_seqs", -1)]


@pytest.mark.parametrize("call", [assign, lambda g: tree(g), lambda g: compact(g)])
@pytest.mark.parametrize("field,bad", BAD_GEOMS)
def test_bad_geometry(call, field, bad):
    assert call(geom(**{field: bad})) == kv.ERR_INVALID_ARG


def test_assign_refuses():
    for name in ("held", "want", "free", "count", "out", "bt", "lens"):
        assert assign(geom(), **{name: None}) == kv.ERR_INVALID_ARG, name
    assert assign(geom(), rows=-1) == kv.ERR_INVALID_ARG
    assert assign(geom(), slots=FAKE + 4) == kv.ERR_INVALID_ARG
    assert assign(geom(num_seqs=B.ASSIGN_MAX_SEQS + 1)) == kv.ERR_UNSUPPORTED


def test_tree_refuses():
    g = geom()
    for name in ("q", "kc", "vc", "ks", "vs", "bt", "ctx", "out"):
        assert tree(g, **{name: None}) == kv.ERR_INVALID_ARG, name
    for name, bad in [("q", FAKE + 2), ("kc", FAKE + 8), ("ks", FAKE + 4), ("out", FAKE + 1), ("mask", FAKE + 4),
                      ("out", FAKE), ("qts", -8), ("qts", 4100), ("qhs", 4), ("ots", -1), ("ohs", -1),
                      ("scale", float("nan")), ("scale", float("inf"))]:
        assert tree(g, **{name: bad}) == kv.ERR_INVALID_ARG, name
    assert tree(g, ws=None) == tree(g, ws=FAKE + 16) == tree(g, wsb=16) == kv.ERR_WORKSPACE
    assert tree(g, heads=0) == tree(g, heads=12) == tree(g, n=-1) == tree(g, most=0) == kv.ERR_INVALID_ARG
    assert tree(g, most=65) == kv.ERR_INVALID_ARG  # two words of mask
    assert tree(g, cu=None, n=3) == kv.ERR_INVALID_ARG  # one draft each: two tokens
    assert tree(g, heads=72) == tree(g, most=B.MAX_DRAFTS + 1, words=5) == tree(g, n=1 << 31) == kv.ERR_UNSUPPORTED
    assert tree(geom(head_dim=96)) == tree(geom(block_size=24)) == kv.ERR_UNSUPPORTED
    assert tree(geom(max_blocks_per_seq=1 << 27)) == kv.ERR_UNSUPPORTED  # positions of 32 bits
    # 2^31 units: 8 heads x 4096 sequences x 8 tiles x 8192 steps
    assert tree(geom(num_seqs=4096, max_blocks_per_seq=1 << 16), most=256, words=4) == kv.ERR_UNSUPPORTED
    assert tree(geom(num_seqs=0), n=0, cu=None) == kv.OK and tree(geom(num_seqs=0), n=1) == kv.ERR_INVALID_ARG
    assert tree(g, n=0, q=None, out=None) == kv.OK


def test_tree_workspace():
    size = lambda g, heads=32, n=5, most=4: kv.kvc8_tree_attention_workspace_bytes(g, heads, n, most)  # noqa: E731
    assert size(geom()) > 0 and size(geom()) % 256 == 0
    assert size(geom(head_dim=96)) == size(geom(), 12) == size(geom(), 32, -1) == size(geom(), 32, 5, 257) == 0


@pytest.mark.parametrize("bf16", [False, True])
def test_compact_refuses(bf16):
    names = ("kc", "vc", "bt", "ctx", "acc", "num") + (() if bf16 else ("ks", "vs"))
    for name in names:
        assert compact(geom(), bf16, **{name: None}) == kv.ERR_INVALID_ARG, name
    assert compact(geom(), bf16, kc=FAKE + 8) == compact(geom(), bf16, most=0) == kv.ERR_INVALID_ARG
    assert compact(geom(), bf16, most=B.MAX_DRAFTS + 1) == kv.ERR_UNSUPPORTED
    assert compact(geom(num_seqs=0), bf16) == kv.OK
    if not bf16:
        assert compact(geom(), ks=FAKE + 4) == kv.ERR_INVALID_ARG


def test_names():
    assert (B.DEV_NO_FREE_BLOCK, B.DEV_BAD_INDEX) == (6, 7) and kv.kvc8_version() >= 10200
    text = open(B.HEADER).read()
    assert f"#define KVC8_ASSIGN_MAX_SEQS {B.ASSIGN_MAX_SEQS}" in text and f"#define KVC8_MAX_DRAFTS {B.MAX_DRAFTS}" in text


def test_tree_refuses_tables_of_more_than_2_26_positions():
    # a tile of query rows may have all its steps in one CTA: its waits must end within their limit
    g = lambda blocks: geom(num_seqs=1, kv_heads=1, max_blocks_per_seq=blocks, block_size=16)  # noqa: E731
    size = lambda blocks: kv.kvc8_tree_attention_workspace_bytes(g(blocks), 4, 1, 4)  # noqa: E731
    assert size(1 << 22) > 0 and size((1 << 22) + 1) == 0
    assert tree(g((1 << 22) + 1), heads=4, n=1) == kv.ERR_UNSUPPORTED


def test_tree_refuses_mask_rows_whose_bits_no_32_bit_count_holds():
    # (no tokens: checks alone)
    assert tree(geom(), n=0, words=1 << 20) == kv.OK
    assert tree(geom(), n=0, words=(1 << 20) + 1) == tree(geom(), words=1 << 30) == kv.ERR_UNSUPPORTED
    assert tree(geom(), n=0, words=1 << 30, mask=None) == kv.OK  # not looked at
