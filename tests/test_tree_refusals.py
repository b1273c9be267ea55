"""Arguments that the tree calls, the appends at positions and the compactions refuse on the host, and
what the mask packing gives: nothing of these touches a device, so they run without a GPU."""
import ctypes
import random

import pytest
import torch

from paged_kv_cache_299_gb300 import binding as pa
from _tree import KINDS, batch_bits, mask_words

P = ctypes.c_void_p
FAKE = P(0x1000)  # never dereferenced
ODD = P(0x1008)
BAD, UNS = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


def desc(nb=4, hkv=8, d=64, bs=16):
    return pa.CacheDesc(nb, hkv, d, bs)


def tree(q8, **kw):
    a = dict(out=FAKE, q=FAKE, mask=FAKE, words=1, qsl=FAKE, tokens=40, mq=20, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
             cd=desc(), bt=FAKE, mb=4, ctx=FAKE, seqs=2, hq=32, scale=0.125, ws=FAKE, wb=1 << 40)
    a.update(kw)
    f = pa.load().pa_tree_attention_q8 if q8 else pa.load().pa_tree_attention
    scales = (a["ks"], a["vs"]) if q8 else ()
    return f(a["out"], a["q"], a["mask"], a["words"], a["qsl"], a["tokens"], a["mq"], a["kc"], a["vc"], *scales, a["cd"],
             a["bt"], a["mb"], a["ctx"], a["seqs"], a["hq"], a["scale"], a["ws"], a["wb"], None, None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(out=None), dict(q=None), dict(mask=None), dict(qsl=None), dict(kc=None), dict(vc=None), dict(bt=None),
    dict(ctx=None), dict(out=ODD), dict(q=ODD), dict(kc=ODD), dict(vc=ODD), dict(mask=P(0x1002)), dict(words=0),
    dict(words=1, mq=33, tokens=60), dict(mq=41), dict(mq=-1), dict(tokens=-1), dict(seqs=-1), dict(mb=0), dict(mb=-4),
    dict(hq=0), dict(hq=30), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(cd=desc(nb=0)), dict(cd=desc(hkv=65))])
def test_tree_refuses(q8, bad):
    assert tree(q8, **bad) == BAD
    assert pa.load().pa_last_error() != b""


@pytest.mark.parametrize("q8", [False, True])
def test_tree_unsupported_and_empty(q8):
    assert tree(q8, hq=24) == UNS and tree(q8, hq=64) == UNS
    assert tree(q8, mq=1025, tokens=2000, words=40) == UNS
    assert tree(q8, cd=desc(d=128)) == UNS and tree(q8, cd=desc(bs=32)) == UNS
    assert tree(q8, cd=desc(nb=1 << 24)) == UNS  # 2^31 rows per pool
    for none in (dict(seqs=0), dict(tokens=0), dict(mq=0)):
        assert tree(q8, out=None, q=None, mask=None, ws=None, wb=0, **none) == pa.PA_OK
    assert tree(True, ks=None) == BAD and tree(True, vs=P(0x1002)) == BAD


@pytest.mark.parametrize("q8", [False, True])
def test_tree_workspace(q8):
    """Without a device there is no size to meet, and no call goes through."""
    for bad in (dict(ws=None), dict(ws=ODD), dict(wb=16)):
        assert tree(q8, **bad) == pa.PA_ERR_WORKSPACE


def append_at(q8, **kw):
    a = dict(q=FAKE, qs=2048, qo=FAKE, qos=2048, hq=32, k=FAKE, ks=512, v=FAKE, vs=512, cs=FAKE, npos=100, inter=0,
             pos=FAKE, axes=3, pairs=0x924924924924, bt=FAKE, mb=4, ctx=FAKE, qsl=FAKE, seqs=2, tokens=5, kc=FAKE,
             vc=FAKE, ksc=FAKE, vsc=FAKE, cd=desc())
    a.update(kw)
    scales = (a["ksc"], a["vsc"]) if q8 else ()
    f = pa.load().pa_rope_append_at_q8 if q8 else pa.load().pa_rope_append_at
    return f(a["q"], a["qs"], a["qo"], a["qos"], a["hq"], a["k"], a["ks"], a["v"], a["vs"], a["cs"], a["npos"],
             a["inter"], a["pos"], a["axes"], a["pairs"], a["bt"], a["mb"], a["ctx"], a["qsl"], a["seqs"], a["tokens"],
             a["kc"], a["vc"], *scales, a["cd"], None, None)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("bad", [
    dict(pos=None), dict(pos=P(0x1001)), dict(axes=0), dict(axes=5), dict(axes=-1), dict(axes=1), dict(axes=2, pairs=2),
    dict(pairs=3 << 62), dict(cs=None), dict(npos=0), dict(k=None), dict(v=None), dict(kc=None), dict(bt=None),
    dict(ctx=None), dict(q=None), dict(qo=None), dict(q=ODD), dict(qs=2044), dict(ks=504), dict(tokens=-1),
    dict(seqs=0), dict(mb=0), dict(qsl=None), dict(qs=4096), dict(cd=desc(nb=0))])
def test_append_at_refuses(q8, bad):
    assert append_at(q8, **bad) == BAD
    assert pa.load().pa_last_error() != b""


def test_append_at_the_rest():
    for q8 in (False, True):
        assert append_at(q8, cd=desc(d=128)) == UNS
        assert append_at(q8, tokens=0, pos=None, k=None) == pa.PA_OK
    assert append_at(True, ksc=None) == BAD and append_at(True, vsc=P(0x1002)) == BAD


def compact(q8, **kw):
    a = dict(kept=FAKE, ksl=FAKE, first=FAKE, n=9, most=5, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, cd=desc(), bt=FAKE, mb=4,
             seqs=2)
    a.update(kw)
    scales = (a["ks"], a["vs"]) if q8 else ()
    f = pa.load().pa_compact_tokens_q8 if q8 else pa.load().pa_compact_tokens
    return f(a["kept"], a["ksl"], a["first"], a["n"], a["most"], a["kc"], a["vc"], *scales, a["cd"], a["bt"], a["mb"],
             a["seqs"], None, None)


@pytest.mark.parametrize("q8", [False, True])
def test_compact_refuses(q8):
    for bad in (dict(kept=None), dict(ksl=None), dict(first=None), dict(kc=None), dict(vc=None), dict(bt=None),
                dict(kc=ODD), dict(vc=ODD), dict(kept=P(0x1002)), dict(n=-1), dict(most=-1), dict(seqs=-1), dict(mb=0),
                dict(cd=desc(nb=0))):
        assert compact(q8, **bad) == BAD, bad
    assert compact(q8, cd=desc(d=32)) == UNS and compact(q8, seqs=1 << 28) == UNS
    for none in (dict(n=0), dict(most=0), dict(seqs=0)):
        assert compact(q8, kept=None, bt=None, **none) == pa.PA_OK
    assert compact(True, ks=None) == BAD and compact(True, vs=P(0x1001)) == BAD


def test_binding_refuses():
    with pytest.raises(ValueError):
        pa.pack_tree_mask(torch.zeros(3, 4))
    with pytest.raises(ValueError):
        pa.pack_tree_mask(torch.zeros(3, dtype=torch.bool))
    for axes in ([0] * 31, [0] * 31 + [4], [0] * 31 + [-1], [0.0] * 32):
        with pytest.raises(ValueError):
            pa._pair_axes(axes, 4)
    with pytest.raises(ValueError):
        pa._pair_axes([0, 1] * 16, 1)
    assert pa._pair_axes([0, 1] * 16, 2) == sum(1 << (4 * i + 2) for i in range(16))
    assert pa._pair_axes(None, 1) == 0 and pa._pair_axes([3] * 32, 4) == (1 << 64) - 1


@pytest.mark.parametrize("n", [1, 31, 32, 33, 64, 100])
def test_packed_masks(n):
    g = torch.Generator().manual_seed(n)
    seen = torch.rand(50, n, generator=g) < 0.5
    packed = pa.pack_tree_mask(seen)
    assert packed.dtype is torch.int32 and packed.shape == (50, -(-n // 32))
    for t in range(50):
        for j in range(n):
            assert bool(int(packed[t, j // 32]) >> (j % 32) & 1) == bool(seen[t, j])
    assert pa.pack_tree_mask(torch.zeros(0, n, dtype=torch.bool)).shape == (0, -(-n // 32))


def test_masks_of_the_tests_agree_with_the_packing():
    for kind in KINDS:
        lens = [5, 40, 0, 70]
        bits = batch_bits(kind, lens, 3)
        seen = torch.zeros(sum(lens), 70, dtype=torch.bool)
        for t, b in enumerate(x for rows in bits for x in rows):
            for j in range(70):
                seen[t, j] = bool(b >> j & 1)
        assert torch.equal(mask_words(bits, lens), pa.pack_tree_mask(seen))


def test_every_mask_kind_has_what_it_is_for():
    rng = random.Random(0)
    from _tree import tree_bits
    assert tree_bits("chain", 3, rng) == [1, 3, 7] and tree_bits("star", 3, rng) == [1, 2, 4]
    assert 0 in tree_bits("mask", 200, rng)  # rows that see nothing drafted
